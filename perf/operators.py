"""The decode-step operators around the W4A16 products, as a user's program calls them: the RMS norm
that feeds a quantized layer, the append to a paged key-value cache with the position rotation, and the
attention of one new token per sequence over that cache.

``run`` computes a case in plain torch operations, or, where ``own`` is true, with the library's kernels.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_BYTES = {"none": 0, "f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
_E4M3_MAX = 448.0
_EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------

def _norm(M, K, x, residual, out, **more):
    return dict(op="rms_norm", M=M, K=K, x=x, residual=residual, out=out, **more)


def _append(T, seqs, Hq, Hkv, D, rot, layout, page, x, q, cache, max_pos, **more):
    return dict(op="kv_append", T=T, seqs=seqs, Hq=Hq, Hkv=Hkv, D=D, rot=rot, layout=layout, page=page, x=x, q=q,
                cache=cache, max_pos=max_pos, **more)


def _attention(B, L, ragged, Hq, Hkv, D, page, q, cache, **more):
    return dict(op="paged_attention", B=B, L=L, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, page=page, q=q, cache=cache, **more)


def listed():
    return [
        # one token of a 7B-shaped layer, between a W4A16 product (fp32 out) and the next (fp16 in)
        _norm(1, 4096, "f32", "f32", "f16", name="norm_1x4096"),
        # an odd batch of the down projection's width, quantized to 8 bits per row
        _norm(37, 11008, "f16", "none", "e4m3", name="norm_37x11008_e4m3"),
        # the calibration batch of the 70B gate+up layer, with its residual stream
        _norm(16384, 8192, "bf16", "bf16", "f16", name="norm_16384x8192"),
        # one token of a 32-head block: QKV straight from the W4A16 product
        _append(1, 1, 32, 32, 128, 128, "half", 16, "f32", "f16", "f16", 4096, name="append_1_mha"),
        # a decode batch with shared key-value heads, far positions, an 8-bit cache
        _append(61, 61, 64, 8, 128, 128, "half", 32, "f32", "f16", "e4m3", 131072, name="append_61_gqa_e4m3"),
        # a prompt batch (8 x 512 tokens), half of each head rotated in interleaved pairs
        _append(4096, 8, 32, 32, 128, 64, "interleaved", 64, "bf16", "bf16", "bf16", 8192, name="append_4096_partial"),
        # the same append from the fp32 product of a prefill, shared heads, a page size of no power of two
        _append(2047, 3, 64, 8, 128, 128, "half", 24, "f32", "bf16", "bf16", 32768, name="append_2047_page24"),
        # the first tokens of one conversation
        _attention(1, 33, False, 32, 32, 128, 16, "f16", "f16", name="attn_1x33_mha"),
        # one long document, shared key-value heads
        _attention(1, 131072, False, 64, 8, 128, 64, "bf16", "bf16", name="attn_1x131072_gqa"),
        # a serving batch of very different lengths, empty padding rows among them
        _attention(67, 8192, True, 64, 8, 128, 16, "bf16", "bf16", name="attn_67_ragged_gqa"),
        # a batch of a 32-head block at one length
        _attention(16, 4096, False, 32, 32, 128, 16, "f16", "f16", name="attn_16x4096_mha"),
        # a serving batch on an 8-bit cache
        _attention(96, 4099, True, 64, 8, 128, 32, "f16", "e4m3", name="attn_96_ragged_e4m3"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_norm", "kv_append", "paged_attention"])
    if op == "rms_norm":
        K = _spread(rng, 64, 16384)
        x, residual = rng.choice(["f32", "f16", "bf16"]), rng.choice(["none", "f16", "bf16", "f32"])
        out = rng.choice(["f16", "bf16", "f32", "e4m3"])
        each = _BYTES[x] + 2 * _BYTES[residual] + _BYTES[out]
        return _norm(_spread(rng, 1, min(16384, (16384 * 8192 * 8) // (K * each))), K, x, residual, out)
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    Hq = Hkv * rng.choice([1, 1, 2, 4, 7, 8] if Hkv <= 8 else [1, 2])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
    cache, q = rng.choice([("f16", "f16"), ("bf16", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")])
    if op == "kv_append":
        most = (4096 * 96 * 128) // ((Hq + 2 * Hkv) * D * 2)
        max_pos = _spread(rng, 4096, min(1 << 20, 8192 * page))
        if rng.random() < 0.5:
            T = seqs = _spread(rng, 1, min(most, 256))
        else:
            T = _spread(rng, 2, min(most, 4096))
            seqs = rng.randint(1, min(T, 16))
        return _append(T, seqs, Hq, Hkv, D, rng.choice([D, D, D // 2, 16, 0]), rng.choice(["half", "interleaved"]), page,
                       rng.choice(["f32", "f16", "bf16"]), q, cache, max_pos)
    most = (16 * 4096 * 32 * 128) // (Hkv * D)
    B = _spread(rng, 1, 256)
    L = _spread(rng, 1, max(1, min(131072, most // B)))
    return _attention(B, L, rng.random() < 0.7, Hq, Hkv, D, page, q, cache)


def _lengths(case):
    """The lengths of an attention case's sequences: all L, or spread below it with an empty row."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    rng = random.Random(B * 1000003 + L)
    lens = [rng.randint(max(1, L // 16), L) for _ in range(B)]
    lens[0] = L
    if B > 2:
        lens[B // 2] = 0
    return lens


# ---- inputs --------------------------------------------------------------------------------

def _randn(shape, g, dtype=torch.float32):
    t = torch.empty(shape, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype, device="cuda")
    t.normal_(generator=g)
    return t.to(dtype)


def _frequencies(rot):
    """theta_i = 10000^(-2i/rot), in radians per position."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -i / rot)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rms_norm":
        M, K = case["M"], case["K"]
        magnitude = torch.exp(0.5 * _randn((K,), g))   # channels of different size, as activations have
        X = (_randn((M, K), g) * magnitude).to(_TYPES[case["x"]])
        state = dict(case, X=X, weight=1.0 + 0.2 * _randn((K,), g), residual_in=None, residual_out=None)
        if case["residual"] != "none":
            state["residual_in"] = _randn((M, K), g, _TYPES[case["residual"]])
            state["residual_out"] = torch.empty_like(state["residual_in"])
        return state
    D, Hq, Hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    ctype = _TYPES[case["cache"]]
    scales = [None, None]
    if case["cache"] == "e4m3":   # a calibrated scale per key-value head
        scales = [torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.01 for _ in range(2)]
    if case["op"] == "kv_append":
        T, seqs = case["T"], case["seqs"]
        rows = _randn((T, (Hq + 2 * Hkv) * D), g, _TYPES[case["x"]])   # the fused [q | k | v] of the QKV product
        q, k, v = rows.split([Hq * D, Hkv * D, Hkv * D], dim=1)
        if T == seqs:   # decode: one token of each sequence
            seq = None
            pos = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda", dtype=torch.int32)
            if T > 8:
                pos[T - 1] = -1   # a padded row of the batch
            first = [int(p) for p in pos.tolist()]
            spans = [(p, p + 1) if p >= 0 else (0, 0) for p in first]
        else:           # prompts: consecutive tokens of each sequence
            share = [T // seqs + (i < T % seqs) for i in range(seqs)]
            starts = torch.randint(0, max(1, case["max_pos"] - max(share)), (seqs,), generator=g, device="cuda").tolist()
            pos = torch.cat([torch.arange(s, s + n, dtype=torch.int32, device="cuda") for s, n in zip(starts, share)])
            seq = torch.repeat_interleave(torch.arange(seqs, dtype=torch.int32, device="cuda"),
                                          torch.tensor(share, device="cuda"))
            spans = [(s, s + n) for s, n in zip(starts, share)]
        width = -(-(case["max_pos"] + 4096) // page)
        table = torch.zeros(seqs, width, dtype=torch.int32)
        used = sum(-(-b // page) - a // page for a, b in spans)
        order = torch.randperm(used, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        at = 0
        for i, (a, b) in enumerate(spans):
            n = -(-b // page) - a // page
            table[i, a // page: a // page + n] = order[at: at + n]
            at += n
        caches = [_randn((max(1, used), page, Hkv, D), g).to(ctype) for _ in range(2)]
        return dict(case, q_in=q.view(T, Hq, D), k_in=k.view(T, Hkv, D), v_in=v.view(T, Hkv, D), positions=pos, seq=seq,
                    table=table.cuda(), k_cache=caches[0], v_cache=caches[1], freqs=_frequencies(case["rot"]) if case["rot"] else None,
                    k_scale=scales[0], v_scale=scales[1])
    lens = _lengths(case)
    B, width = case["B"], max(1, -(-case["L"] // page))
    pages = sum(-(-n // page) for n in lens) + 1
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    need = torch.tensor([-(-n // page) for n in lens], device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    rank = (torch.cumsum(need, 0) - need)[:, None] + slot
    table = torch.where(slot < need[:, None], order[rank.clamp(max=pages - 1)], 0).to(torch.int32)
    caches = [_randn((pages, page, Hkv, D), g, torch.float16 if case["cache"] == "e4m3" else ctype) for _ in range(2)]
    if case["cache"] == "e4m3":
        caches = [(c * 60.0).to(ctype) for c in caches]
    return dict(case, q_in=_randn((B, Hq, D), g, _TYPES[case["q"]]) * 2.0, k_cache=caches[0], v_cache=caches[1], table=table,
                lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), k_scale=scales[0], v_scale=scales[1])


# ---- the plain forms -----------------------------------------------------------------------

def _plain_norm(s):
    h = s["X"].float()
    if s["residual_in"] is not None:
        h = h + s["residual_in"].float()
        s["residual_out"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + _EPS) * s["weight"]
    if s["out"] != "e4m3":
        return y.to(_TYPES[s["out"]])
    peak = y.abs().amax(dim=1, keepdim=True)
    scale = torch.where(peak > 0, peak / _E4M3_MAX, torch.ones_like(peak))
    return (y / scale).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn), scale.squeeze(1)


def _rotated(x, cos, sin, rot, layout):
    x = x.float()
    if rot == 0:
        return x
    head, tail = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return torch.cat([head, tail], dim=-1)


def _to_cache(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x / scale[None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(dtype)


def _put(cache, page, slot, rows, live):
    """cache[page, slot] = rows[live], moved as plain bytes or halves."""
    as_bits = {1: torch.uint8, 2: torch.int16}[cache.element_size()]
    cache.view(as_bits)[page, slot] = rows.view(as_bits)[live]


def _plain_append(s):
    pos = s["positions"].long()
    cos = sin = None
    if s["rot"]:
        angle = pos.double()[:, None] * s["freqs"]   # far positions times a frequency need 64 bits
        cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    q = _rotated(s["q_in"], cos, sin, s["rot"], s["layout"]).to(_TYPES[s["q"]])
    k = _to_cache(_rotated(s["k_in"], cos, sin, s["rot"], s["layout"]), s["k_scale"], s["k_cache"].dtype)
    v = _to_cache(s["v_in"].float(), s["v_scale"], s["v_cache"].dtype)
    seq = torch.arange(pos.numel(), device=pos.device) if s["seq"] is None else s["seq"].long()
    live = pos >= 0
    at = pos.clamp(min=0)
    page, slot = s["table"][seq, at // s["page"]].long()[live], (at % s["page"])[live]
    _put(s["k_cache"], page, slot, k, live)
    _put(s["v_cache"], page, slot, v, live)
    return q.masked_fill(~live[:, None, None], 0.0), s["k_cache"], s["v_cache"]


def _gathered(cache, table, scale):
    """(B, Hkv, positions, D) in 32 bits: the pages of each sequence side by side."""
    rows = cache.view(torch.uint8)[table.long()].view(cache.dtype).float()
    B, n, page, H, D = rows.shape
    rows = rows.view(B, n * page, H, D).transpose(1, 2)
    return rows if scale is None else rows * scale[None, :, None, None]


def _plain_attention(s):
    B, Hq, Hkv, D = s["B"], s["Hq"], s["Hkv"], s["D"]
    k, v = _gathered(s["k_cache"], s["table"], s["k_scale"]), _gathered(s["v_cache"], s["table"], s["v_scale"])
    q = s["q_in"].float().view(B, Hkv, Hq // Hkv, D)
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    live = torch.arange(k.shape[2], device=q.device)[None, :] < s["lengths"][:, None]
    score = score.masked_fill(~live[:, None, None, :], -math.inf)
    peak = score.amax(dim=-1, keepdim=True)
    weight = torch.exp(score - torch.where(peak == -math.inf, 0.0, peak))
    total = weight.sum(dim=-1, keepdim=True)
    out = torch.matmul(weight, v.masked_fill(~live[:, None, :, None], 0.0)) / torch.where(total > 0, total, 1.0)
    return out.reshape(B, Hq, D).to(_TYPES[s["q"]])


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        import post_quantization_column_b200 as awq
        if s["op"] == "rms_norm":
            out = awq.rms_norm(s["X"], s["weight"], _EPS, residual=s["residual_in"], residual_out=s["residual_out"],
                               out_dtype=_TYPES[s["out"]])
        elif s["op"] == "kv_append":
            out = awq.kv_append(s["q_in"], s["k_in"], s["v_in"], s["k_cache"], s["v_cache"], s["table"], s["positions"],
                                s["freqs"], seqs=s["seq"], interleaved=s["layout"] == "interleaved",
                                k_scale=s["k_scale"], v_scale=s["v_scale"], q_dtype=_TYPES[s["q"]])
            out = (out, s["k_cache"], s["v_cache"])
        else:
            out = awq.paged_attention(s["q_in"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
    elif s["op"] == "rms_norm":
        out = _plain_norm(s)
    elif s["op"] == "kv_append":
        out = _plain_append(s)
    else:
        out = _plain_attention(s)
    if s["op"] == "rms_norm":
        out = tuple(out) if isinstance(out, tuple) else (out,)
        out = out if s["residual_out"] is None else out + (s["residual_out"],)
    return out


def work(case):
    if case["op"] == "rms_norm":
        M, K, r = case["M"], case["K"], _BYTES[case["residual"]]
        return {"bytes": M * K * (_BYTES[case["x"]] + 2 * r + _BYTES[case["out"]]) + 4 * K + (4 * M if case["out"] == "e4m3" else 0),
                "flops": 5 * M * K}
    D, Hq, Hkv, c, q = case["D"], case["Hq"], case["Hkv"], _BYTES[case["cache"]], _BYTES[case["q"]]
    if case["op"] == "kv_append":
        T = case["T"]
        return {"bytes": T * D * ((Hq + 2 * Hkv) * _BYTES[case["x"]] + Hq * q + 2 * Hkv * c) + 8 * T + 4 * case["rot"],
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    total = sum(_lengths(case))
    return {"bytes": 2 * total * Hkv * D * c + 2 * case["B"] * Hq * D * q + 4 * sum(-(-n // case["page"]) for n in _lengths(case)),
            "flops": 4 * total * Hq * D}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rms_norm":
        h = s["X"].double()
        if s["residual_in"] is not None:
            h += s["residual_in"].double()
        y = h * s["weight"].double() / torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["K"] + _EPS)
        outs = [y]
        if case["out"] == "e4m3":
            scale = y.abs().max(dim=1).values / _E4M3_MAX
            scale[scale == 0] = 1.0
            outs = [y / scale[:, None], scale]
        return tuple(outs + ([h] if s["residual_in"] is not None else []))
    if case["op"] == "kv_append":
        T, D, rot = case["T"], case["D"], case["rot"]
        pos = s["positions"].double()
        first, second = torch.arange(D, device="cuda"), torch.arange(D, device="cuda")
        cos = torch.ones(T, 1, D, dtype=torch.float64, device="cuda")
        sin = torch.zeros_like(cos)
        if rot:   # out[d] = x[d] cos + x[partner(d)] (+-sin)
            pair = torch.arange(rot // 2, device="cuda")
            lo, hi = (pair, pair + rot // 2) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
            second[lo], second[hi] = first[hi], first[lo]
            theta = torch.outer(pos, s["freqs"])[:, None, :]
            cos[..., lo], cos[..., hi] = torch.cos(theta), torch.cos(theta)
            sin[..., lo], sin[..., hi] = -torch.sin(theta), torch.sin(theta)
        turn = lambda x: x.double() * cos + x.double()[..., second] * sin  # noqa: E731
        q, k, v = turn(s["q_in"]), turn(s["k_in"]), s["v_in"].double()
        if case["cache"] == "e4m3":
            k = (k / s["k_scale"].double()[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
            v = (v / s["v_scale"].double()[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
        q[s["positions"] < 0] = 0.0
        caches = [s["k_cache"].double(), s["v_cache"].double()]
        where = [(t, int(p)) for t, p in enumerate(s["positions"].tolist()) if p >= 0]
        seqs = range(T) if s["seq"] is None else s["seq"].tolist()
        table = s["table"].cpu()
        rows = torch.tensor([int(table[seqs[t], p // case["page"]]) * case["page"] + p % case["page"] for t, p in where],
                            device="cuda", dtype=torch.long)
        kept = torch.tensor([t for t, _ in where], device="cuda", dtype=torch.long)
        for c, x in zip(caches, (k, v)):
            c.view(-1, case["Hkv"], D).index_copy_(0, rows, x.index_select(0, kept))
        return q, caches[0], caches[1]
    B, Hq, Hkv, D, page = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        ids = s["table"][b, : -(-n // page)].long()
        k, v = (c.view(torch.uint8)[ids].view(c.dtype).reshape(-1, Hkv, D)[:n].double().permute(1, 0, 2) for c in (s["k_cache"], s["v_cache"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
        logits = torch.bmm(s["q_in"][b].double().view(Hkv, -1, D), k.transpose(1, 2)) / math.sqrt(D)
        out[b] = torch.bmm(torch.softmax(logits, dim=-1), v).view(Hq, D)
    return out
