"""The decode-step operators against their oracle (B200 only).

Tolerances, with u = 2^-24 (half a step of fp32) and eta(t) = finfo(t).eps / 2, the half step of
an output type relative to the value (tiny(t) / 2 absolute below its normal range):

* RMS norm: h is one fp32 addition (u); sum h^2 adds at most K / 32 terms one after the other in
  a thread and fewer than 64 partial sums, each product and addition rounded once, and the square
  root halves the relative error: (K / 32 + 66) u / 2; h w, the quotient, the root, the
  reciprocal, the last product and the quotient by a scale add fewer than 10 roundings. Then eta of
  the output.
* Rotation: the fraction of a turn is rounded to fp32 (at most 2^-26 turns = 2 pi 2^-26), sine
  and cosine of it are within 2 ulp (2^-23), the magnitude and the two products and the sum add
  3 roundings: a pair (x, y) comes within (|x| + |y|) |m| (2 pi 2^-26 + 2^-23 + 3 u), plus eta. The
  quotient by an e4m3 scale is a product with the rounded reciprocal: 2 u, and 1 for their product.
* Attention: a score is an fp32 sum of D exact products: it is off by at most 2 D u scale
  sum |q k| (twice the bound of D rounded additions, since a tensor-core step may truncate),
  plus 4 u |s| for the scale in base 2; a weight is then off by that (as a factor), by the
  exponential (2^-21 with its argument's rounding, 4 u |s - max|) and by its 16-bit rounding
  eta(weight type), together E, so that the output is off by E sum p |v - o| / (1 - E), by the fp32
  sums over the tokens (n / 32 + 64) 2 u sum p |v|, and by eta of the output.
"""
import numpy as np
import pytest
import torch

import oracle as O
import oracle.awq_decode as D
import oracle.awq_w4a16 as Q
import post_quantization_column_b200 as awq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _np(t):
    return t.detach().cpu().double().numpy()


def _eta(dtype, value):
    """Half a step of `dtype` at `value`."""
    info = torch.finfo(dtype)
    return np.maximum(info.eps / 2 * np.abs(value), info.smallest_normal * info.eps / 2)


def _randn(*shape, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _close(got, ref, bound, what=""):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], np.broadcast_to(bound, got.shape)[bad][:4])


# ---- RMS norm ------------------------------------------------------------------------------

def _norm_bound(K):
    return ((K / 32 + 66) / 2 + 10) * U


def _check_norm(X, w, out, residual=None, new_residual=None, eps=1e-6, rows=slice(None)):
    y, h = D.rms_norm(_np(X), None if residual is None else _np(residual), _np(w), eps)
    if isinstance(out, tuple):
        codes, scales = _np(out[0]), _np(out[1])
        ref = D.row_scales(y)
        _close(scales[rows], ref[rows], (_norm_bound(y.shape[1]) + 2 * U) * ref[rows], "scale")
        z = y / scales[:, None]
        _close(codes[rows], z[rows], (_eta(E4M3, z) * (1 + 2.0 ** -20) + 2 * _norm_bound(y.shape[1]) * np.abs(z))[rows], "codes")
    else:
        tol = _norm_bound(y.shape[1])
        _close(_np(out)[rows], y[rows], (_eta(out.dtype, y) * (1 + 2.0 ** -10) + 2 * tol * np.abs(y))[rows], "y")
    if residual is not None:
        _close(_np(new_residual)[rows], h[rows], (_eta(new_residual.dtype, h) * (1 + 2.0 ** -10) + U * np.abs(h))[rows], "h")


@pytest.mark.parametrize("out", [F16, BF16, F32, E4M3])
@pytest.mark.parametrize("x,r", [(F32, None), (F32, F32), (F16, F16), (BF16, BF16), (F16, None), (BF16, F32), (F32, BF16), (F16, BF16)])
def test_norm_types(x, r, out):
    for M, K in ((3, 256), (5, 4096), (2, 11008)):
        X, w = _randn(M, K, dtype=x, seed=1), _randn(K, seed=2)
        R = None if r is None else _randn(M, K, dtype=r, seed=3, scale=3.0)
        new = None if r is None else torch.full_like(R, 7.0)
        got = awq.rms_norm(X, w, residual=R, residual_out=new, out_dtype=out)
        _check_norm(X, w, got, R, new)
        if r is not None:   # in place, the same bits
            again = awq.rms_norm(X, w, residual=R, out_dtype=out)
            assert torch.equal(R, new)
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got if out == E4M3 else [got], again if out == E4M3 else [again]))


@pytest.mark.parametrize("K", [1, 2, 7, 8, 31, 64, 72, 130, 255, 256, 264, 1000, 1024, 1032, 2049, 4104, 8192, 8200, 12151, 16384, 16392, 28672, 57344])
@pytest.mark.parametrize("M", [1, 3, 700])
def test_norm_sizes(M, K):
    if M * K > 3e7:
        M = 40
    X, w, R = _randn(M, K, dtype=BF16, seed=K), _randn(K, dtype=BF16, seed=2), _randn(M, K, dtype=BF16, seed=3)
    new = torch.empty_like(R)
    _check_norm(X, w, awq.rms_norm(X, w, residual=R, residual_out=new), R, new)
    _check_norm(X, w, awq.rms_norm(X, w, out_dtype=E4M3))


@pytest.mark.parametrize("out", [F16, E4M3])
@pytest.mark.parametrize("x,r", [(BF16, None), (F16, BF16), (F32, None), (F32, F32)])
@pytest.mark.parametrize("K", [8, 64, 65, 120, 250, 500, 1001, 1032, 2047, 4096, 4104, 5000, 8190])
def test_norm_many_rows(x, r, out, K):
    """More rows than a grid holds several times over."""
    M = 1500 if K > 1000 else 5003
    X, w, R = _randn(M, K, dtype=x, seed=K), _randn(K, seed=2), None if r is None else _randn(M, K, dtype=r, seed=3)
    new = None if r is None else torch.empty_like(R)
    _check_norm(X, w, awq.rms_norm(X, w, residual=R, residual_out=new, out_dtype=out), R, new)


@pytest.mark.parametrize("K,pitch,offset", [(256, 264, 0), (256, 257, 0), (256, 264, 1), (4096, 4104, 8), (100, 128, 4), (2048, 2050, 2), (12288, 12296, 0)])
def test_norm_strides_and_offsets(K, pitch, offset):
    M = 9
    base, rbase = _randn(M, pitch + offset, dtype=F16, seed=4), _randn(M, pitch + offset, seed=5)
    X, R, w = base[:, offset:offset + K], rbase[:, offset:offset + K], _randn(K, dtype=F16, seed=6)
    before, kept = rbase.clone(), base.clone()
    out = awq.rms_norm(X, w, residual=R, out_dtype=BF16)
    _check_norm(X, w, out, before[:, offset:offset + K], R)
    rbase[:, offset:offset + K] = before[:, offset:offset + K]
    assert torch.equal(rbase, before) and torch.equal(base, kept)   # nothing beside the rows was written
    Xt = _randn(K, M, dtype=F16, seed=7).t()                        # rows that are not contiguous
    _check_norm(Xt, w, awq.rms_norm(Xt, w))
    Xe = _randn(1, K, dtype=F16, seed=8).expand(M, K)               # one row M times
    _check_norm(Xe, w, awq.rms_norm(Xe, w))


@pytest.mark.parametrize("K", [96, 515])
def test_norm_columns_of_one_buffer(K):
    """X and a residual that is replaced in place, side by side in one buffer; rows that overlap."""
    M, w = 40, _randn(K, seed=6)
    for pitch, at in ((2 * K, K), (3 * K + 5, K), (2 * K + 64, K + 64)):
        buf = _randn(M, pitch, seed=5)
        before = buf.clone()
        X, R = buf[:, :K], buf[:, at:at + K]
        _check_norm(before[:, :K], w, awq.rms_norm(X, w, residual=R), before[:, at:at + K], R)
        kept = torch.ones(pitch, dtype=torch.bool, device="cuda")
        kept[at:at + K] = False
        assert torch.equal(buf[:, kept], before[:, kept])
        with pytest.raises(awq.AwqError):
            awq.rms_norm(X, w, residual=buf[:, K - 1:2 * K - 1])
        with pytest.raises(awq.AwqError):
            awq.rms_norm(buf[:, 1:1 + K], w, residual=buf[:, :K])
    flat = _randn(M + K, seed=7)
    for step in (1, K % 8 or 8):
        Xh = torch.as_strided(flat, (1 + M // step, K), (step, 1))
        _check_norm(Xh, w, awq.rms_norm(Xh, w))
    with pytest.raises(awq.AwqError):
        awq.rms_norm(_randn(M, K, seed=8), buf[3, :K], residual=buf[:, :K])


@pytest.mark.parametrize("K", [512, 515])
def test_norm_special_rows(K):
    X, w = _randn(6, K, seed=9), _randn(K, seed=10)
    X[1] = 0.0
    X[2, 3] = float("nan")
    X[3, 5] = float("inf")
    X[4] *= 1e-15
    good = [0, 1, 4, 5]
    out = awq.rms_norm(X, w, eps=1e-6, out_dtype=F32)
    _check_norm(X[good], w, out[good])
    assert torch.isnan(out[2]).all() and torch.isnan(out[3, 5])
    codes, scales = awq.rms_norm(X, w, eps=1e-6, out_dtype=E4M3)
    assert scales[1] == 1.0 and (codes[1].float() == 0).all()
    assert torch.isnan(scales[2]) and torch.isnan(scales[3])
    assert torch.isnan(codes[2].float()).all()
    for i in good:
        _check_norm(X[i:i + 1], w, (codes[i:i + 1], scales[i:i + 1]))
    assert awq.rms_norm(X[:0], w).shape == (0, K)
    assert awq.rms_norm(X[:0], w, out_dtype=E4M3)[1].shape == (0,)


def test_norm_refusals():
    X, w = _randn(4, 64), _randn(64)
    R = _randn(4, 64)
    for bad in (lambda: awq.rms_norm(X[0], w), lambda: awq.rms_norm(X, w[:-1]), lambda: awq.rms_norm(X, w, residual=R[:2]),
                lambda: awq.rms_norm(X, w, residual_out=R), lambda: awq.rms_norm(X, w.cpu()),
                lambda: awq.rms_norm(X, w, residual=R, residual_out=R.half()),
                lambda: awq.rms_norm(X, w, residual=R.t().contiguous().t()),
                lambda: awq.rms_norm(X, w.clone().requires_grad_())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: awq.rms_norm(X.double(), w), lambda: awq.rms_norm(X, w, out_dtype=torch.int8)):
        with pytest.raises(TypeError):
            bad()
    big = _randn(8, 64)
    for bad in (lambda: awq.rms_norm(X, w, residual=big[:4], residual_out=big[2:6]), lambda: awq.rms_norm(X, w, residual=R, residual_out=X),
                lambda: awq.rms_norm(X, w, residual=R[:1].expand(4, 64)), lambda: awq.rms_norm(X, w, eps=-1.0)):
        with pytest.raises(awq.AwqError):
            bad()


# ---- append to the paged cache ---------------------------------------------------------------

def _cache(pages, page, heads, dim, dtype, order="pshd", seed=0, values=None):
    """A cache tensor (pages, page, heads, dim) whose memory holds the dims in `order`."""
    sizes = dict(p=pages, s=page, h=heads, d=dim)
    t = (_randn(*[sizes[c] for c in order], seed=seed) if values is None else torch.full([sizes[c] for c in order], values).cuda()).to(dtype)
    return t.permute(*[order.index(c) for c in "pshd"])


def _table(rng, seqs, max_pages, pages):
    """Distinct random pages for every entry."""
    return torch.from_numpy(rng.permutation(pages)[: seqs * max_pages].reshape(seqs, max_pages).astype(np.int32)).cuda()


def _check_append(q, k, v, before, caches, table, positions, freqs, out, seqs=None, interleaved=False, magnitude=1.0, scales=(None, None)):
    page, pages = caches[0].shape[1], caches[0].shape[0]
    f = np.zeros(0) if freqs is None else _np(freqs)
    pos = positions.cpu().numpy()
    R = 2 * len(f)

    def turned(x):
        ref = D.rotate(_np(x), pos, f, interleaved, magnitude)
        size = np.abs(_np(x))
        pair = size.copy()
        if R:
            i = np.arange(R // 2)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            pair[..., a] = pair[..., b] = size[..., a] + size[..., b]
        tol = pair * abs(magnitude) * (2 * np.pi * 2.0 ** -26 + 2.0 ** -23 + 3 * U)
        if R < size.shape[-1]:
            tol[..., R:] = 0.0
        return ref, tol

    if q is not None:
        ref, tol = turned(q)
        ref[pos < 0], tol[pos < 0] = 0.0, 0.0
        _close(_np(out), ref, tol + _eta(out.dtype, np.abs(ref) + tol), "q")
    at = D.places(table.cpu().numpy(), page, pages, pos, None if seqs is None else seqs.cpu().numpy())
    for x, old, new, scale, turn in ((k, before[0], caches[0], scales[0], True), (v, before[1], caches[1], scales[1], False)):
        ref, tol = turned(x) if turn else (_np(x), np.zeros(x.shape))
        s = np.ones(x.shape[1]) if scale is None else _np(scale)
        ref, tol = ref / s[:, None], tol / s[:, None] + (0 if scale is None else 3 * U * np.abs(ref / s[:, None]))
        got, want = _np(new), _np(old)
        touched = np.zeros(want.shape[:2], dtype=bool)
        for t, (p, slot) in enumerate(at):
            if p < 0:
                continue
            r = np.clip(ref[t], -D.E4M3_MAX, D.E4M3_MAX) if new.dtype == E4M3 else ref[t]
            _close(got[p, slot], r, tol[t] + _eta(new.dtype, np.abs(r) + tol[t]), ("cache", t))
            touched[p, slot] = True
        assert np.array_equal(got[~touched], want[~touched])   # every other place as it was


@pytest.mark.parametrize("x,cache,qt", [(F32, F16, F16), (F32, E4M3, BF16), (F16, F16, F16), (BF16, BF16, BF16), (BF16, E4M3, F16), (F32, BF16, F16)])
@pytest.mark.parametrize("Dh,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 64, False), (64, 16, True), (64, 64, False), (256, 256, True), (256, 128, False), (128, 0, False)])
def test_append_types_and_layouts(x, cache, qt, Dh, rot, interleaved):
    rng = np.random.default_rng(Dh + rot)
    T, seqs, Hq, H, page, mp = 11, 11, 6, 3, 7, 5
    rows = _randn(T, (Hq + 2 * H) * Dh, dtype=x, seed=rot)
    q, k, v = (t.view(T, -1, Dh) for t in rows.split([Hq * Dh, H * Dh, H * Dh], dim=1))
    caches = [_cache(seqs * mp + 3, page, H, Dh, cache, seed=i) for i in (1, 2)]
    scales = [torch.rand(H, device="cuda") * 0.01 + 0.004 for _ in range(2)] if cache == E4M3 else [None, None]
    before = [c.clone() for c in caches]
    table = _table(rng, seqs, mp, seqs * mp + 3)
    pos = torch.from_numpy(rng.integers(0, page * mp, T).astype(np.int32)).cuda()
    pos[4] = -1
    freqs = awq.rope_frequencies(rot)[0] if rot else None
    out = awq.kv_append(q, k, v, *caches, table, pos, freqs, interleaved=interleaved, k_scale=scales[0], v_scale=scales[1], q_dtype=qt)
    assert out.dtype == qt and out.is_contiguous()
    _check_append(q, k, v, before, caches, table, pos, freqs, out, None, interleaved, 1.0, scales)


@pytest.mark.parametrize("order", ["pshd", "phsd", "hpsd", "sphd"])
@pytest.mark.parametrize("page,T,Hq,H", [(1, 1, 1, 1), (16, 40, 8, 1), (5, 300, 4, 4), (64, 513, 64, 8), (100, 7, 71, 71)])
def test_append_prompts_and_cache_orders(order, page, T, Hq, H):
    rng = np.random.default_rng(page + T)
    seqs = max(1, T // 100)
    lens = np.diff(np.linspace(0, T, seqs + 1).astype(int))
    starts = rng.integers(0, 50, size=seqs)
    mp = -(-int(max(starts + lens)) // page)
    pos = torch.from_numpy(np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)]).astype(np.int32)).cuda()
    sq = torch.from_numpy(np.repeat(np.arange(seqs), lens).astype(np.int32)).cuda()
    q, k, v = (_randn(T, h, 128, dtype=BF16, seed=i) for i, h in enumerate((Hq, H, H)))
    caches = [_cache(seqs * mp, page, H, 128, BF16, order, seed=i) for i in (1, 2)]
    before = [c.clone() for c in caches]
    table = _table(rng, seqs, mp, seqs * mp)
    freqs, mag = awq.rope_frequencies(128, scaling="ramp", factor=4.0, original_len=1024.0)
    out = awq.kv_append(q, k, v, *caches, table, pos, freqs, seqs=sq, magnitude=mag)
    _check_append(q, k, v, before, caches, table, pos, freqs, out, sq, False, mag)
    # without queries, the same cache
    again = [c.clone() for c in before]
    assert awq.kv_append(None, k, v, *again, table, pos, freqs, seqs=sq, magnitude=mag) is None
    assert all(torch.equal(a, b) for a, b in zip(again, caches))


def test_append_far_positions_and_strided_inputs():
    T, H, Dh, page = 6, 2, 128, 4096
    pos = torch.tensor([0, 4095, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) + 4097], dtype=torch.int32, device="cuda")
    mp = int(pos.max()) // page + 1
    table = torch.full((T, mp), -1, dtype=torch.int32, device="cuda")
    for t in range(T):
        table[t, int(pos[t]) // page] = t
    wide = _randn(Dh, T, 4 * H + 1, seed=3).permute(1, 2, 0)          # rows that are not contiguous
    q, k, v = wide[:, :2 * H], wide[:, 2 * H:3 * H], wide[:, 3 * H:4 * H]
    caches = [_cache(T, page, H, Dh, F16, seed=i) for i in (1, 2)]
    before = [c.clone() for c in caches]
    freqs = awq.rope_frequencies(Dh)[0]
    out = awq.kv_append(q, k, v, *caches, table, pos, freqs)
    _check_append(q, k, v, before, caches, table, pos, freqs, out)


def test_append_tokens_without_a_place():
    T, H, Dh, page = 8, 2, 64, 8
    q, k, v = _randn(T, H, Dh, seed=1), _randn(T, H, Dh, seed=2), _randn(T, H, Dh, seed=3)
    caches = [_cache(4, page, H, Dh, F16, seed=i) for i in (1, 2)]
    before = [c.clone() for c in caches]
    table = torch.tensor([[0, 1], [-1, 7], [2, 3], [4, 3]], dtype=torch.int32, device="cuda")
    #                     fine    page -1  page 7  fine     page 4   beyond the table, no such sequence (2)
    seqs = torch.tensor([0, 1, 1, 2, 3, 0, 4, -1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([9, 3, 8, 15, 0, 16, 1, 1], dtype=torch.int32, device="cuda")
    freqs = awq.rope_frequencies(Dh)[0]
    for status in (torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32).pin_memory()):
        out = awq.kv_append(q, k, v, *caches, table, pos, freqs, seqs=seqs, status=status)
        torch.cuda.synchronize()
        _check_append(q, k, v, before, caches, table, pos, freqs, out, seqs)
        with pytest.raises(awq.AwqError):
            awq.check_status(status)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    awq.kv_append(q[:1], k[:1], v[:1], *caches, table, pos[:1], freqs, status=status)
    awq.check_status(status)


# ---- attention over the paged cache ------------------------------------------------------------

def _check_attention(q, k_cache, v_cache, table, lengths, out, scale=None, k_scale=None, v_scale=None, rows=None):
    B, Hq, Dh = q.shape
    page, H = k_cache.shape[1], k_cache.shape[2]
    scale = Dh ** -0.5 if scale is None else scale
    wt = F16 if k_cache.dtype == E4M3 else k_cache.dtype
    tab, lens = table.cpu().numpy(), lengths.cpu().numpy()
    for b in range(B) if rows is None else rows:
        n = max(0, int(lens[b]))
        got = _np(out[b])
        if n == 0:
            assert np.array_equal(got, np.zeros((Hq, Dh)))
            continue
        ids = torch.from_numpy(tab[b, : -(-n // page)].astype(np.int64)).cuda()
        bits = torch.uint8 if k_cache.element_size() == 1 else torch.int16
        k, v = (_np(c.view(bits)[ids].view(c.dtype).reshape(-1, H, Dh)[:n]) for c in (k_cache, v_cache))
        if k_scale is not None:
            k, v = k * _np(k_scale)[:, None], v * _np(v_scale)[:, None]
        qb = _np(q[b])
        ref = D.attention(qb, k, v, scale)
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
            s = scale * (kh @ qb[h])
            p = np.exp(s - s.max())
            p /= p.sum()
            off = 2 * Dh * U * abs(scale) * (np.abs(kh) @ np.abs(qb[h])) + 4 * U * np.abs(s)
            E = 2 * off.max() + 2.0 ** -21 + float((4 * U * np.abs(s - s.max()) * (p > 1e-12)).max()) + torch.finfo(wt).eps / 2
            assert E < 0.1
            tol = E / (1 - E) * (p @ np.abs(vh - ref[h])) + (n / 32 + 64) * 2 * U * (p @ np.abs(vh))
            _close(got[h], ref[h], tol + _eta(out.dtype, np.abs(ref[h]) + tol), (b, h, n))


def _attn_case(lens, Hq, H, Dh, page, qt, cache, order="pshd", seed=0, spread=2.0, extra_pages=2):
    rng = np.random.default_rng(seed)
    B, mp = len(lens), max(1, -(-max(max(lens), 1) // page))
    pages = B * mp + extra_pages
    caches = [_cache(pages, page, H, Dh, cache, order, seed=seed + i) for i in (1, 2)]
    scales = [None, None]
    if cache == E4M3:
        caches = [_cache(pages, page, H, Dh, F32, order, seed=seed + i).mul_(50.0).to(E4M3) for i in (1, 2)]
        scales = [torch.rand(H, device="cuda") * 0.01 + 0.015 for _ in range(2)]
    q = _randn(B, Hq, Dh, dtype=qt, seed=seed + 3, scale=spread)
    return q, caches[0], caches[1], _table(rng, B, mp, pages), torch.tensor(lens, dtype=torch.int32, device="cuda"), scales


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 128, 129, 200, 0, 511, 512, 513]


@pytest.mark.parametrize("qt,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("Dh", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(1, 1), (6, 6), (8, 1), (14, 2), (9, 1), (32, 2), (71, 1)])
def test_attention_heads_types_lengths(qt, cache, Dh, Hq, H):
    q, kc, vc, table, lens, (ks, vs) = _attn_case(EDGES, Hq, H, Dh, 16, qt, cache, seed=Dh + Hq)
    out = awq.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs)
    _check_attention(q, kc, vc, table, lens, out, None, ks, vs)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 1024])
@pytest.mark.parametrize("order", ["pshd", "phsd", "hpsd"])
def test_attention_pages_and_orders(page, order):
    q, kc, vc, table, lens, _ = _attn_case([700, 1, 65, 0, 333], 8, 2, 128, page, BF16, BF16, order, seed=page)
    out = awq.paged_attention(q, kc, vc, table, lens)
    _check_attention(q, kc, vc, table, lens, out)


@pytest.mark.parametrize("lens", [[1], [64], [65], [5000], [40000], [0], [0, 0, 0], [3, 0, 20000, 0, 1], [130] * 300, [0] * 200 + [70] * 333 + [0] * 9])
def test_attention_batches(lens):
    q, kc, vc, table, lt, _ = _attn_case(lens, 8, 2, 128, 32, F16, F16, seed=len(lens))
    out = awq.paged_attention(q, kc, vc, table, lt)
    rows = sorted(set(range(0, len(lens), max(1, len(lens) // 12))) | {len(lens) - 1, len(lens) // 2})
    _check_attention(q, kc, vc, table, lt, out, rows=rows)
    assert torch.equal(out, awq.paged_attention(q, kc, vc, table, lt))   # the same bits again


@pytest.mark.parametrize("lens,Hq,H,Dh,page,qt,cache", [
    ([35000] * 4 + [0] + [36001] * 4, 16, 8, 128, 32, F16, E4M3),        # few segments, heads in fours
    ([4400 + 37 * (i % 9) for i in range(65)], 8, 8, 128, 16, BF16, E4M3),  # more segments than runs
    ([130000, 0, 100001, 150000], 6, 6, 64, 64, F16, F16),               # rows of 128 bytes, heads in twos
    ([90000, 60000, 80000], 20, 20, 64, 24, BF16, E4M3),                 # a page that ends inside a block of 16
    ([200000, 230001], 5, 5, 64, 16, F16, E4M3)])                        # heads that do not pair
def test_attention_long_batches_of_short_rows(lens, Hq, H, Dh, page, qt, cache):
    """Enough work that the heads of short rows lie side by side in a CTA where they can."""
    g = torch.Generator("cuda").manual_seed(Hq + Dh)
    rng = np.random.default_rng(Dh)
    B, need = len(lens), [-(-n // page) for n in lens]
    pages = sum(need) + 1
    scales = [torch.rand(H, device="cuda", generator=g) * 0.01 + 0.015 for _ in range(2)] if cache == E4M3 else [None, None]
    caches = [(torch.randn(pages, page, H, Dh, device="cuda", generator=g, dtype=F16) * (50 if cache == E4M3 else 1)).to(cache) for _ in range(2)]
    order, table, at = rng.permutation(pages).astype(np.int32), np.zeros((B, max(need)), dtype=np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = _randn(B, Hq, Dh, dtype=qt, seed=3, scale=2.0)
    lt, tab = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(table).cuda()
    out = awq.paged_attention(q, *caches, tab, lt, k_scale=scales[0], v_scale=scales[1])
    _check_attention(q, *caches, tab, lt, out, None, *scales, rows=sorted({0, B // 2, B - 1}))
    assert torch.isfinite(out.float()).all()
    # every row again, alone: another split of the same sums. Both are within E sum p |v - o| of the
    # exact value, E < 1e-3 (an fp16 weight's half step and the score's error) and |v| about 1, and
    # rounded to at most a half step of bf16
    for b in range(B):
        alone = awq.paged_attention(q[b:b + 1], *caches, tab[b:b + 1], lt[b:b + 1], k_scale=scales[0], v_scale=scales[1])
        assert torch.allclose(alone[0].float(), out[b].float(), atol=2e-3, rtol=2e-2), b


@pytest.mark.parametrize("order", ["pshd", "phsd", "hpsd"])
@pytest.mark.parametrize("qt,cache,Dh,Hq,H,page", [(F16, F16, 64, 32, 32, 16), (BF16, E4M3, 128, 32, 8, 8), (F16, E4M3, 64, 20, 10, 24), (BF16, E4M3, 128, 90, 9, 16)])
@pytest.mark.parametrize("width", [None, 4096])
def test_attention_many_short_sequences_over_short_rows(order, qt, cache, Dh, Hq, H, page, width):
    """No sequence longer than one unit of work, and many of them: the heads of a token go side by
    side where they go in fours or twos. `width`: the tokens that a row of the table has room for."""
    unit = 32768 // (2 * Dh * (2 if cache == F16 else 1))
    lens = [min(n, unit) for n in (0, 1, 15, 16, 17, 31, 33, unit // 4, unit // 4 + 1, unit // 2 - 1, unit // 2 + 1, unit - 1, unit, 0)] * 20
    q, kc, vc, table, lt, (ks, vs) = _attn_case(lens, Hq, H, Dh, page, qt, cache, order, seed=Hq)
    if width is not None:
        table = torch.nn.functional.pad(table, (0, width // page - table.shape[1]), value=-1)
    out = awq.paged_attention(q, kc, vc, table, lt, k_scale=ks, v_scale=vs)
    _check_attention(q, kc, vc, table, lt, out, None, ks, vs, rows=range(14))
    for b in (50, 133, 279):
        _check_attention(q, kc, vc, table, lt, out, None, ks, vs, rows=[b])
    assert torch.isfinite(out.float()).all()
    assert torch.equal(out, awq.paged_attention(q, kc, vc, table, lt, k_scale=ks, v_scale=vs))


def test_attention_peaked_and_flat_scores():
    q, kc, vc, table, lens, _ = _attn_case([900, 130, 40], 4, 4, 128, 16, F16, F16, seed=5, spread=20.0)
    out = awq.paged_attention(q, kc, vc, table, lens)
    _check_attention(q, kc, vc, table, lens, out)
    for scale in (0.0, -0.05, 1e-3):
        out = awq.paged_attention(q, kc, vc, table, lens, scale)
        _check_attention(q, kc, vc, table, lens, out, scale)


@pytest.mark.parametrize("qt,cache", [(BF16, E4M3), (BF16, BF16)])
def test_attention_queries_of_every_size(qt, cache):
    # queries far beyond and below fp16's range, whose scores a scale brings back
    q, kc, vc, table, lens, (ks, vs) = _attn_case([300, 70], 8, 2, 128, 16, qt, cache, seed=6, spread=1.0)
    for size in (2.0 ** 30, 2.0 ** -30):
        qs = q * size
        out = awq.paged_attention(qs, kc, vc, table, lens, 0.1 / size, k_scale=ks, v_scale=vs)
        _check_attention(qs, kc, vc, table, lens, out, 0.1 / size, ks, vs)


@pytest.mark.parametrize("qt,cache", [(F16, F16), (BF16, BF16), (F16, E4M3)])
def test_attention_does_not_see_what_lies_beyond(qt, cache):
    """NaN and infinities in unused pages, in the rest of a last page and in a zero-length sequence's
    pages; table entries beyond the need that name no page."""
    lens = [70, 0, 17, 33]
    q, kc, vc, table, lt, (ks, vs) = _attn_case(lens, 8, 2, 128, 16, qt, cache, seed=7)
    clean = awq.paged_attention(q, kc, vc, table, lt, k_scale=ks, v_scale=vs)
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    tab = table.cpu()
    for b, n in enumerate(lens):
        for p in range(n):
            used[int(tab[b, p // 16]), p % 16] = True
    for c, bad in ((kc, float("nan")), (vc, float("nan") if cache == E4M3 else float("inf"))):
        f = c.float()
        f[~used.cuda()] = bad
        c.copy_(f.to(cache))
    for b, n in enumerate(lens):
        table[b, -(-n // 16):] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = awq.paged_attention(q, kc, vc, table, lt, k_scale=ks, v_scale=vs, status=status)
    assert torch.equal(out, clean)
    awq.check_status(status)


def test_attention_nonfinite_inside():
    """What softmax gives: a NaN key or query makes its heads NaN, a -inf score has no weight."""
    q, kc, vc, table, lens, _ = _attn_case([100, 100, 100, 100], 4, 2, 64, 16, F16, F16, seed=8)
    clean = awq.paged_attention(q, kc, vc, table, lens)
    at = lambda b, p: (int(table[b, p // 16]), p % 16)  # noqa: E731
    kc[at(0, 37)][1, 5] = float("nan")
    kc[at(1, 37)][0] = float("-inf")     # scores -inf or +inf by the query's signs: made one sign below
    q[1, :2] = q[1, :2].abs() + 0.01
    vc[at(2, 3)][0, 7] = float("nan")
    ref = awq.paged_attention(q, kc, vc, table, lens)
    assert torch.isnan(ref[0, 2:]).all() and torch.equal(ref[0, :2], clean[0, :2])
    kept = kc.clone()
    kept[at(1, 37)][0] = 0.0
    assert torch.isfinite(ref[1]).all() and torch.equal(ref[1, 2:], clean[1, 2:])
    s = (_np(q[1, :2]) @ np.stack([_np(kept[at(1, p)][0]) for p in range(100)]).T) / 8.0
    s[:, 37] = -np.inf
    p = np.exp(s - s.max(axis=1, keepdims=True))
    v = np.stack([_np(vc[at(1, t)][0]) for t in range(100)])
    want = p @ v / p.sum(axis=1, keepdims=True)
    assert np.all(np.abs(_np(ref[1, :2]) - want) <= 2 ** -9 * (np.abs(want) + (p @ np.abs(v)) / p.sum(axis=1, keepdims=True)))
    assert torch.isnan(ref[2, :2, 7]).all() and torch.equal(ref[2, :2, :7], clean[2, :2, :7]) and torch.equal(ref[3], clean[3])


def test_attention_bad_pages_and_lengths():
    lens = [70, 200, 129, 40, 64]
    q, kc, vc, table, lt, _ = _attn_case(lens, 8, 2, 128, 16, BF16, BF16, seed=9)
    clean = awq.paged_attention(q, kc, vc, table, lt)
    table[1, 7] = kc.shape[0]
    table[2, 0] = -1
    lt[3] = table.shape[1] * 16 + 1
    table[3] = table[0, 0]
    lt[4] = -3
    for status in (torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32).pin_memory()):
        out = awq.paged_attention(q, kc, vc, table, lt, status=status)
        torch.cuda.synchronize()
        assert torch.isnan(out[1:4].float()).all() and torch.equal(out[0], clean[0]) and (out[4] == 0).all()
        with pytest.raises(awq.AwqError):
            awq.check_status(status)
    assert torch.isnan(awq.paged_attention(q, kc, vc, table, lt)[1].float()).all()   # and without a status word


@pytest.mark.parametrize("lens,Hq,H,Dh,cache", [([5000] * 4, 8, 8, 128, F16), ([700] * 70, 8, 8, 128, E4M3), ([9000] * 66, 8, 8, 128, E4M3),
                                                ([40000], 32, 2, 64, F16), ([900] * 100, 20, 5, 256, F16), ([65], 16, 1, 128, BF16)])
def test_attention_stays_in_its_work_space(lens, Hq, H, Dh, cache):
    """Through the C ABI, in exactly the bytes it asks for: what lies behind them stays."""
    import ctypes
    import struct
    qt = F16 if cache == E4M3 else cache
    q, kc, vc, table, lt, (ks, vs) = _attn_case(lens, Hq, H, Dh, 16, qt, cache, seed=Dh)
    lib, code = awq.library(), {BF16: 0, F16: 2, E4M3: 3}
    size = lib.awq_paged_attention_workspace(Hq, H, Dh, code[cache])
    ws = torch.full((size + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((len(lens) * Hq * Dh + 512,), 7.0, dtype=qt, device="cuda")
    desc = struct.pack("@16q", kc.data_ptr(), vc.data_ptr(), code[cache], *kc.shape, *kc.stride()[:3], ks.data_ptr() if ks is not None else 0,
                       vs.data_ptr() if vs is not None else 0, table.data_ptr(), *table.shape, table.stride(0))
    torch.cuda.synchronize()
    st = lib.awq_paged_attention(q.data_ptr(), q.stride(0), q.stride(1), code[qt], Hq, desc, lt.data_ptr(), Dh ** -0.5, out.data_ptr(),
                                 ws.data_ptr(), size, None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, lib.awq_last_error_message()
    torch.cuda.synchronize()
    assert (ws[size:] == 0x5A).all() and (out[len(lens) * Hq * Dh:] == 7.0).all()
    want = awq.paged_attention(q, kc, vc, table, lt, k_scale=ks, v_scale=vs)
    assert torch.equal(out[: len(lens) * Hq * Dh].view_as(want), want)


def test_attention_shared_pages_and_expanded_queries():
    q, kc, vc, table, lens, _ = _attn_case([90, 90, 55], 4, 4, 128, 16, F16, F16, seed=11)
    table[1] = table[0]                                   # two sequences on one prefix
    qe = q[:1].expand(3, -1, -1)
    out = awq.paged_attention(qe, kc, vc, table, lens)
    _check_attention(qe, kc, vc, table, lens, out)
    wide = _randn(3, 12, 128, dtype=F16, seed=12)[:, 4:8]  # a part of wider rows
    out = awq.paged_attention(wide, kc, vc, table, lens)
    _check_attention(wide, kc, vc, table, lens, out)
    odd = _randn(3 * 4 * 128 + 1, dtype=F16, seed=13)[1:].view(3, 4, 128)   # not 16-byte aligned
    _check_attention(odd, kc, vc, table, lens, awq.paged_attention(odd, kc, vc, table, lens))


def test_cache_offsets_beyond_32_bits():
    """Pages behind element 2^32 of a cache; keys and values share one buffer, so that it stays
    within a few GB."""
    H, Dh, page = 8, 128, 256
    pages = (1 << 32) // (page * H * Dh) + 8
    buf = torch.empty(pages, page, H, Dh, dtype=torch.uint8, device="cuda").view(E4M3)
    assert buf.numel() > 1 << 32
    one = torch.ones(H, device="cuda") * 0.01
    T = 300
    k = _randn(T, H, Dh, dtype=F16, seed=1)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    pos, sq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    awq.kv_append(None, k, k, buf, buf, table, pos, None, seqs=sq, k_scale=one, v_scale=one)
    got = torch.cat([buf.view(torch.uint8)[pages - 1], buf.view(torch.uint8)[pages - 3, : T - page]]).view(E4M3)
    assert torch.equal(got.view(torch.uint8), (k.float() / one[0]).clamp(-448, 448).to(E4M3).view(torch.uint8))
    q = _randn(1, 16, Dh, dtype=F16, seed=2)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    small = torch.stack([buf.view(torch.uint8)[pages - 1], buf.view(torch.uint8)[pages - 3]]).view(E4M3)
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    assert torch.equal(awq.paged_attention(q, buf, buf, table, lens, k_scale=one, v_scale=one),
                       awq.paged_attention(q, small, small, near, lens, k_scale=one, v_scale=one))


def test_cache_refusals():
    q, kc, vc, table, lens, _ = _attn_case([20, 20], 4, 2, 128, 16, F16, F16, seed=14)
    k = _randn(2, 2, 128, dtype=F16)
    pos = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    att = awq.paged_attention
    for bad in (lambda: att(q, kc, vc[:, :8], table, lens), lambda: att(q, kc, vc, table[:1], lens), lambda: att(q, kc, vc, table.long(), lens),
                lambda: att(q, kc, vc, table, lens.long()), lambda: att(q, kc, vc, table, lens[:1]), lambda: att(q[:, :3], kc, vc, table, lens),
                lambda: att(q[0], kc, vc, table, lens), lambda: att(q[..., :64], kc, vc, table, lens), lambda: att(q.float(), kc, vc, table, lens),
                lambda: att(q, kc.to(E4M3), vc.to(E4M3), table, lens), lambda: att(q, kc, vc, table, lens, k_scale=torch.ones(2, device="cuda")),
                lambda: att(q, kc, vc.cpu(), table, lens), lambda: att(q, kc, vc, table, lens, status=torch.zeros(1, dtype=torch.int64, device="cuda")),
                lambda: awq.kv_append(q, k, k, kc, vc, table, pos.long()), lambda: awq.kv_append(q, k[:1], k, kc, vc, table, pos),
                lambda: awq.kv_append(q.float(), k, k, kc, vc, table, pos), lambda: awq.kv_append(q, k, k, kc, vc, table, pos, torch.ones(8, device="cuda")),
                lambda: awq.kv_append(q, k[..., :64], k, kc, vc, table, pos), lambda: att(q, kc, vc, table, lens, status=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        att(q.bfloat16(), kc, vc, table, lens)
    with pytest.raises(TypeError):
        att(q, kc.float(), vc.float(), table, lens)
    for bad in (lambda: att(q, kc, vc, table, lens, float("inf")), lambda: awq.kv_append(q, k, k, kc, vc, table, pos, torch.ones(12, dtype=torch.float64, device="cuda")),
                lambda: awq.kv_append(q, k, k, kc[:1].expand(4, -1, -1, -1), vc[:1].expand(4, -1, -1, -1), table, pos)):
        with pytest.raises(awq.AwqError):
            bad()
    assert att(q[:0], kc, vc, table[:0], lens[:0]).shape == (0, 4, 128)


# ---- together, as a decode step uses them -------------------------------------------------------

class _Block:
    """One quantized attention block: norm, QKV and output products, cache."""

    def __init__(self, K, Hq, H, batch, page, max_len, cache, seed):
        rng = np.random.default_rng(seed)
        self.K, self.Hq, self.H, self.page = K, Hq, H, page
        N = (Hq + 2 * H) * 128
        self.host = {}
        for name, (k, n) in {"qkv": (K, N), "o": (Hq * 128, K)}.items():
            codes = O.pack_codes(rng.integers(0, 16, size=(k, n)))
            steps = (rng.random((k // 128, n)) * 0.008 + 1e-3).astype(np.float16)
            zeros = rng.integers(6, 10, size=(k // 128, n)).astype(np.float16)
            self.host[name] = (codes, steps, zeros)
            c, st, zr = (torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (codes, steps, zeros))
            setattr(self, name, (awq.w4a16_repack(c), st, zr))
        self.w1, self.w2 = _randn(K, seed=seed + 1, scale=0.2) + 1, _randn(K, seed=seed + 2, scale=0.2) + 1
        mp = -(-max_len // page)
        self.table = _table(rng, batch, mp, batch * mp)
        dtype = E4M3 if cache == "e4m3" else F16
        self.caches = [torch.zeros(batch * mp, page, H, 128, dtype=F16, device="cuda").to(dtype) for _ in range(2)]
        self.scales = [torch.full((H,), s, device="cuda") for s in (0.05, 0.04)] if cache == "e4m3" else [None, None]
        self.freqs = awq.rope_frequencies(128, 5e5)[0]

    def step(self, X, residual, positions, lengths):
        M = X.shape[0]
        A = awq.rms_norm(X, self.w1, residual=residual)
        Y = awq.w4a16_matmul_packed(A, *self.qkv)
        q, k, v = (t.view(M, -1, 128) for t in Y.split([self.Hq * 128, self.H * 128, self.H * 128], dim=1))
        qr = awq.kv_append(q, k, v, *self.caches, self.table, positions, self.freqs, k_scale=self.scales[0], v_scale=self.scales[1])
        o = awq.paged_attention(qr, *self.caches, self.table, lengths, k_scale=self.scales[0], v_scale=self.scales[1])
        Z = awq.w4a16_matmul_packed(o.view(M, -1), *self.o)
        return awq.rms_norm(Z, self.w2, residual=residual), A, Y, qr, o, Z


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_decode_steps_together(cache):
    """Several tokens through a block with a growing cache: each operator's output against its
    oracle on the inputs that it got, every token's keys and values found again by the attention."""
    M, K = 3, 256
    blk = _Block(K, 4, 2, M, 16, 64, cache, seed=21)
    residual = _randn(M, K, seed=22)
    base = torch.tensor([0, 5, 30], dtype=torch.int32, device="cuda")
    if base.max() > 0:   # a past for the longer sequences
        for c in blk.caches:
            c.copy_((torch.randn(c.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(4)) * (10 if cache == "e4m3" else 1)).to(c.dtype))
    for i in range(20):
        X = _randn(M, K, seed=100 + i)
        r0 = residual.clone()
        pos = base + i
        before = [c.clone() for c in blk.caches]
        out, A, Y, qr, o, Z = blk.step(X, residual, pos, pos + 1)
        q, k, v = (t.view(M, -1, 128) for t in Y.split([512, 256, 256], dim=1))
        h = r0 + X
        _check_norm(X, blk.w1, A, r0, h)
        _close(_np(Y), Q.w4a16_matmul(A.cpu().numpy(), *blk.host["qkv"], 128), 2e-5 * (np.abs(_np(A)) @ np.abs(Q.dequant_operand(*blk.host["qkv"], 128, 1024).astype(np.float64))) + 1e-30)
        _check_append(q, k, v, before, blk.caches, blk.table, pos, blk.freqs, qr, None, False, 1.0, blk.scales)
        _check_attention(qr, *blk.caches, blk.table, pos + 1, o, None, *blk.scales)
        _check_norm(Z, blk.w2, out, h, residual)


def test_decode_step_captured_and_replayed():
    """A step captured once and replayed with new inputs and positions equals the eager steps; two
    captured graphs replayed on two streams at once do not disturb one another."""
    M, K, n = 3, 256, 12
    eager = [_Block(K, 8, 1, M, 16, 256, "f16", seed=s) for s in (31, 32)]
    graphs = [_Block(K, 8, 1, M, 16, 256, "f16", seed=s) for s in (31, 32)]
    states = []
    for blk in graphs:
        X, residual = torch.zeros(M, K, device="cuda"), torch.zeros(M, K, device="cuda")
        pos, lens = (torch.zeros(M, dtype=torch.int32, device="cuda") for _ in range(2))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.step(X, residual, pos, lens)
        torch.cuda.current_stream().wait_stream(side)
        for c in blk.caches:
            c.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = blk.step(X, residual, pos, lens)[0]
        states.append((g, X, residual, pos, lens, out, torch.cuda.Stream()))
    want = [[], []]
    start = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    for j, blk in enumerate(eager):
        residual = torch.zeros(M, K, device="cuda")
        for i in range(n):
            want[j].append(blk.step(_randn(M, K, seed=1000 * j + i), residual, start + i, start + i + 1)[0].clone())
    got = [[], []]
    for (g, X, residual, *_r) in states:
        residual.zero_()
    torch.cuda.synchronize()
    inputs = [[_randn(M, K, seed=1000 * j + i) for i in range(n)] for j in range(2)]
    torch.cuda.synchronize()
    for i in range(n):
        for j, (g, X, residual, pos, lens, out, stream) in enumerate(states):
            with torch.cuda.stream(stream):
                X.copy_(inputs[j][i])
                pos.copy_(start + i)
                lens.copy_(start + i + 1)
                g.replay()
                got[j].append(out.clone())
    torch.cuda.synchronize()
    for j in range(2):
        for i in range(n):
            assert torch.equal(got[j][i], want[j][i]), (j, i)
        assert all(torch.equal(a, b) for a, b in zip(eager[j].caches, graphs[j].caches))


def test_streams_and_threads():
    """A side stream waits for the inputs made on the current one; calls of several host threads on
    streams of their own overlap."""
    import threading
    q, kc, vc, table, lens, _ = _attn_case([5000, 300, 0, 77], 8, 2, 128, 16, F16, F16, seed=41)
    X, w = _randn(64, 4096, seed=42), _randn(4096, seed=43)
    want, norm = awq.paged_attention(q, kc, vc, table, lens), awq.rms_norm(X, w)
    side = torch.cuda.Stream()
    big = torch.zeros(1 << 26, device="cuda")
    late = torch.empty_like(q)
    for _ in range(20):
        big.add_(1.0)
    late.copy_(q)
    got = awq.paged_attention(late, kc, vc, table, lens, stream=side)
    gn = awq.rms_norm(X * 1.0, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(gn, norm)
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                if not torch.equal(awq.paged_attention(q, kc, vc, table, lens), want) or not torch.equal(awq.rms_norm(X, w), norm):
                    bad.append(1)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
