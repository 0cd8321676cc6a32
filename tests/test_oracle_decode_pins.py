"""Pins of the decode-step operators' oracle, and their library's host side (CPU only)."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import oracle.awq_decode as D
import post_quantization_column_b200 as awq


def test_rms_norm_by_hand():
    # h = (3, 4): mean square 12.5; with eps 0 the norm divides by sqrt(12.5)
    y, h = D.rms_norm([[1.0, 4.0]], [[2.0, 0.0]], [1.0, 2.0], 0.0)
    assert np.array_equal(h, [[3.0, 4.0]])
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]], rtol=1e-15)
    assert np.array_equal(D.row_scales(np.array([[0.0, 0.0], [-896.0, 1.0]])), [1.0, 2.0])


def test_rotation_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    quarter = [math.pi / 2]   # one pair, a quarter turn per position: (a, b) -> (-b, a)
    assert np.allclose(D.rotate(x, [1], quarter, False), [[[-2, 1, 3, 4, 5]]], atol=1e-15)
    two = [math.pi / 2, 0.0]
    assert np.allclose(D.rotate(x, [1], two, False), [[[-3, 2, 1, 4, 5]]], atol=1e-15)
    assert np.allclose(D.rotate(x, [1], two, True), [[[-2, 1, 3, 4, 5]]], atol=1e-15)
    assert np.allclose(D.rotate(x, [2], quarter, True, 0.5), [[[-0.5, -1, 3, 4, 5]]], atol=1e-15)


def test_rotation_keeps_relative_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f, _ = D.frequencies(16)
    dot = lambda p, r: float(np.sum(D.rotate(q, [p], f, True) * D.rotate(k, [r], f, True)))  # noqa: E731
    assert abs(dot(7, 3) - dot(1007, 1003)) < 1e-9


def test_places_of_a_paged_cache():
    table = np.array([[4, 2], [0, 9]], dtype=np.int32)
    assert D.places(table, 8, 5, [9, 3]) == [(2, 1), (0, 3)]
    assert D.places(table, 8, 5, [-1, 8]) == [(-1, -1), (-1, -1)]           # padded; page 9 of 5
    assert D.places(table, 8, 5, [16, 0, 7], [0, 2, 1]) == [(-1, -1), (-1, -1), (0, 7)]


def test_attention_by_hand():
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    k = np.zeros((2, 1, 2))
    assert np.allclose(D.attention(np.ones((3, 2)), k, v, 1.0), 0.5)
    k[1, 0, 0] = math.log(3.0)
    assert np.allclose(D.attention(np.array([[1.0, 0.0]]), k, v, 1.0), [[0.25, 0.75]])
    assert np.array_equal(D.attention(np.ones((2, 2)), k[:0], v[:0], 1.0), np.zeros((2, 2)))


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                dict(scaling="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
                                dict(scaling="ramp", factor=16.0, original_len=4096.0, low=1.0, high=32.0)])
@pytest.mark.parametrize("R,base", [(128, 1e4), (64, 5e5), (16, 1e4), (256, 1e6)])
def test_library_frequencies_match_the_oracle(R, base, kw):
    got, mag = awq.rope_frequencies(R, base, device="cpu", **kw)
    ref, ref_mag = D.frequencies(R, base, **kw)
    assert got.dtype == torch.float64 and got.shape == (R // 2,)
    # two pow, a product and a blend of correctly scaled fp64 values: a few units of 2^-53, and
    # the exponent's own rounding (|log f| <= 21) in front of exp
    assert np.all(np.abs(got.numpy() - ref) <= 64 * 2.0 ** -53 * ref)
    assert abs(mag - ref_mag) < 1e-15


def test_frequency_refusals():
    for kw in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, base=math.nan),
               dict(rotary_dim=8, scaling="linear", factor=0.5), dict(rotary_dim=2, scaling="base", factor=2.0),
               dict(rotary_dim=8, scaling="bands", factor=2.0), dict(rotary_dim=8, scaling="ramp", factor=2.0, original_len=64.0, low=4.0, high=4.0)):
        with pytest.raises(awq.AwqError):
            awq.rope_frequencies(device="cpu", **kw)
    with pytest.raises(ValueError):
        awq.rope_frequencies(8, scaling="other", device="cpu")


# ---- refusals of the C ABI: decided on the host, before any device call --------------------

NULL = None
BUF = ctypes.create_string_buffer(4096)
P = (ctypes.addressof(BUF) + 255) // 256 * 256   # an aligned address that nothing reads


def _norm(**kw):
    a = dict(X=P, xt=1, xs=128, r=NULL, rt=1, rs=128, ro=NULL, ros=128, w=P, wt=1, M=2, K=128, eps=1e-6, out=P + 2048, ot=2,
             sc=NULL, s=NULL)
    a.update(kw)
    return awq.library().awq_rms_norm(*a.values())


def test_rms_norm_refusals():
    lib = awq.library()
    for kw, st in ((dict(X=NULL), 1), (dict(w=NULL), 1), (dict(out=NULL), 1), (dict(M=-1), 2), (dict(K=0), 2), (dict(K=57345), 2),
                   (dict(M=1 << 31), 2), (dict(xt=3), 1), (dict(wt=4), 1), (dict(ot=4), 1), (dict(ot=3), 1), (dict(eps=-1.0), 1),
                   (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(r=P), 1), (dict(ro=P), 1), (dict(X=P + 2), 1),
                   (dict(out=P + 1), 1), (dict(xs=-1), 1), (dict(r=P + 512, ro=P + 512, ros=100), 1),
                   (dict(r=P, ro=P + 64), 1), (dict(r=P + 1024, ro=P), 1), (dict(r=P + 1024, rt=7, ro=P + 1024), 1),
                   (dict(out=P + 1000), 1), (dict(r=P + 1024, ro=P + 1024, out=P + 1536), 1)):
        assert _norm(**kw) == st, kw
        assert lib.awq_last_error_message()
    assert _norm(M=0, X=NULL, out=NULL) == 0


CACHE = dict(k=P, v=P, dtype=2, num_pages=4, page_size=16, heads=2, head_dim=128, ps=4096, ss=256, hs=128, ks=0, vs=0, table=P,
             seqs=3, max_pages=4, ts=4)
BAD_CACHES = ((dict(k=0), 1), (dict(v=0), 1), (dict(table=0), 1), (dict(dtype=1), 1), (dict(dtype=3), 1), (dict(head_dim=80), 2),
              (dict(heads=0), 2), (dict(page_size=0), 2), (dict(num_pages=0), 2), (dict(seqs=0), 2), (dict(max_pages=0), 2),
              (dict(max_pages=1 << 30), 2), (dict(k=P + 16), 1), (dict(ps=4097), 1), (dict(ss=8), 1), (dict(hs=-128), 1),
              (dict(table=P + 2), 1), (dict(num_pages=1 << 31), 2), (dict(ps=1 << 35), 2), (dict(ps=1 << 62), 2))


def _cache(**kw):
    return struct.pack("@16q", *{**CACHE, **kw}.values())   # awq_paged_cache


def _append(cache=None, **kw):
    a = dict(q=P, qs=512, qh=128, k=P, ks=256, kh=128, v=P, vs=256, vh=128, it=2, T=2, Hq=4, qo=P, qt=2, pos=P, seq=NULL, f=P,
             rot=128, il=0, mag=1.0, c=_cache() if cache is None else cache, st=NULL, s=NULL)
    a.update(kw)
    return awq.library().awq_kv_append(*a.values())


def test_kv_append_refusals():
    for kw, st in BAD_CACHES:
        assert _append(_cache(**kw)) == st, kw
    for kw, st in ((dict(k=NULL), 1), (dict(v=NULL), 1), (dict(pos=NULL), 1), (dict(q=NULL), 1), (dict(qo=NULL), 1), (dict(it=3), 1),
                   (dict(qt=1), 1), (dict(T=-1), 2), (dict(Hq=-1), 2), (dict(rot=24), 2), (dict(rot=144), 2), (dict(rot=-16), 2),
                   (dict(f=NULL), 1), (dict(mag=math.inf), 1), (dict(T=4), 2), (dict(qs=4), 1), (dict(k=P + 8), 1),
                   (dict(vh=-128), 1), (dict(kh=1 << 29), 2), (dict(pos=P + 2), 1), (dict(f=P + 4), 1), (dict(st=P + 1), 1), (dict(c=NULL), 1)):
        assert _append(**kw) == st, kw
    for kw in (dict(ps=0), dict(ss=64), dict(hs=0)):   # a written cache with rows on one another
        assert _append(_cache(**kw)) == 1
    assert _append(T=0) == 0


def _attention(cache=None, **kw):
    a = dict(q=P, qs=512, qh=128, qt=2, Hq=4, c=_cache() if cache is None else cache, len=P, scale=0.1, out=P, ws=P, wb=1 << 30, st=NULL,
             s=NULL)
    a.update(kw)
    return awq.library().awq_paged_attention(*a.values())


def test_paged_attention_refusals():
    for kw, st in BAD_CACHES:
        assert _attention(_cache(**kw)) == st, kw
    for kw, st in ((dict(q=NULL), 1), (dict(len=NULL), 1), (dict(out=NULL), 1), (dict(ws=NULL), 1), (dict(qt=0), 1), (dict(qt=1), 1),
                   (dict(Hq=5), 2), (dict(Hq=0), 2), (dict(scale=math.nan), 1), (dict(wb=100), 1), (dict(q=P + 8), 1), (dict(qs=4), 1),
                   (dict(ws=P + 4), 1), (dict(len=P + 2), 1), (dict(qh=-128), 1), (dict(c=NULL), 1)):
        assert _attention(**kw) == st, kw
    lib = awq.library()
    assert lib.awq_paged_attention_workspace(4, 2, 128, 2) > 0
    for bad in ((5, 2, 128, 2), (4, 0, 128, 2), (4, 2, 80, 2), (4, 2, 128, 1)):
        assert lib.awq_paged_attention_workspace(*bad) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.float16)
    c = torch.zeros(4, 16, 2, 128, dtype=torch.float16)
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        awq.rms_norm(x, x[0])
    with pytest.raises(ValueError):
        awq.kv_append(None, x.view(1, 2, 128), x.view(1, 2, 128), c, c, i, i[0, :1])
    with pytest.raises(ValueError):
        awq.paged_attention(x.view(1, 2, 128), c, c, i, i[0, :1])


def test_runs_of_units_cover_every_segment_once():
    """The attention's dealing of units to runs (the formulas of its kernels, restated): every run
    has a unit, a segment's runs are consecutive, and a run leaves at most one partial that began
    before it (slot 1) and one that goes on after it (slot 0)."""
    rng = np.random.default_rng(3)
    for _ in range(300):
        B, HH, ctas = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 297))
        nblk = rng.integers(0, int(rng.choice([2, 5, 200])), size=B)
        units = int(nblk.sum()) * HH
        if units == 0:
            continue
        C = min(ctas, units)
        start = [c * units // C for c in range(C + 1)]
        assert all(a < b for a, b in zip(start, start[1:]))
        owner = lambda u: ((u + 1) * C - 1) // units  # noqa: E731
        slots, s0 = set(), 0
        for b in range(B):
            for _ in range(HH):
                s1 = s0 + int(nblk[b])
                if s1 == s0:
                    continue
                c0, c1 = owner(s0), owner(s1 - 1)
                assert start[c0] <= s0 < start[c0 + 1] and start[c1] < s1 <= start[c1 + 1]
                for p, c in enumerate(range(c0, c1 + 1)):
                    if c0 != c1:
                        slot = 2 * c + (1 if s0 < start[c] else 0)     # what the run writes
                        assert slot == 2 * c + (1 if p > 0 else 0)     # what the join reads
                        assert slot not in slots
                        slots.add(slot)
                s0 = s1
