"""Host side of the decode-step operators (CPU only): arguments that are refused before any device
call. An address is never followed here; without a device an accepted call ends in a CUDA error."""
import ctypes
import struct

import pytest

import post_quantization_column_b200 as awq

BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) // 256 * 256   # an aligned address that nothing reads
REFUSED = 1                                      # AWQ_ERR_INVALID_ARG


def _cache(**kw):
    d = dict(k=P, v=P, dtype=2, num_pages=4, page_size=16, heads=2, head_dim=128, ps=4096, ss=256, hs=128, ks=0, vs=0, table=P, seqs=3,
             max_pages=4, ts=4)
    d.update(kw)
    return struct.pack("@16q", *d.values())


def _append(cache=None, **kw):
    a = dict(q=P + 4096, qs=512, qh=128, k=P, ks=256, kh=128, v=P, vs=256, vh=128, it=2, T=2, Hq=4, qo=P + 16384, qt=2, pos=P, seq=None,
             f=P, rot=128, il=0, mag=1.0, c=_cache() if cache is None else cache, st=None, s=None)
    a.update(kw)
    return awq.library().awq_kv_append(*a.values())


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="addresses of nothing: only without a device")
def test_append_refuses_caches_whose_rows_overlap():
    """Two tokens' rows on one another would be a race of their writes."""
    for kw in (dict(ps=256, ss=256), dict(ps=256, ss=128, hs=2048), dict(ss=128), dict(ps=4096 - 16), dict(hs=256, ss=128, page_size=3),
               dict(ps=128, ss=512, hs=256)):
        assert _append(_cache(**kw)) == REFUSED, kw
        assert b"overlap" in awq.library().awq_last_error_message()
    for kw in (dict(), dict(ps=4096, hs=2048, ss=128), dict(hs=8192, ps=2048, ss=128), dict(ss=1024, ps=256, hs=128), dict(ps=0, num_pages=1),
               dict(hs=0, heads=1), dict(ps=8192, ss=512, hs=256)):
        assert _append(_cache(**kw)) > 2, kw   # taken: what fails is the device
