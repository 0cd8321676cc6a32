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
    d = dict(k=P + (1 << 22), v=P + (1 << 23), dtype=2, num_pages=4, page_size=16, heads=2, head_dim=128, ps=4096, ss=256, hs=128, ks=0, vs=0, table=P, seqs=3,
             max_pages=4, ts=4)
    d.update(kw)
    return struct.pack("@16q", *d.values())


def _append(cache=None, **kw):
    a = dict(q=P + 4096, qs=512, qh=128, k=P, ks=256, kh=128, v=P, vs=256, vh=128, it=2, T=2, Hq=4, qo=P + 16384, qt=2, pos=P, seq=None,
             f=P, rot=128, il=0, mag=1.0, c=_cache() if cache is None else cache, st=None, s=None)
    a.update(kw)
    return awq.library().awq_kv_append(*a.values())


def _attention(cache=None, **kw):
    a = dict(q=P + 16384, qs=512, qh=128, qt=2, Hq=4, c=_cache(seqs=2, num_pages=1) if cache is None else cache, len=P, scale=0.1,
             out=P + 24576, ws=P + (1 << 20), wb=1 << 30, st=None, s=None)
    a.update(kw)
    return awq.library().awq_paged_attention(*a.values())


def _norm(**kw):
    a = dict(X=P, xt=1, xs=128, r=None, rt=1, rs=128, ro=None, ros=128, w=P + 8192, wt=1, M=4, K=128, eps=1e-6, out=P + 16384, ot=3,
             sc=P + 20480, s=None)
    a.update(kw)
    return awq.library().awq_rms_norm(*a.values())


pytestmark = pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="addresses of nothing: only without a device")


def test_append_refuses_caches_whose_rows_overlap():
    """Two tokens' rows on one another would be a race of their writes."""
    for kw in (dict(ps=256, ss=256), dict(ps=256, ss=128, hs=2048), dict(ss=128), dict(ps=4096 - 16), dict(hs=256, ss=128, page_size=3),
               dict(ps=128, ss=512, hs=256)):
        assert _append(_cache(**kw)) == REFUSED, kw
        assert b"overlap" in awq.library().awq_last_error_message()
    for kw in (dict(), dict(ps=4096, hs=2048, ss=128), dict(hs=8192, ps=2048, ss=128), dict(ss=1024, ps=256, hs=128), dict(ps=0, num_pages=1),
               dict(hs=0, heads=1), dict(ps=8192, ss=512, hs=256)):
        assert _append(_cache(**kw)) > 2, kw   # taken: what fails is the device


def test_outputs_that_overlap_other_arguments_are_refused():
    one = dict(cache=_cache(num_pages=1, k=P + (1 << 17), v=P + (1 << 18)))
    kb, vb = P + (1 << 17), P + (1 << 18)
    for call, bad, good in (
            (lambda **kw: _append(**one, **kw),
             (dict(qo=P + 4096 + 1024), dict(qo=P), dict(v=P + 8192, qo=P + 8192 + 256), dict(qo=kb + 512), dict(qo=vb - 16), dict(qo=P + 4096, qs=1024),
              dict(qo=P + 4096, qt=0), dict(q=P + 4096, qo=P + 4096, qh=256, qs=1024), dict(qo=P + 4096 + 2032)),
             (dict(), dict(qo=P + 4096), dict(qo=P + 4096 + 2048), dict(Hq=0, q=None, qo=None), dict(T=1, qo=P + 4096, qs=4096))),
            (lambda **kw: _attention(cache=_cache(num_pages=1, seqs=2, k=kb, v=vb), **kw),
             (dict(out=P + 16384 + 512), dict(out=kb), dict(out=vb + 8176), dict(ws=P + 16384 + 16), dict(ws=P + 24576 - 32), dict(ws=kb - 64),
              dict(out=P + 16384, qs=1024), dict(out=P + 16384 - 2032)),
             (dict(), dict(out=P + 16384), dict(out=P + 16384 + 2048), dict(ws=P + (1 << 21), out=P + (1 << 29)))),   # in a larger buffer
            (_norm,
             (dict(sc=P), dict(sc=P + 2044), dict(sc=P + 8192 + 508), dict(sc=P + 16384 + 508), dict(r=P + 32768, ro=P + 32768, sc=P + 32768 + 64)),
             (dict(), dict(sc=P + 2048), dict(sc=P + 16384 + 512), dict(ot=2, sc=P)))):
        for kw in bad:
            assert call(**kw) == REFUSED, kw
            assert b"overlap" in awq.library().awq_last_error_message(), kw
        for kw in good:
            assert call(**kw) > 2, (kw, awq.library().awq_last_error_message())


# ---- the build ---------------------------------------------------------------------------------------

def _binding_builds(monkeypatch):
    """What build_binding() would compile: its commands, which are not run."""
    from post_quantization_column_b200 import build
    ran = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd))
    build.build_binding()
    return ran


def test_binding_is_built_again_when_what_it_was_built_for_changes(monkeypatch, tmp_path):
    import os
    import shutil

    import torch
    from post_quantization_column_b200 import build
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_decode.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "_decode.key"))
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("decode_binding.cpp", "decode_entry.h"):
        shutil.copy(os.path.join(build.CSRC, name), csrc / name)
    monkeypatch.setattr(build, "CSRC", str(csrc))
    assert len(_binding_builds(monkeypatch)) == 1
    (tmp_path / "_decode.so").write_bytes(b"")
    assert _binding_builds(monkeypatch) == []
    late = os.path.getmtime(tmp_path / "_decode.so") + 10
    os.utime(csrc / "decode_entry.h", (late, late))
    assert len(_binding_builds(monkeypatch)) == 1
    os.utime(tmp_path / "_decode.so", (late + 10, late + 10))
    assert _binding_builds(monkeypatch) == []
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert len(_binding_builds(monkeypatch)) == 1
    assert _binding_builds(monkeypatch) == []


def test_entry_points_are_declared_in_one_place():
    import os
    import re
    csrc = os.path.join(os.path.dirname(awq.__file__), "csrc")
    for name in ("decode_binding.cpp", "awq_decode.cu"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert '#include "decode_entry.h"' in text
        assert not re.search(r"^int awq_\w+_on\([^;{}]*\);$", text, re.M), name   # no declaration of its own


@pytest.mark.parametrize("lacking", ["torch", "headers", "compiler"])
def test_the_library_is_built_where_the_binding_cannot_be(monkeypatch, capsys, lacking):
    import sys
    import sysconfig

    from post_quantization_column_b200 import build
    build.build()   # nothing left to compile
    if lacking == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif lacking == "headers":
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    else:
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build.build() == build.LIB
    assert "_decode.so is not built" in capsys.readouterr().err
