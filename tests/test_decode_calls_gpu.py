"""Calls of the decode-step operators that their other tests do not make (B200 only): the C ABI
with addresses that it has to refuse, and the binding under autograd, threads and streams."""
import ctypes
import struct

import pytest
import torch

import post_quantization_column_b200 as awq
from tests.test_decode_ops_gpu import _check_norm

pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _randn(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


class _Step:
    """One append and one attention of two sequences, four query heads on two, through the C ABI."""

    def __init__(self, page=16, pages=4, **cache):
        self.k, self.v = (_randn(2, 2, 128, dtype=F16, seed=i) for i in (1, 2))
        self.q = _randn(2, 4, 128, dtype=F16, seed=3)
        self.caches = [_randn(pages, page, 2, 128, dtype=F16, seed=i) for i in (4, 5)]
        self.table = torch.tensor([[1], [3]], dtype=torch.int32, device="cuda")
        self.pos = torch.tensor([4, 9], dtype=torch.int32, device="cuda")
        self.lens = self.pos + 1
        self.out = torch.full((2, 4, 128), 7.0, dtype=F16, device="cuda")
        self.freqs = awq.rope_frequencies(128)[0]
        size = awq.library().awq_paged_attention_workspace(4, 2, 128, 2)
        self.ws, self.ws_bytes = torch.empty(size, dtype=torch.uint8, device="cuda"), size
        d = dict(k=self.caches[0].data_ptr(), v=self.caches[1].data_ptr(), dtype=2, num_pages=pages, page_size=page, heads=2, head_dim=128,
                 ps=page * 256, ss=256, hs=128, ks=0, vs=0, table=self.table.data_ptr(), seqs=2, max_pages=1, ts=1)
        self.desc = struct.pack("@16q", *{**d, **cache}.values())
        torch.cuda.synchronize()

    def append(self, status=None, **kw):
        a = dict(q=self.q.data_ptr(), qs=512, qh=128, k=self.k.data_ptr(), ks=256, kh=128, v=self.v.data_ptr(), vs=256, vh=128, it=2,
                 T=2, Hq=4, qo=self.out.data_ptr(), qt=2, pos=self.pos.data_ptr(), seq=None, f=self.freqs.data_ptr(), rot=128, il=0, mag=1.0,
                 c=self.desc, st=status, s=ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        a.update(kw)
        return awq.library().awq_kv_append(*a.values())

    def attend(self, status=None, **kw):
        a = dict(q=self.q.data_ptr(), qs=512, qh=128, qt=2, Hq=4, c=self.desc, len=self.lens.data_ptr(), scale=0.1, out=self.out.data_ptr(),
                 ws=self.ws.data_ptr(), wb=self.ws_bytes, st=status, s=ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        a.update(kw)
        return awq.library().awq_paged_attention(*a.values())


def test_status_of_memory_that_a_kernel_cannot_reach_is_refused():
    """A plain host int as the status word: the store that reports a bad page would go astray, so the
    call is refused before any launch (every page here is good, and nothing is written)."""
    step = _Step()
    before = [c.clone() for c in step.caches]
    word = (ctypes.c_int32 * 4)()
    for call in (step.append, step.attend):
        assert call(ctypes.c_void_p(ctypes.addressof(word))) == 1
        assert b"status" in awq.library().awq_last_error_message()
    torch.cuda.synchronize()
    assert (step.out == 7.0).all() and all(torch.equal(a, b) for a, b in zip(before, step.caches)) and not any(word)
    for status in (torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32).pin_memory()):
        assert step.append(status.data_ptr()) == 0 and step.attend(status.data_ptr()) == 0
        torch.cuda.synchronize()
        assert int(status) == 0


def test_rotated_queries_and_attention_in_place():
    """q_out = q and out = q, as the header allows, against outputs of their own."""
    for lens in ([5, 10], [16, 1]):
        a, b = _Step(), _Step()
        for s in (a, b):
            s.lens.copy_(torch.tensor(lens))
        assert a.append() == 0 and b.append(qo=b.q.data_ptr()) == 0
        assert torch.equal(a.out, b.q) and all(torch.equal(x, y) for x, y in zip(a.caches, b.caches))
        assert a.attend(out=a.q.data_ptr(), q=a.out.data_ptr()) == 0 and b.attend(out=b.q.data_ptr()) == 0
        assert torch.equal(a.q, b.q)


# ---- forms of the RMS norm that take rows too long for registers, value by value or in pairs ----------

@pytest.mark.parametrize("K", [16385, 20001, 57343, 16386, 30002, 57342])
@pytest.mark.parametrize("M", [3, 170])
def test_long_rows_of_odd_and_even_length(M, K):
    X, w, R = _randn(M, K, dtype=BF16, seed=K), _randn(K, dtype=BF16, seed=2), _randn(M, K, seed=3)
    new = torch.empty_like(R)
    _check_norm(X, w, awq.rms_norm(X, w, residual=R, residual_out=new), R, new)
    _check_norm(X, w, awq.rms_norm(X, w, out_dtype=E4M3))


@pytest.mark.parametrize("offset", [1, 2])
def test_long_rows_that_start_between_vectors(offset):
    M, K = 5, 28672
    base, rbase, w = _randn(M, K + 2, dtype=F16, seed=4), _randn(M, K + 2, dtype=BF16, seed=5), _randn(K, seed=6)
    X, R = base[:, offset:offset + K], rbase[:, offset:offset + K]
    before = rbase.clone()
    for out in (F16, E4M3):
        R.copy_(before[:, offset:offset + K])
        _check_norm(X, w, awq.rms_norm(X, w, residual=R, out_dtype=out), before[:, offset:offset + K], R)
    rbase[:, offset:offset + K] = before[:, offset:offset + K]
    assert torch.equal(rbase, before)   # nothing beside the rows was written


@pytest.mark.parametrize("K", [512, 515, 4096, 20001])
def test_norm_at_the_ends_of_its_range(K):
    """What the header says of sums beyond fp32 and of eps = 0; within the range, the formula."""
    w = _randn(K, seed=1)
    X = _randn(5, K, seed=2)
    X[1] *= 1e16                      # K 1e32 < 3.4e38
    X[2] *= 1e20                      # its sum is beyond fp32
    X[3] = 0.0
    X[4] *= 1e-15
    for M in (5, 300):
        rows = X.repeat(M // 5, 1)
        fine = [m for m in range(M) if m % 5 != 2]
        out = awq.rms_norm(rows, w, out_dtype=F32)
        _check_norm(rows[fine], w, out[fine])
        assert (out[2] == 0).all()
        codes, scales = awq.rms_norm(rows, w, out_dtype=E4M3)
        _check_norm(rows[fine], w, (codes[fine], scales[fine]))
        assert (codes[2].float() == 0).all() and scales[2] == 1.0
        fine = [m for m in range(M) if m % 5 not in (2, 3)]
        out = awq.rms_norm(rows, w, 0.0, out_dtype=F32)
        _check_norm(rows[fine], w, out[fine], eps=0.0)
        assert torch.isnan(out[3]).all()
        codes, scales = awq.rms_norm(rows, w, 0.0, out_dtype=E4M3)
        assert torch.isnan(scales[3]) and torch.isnan(codes[3].float()).all()
    tiny = torch.full((2, K), 1e-25, device="cuda")
    assert torch.isinf(awq.rms_norm(tiny, torch.ones(K, device="cuda"), 0.0, out_dtype=F32)).all()


# ---- the binding -----------------------------------------------------------------------------------

def _decode_inputs():
    k, v, q = _randn(2, 2, 128, dtype=F16, seed=1), _randn(2, 2, 128, dtype=F16, seed=2), _randn(2, 4, 128, dtype=F16, seed=3)
    kc, vc = (_randn(4, 16, 2, 128, dtype=F16, seed=i) for i in (4, 5))
    table = torch.tensor([[1], [3]], dtype=torch.int32, device="cuda")
    return q, k, v, kc, vc, table, torch.tensor([4, 9], dtype=torch.int32, device="cuda")


def test_status_of_a_call_on_another_stream():
    """check_status waits for the device, whichever stream the reporting call is on."""
    q, k, v, kc, vc, table, pos = _decode_inputs()
    table.fill_(99)
    status, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    awq.paged_attention(q, kc, vc, table, pos + 1)   # what a first call loads is loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)               # 0.2 s
    awq.paged_attention(q, kc, vc, table, pos + 1, status=status, stream=side)
    with pytest.raises(awq.AwqError):
        awq.check_status(status)


def test_tensors_that_autograd_saved_are_written_openly():
    """An in-place write of a tensor that a backward pass still needs makes that pass an error."""
    q, k, v, kc, vc, table, pos = _decode_inputs()
    X, w, r = _randn(4, 64, seed=6), _randn(64, seed=7), _randn(4, 64, seed=8)
    for write, saved in ((lambda: awq.rms_norm(X, w, residual=r), [r]),
                         (lambda: awq.rms_norm(X, w, residual=X * 2, residual_out=r), [r]),
                         (lambda: awq.kv_append(q, k, v, kc, vc, table, pos), [kc, vc]),
                         (lambda: awq.kv_append(q, k, v, kc[:], vc[:], table, pos), [kc, vc])):
        for t in saved:
            leaf = torch.ones_like(t, requires_grad=True)
            loss = (t * leaf).sum()
            write()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
    versions = [t._version for t in (X, w, q, k, v, table, pos)]
    awq.kv_append(q, k, v, kc, vc, table, pos)
    awq.rms_norm(X, w)
    awq.paged_attention(q, kc, vc, table, pos + 1)
    assert versions == [t._version for t in (X, w, q, k, v, table, pos)]   # inputs that are only read
    with torch.inference_mode():                       # tensors without a version
        ri, kci, vci = r.clone(), kc.clone(), vc.clone()
        awq.rms_norm(X, w, residual=ri)
        awq.kv_append(q, k, v, kci, vci, table, pos)
    assert torch.equal(kci, kc) and torch.equal(vci, vc)


def test_forward_mode_tangents_are_refused():
    import torch.autograd.forward_ad as fwd
    q, k, v, kc, vc, table, pos = _decode_inputs()
    X, w, r = _randn(4, 64, seed=6), _randn(64, seed=7), _randn(4, 64, seed=8)
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))  # noqa: E731
        for bad in (lambda: awq.rms_norm(dual(X), w), lambda: awq.rms_norm(X, dual(w)), lambda: awq.rms_norm(X, w, residual=dual(r)),
                    lambda: awq.kv_append(dual(q), k, v, kc, vc, table, pos), lambda: awq.kv_append(q, k, dual(v), kc, vc, table, pos),
                    lambda: awq.paged_attention(dual(q), kc, vc, table, pos + 1), lambda: awq.paged_attention(q, dual(kc), vc, table, pos + 1)):
            with torch.no_grad(), pytest.raises(ValueError):   # no_grad leaves forward mode on
                bad()
        awq.rms_norm(X, w)


def test_other_threads_run_while_a_call_waits_for_the_queue():
    """A call that finds the launch queue full waits without the interpreter lock."""
    import threading
    import time
    X, w = _randn(1, 64, seed=1), _randn(64, seed=2)
    awq.rms_norm(X, w)
    torch.cuda.synchronize()
    gaps, stop = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    other = threading.Thread(target=tick)
    other.start()
    time.sleep(0.05)
    torch.cuda._sleep(2_000_000_000)   # about 1 s
    start = time.perf_counter()
    for _ in range(4000):
        awq.rms_norm(X, w)
    took = time.perf_counter() - start
    stop.set()
    other.join()
    torch.cuda.synchronize()
    if took > 0.5:   # the queue was full, and the calls waited
        assert max(gaps) < took / 2, (max(gaps), took)


def test_launch_counts_are_the_calling_thread_s():
    import threading
    X, W = _randn(128, 256, seed=1), _randn(256, 256, seed=2)
    awq.search(X, W, n_grid=4)
    made = awq.last_launch_count()
    seen = []

    def work():
        x, w = _randn(4, 64, seed=1), _randn(64, seed=2)
        for _ in range(20):
            awq.rms_norm(x, w)
        seen.append(awq.last_launch_count())

    other = threading.Thread(target=work)
    other.start()
    other.join()
    assert made > 1 and seen == [1] and awq.last_launch_count() == made


def test_a_step_without_tokens():
    q, k, v, kc, vc, table, pos = _decode_inputs()
    before = [kc.clone(), vc.clone()]
    assert awq.kv_append(q[:0], k[:0], v[:0], kc, vc, table[:0], pos[:0]).shape == (0, 4, 128)
    assert awq.kv_append(None, k[:0], v[:0], kc, vc, table[:0], pos[:0]) is None
    assert awq.paged_attention(q[:0], kc, vc, table[:0], pos[:0]).shape == (0, 4, 128)
    assert awq.rms_norm(q[:0].view(0, 128), torch.ones(128, device="cuda")).shape == (0, 128)
    assert torch.equal(before[0], kc) and torch.equal(before[1], vc)


_CAPTURED_FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import post_quantization_column_b200 as awq
g = torch.Generator().manual_seed(0)
X, w = torch.randn(3, 20002, generator=g).cuda(), torch.randn(20002, generator=g).cuda()
rows = torch.randn(2, 8, 128, generator=g).half().cuda()
caches = [torch.randn(4, 16, 2, 128, generator=g).half().cuda() for _ in range(2)]
kept = [c.clone() for c in caches]
table, pos = torch.tensor([[1], [3]], dtype=torch.int32).cuda(), torch.tensor([4, 9], dtype=torch.int32).cuda()
lens, freqs = pos + 1, awq.rope_frequencies(128)[0]

def step(kc, vc):
    q = awq.kv_append(rows[:, :4], rows[:, 4:6], rows[:, 6:], kc, vc, table, pos, freqs)
    return awq.rms_norm(X, w), q, awq.paged_attention(q, kc, vc, table, lens)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step(*caches)
graph.replay()
torch.cuda.synchronize()
want = step(*kept)
assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(caches, kept))
print("captured first: ok")
"""


def test_a_first_call_may_be_a_captured_one():
    """In a new process, with nothing of the library used before the capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", _CAPTURED_FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured first: ok" in done.stdout, done.stdout + done.stderr


# ---- the attention's weights ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Dh,Hq,H", [(128, 8, 2), (128, 32, 2), (64, 12, 4), (256, 4, 4)])
def test_attention_weights_keep_the_bits_of_fp32(dtype, Dh, Hq, H):
    """Against 64 bits, with nothing allowed for a rounding of the weights to 16 bits. Keys and queries
    are -1, 0 or 1 and the scale 1/8, so that every score is exact. With u = 2^-24 and h half a step
    of the dtype at 1, a weight (as a factor) is off by 4 u |s| for the scale in base 2, twice for its
    difference from the maximum, by 2^-21 for the exponential and by h^2 for the rest's rounding, together
    E; in fp16 weights below 2^-14, of a sum of at least 2^7, are off by 2^-25 each. The fp32 sums
    over n tokens add (n / 32 + 64) 2 u, and the output is rounded once."""
    lens = [1, 17, 40, 63, 64, 65, 300, 1000, 0, 5000]
    g = torch.Generator().manual_seed(Dh + Hq)
    pages = sum(-(-n // 16) for n in lens)
    signs = lambda *shape: torch.randint(-1, 2, shape, generator=g).to(dtype).cuda()  # noqa: E731
    q, kc = signs(len(lens), Hq, Dh), signs(pages, 16, H, Dh)
    vc = torch.randn(pages, 16, H, Dh, generator=g).to(dtype).cuda()
    order, table, at = torch.randperm(pages, generator=g).to(torch.int32), torch.zeros(len(lens), 5000 // 16 + 1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        need = -(-n // 16)
        table[b, :need] = order[at:at + need]
        at += need
    out = awq.paged_attention(q, kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125)
    u, h = 2.0 ** -24, torch.finfo(dtype).eps / 2
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        ids = table[b, : -(-n // 16)].long().cuda()
        k, v = (c[ids].reshape(-1, H, Dh)[:n].double().repeat_interleave(Hq // H, dim=1).transpose(0, 1) for c in (kc, vc))
        s = 0.125 * (k @ q[b].double()[:, :, None])[..., 0]                     # (Hq, n)
        p = torch.softmax(s, dim=1)
        want = (p[:, None] @ v)[:, 0]
        E = 8 * u * s.abs().amax(dim=1) + 4 * u * (s.amax(dim=1, keepdim=True) - s).amax(dim=1) + 2.0 ** -21 + h * h
        off = (p[:, None] @ (v - want[:, None]).abs())[:, 0] * (E / (1 - E))[:, None]
        off += (n / 32 + 64) * 2 * u * (p[:, None] @ v.abs())[:, 0]
        if dtype == F16:
            off += n * 2.0 ** -32 * (v - want[:, None]).abs().amax(dim=1)
        off += torch.maximum(h * (want.abs() + off), torch.tensor(torch.finfo(dtype).smallest_normal * h, dtype=torch.float64, device="cuda"))
        bad = ~((out[b].double() - want).abs() <= off)
        assert not bad.any(), (n, int(bad.sum()), float(((out[b].double() - want).abs() / off).max()))
