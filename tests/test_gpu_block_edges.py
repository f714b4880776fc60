"""The linear layers and the norm where calls are unusual: tensors past 2^31 elements, a first call
inside a graph capture, a captured backward beside a living eager graph, several streams and host
threads at once, a second backward, many short sequences."""
import subprocess
import sys
import threading
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _block_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_attention_gb300.build import build
    sa.load_library(build())


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def test_offsets_past_32_bits():
    """Outputs of 2.4e9 elements: rows at the start, around 2^31 elements and at the end."""
    g = _gen("big")
    M, K, N = 300_001, 64, 8192
    x, w, dy_w = _randn(g, M, K), _randn(g, K, N, std=K ** -0.5), _randn(g, N, K)
    bias = _randn(g, N, dtype=torch.float32)
    pick = torch.tensor([0, 1, 262_143, 262_144, 262_145, M - 2, M - 1], device="cuda")
    y, z = sa.linear_forward(x, w, bias, None, "gelu", keep_z=True)
    ry, rz, ty, tz = ref.linear(x[pick], w, bias, None, "gelu")
    ref.check("y", y[pick], ry, ty)
    ref.check("z", z[pick], rz, tz)
    # y as a gradient: dx and dw of a layer whose output is that large
    dx, dw, db = sa.linear_backward(x, w, y, z, "gelu")
    want = ref.linear_bwd(x[pick], w, y[pick], z[pick], "gelu")["dx"]
    ref.check("dx", dx[pick], *want)
    cols = slice(0, 64)
    want = ref.linear_bwd(x, w[:, cols].contiguous(), y[:, cols].contiguous(), z[:, cols].contiguous(), "gelu")
    ref.check("dw", dw[:, cols], *want["dw"])
    ref.check("db", db[cols], *want["db"])
    del z, dx, dw
    # the norm and the 8-bit product over the same rows
    g1 = torch.ones(N, device="cuda")
    n, _, rstd = sa.rms_norm_forward(y, g1)
    rn, _, rr = ref.rms_norm(y[pick], g1)
    ref.check("norm", n[pick], rn, 1.02 * ref.U8 * rn.abs() + 1e-6)
    del n
    q, s = sa.quantize_q8(y)
    wq, ws = sa.quantize_q8(dy_w.t().contiguous())      # [K, N] rows: a product of N down to K
    out = sa.linear_q8(q, s, wq, ws)
    ro, _, to, _ = ref.linear(q[pick].double() * s[pick].double()[:, None],
                              (wq.double() * ws.double()[:, None]).T)
    ref.check("q8", out[pick], ro, to)
    assert sa.attn_get_device_status() == 0


def test_first_call_inside_a_capture():
    """A fresh process whose first calls are captured (forward, backward, norm, 8 bits) and replayed."""
    code = """
import torch, self_attention_gb300 as sa
x, w = torch.randn(300, 256, device='cuda').bfloat16(), torch.randn(256, 520, device='cuda').bfloat16()
one, g = torch.ones(256, device='cuda'), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
def run():
    y, z = sa.linear_forward(x, w, None, None, 'gelu', keep_z=True)
    n, h, r = sa.rms_norm_forward(x, one, x)
    q, s, _ = sa.rms_norm_q8(x, one, x)
    wq, ws = sa.quantize_q8(w[:, :512].t().contiguous())
    return (y, z, *sa.linear_backward(x, w, y, z, 'gelu'), n, r, *sa.rms_norm_backward(n, h, one, r),
            q.float(), s, sa.linear_q8(q, s, wq, ws), sa.linear_forward(x[:3], w))
with torch.cuda.graph(g):
    out = run()
g.replay()
for a, b in zip(out, run()):
    assert torch.equal(a, b)
assert sa.attn_get_device_status() == 0
print('same')
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_captured_backward_beside_a_living_eager_graph():
    """The captured pass runs on leaves of its own (the same memory, detached): PyTorch refuses to
    capture a backward whose leaves a living eager graph holds, with its own operators too."""
    g = _gen("alive")
    x, w = _randn(g, 130, 128).requires_grad_(), _randn(g, 128, 264, std=0.1).requires_grad_()
    gw = (1 + _randn(g, 128, std=0.1, dtype=torch.float32)).requires_grad_()
    dy = _randn(g, 130, 264)

    leaves = [t.detach().requires_grad_() for t in (x, w, gw)]

    def step():
        y = sa.linear(sa.rms_norm(leaves[0], leaves[2]), leaves[1], None, None, "silu")
        return torch.autograd.grad(y, leaves, dy)

    eager = sa.linear(sa.rms_norm(x, gw), w, None, None, "silu")     # its graph stays alive
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    gr.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for a, b in zip(want, torch.autograd.grad(eager, (x, w, gw), dy)):
        assert torch.equal(a, b)


def test_streams_and_host_threads_at_once():
    """Different calls from four host threads, each on its own stream, all at once, many times: the
    results each gets alone."""
    g = _gen("threads")
    jobs = []
    for M, K, N in ((1, 512, 1032), (70, 256, 520), (513, 320, 264), (1500, 128, 776)):
        x, w, dy = _randn(g, M, K), _randn(g, K, N, std=0.1), _randn(g, M, N)
        one, res = torch.ones(K, device="cuda"), _randn(g, M, K)

        def run(stream=None, x=x, w=w, dy=dy, one=one, res=res):
            n, h, r = sa.rms_norm_forward(x, one, res, stream=stream)
            y, z = sa.linear_forward(x, w, None, dy, "gelu", keep_z=True, stream=stream)
            return (n, h, r, y, z, *sa.linear_backward(x, w, dy, z, "gelu", stream=stream),
                    *sa.rms_norm_backward(n, h, one, r, stream=stream))

        jobs.append((run, run()))
    torch.cuda.synchronize()
    wrong = []

    def work(run, want):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(40):
                got = run()
            st.synchronize()
        if not all(torch.equal(a, b) for a, b in zip(want, got)):
            wrong.append(want[0].shape)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and sa.attn_get_device_status() == 0


def test_streams_by_handle():
    """A stream may be given as a torch stream or as its handle, the default stream's 0 included."""
    g = _gen("handles")
    x, w = _randn(g, 33, 64), _randn(g, 64, 72)
    one, want = torch.ones(64, device="cuda"), sa.linear_forward(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (0, side.cuda_stream, side, torch.cuda.current_stream()):
        y = sa.linear_forward(x, w, stream=st)
        n, _, _ = sa.rms_norm_forward(x, one, stream=st)
        q, s = sa.quantize_q8(x, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(n, sa.rms_norm_forward(x, one)[0]) and torch.equal(s, sa.quantize_q8(x)[1])


def test_an_allocation_that_fails():
    """An output of 1.1 TB: PyTorch's own error, and the next call works."""
    x, w = torch.zeros(1 << 20, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 524_288, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        sa.linear_forward(x, w)
    assert not bool(sa.linear_forward(x[:3].contiguous(), w).any())


def test_no_second_derivative():
    x, w = (torch.ones(8, 8, dtype=torch.bfloat16, device="cuda", requires_grad=True) for _ in range(2))
    y = sa.linear(x, w, None, None, "gelu")
    (gx,) = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.float().sum().backward()


@pytest.mark.parametrize("B,H,N,d", [(700, 2, 3, 64), (1000, 2, 1, 128), (64, 4, 33, 64), (9, 1, 40, 128)])
def test_many_short_sequences(B, H, N, d):
    g = _gen("short", B, H, N, d)
    o, w, dy = _randn(g, B, H, N, d), _randn(g, H * d, 264, std=0.1), _randn(g, B, N, 264)
    rows = ref.heads_to_rows(o)
    y, _, ty, _ = ref.linear(rows, w, None, dy.view(B * N, 264))
    ref.check("y", sa.out_proj_forward(o, w, None, dy).view(B * N, 264), y, ty)
    do, dw, db = sa.out_proj_backward(o, w, dy)
    want = ref.linear_bwd(rows, w, dy.view(B * N, 264))
    ref.check("do", do, *(ref.rows_to_heads(t, B, H, N, d) for t in want["dx"]))
    ref.check("dw", dw, *want["dw"])
    ref.check("db", db, *want["db"])


def test_a_row_is_the_same_in_any_batch_of_its_plan():
    """Rows do not see one another: a row's outputs do not depend on the other rows' values."""
    g = _gen("rows")
    for M in (12, 200, 1000):
        x, w, dy = _randn(g, M, 256), _randn(g, 256, 136, std=0.1), _randn(g, M, 136)
        y, (dx, _, _) = sa.linear_forward(x, w), sa.linear_backward(x, w, dy)
        x2, dy2 = x.clone(), dy.clone()
        x2[1:], dy2[1:] = x2[1:] * 3, dy2[1:] * 3
        assert torch.equal(sa.linear_forward(x2, w)[0], y[0])
        assert torch.equal(sa.linear_backward(x2, w, dy2)[0][0], dx[0])


def test_a_flag_without_a_truth_value():
    """Its own error comes through, from before anything is launched."""
    class NoTruth:
        def __bool__(self):
            raise KeyError("no truth value")

    x, w = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(64, 32, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(KeyError):
        sa.linear_forward(x, w, keep_z=NoTruth())
    with pytest.raises(KeyError):
        sa.linear_backward(x, w, torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16), need_dw=NoTruth())


@pytest.mark.parametrize("N,d", [(1024, 64), (2048, 128)])
def test_beside_attention_on_another_stream(N, d):
    """Attention's kernels and these share the SMs' tensor memory when they run at once; each gives what it
    gives alone."""
    g = _gen("beside", N, d)
    q, k, v = (_randn(g, 2, 8, N, d) for _ in range(3))
    few, many = _randn(g, 24, 1024), _randn(g, 4096, 1024)
    w, gain = _randn(g, 1024, 1024, std=0.05), torch.rand(1024, device="cuda") + 0.5

    def attend():
        return list(sa.forward(q, k, v, d ** -0.5))

    def rows():
        out = []
        for x in (few, many):
            y, h, rstd = sa.rms_norm_forward(x, gain, x)
            z = sa.linear_forward(y, w, None, h, "gelu")
            out += [z, *sa.linear_backward(y, w, z), *sa.rms_norm_backward(z, h, gain, rstd)]
        return out

    want = attend(), rows()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [], []
    for _ in range(12):
        for st, fn, to in zip(streams, (attend, rows), got):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                to.append(fn())
    torch.cuda.synchronize()
    for results, alone in zip(got, want):
        for r in results:
            for a, b in zip(r, alone):
                assert torch.equal(a, b)
