"""INT8 matmuls whose tiles have their K split between CTAs that wait for one another's sums: on competing streams, each
with its own workspace, and captured into graphs.  Every shape here is asked for its workspace, which only a split
shape needs, so a change of the kernels' choice fails these tests instead of emptying them."""
import pytest
import torch

import group_wise_weight_b200 as wq
from group_wise_weight_b200 import build as wqbuild

SHAPES = [(100, 1000, 28672), (30, 999, 28672), (64, 512, 28672), (300, 1000, 28672), (1, 1000, 28672), (128, 2048, 28672),
          (8, 2304, 28672), (16, 1000, 20000)]
COUNTERS = 65536


@pytest.fixture(scope="module", autouse=True)
def _lib():
    wqbuild.build()
    wq.lib()


@pytest.fixture(autouse=True)
def _no_device_timeouts(request):
    yield
    if "gpu" in request.keywords:
        assert wq.wq_device_status() == wq.WQ_OK, "a kernel recorded a bounded-wait timeout"


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes_are_split(M, N, K):
    assert wq.wq_gemm_w8a8_int8_workspace_bytes(M, N, K) > COUNTERS


def job(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, w = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((M, K), (N, K)))
    sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda").to(torch.bfloat16)
    return a, sx, w, sw


def reference(a, sx, w, sw):
    """The exact sum, rounded to binary32, times RN(sx sw), rounded to bf16."""
    acc = a.double() @ w.double().t()
    return (acc.float() * (sx[:, None] * sw.float()[None, :])).to(torch.bfloat16)


def space():
    need = max(wq.wq_gemm_w8a8_int8_workspace_bytes(*s) for s in SHAPES)
    assert need > COUNTERS
    return torch.zeros(need, dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
def test_shapes_in_turn_on_one_workspace():
    ws = space()
    for i, s in enumerate(SHAPES + SHAPES[::-1]):
        d = job(*s, i)
        assert torch.equal(wq.wq_gemm_w8a8_int8(*d, workspace=ws), reference(*d)), s
        assert int(ws[:COUNTERS].max()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("priorities", [(0, 0), (0, -1, 0)])
def test_split_calls_on_every_stream_at_once(priorities):
    """Each step gives every stream a split call, so several of them compete for the SMs that their CTAs wait on."""
    jobs = [job(*s, i) for i, s in enumerate(SHAPES)]
    want = [reference(*d) for d in jobs]
    fill = torch.randn(1 << 22, device="cuda")
    streams = [torch.cuda.Stream(priority=p) for p in priorities]
    spaces = [space() for _ in streams]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for i in range(48):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                if (i + s) % 5 == 0:
                    fill.mul(1.5)
                got[s].append(wq.wq_gemm_w8a8_int8(*jobs[(i + 3 * s) % len(jobs)], workspace=spaces[s]))
    torch.cuda.synchronize()
    for s in range(len(streams)):
        assert all(torch.equal(y, want[(i + 3 * s) % len(jobs)]) for i, y in enumerate(got[s]))
        assert int(spaces[s][:COUNTERS].max()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_captured_and_replayed(M, N, K):
    """The activations' quantiser and a split matmul as one graph: replays with other inputs, and again with no wait between
    them, find the counters as the replay before left them."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    _, _, w, sw = job(M, N, K, 1)
    ws = space()
    q, s = wq.wq_quantize_int8_tokens(x)
    y = wq.wq_gemm_w8a8_int8(q, s, w, sw, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_quantize_int8_tokens(x, q, s)
        wq.wq_gemm_w8a8_int8(q, s, w, sw, y=y, workspace=ws)
    for _ in range(3):
        x.copy_(torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16))
        y.zero_()
        for _ in range(4):
            graph.replay()
        torch.cuda.synchronize()
        qr, sr = wq.wq_quantize_int8_tokens(x)
        assert torch.equal(q, qr) and torch.equal(y, reference(qr, sr, w, sw))
        assert int(ws[:COUNTERS].max()) == 0


@pytest.mark.gpu
def test_two_graphs_and_eager_calls_share_a_workspace_on_one_stream():
    ws = space()
    jobs = [job(*s, 7 + i) for i, s in enumerate(SHAPES[:3])]
    want = [reference(*d) for d in jobs]
    out = [wq.wq_gemm_w8a8_int8(*d, workspace=ws) for d in jobs]
    torch.cuda.synchronize()
    graphs = []
    for d, y in zip(jobs[:2], out):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            wq.wq_gemm_w8a8_int8(*d, y=y, workspace=ws)
    for y in out:
        y.zero_()
    for _ in range(6):
        graphs[0].replay()
        graphs[1].replay()
        wq.wq_gemm_w8a8_int8(*jobs[2], y=out[2], workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_workspace_allocated_by_the_call_inside_a_capture():
    """Without a workspace the call makes a zeroed one, inside a capture too."""
    d = job(64, 512, 28672, 3)
    want = reference(*d)
    y = torch.empty_like(want)
    wq.wq_gemm_w8a8_int8(*d, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_gemm_w8a8_int8(*d, y=y)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
