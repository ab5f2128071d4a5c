"""The prompt-side calls on streams that are not the current one, with and without given outputs, interleaved on two
streams, and their results unchanged by what runs beside them."""
import pytest
import torch

import group_wise_weight_b200 as wq
from group_wise_weight_b200 import build as wqbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    wqbuild.build()
    wq.lib()
    torch.cuda.init()


@pytest.fixture(autouse=True)
def _no_device_timeouts():
    yield
    assert wq.wq_device_status() == wq.WQ_OK, "a kernel recorded a bounded-wait timeout"


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = torch.randn(333, 12, 128, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = fused.split([8, 2, 2], dim=1)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    return {"x": fused.view(333, -1), "q": q, "k": k, "v": v, "pos": torch.arange(333, device="cuda", dtype=torch.int32),
            "freq": (10000.0 ** (-torch.arange(64, device="cuda").double() / 64)).float(),
            "slots": torch.randperm(400, generator=g, device="cuda")[:333],
            "starts": torch.tensor([0, 100, 101, 333], device="cuda", dtype=torch.int32),
            "w": codes(700, 8192), "ws": torch.rand(700, generator=g, device="cuda").to(torch.bfloat16),
            "a": codes(5, 8192), "as": torch.rand(5, generator=g, device="cuda"), "one": torch.full((1,), 0.05, device="cuda")}


def run(d, stream=None):
    """Every call once; with `stream` as its argument."""
    kc, vc = (torch.zeros(4, 100, 2, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    k4, v4 = (torch.zeros(4, 100, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    par = [torch.zeros(4, 100, 2, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    if stream is not None:  # the zeros above are the current stream's
        torch.cuda.current_stream().synchronize()
    out = [*wq.wq_quantize_int8_tokens(d["x"], stream=stream),
           wq.wq_gemm_w8a8_int8(d["a"], d["as"], d["w"], d["ws"], stream=stream),
           *wq.wq_qk_norm_rope(d["q"], d["k"], d["pos"], d["freq"], stream=stream),
           wq.wq_prompt_attention(d["q"], d["k"], d["v"], d["starts"], stream=stream)]
    wq.wq_kv_store_fp8(d["k"], d["v"], d["slots"], kc, d["one"], vc, d["one"], stream=stream)
    wq.wq_kv_store_int4(d["k"], d["v"], d["slots"], k4, par[0], par[1], v4, par[2], par[3], stream=stream)
    return out + [kc, vc, k4, v4, *par]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_given_stream():
    d = make(1)
    want = run(d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream, torch.cuda.default_stream(), 0):
        got = run(d, stream=handle)
        torch.cuda.synchronize()
        assert same(got, want)


def test_a_given_stream_orders_the_calls():
    """On the given stream behind work that is still running there: the calls must read what that work writes."""
    d = make(2)
    want = run(d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fresh = {n: torch.zeros_like(t) if n in ("x", "a", "w") else t for n, t in d.items()}
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            big = big @ big * 1e-3
        for n in ("x", "a", "w"):
            fresh[n].copy_(d[n])
    q, sc = wq.wq_quantize_int8_tokens(fresh["x"], stream=s)
    y = wq.wq_gemm_w8a8_int8(fresh["a"], d["as"], fresh["w"], d["ws"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(sc, want[1]) and torch.equal(y, want[2])


def test_two_streams_interleaved():
    data = [make(3), make(4)]
    want = [run(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got[i % 2].append(run(data[i % 2]))
    torch.cuda.synchronize()
    assert all(same(g, want[i]) for i in range(2) for g in got[i])


def test_matmul_right_behind_the_weight_quantiser():
    """The weights quantised by the call just before on the stream: the matmul, which is launched while its predecessor
    ends, must see all of them."""
    g = torch.Generator(device="cuda").manual_seed(6)
    w = [torch.randn(4096, 4096, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    a, s = wq.wq_quantize_int8_tokens(torch.randn(3, 4096, generator=g, device="cuda"))
    space = torch.zeros(max(16, wq.wq_gemm_w8a8_int8_workspace_bytes(3, 4096, 4096)), dtype=torch.uint8, device="cuda")
    want = []
    for t in w:
        q, sc = wq.wq_quantize_int8(t)
        torch.cuda.synchronize()
        want.append(wq.wq_gemm_w8a8_int8(a, s, q, sc))
    q, sc = torch.empty_like(q), torch.empty_like(sc)
    for i in range(20):
        wq.wq_quantize_int8(w[i % 2], qweight=q, scales=sc)
        y = wq.wq_gemm_w8a8_int8(a, s, q, sc, workspace=space)
        assert torch.equal(y, want[i % 2])


def test_matmuls_whose_parts_wait_on_streams_of_two_priorities():
    """Shapes that fill every SM with CTAs that add up a tile together, on streams that compete for the SMs, with calls of
    other sizes between: nobody may wait for a CTA that cannot start."""
    g = torch.Generator(device="cuda").manual_seed(7)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    jobs = []
    for M, N, K in ((100, 8192, 4096), (64, 9472, 2048), (32, 1280, 8192), (1, 1000, 28672)):
        a, w = codes(M, K), codes(N, K)
        sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda").to(torch.bfloat16)
        jobs.append((a, sx, w, sw, wq.wq_gemm_w8a8_int8(a, sx, w, sw)))
    fill = torch.randn(1 << 22, device="cuda")
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, 0)]
    space = [torch.zeros(max(wq.wq_gemm_w8a8_int8_workspace_bytes(a.shape[0], w.shape[0], a.shape[1]) for a, _, w, _, _ in jobs),
                         dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for i in range(60):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                if (i + s) % 5 == 0:
                    fill.mul(1.5)
                a, sx, w, sw, _ = jobs[(i + s) % len(jobs)]
                got[s].append(wq.wq_gemm_w8a8_int8(a, sx, w, sw, workspace=space[s]))
    torch.cuda.synchronize()
    for s in range(len(streams)):
        for i, y in enumerate(got[s]):
            assert torch.equal(y, jobs[(i + s) % len(jobs)][4])


def test_weights_made_two_calls_before_a_kernel_that_reads_them_early():
    """wq_gemm_w4a16 may read its weights before the call just before it has ended, so another call goes between the
    quantiser and it: the INT8 matmul, which starts early itself, must be such a call."""
    g = torch.Generator(device="cuda").manual_seed(8)
    N, K = 28672, 8192
    w = [torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    x = torch.randn(1, K, generator=g, device="cuda").to(torch.bfloat16)
    a, sx = wq.wq_quantize_int8_tokens(x[:, :512].contiguous())
    small = torch.randint(-127, 128, (64, 512), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    want = []
    for t in w:
        q, s, z = wq.wq_quantize_int4(t, 128)
        torch.cuda.synchronize()
        want.append(wq.wq_gemm_w4a16(x, q, s, z, 128))
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    space = torch.zeros(wq.wq_gemm_workspace_bytes(1, N, K, 128, 4), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for i in range(10):
        wq.wq_quantize_int4(w[i % 2], 128, qweight=q, scales=s, zeros=z)
        wq.wq_gemm_w8a8_int8(a, sx, small, sw)
        assert torch.equal(wq.wq_gemm_w4a16(x, q, s, z, 128, workspace=space), want[i % 2])
