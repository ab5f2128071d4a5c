"""Per-token INT8 quantisation and the INT8 W8A8 matmul on the GPU: both are defined bit by bit, so both are
compared for equality with 64-bit arithmetic on the CPU."""
import numpy as np
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


def tokens_ref(x: torch.Tensor):
    """s = RN(max|x| / 127) (1 if 0), q = clip(rint(RN(x / s))): binary64 quotients rounded to binary32."""
    v = x.double().numpy()
    s = (np.abs(v).max(axis=1) / 127).astype(np.float32)
    s[s == 0] = 1
    q = np.clip(np.rint((v / s.astype(np.float64)[:, None]).astype(np.float32)), -127, 127)
    return q.astype(np.int8), s


def check_tokens(x_cpu: torch.Tensor, x_gpu: torch.Tensor):
    q, s = wq.wq_quantize_int8_tokens(x_gpu)
    qr, sr = tokens_ref(x_cpu)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 256), (9, 512), (8, 544), (17, 1024), (5, 2048), (4, 2080), (3, 4096),
                                 (2, 4128), (2, 8192), (1, 8224), (2, 16384), (3, 28672), (2, 32768), (2, 32800),
                                 (1, 70016)])
def test_tokens_bit_exact(M, K, dtype):
    g = torch.Generator().manual_seed(M * 100003 + K)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g) * 3)
    x = (x * (1 + 19 * (torch.rand(K, generator=g) < 0.01).float())).to(dtype)
    check_tokens(x, x.cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens_borders(dtype):
    """Rows of zeros (both signs), one value, powers of two (quotients of 63.5 and 31.75), the type's largest and
    smallest values, and scales outside the reciprocal's range."""
    K = 96
    rows = [torch.zeros(K), -torch.zeros(K), torch.full((K,), 3.0), torch.full((K,), -1e-30)]
    ties = torch.ones(K)
    ties[::2], ties[1::4] = 0.5, -0.25
    rows.append(ties)
    top = torch.linspace(-1, 1, K) * 3.0e38
    rows += [top, torch.linspace(-1, 1, K) * 2.0 ** -126, torch.linspace(-3, 3, K) * 1e-36, torch.linspace(-2, 5, K) * 2e33]
    tiny = torch.zeros(K)
    tiny[5], tiny[7], tiny[9] = 9.2e-41, -9.2e-41, 4.6e-41  # multiples of the smallest binary32 subnormal
    rows.append(tiny)
    x = torch.stack(rows).to(dtype)
    check_tokens(x, x.cuda())


def test_tokens_strides_and_given_outputs():
    g = torch.Generator().manual_seed(5)
    for dtype, pad in ((torch.bfloat16, 8), (torch.float32, 40)):
        wide = torch.randn(37, 640 + pad, generator=g).to(dtype)
        check_tokens(wide[:, :640], wide.cuda()[:, :640])
        x = wide.cuda()[::2, :640]  # a row stride of two rows
        check_tokens(wide[::2, :640], x)
        q, s = torch.full((19, 640), 99, dtype=torch.int8).cuda(), torch.zeros(19).cuda()
        r = wq.wq_quantize_int8_tokens(x, q, s)
        assert r[0] is q and r[1] is s and torch.equal(q, wq.wq_quantize_int8_tokens(x)[0])


def test_tokens_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16).cuda()
    for bad, err in ((x.half(), TypeError), (x.t(), ValueError), (x[:, :40], wq.WQError), (x[:0], wq.WQError),
                     (x[:, 4:36], wq.WQError)):
        with pytest.raises(err):
            wq.wq_quantize_int8_tokens(bad)
    with pytest.raises(ValueError):
        wq.wq_quantize_int8_tokens(x, scales=torch.zeros(5).cuda())
    with pytest.raises(TypeError):
        wq.wq_quantize_int8_tokens(x, q=torch.zeros(4, 256, dtype=torch.uint8).cuda())


def operands(M, N, K, seed, low=-127):
    g = torch.Generator().manual_seed(seed)
    xq = torch.randint(low, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(low, 128, (N, K), generator=g, dtype=torch.int8)
    xs = torch.exp(torch.randn(M, generator=g))
    ws = (torch.exp(torch.randn(N, generator=g)) * 0.01).to(torch.bfloat16)
    return xq, xs, w, ws


def matmul_ref(xq, xs, w, ws):
    """The exact sum (below 2^53 in binary64), rounded to binary32, times RN(xs ws), rounded to bf16."""
    acc = (xq.cuda().double() @ w.cuda().double().t()).cpu()
    return (acc.float() * (xs[:, None] * ws.float()[None, :])).to(torch.bfloat16)


def check_matmul(M, N, K, seed, workspace=None, low=-127):
    xq, xs, w, ws = operands(M, N, K, seed, low)
    y = wq.wq_gemm_w8a8_int8(xq.cuda(), xs.cuda(), w.cuda(), ws.cuda(), workspace=workspace)
    ref = matmul_ref(xq, xs, w, ws)
    assert torch.equal(y.cpu().view(torch.int16), ref.view(torch.int16)), (M, N, K)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 511])
def test_matmul_rows(M):
    check_matmul(M, 1024, 2048, M)


@pytest.mark.parametrize("N", [1, 2, 15, 127, 129, 255, 257, 1000, 4099])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_matmul_columns(M, N):
    check_matmul(M, N, 544, 7 * N + M)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 352, 1024, 1056, 4064, 28672])
@pytest.mark.parametrize("M", [1, 16, 90, 260])
def test_matmul_depths(M, K):
    check_matmul(M, 384, K, K + M)


@pytest.mark.parametrize("M,N,K", [(1, 10240, 8192), (100, 8192, 28672), (1000, 10240, 8192), (2049, 57344, 1024),
                                   (8190, 2000, 4096), (3, 57344, 8192), (640, 130, 28672)])
def test_matmul_model_shapes(M, N, K):
    check_matmul(M, N, K, M + N + K)


# Weight rows shared out: one to eight pieces of K per stage, one to several tiles of tokens and rounds, odd everything
@pytest.mark.parametrize("M,N,K", [(1, 1000, 8192), (2, 130, 4000), (128, 4099, 1056), (65, 10247, 512), (127, 19001, 288),
                                   (128, 57343, 160), (129, 2048, 8192), (300, 1001, 4096), (384, 5003, 1024), (700, 513, 544),
                                   (1000, 70, 2080), (2049, 130, 1024), (64, 40000, 352), (150, 130, 131040)])
def test_matmul_shared_rows(M, N, K):
    check_matmul(M, N, K, M + N + K)


# Tiles of 256 tokens by 160 to 256 weight rows on pairs of SMs, one to several rounds of them
@pytest.mark.parametrize("M,N,K", [(700, 8191, 1056), (300, 57345, 160), (1821, 17124, 128), (1000, 10242, 96), (100, 4100, 512), (256, 10243, 512), (1500, 4099, 2080), (513, 14337, 288),
                                   (2000, 20011, 96), (150, 40001, 1024), (129, 57344, 544), (4097, 1001, 2048)])
def test_matmul_pair_tiles(M, N, K):
    check_matmul(M, N, K, M + N + K)


# Tiles of 128 weight rows by 16, 32, 64 and 128 tokens, whole and with their K split between CTAs
@pytest.mark.parametrize("M,N,K", [(5, 17, 96), (33, 300, 160), (3, 28671, 1056), (20, 28672, 1024), (40, 14336, 1024),
                                   (16, 57344, 512), (2, 130, 28672), (1, 1, 16384), (16, 1000, 20000), (30, 999, 28672),
                                   (67, 14420, 96), (64, 257, 28640), (100, 1000, 28672), (300, 1000, 28672),
                                   (129, 1001, 28672)])
def test_matmul_streamed_tiles(M, N, K):
    check_matmul(M, N, K, M + N + K)


@pytest.mark.parametrize("M", [1, 5, 300])
def test_matmul_largest_sums(M):
    """Every code -128 at the greatest depth: 2^14 * 131040 is the largest sum, just below 2^31."""
    K, N = 131040, 130
    xq, w = torch.full((M, K), -128, dtype=torch.int8), torch.full((N, K), -128, dtype=torch.int8)
    w[::2] = 127
    xs, ws = torch.full((M,), 2.0 ** -20), torch.full((N,), 2.0 ** -5, dtype=torch.bfloat16)
    y = wq.wq_gemm_w8a8_int8(xq.cuda(), xs.cuda(), w.cuda(), ws.cuda())
    assert torch.equal(y.cpu(), matmul_ref(xq, xs, w, ws))


def test_matmul_codes_with_minus_128():
    check_matmul(33, 300, 4096, 3, low=-128)


def test_matmul_one_workspace_for_every_shape():
    shapes = [(1, 8192, 8192), (300, 1000, 4096), (64, 512, 28672), (1, 300, 28672), (1500, 900, 512), (17, 8192, 1024),
              (130, 130, 130 * 32), (1, 8192, 8192)]
    need = max(wq.wq_gemm_w8a8_int8_workspace_bytes(*s) for s in shapes)
    ws = torch.zeros(need, dtype=torch.uint8).cuda()
    for i, s in enumerate(shapes):
        check_matmul(*s, seed=i, workspace=ws)


def test_matmul_given_output_and_scale_shape():
    xq, xs, w, ws = (t.cuda() for t in operands(5, 70, 64, 1))
    y = torch.zeros(5, 70, dtype=torch.bfloat16).cuda()
    assert wq.wq_gemm_w8a8_int8(xq, xs, w, ws.view(70, 1), y=y) is y
    assert torch.equal(y, wq.wq_gemm_w8a8_int8(xq, xs, w, ws))


def test_matmul_refusals():
    xq, xs, w, ws = (t.cuda() for t in operands(4, 64, 64, 1))
    for args, err in (((xq.view(torch.uint8), xs, w, ws), TypeError), ((xq, xs[:3], w, ws), ValueError),
                      ((xq, xs, w[:, :32], ws), ValueError), ((xq, xs, w, ws.float()), TypeError),
                      ((xq, xs, w, ws[:5]), ValueError), ((xq[:, :40].contiguous(), xs, w[:, :40].contiguous(), ws), wq.WQError),
                      ((xq, xs.cpu(), w, ws), TypeError)):
        with pytest.raises(err):
            wq.wq_gemm_w8a8_int8(*args)
    args = [t.cuda() for t in operands(1, 1000, 28672, 1)]
    assert wq.wq_gemm_w8a8_int8_workspace_bytes(1, 1000, 28672) > 0
    with pytest.raises(wq.WQError):
        wq.wq_gemm_w8a8_int8(*args, workspace=torch.zeros(16, dtype=torch.uint8).cuda())


def test_quantised_linear_against_the_full_precision_product():
    """Weights and activations through the quantisers and the matmul: each operand is off by at most half a step,
    |x - s q| <= s / 2 (1 + 2^-10) and the same for w (a bf16 scale below max|w| / 127 clips by up to 2^-8 of the
    maximum more), so |y - x w^T| <= sum_k dx |w| + |x| dw + dx dw, then bf16."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(70, 1024, generator=g).to(torch.bfloat16)
    w = (torch.randn(520, 1024, generator=g) * 0.02).to(torch.bfloat16)
    xq, xs = wq.wq_quantize_int8_tokens(x.cuda())
    wqt, ws = wq.wq_quantize_int8(w.cuda())
    y = wq.wq_gemm_w8a8_int8(xq, xs, wqt, ws).double().cpu()
    xd, wd = x.double(), w.double()
    dx = (xs.double().cpu() / 2 * (1 + 2 ** -10))[:, None]
    dw = (ws.double().cpu().flatten() / 2 * (1 + 2 ** -10))[:, None] + wd.abs().amax(1, keepdim=True) * 2 ** -8
    bound = dx * wd.abs().sum(1)[None] + xd.abs().sum(1)[:, None] * dw.t() + 1024 * dx * dw.t()
    ref = xd @ wd.t()
    assert ((y - ref).abs() <= bound + 2 ** -8 * (ref.abs() + bound)).all()


def test_two_streams_with_their_own_workspaces():
    xq, xs, w, ws = (t.cuda() for t in operands(40, 2000, 8192, 2))
    want = wq.wq_gemm_w8a8_int8(xq, xs, w, ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = wq.wq_gemm_w8a8_int8_workspace_bytes(40, 2000, 8192)
    spaces = [torch.zeros(need, dtype=torch.uint8).cuda() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(wq.wq_gemm_w8a8_int8(xq, xs, w, ws, workspace=spaces[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_captured_and_replayed():
    x = torch.randn(6, 1024, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    _, _, w, ws = (t.cuda() for t in operands(6, 500, 1024, 3))
    space = torch.zeros(wq.wq_gemm_w8a8_int8_workspace_bytes(6, 500, 1024), dtype=torch.uint8).cuda()
    q, s = wq.wq_quantize_int8_tokens(x)
    y = wq.wq_gemm_w8a8_int8(q, s, w, ws, workspace=space)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_quantize_int8_tokens(x, q, s)
        wq.wq_gemm_w8a8_int8(q, s, w, ws, y=y, workspace=space)
    for seed in (2, 3):
        x.copy_(torch.randn(6, 1024, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        qr, sr = wq.wq_quantize_int8_tokens(x)
        assert torch.equal(q, qr) and torch.equal(y, wq.wq_gemm_w8a8_int8(qr, sr, w, ws))
