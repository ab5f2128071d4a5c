"""Per-head norms and rotary positions on the GPU against binary64.

Bound, per value y = a cos t - b sin t (or b cos t + a sin t) of the normed pair (a, b): the output's rounding to
bf16, at most 2^-8 |y|, and the binary32 arithmetic before it.  With u = 2^-24: the mean of D squares is off by at
most (D / 2 + 1) u of itself under the square root (D additions halved by it; the shuffle's tree does fewer), the
square root, division, two products and the weight add 5 u, the rotation's products and sum 2 u, the sine and
cosine 2 units in the last place and the fraction of a turn pi 2^-25: together below (D / 2 + 24) u (|a| + |b|).
"""
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


def reference(x, weight, eps, positions, inv_freq, interleaved):
    """(y, |a| + |b|) in binary64."""
    x = x.cpu().double()
    D, rot = x.shape[-1], 2 * inv_freq.numel()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.cpu().double()
    y, size = x.clone(), x.abs()
    t = positions.cpu().double()[:, None] * inv_freq.cpu().double()
    c, s = t.cos()[:, None], t.sin()[:, None]
    i = torch.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = a.abs() + b.abs()
    assert D >= rot
    return y, size


def check(out, x, weight, eps, positions, inv_freq, interleaved):
    y, size = reference(x, weight, eps, positions, inv_freq, interleaved)
    bound = 2 ** -8 * y.abs() * (1 + 2 ** -10) + (x.shape[-1] / 2 + 24) * 2 ** -24 * size
    err = (out.double().cpu() - y).abs()
    assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())


def inputs(M, Hq, H, D, seed, far=8000, rot=None, theta=500000.0):
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn(M, Hq + 2 * H, D, generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, far, (M,), generator=g, dtype=torch.int32).cuda()
    rot = rot or D
    f = (theta ** (-2 * torch.arange(rot // 2).double() / rot)).float().cuda()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    return fused, pos, f, w


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("M,Hq,H,D,rot", [(1, 64, 8, 128, 128), (5, 1, 1, 128, 64), (33, 3, 1, 64, 64), (7, 40, 8, 128, 16),
                                          (2, 71, 1, 64, 48), (300, 4, 4, 128, 112), (1300, 2, 1, 64, 16),
                                          (19, 128, 16, 128, 128)])
def test_shapes(M, Hq, H, D, rot, norm, interleaved):
    fused, pos, f, w = inputs(M, Hq, H, D, M + Hq + rot, rot=rot)
    q, k, _ = fused.split([Hq, H, H], dim=1)
    qw, kw = w if norm else (None, None)
    qo, ko = wq.wq_qk_norm_rope(q, k, pos, f, qw, kw, 1e-6, interleaved)
    check(qo, q, qw, 1e-6, pos, f, interleaved)
    check(ko, k, kw, 1e-6, pos, f, interleaved)


def test_far_and_negative_positions():
    fused, pos, f, w = inputs(64, 4, 2, 128, 1)
    pos[:8] = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 1000003, 123456789, -77777], dtype=torch.int32).cuda()
    q, k, _ = fused.split([4, 2, 2], dim=1)
    qo, ko = wq.wq_qk_norm_rope(q, k, pos, f, *w)
    check(qo, q, w[0], 1e-6, pos, f, False)
    check(ko, k, w[1], 1e-6, pos, f, False)


def test_rows_of_zeros_and_extremes():
    """A zero vector stays zero for any eps > 0; large and tiny magnitudes are normed without overflow of the sum of
    squares (up to 2^60) or loss of it (down to 2^-60, where eps decides)."""
    fused, pos, f, w = inputs(6, 2, 1, 128, 2)
    fused[0] = 0
    fused[1] *= 2.0 ** 58
    fused[2] *= 2.0 ** -60
    fused[3] = 0
    fused[3, :, 17] = -3.0
    q, k, _ = fused.split([2, 1, 1], dim=1)
    for eps in (1e-6, 1e-5, 0.25):
        qo, ko = wq.wq_qk_norm_rope(q, k, pos, f, w[0], w[1], eps)
        check(qo, q, w[0], eps, pos, f, False)
        check(ko, k, w[1], eps, pos, f, False)
        assert (qo[0] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_on_the_fused_projection(interleaved):
    fused, pos, f, w = inputs(517, 8, 2, 128, 3, rot=96)
    q, k, v = fused.split([8, 2, 2], dim=1)
    want = wq.wq_qk_norm_rope(q, k, pos, f, *w, interleaved=interleaved)
    kept = v.clone()
    got = wq.wq_qk_norm_rope(q, k, pos, f, *w, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


def test_refusals():
    fused, pos, f, w = inputs(4, 4, 2, 128, 4)
    q, k, _ = fused.split([4, 2, 2], dim=1)
    for args, kw, err in (((q.float(), k, pos, f), {}, TypeError), ((q, k[:3], pos, f), {}, ValueError),
                          ((q, k, pos.long(), f), {}, TypeError), ((q, k, pos[:2], f), {}, ValueError),
                          ((q, k, pos, f.double()), {}, TypeError), ((q, k, pos, f[:5]), {}, wq.WQError),
                          ((q, k, pos, f, w[0]), {}, wq.WQError), ((q, k, pos, f, w[0][:64], w[1]), {}, ValueError),
                          ((q.transpose(0, 1), k, pos, f), {}, ValueError), ((q, k, pos, f), dict(q_out=k), ValueError),
                          ((q[:0], k[:0], pos[:0], f), {}, wq.WQError), ((q, k, pos, f), dict(k_out=q[:, :2]), wq.WQError)):
        with pytest.raises(err):
            wq.wq_qk_norm_rope(*args, **kw)


def test_captured_and_replayed_on_another_stream():
    fused, pos, f, w = inputs(9, 8, 2, 128, 5)
    q, k, _ = fused.split([8, 2, 2], dim=1)
    qo, ko = wq.wq_qk_norm_rope(q, k, pos, f, *w)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        wq.wq_qk_norm_rope(q, k, pos, f, *w, q_out=qo, k_out=ko)
    pos += 1000
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(qo, q, w[0], 1e-6, pos, f, False)
    check(ko, k, w[1], 1e-6, pos, f, False)
