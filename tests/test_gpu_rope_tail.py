"""Values rot .. D - 1 of a head pass the rotary positions unturned: without norms they keep their bits, and with norms each
is its own value scaled, whatever the others hold."""
import math

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


def inputs(M, Hq, H, D, rot, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, Hq + H, D, generator=g).to(torch.bfloat16)
    x[torch.rand(x.shape, generator=g) < 0.2] = 0.0
    x[torch.rand(x.shape, generator=g) < 0.2] = -0.0
    pos = torch.randint(0, 5000, (M,), generator=g, dtype=torch.int32)
    f = (10000.0 ** (-2 * torch.arange(rot // 2).double() / rot)).float()
    return x, pos.cuda(), f.cuda()


def bits(t):
    return t.cpu().view(torch.int16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,Hq,H,D,rot", [(3, 5, 1, 128, 64), (40, 8, 2, 128, 16), (7, 4, 4, 64, 48), (2500, 2, 1, 64, 16),
                                          (1, 71, 8, 128, 112)])
def test_unturned_values_keep_their_bits(M, Hq, H, D, rot, interleaved):
    x, pos, f = inputs(M, Hq, H, D, rot, M + rot)
    g = torch.Generator().manual_seed(1)
    tail = x[..., rot:]  # in a third of the heads one infinity or NaN
    where = torch.randint(0, D - rot, (M, Hq + H, 1), generator=g)
    special = torch.tensor([math.inf, -math.inf, math.nan])[torch.randint(0, 3, (M, Hq + H, 1), generator=g)].to(torch.bfloat16)
    chosen = torch.rand(M, Hq + H, 1, generator=g) < 0.33
    tail.scatter_(2, where, torch.where(chosen, special, tail.gather(2, where)))
    q, k = x.cuda().split([Hq, H], dim=1)
    for o, src in zip(wq.wq_qk_norm_rope(q, k, pos, f, interleaved=interleaved), (x[:, :Hq], x[:, Hq:])):
        got, want = o.cpu()[..., rot:], src[..., rot:]
        number = ~want.isnan()
        assert torch.equal(bits(got.contiguous())[number], bits(want.contiguous())[number])
        assert got[~number].isnan().all()
        assert torch.isfinite(o.cpu()[..., :rot]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_unturned_zeros_keep_their_sign_under_norms(interleaved):
    x, pos, f = inputs(50, 6, 2, 128, 32, 5)
    w = (1 + 0.2 * torch.rand(128, generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    q, k = x.cuda().split([6, 2], dim=1)
    for o, src in zip(wq.wq_qk_norm_rope(q, k, pos, f, w.cuda(), w.cuda(), interleaved=interleaved), (x[:, :6], x[:, 6:])):
        zero = src[..., 32:] == 0
        assert zero.any() and (o.cpu()[..., 32:][zero] == 0).all()
        assert torch.equal(torch.signbit(o.cpu()[..., 32:]), torch.signbit(src[..., 32:]))
