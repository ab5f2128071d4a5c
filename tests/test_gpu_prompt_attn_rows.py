"""Outputs of the prompt attention depend on their own token's query and on the keys and values it sees, to the bit: not on
what other rows of a tile hold, be it the next sequence, later tokens or what an earlier kernel left in shared memory.

Equality needs no tolerance: the arithmetic of a row is the same in both calls, and what differs lies in other rows or
behind p = 0 (a finite value times 0 adds nothing)."""
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


def qkv(M, Hq, H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = torch.randn(M, Hq + 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    return fused.split([Hq, H, H], dim=1)


def attend(q, k, v, starts):
    return wq.wq_prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32).cuda())


def bits(t):
    return t.view(torch.int16)


# Items of one tile (few heads) and of two (64 heads), both head sizes, groups that divide a tile's 128 rows and not
SHAPES = [(8, 1, 128), (8, 2, 64), (5, 1, 128), (7, 1, 64), (64, 8, 128), (60, 12, 64), (3, 3, 128), (128, 128, 64)]


@pytest.mark.parametrize("Hq,H,D", SHAPES)
@pytest.mark.parametrize("n", [999, 515, 130])
def test_the_next_sequence_changes_no_bit(Hq, H, D, n):
    M = n + 300
    q, k, v = qkv(M, Hq, H, D, n + Hq)
    found = []
    for scale in (0.0, 1.0, 100.0):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[n:] = (t[n:] * scale).abs()
        found.append(attend(q2, k2, v2, [0, n, M])[:n].clone())
    assert torch.equal(bits(found[0]), bits(found[1])) and torch.equal(bits(found[0]), bits(found[2]))


@pytest.mark.parametrize("Hq,H,D", SHAPES)
def test_later_tokens_change_no_bit(Hq, H, D):
    n, seen = 1000, 701
    q, k, v = qkv(n, Hq, H, D, Hq)
    want = attend(q, k, v, [0, n])[:seen].clone()
    for scale in (0.0, 100.0):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[seen:] *= scale
        assert torch.equal(bits(attend(q2, k2, v2, [0, n])[:seen]), bits(want))


@pytest.mark.parametrize("Hq,H,D", [(5, 1, 128), (6, 2, 64), (7, 1, 128), (70, 14, 64), (33, 1, 128), (66, 6, 128)])
def test_what_an_earlier_kernel_left_changes_no_bit(Hq, H, D):
    """Groups that do not divide a tile's 128 rows: the rows past the last whole token are in no copy."""
    n = 1200
    q, k, v = qkv(n, Hq, H, D, Hq)
    zeros = torch.zeros(n, Hq + 2 * H, D, dtype=torch.bfloat16, device="cuda").split([Hq, H, H], dim=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    a, w = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((2048, 2048), (8192, 2048)))
    sx, sw = torch.ones(2048, device="cuda"), torch.ones(8192, device="cuda", dtype=torch.bfloat16)
    attend(*zeros, [0, n])
    want = attend(q, k, v, [0, n])
    for _ in range(3):
        wq.wq_gemm_w8a8_int8(a, sx, w, sw)
        assert torch.equal(bits(attend(q, k, v, [0, n])), bits(want))
    attend(*zeros, [0, n])
    assert torch.equal(bits(attend(q, k, v, [0, n])), bits(want))


@pytest.mark.parametrize("Hq,H,D,lengths", [(64, 8, 128, [1, 70, 331, 200, 45] * 8), (64, 8, 128, [6000]), (20, 4, 64, [2048, 1900, 777]),
                                            (40, 8, 128, [900, 1000])])
def test_repeated_calls_give_identical_bytes(Hq, H, D, lengths):
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    q, k, v = qkv(starts[-1], Hq, H, D, 3)
    want = attend(q, k, v, starts)
    for _ in range(10):
        assert torch.equal(bits(attend(q, k, v, starts)), bits(want))
