"""Stores into the quantised KV caches: bit for bit what the library's quantisers and the oracle give for the same
vectors, at the slots asked for, and nothing anywhere else."""
import numpy as np
import pytest
import torch

import group_wise_weight_b200 as wq
import oracle
import oracle.kv_cache as kv
from group_wise_weight_b200 import build as wqbuild

pytestmark = pytest.mark.gpu
NAMES = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales", "v_zeros")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    wqbuild.build()
    wq.lib()
    torch.cuda.init()


def int4_cache(B, T, H, seed=0):
    g = torch.Generator().manual_seed(seed)
    return {n: torch.randint(0, 256, (B, T, H, 64), generator=g, dtype=torch.uint8).cuda() if n.endswith("codes")
            else torch.randn(B, T, H, generator=g).to(torch.bfloat16).cuda() for n in NAMES}


def rows(M, H, seed):
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn(M, 3 * H, 128, generator=g).to(torch.bfloat16)
    special = [torch.zeros(128), torch.full((128,), -2.5), torch.full((128,), 1e-3) + torch.arange(128) * 2e-5,
               torch.linspace(100, 101, 128), torch.linspace(-1, 1, 128) * 3e38, torch.linspace(-1, 1, 128) * 2.0 ** -126,
               torch.arange(128).float() / 15 * 15, -torch.zeros(128)]
    for i, s in enumerate(special):
        if i < M:
            fused[i, H + i % H] = s.to(torch.bfloat16)
            fused[M - 1 - i, 2 * H + i % H] = s.to(torch.bfloat16)
    return fused


@pytest.mark.parametrize("M,B,T,H", [(1, 1, 1, 1), (1, 3, 7, 8), (5, 2, 9, 1), (64, 8, 33, 3), (257, 5, 100, 8), (1000, 1, 1003, 5)])
def test_int4_bit_exact(M, B, T, H):
    fused = rows(M, H, M + H)
    dev = fused.cuda()
    k, v = dev[:, H:2 * H], dev[:, 2 * H:]
    g = torch.Generator().manual_seed(M)
    slots = torch.randperm(B * T, generator=g)[:M]
    slots[::4] = torch.tensor([-1, B * T, -2**62, 2**62])[torch.arange(len(slots[::4])) % 4] if M > 1 else slots[::4]
    cache = int4_cache(B, T, H, M)
    before = {n: t.clone() for n, t in cache.items()}
    wq.wq_kv_store_int4(k, v, slots.cuda(), *(cache[n] for n in NAMES))
    torch.cuda.synchronize()
    kept = (slots >= 0) & (slots < B * T)
    for name, t in (("k", k), ("v", v)):
        dense = t.contiguous()[kept.cuda()]
        codes, s, z = kv.quantize_kv_int4(dense.float().cpu().numpy()[:, None])  # [m][1][H][D]
        m = dense.shape[0]
        want = {"codes": torch.from_numpy(oracle.pack_int4(codes.reshape(-1, 128))).view(m, H, 64)}
        for part, values in (("scales", s), ("zeros", z)):
            want[part] = torch.from_numpy(oracle.bf16_bits(values).astype(np.int16)).view(torch.bfloat16).view(m, H)
        q, qs, qz = wq.wq_quantize_int4(dense.reshape(-1, 128), 128)
        assert torch.equal(q.cpu().view(m, H, 64), want["codes"])
        for part in ("codes", "scales", "zeros"):
            whole = before[f"{name}_{part}"].cpu().flatten(0, 1)
            whole[slots[kept]] = want[part]
            got = cache[f"{name}_{part}"].cpu().flatten(0, 1)
            assert torch.equal(got.view(torch.int16) if got.dtype == torch.bfloat16 else got,
                               whole.view(torch.int16) if whole.dtype == torch.bfloat16 else whole), (name, part)


def fp8_ref(x, s):
    """Nearest E4M3 to RN(x / s), ties to even, saturated."""
    q = (x.double() / float(s)).float().clamp(-448, 448)
    return q.to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("scales", [(0.031, 0.011), (1.0, 2.0 ** -7), (3e-20, 1e20), (2.0 ** -120, 1e35)])
@pytest.mark.parametrize("M,B,T,H", [(1, 2, 3, 1), (130, 4, 40, 5)])
def test_fp8_bit_exact(M, B, T, H, scales):
    fused = rows(M, H, M + H)
    fused[0, H, :4] = torch.tensor([-0.0, 0.0, -1e-30, 1e-30])
    dev = fused.cuda()
    k, v = dev[:, H:2 * H], dev[:, 2 * H:]
    slots = torch.randperm(B * T, generator=torch.Generator().manual_seed(3))[:M]
    if M > 1:
        slots[5] = -1
    kc, vc = (torch.full((B, T, H, 128), 7, dtype=torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.tensor([s], dtype=torch.float32) for s in scales)
    wq.wq_kv_store_fp8(k, v, slots.cuda(), kc, ks.cuda(), vc, vs.cuda())
    for t, s, c in ((k, ks, kc), (v, vs, vc)):
        want = torch.full((B * T, H, 128), 7, dtype=torch.uint8)
        want[slots[slots >= 0]] = fp8_ref(t.cpu()[slots >= 0], s)
        assert torch.equal(c.cpu().flatten(0, 1), want)


def test_fp8_agrees_with_the_tensor_quantiser():
    x = torch.randn(50, 2, 128, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    q, s = wq.wq_quantize_fp8_tensor(x.reshape(100, 128))
    kc, vc = (torch.zeros(1, 50, 2, 128, dtype=torch.uint8).cuda() for _ in range(2))
    wq.wq_kv_store_fp8(x, x, torch.arange(50).cuda(), kc, s, vc, s)
    assert torch.equal(kc.view(100, 128), q) and torch.equal(vc, kc)


def test_slots_beyond_32_bits_of_bytes():
    """A cache whose code offsets pass 2^32 (4.3 GB of codes): its last and first slots."""
    T, H = 8_400_000, 8
    kc, vc = (torch.zeros(1, T, H, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    par = [torch.zeros(1, T, H, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    x = torch.randn(2, H, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    wq.wq_kv_store_int4(x, x, torch.tensor([T - 1, 0]).cuda(), kc, par[0], par[1], vc, par[2], par[3])
    q, s, _ = wq.wq_quantize_int4(x.reshape(-1, 128), 128)
    for c in (kc, vc):
        assert torch.equal(c[0, T - 1], q.view(2, H, 64)[0]) and torch.equal(c[0, 0], q.view(2, H, 64)[1])
        assert int(c[0, 1:1000].max()) == 0 and int(c[0, -1000:-1].max()) == 0
    assert torch.equal(par[0][0, T - 1], s.view(2, H)[0])


def test_refusals():
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16).cuda()
    slots = torch.arange(3).cuda()
    c = int4_cache(1, 4, 2)
    args = [c[n] for n in NAMES]
    for bad, err in (((x, x[:2], slots, *args), ValueError), ((x, x, slots.int(), *args), TypeError),
                     ((x, x, slots[:2], *args), ValueError), ((x[:, :1], x[:, :1], slots, *args), ValueError),
                     ((x, x, slots, args[0], args[1].float(), *args[2:]), TypeError),
                     ((x, x, slots, args[0], args[1][:, :2], *args[2:]), ValueError),
                     ((x, x, slots, args[0], args[1], args[1], *args[3:]), wq.WQError),
                     ((x[..., :64], x[..., :64], slots, *args), (ValueError, wq.WQError)),
                     ((x[:0], x[:0], slots[:0], *args), wq.WQError)):
        with pytest.raises(err):
            wq.wq_kv_store_int4(*bad)
    code = torch.zeros(1, 4, 2, 128, dtype=torch.uint8).cuda()
    one = torch.ones(1).cuda()
    with pytest.raises(wq.WQError):
        wq.wq_kv_store_fp8(x, x, slots, code, one, code, one)
    with pytest.raises(ValueError):
        wq.wq_kv_store_fp8(x, x, slots, code, torch.ones(2).cuda(), code.clone(), one)
