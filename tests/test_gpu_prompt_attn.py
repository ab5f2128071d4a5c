"""Causal attention over packed prompts on the GPU against binary64.

Bound per output o = sum_u p_u v_u, with A = sum_u p_u |v_u|: p rounded to bf16 (2^-8 A), the output rounded to bf16
(2^-8 |o|), and the binary32 part.  A score is off by at most (D + 8) 2^-24 S with S the row's largest
sum_d |q_d k_d| / sqrt(D) (D products and additions, the scaling, the subtraction of the maximum); an exponential is
within 2^-16 of itself beyond that; both enter p and the sum below it: 2 ((D + 8) 2^-24 S + 2^-16) A; the sums of
up to L terms in binary32 and the scalings by e^(m_old - m_new), one for each block of keys, add 2 L 2^-24 A.
"""
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


@pytest.fixture(autouse=True)
def _no_device_timeouts():
    yield
    assert wq.wq_device_status() == wq.WQ_OK, "a kernel recorded a bounded-wait timeout"


def qkv(M, Hq, H, D, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = torch.randn(M, Hq + 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = fused.split([Hq, H, H], dim=1)
    q.mul_(scale)
    return q, k, v


def starts_of(lengths, first=0):
    s = [first]
    for n in lengths:
        s.append(s[-1] + n)
    return s


def check(o, q, k, v, starts):
    Hq, D = q.shape[1:]
    r = Hq // k.shape[1]
    worst = 0.0
    for a, b in zip(starts[:-1], starts[1:]):
        n = b - a
        if n == 0:
            continue
        mask = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for j in range(Hq):
            qd, kd, vd = q[a:b, j].double(), k[a:b, j // r].double(), v[a:b, j // r].double()
            s = (qd @ kd.t() / math.sqrt(D)).masked_fill(~mask, -math.inf)
            p = torch.softmax(s, dim=1)
            size = ((qd.abs() @ kd.abs().t()) / math.sqrt(D)).masked_fill(~mask, 0).amax(1, keepdim=True)
            ref, top = p @ vd, p @ vd.abs()
            bound = (2 ** -8 + 2 * ((D + 8) * 2 ** -24 * size + 2 ** -16) + 2 * n * 2 ** -24) * top + 2 ** -8 * ref.abs()
            err = (o[a:b, j].double() - ref).abs()
            assert torch.isfinite(o[a:b, j]).all()
            worst = max(worst, float((err / bound.clamp_min(1e-300)).max()))
    assert worst <= 1, worst
    return worst


def run(lengths, Hq, H, D, seed, scale=1.0):
    starts = starts_of(lengths)
    q, k, v = qkv(starts[-1], Hq, H, D, seed, scale)
    o = wq.wq_prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32).cuda())
    check(o, q, k, v, starts)
    return o


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 384, 385, 513, 1000])
def test_one_sequence(n, D):
    run([n], 4, 2, D, n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (2, 1), (3, 1), (10, 2), (6, 1), (7, 1), (64, 8), (16, 1), (33, 1), (64, 1)])
def test_groups(Hq, H, D):
    run([70, 1, 200, 33], Hq, H, D, Hq + H)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 127, 128, 129, 255, 256, 257, 385, 513, 700])
def test_two_tiles_to_an_item(n, D):
    """More work than SMs: a CTA takes two tiles at a time, the second of them absent, cut short or whole."""
    run([n, 0, 300], 64, 64, D, n)


@pytest.mark.parametrize("D", [64, 128])
def test_ragged_pack_with_empty_sequences(D):
    run([0, 5, 0, 0, 129, 1, 1, 1, 300, 0, 64, 127, 2, 0], 8, 2, D, 3)


def test_many_sequences():
    g = torch.Generator().manual_seed(0)
    lengths = [int(x) for x in torch.randint(0, 40, (300,), generator=g)]
    run(lengths, 8, 2, 128, 4)


def test_long_runs_of_empty_sequences():
    """Far more CTAs than items: few short sequences among thousands of empty ones, at the end of the batch."""
    for B, heads in ((3000, 4), (16384, 64)):
        starts = [0] * (B - 4) + [5, 5, 40, 41, 300]
        q, k, v = qkv(300, heads, heads, 64, 9)
        o = wq.wq_prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32).cuda())
        check(o, q, k, v, [0, 5, 40, 41, 300])


def test_long_sequences():
    run([4100, 3000], 8, 1, 128, 5)
    run([5003], 2, 2, 64, 6)


@pytest.mark.parametrize("scale", [0.0, 0.01, 8.0, 40.0])
def test_flat_and_sharp_softmax(scale):
    run([500, 77], 8, 4, 128, 7, scale)


def test_running_maximum_that_rises_and_falls():
    """Keys whose scores climb with the position (every block raises the maximum) and fall with it (the first
    block holds it; later terms vanish)."""
    n, D = 900, 128
    for sign in (1.0, -1.0):
        q, k, v = qkv(n, 4, 2, D, 8)
        ramp = sign * torch.linspace(-30, 30, n, device="cuda")[:, None]
        q[..., 0] = 8.0
        k[..., 0] = (ramp * math.sqrt(D) / 8).to(torch.bfloat16)
        o = wq.wq_prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32).cuda())
        check(o, q, k, v, [0, n])


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_no_sequence(D):
    """Rows before the first sequence and behind the last keep what they held, and infinities and NaN in them, or in
    any row after a sequence's end, change nothing."""
    lengths, first, M = [100, 45, 130], 37, 400
    starts = starts_of(lengths, first)
    q, k, v = qkv(M, 8, 2, D, 9)
    o = torch.full((M, 8, D), 5.0, dtype=torch.bfloat16, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    wq.wq_prompt_attention(q, k, v, st, o=o)
    check(o, q, k, v, starts)
    assert (o[:first] == 5).all() and (o[starts[-1]:] == 5).all()
    want = o.clone()
    for t in (q, k, v):
        t[:first] = math.nan
        t[starts[-1]:] = math.inf
        t[starts[-1] + 1::2] = math.nan
    wq.wq_prompt_attention(q, k, v, st, o=o)
    assert torch.equal(o, want)
    # the last sequence alone, right behind rows of NaN, and a sequence that ends in the middle of a block of keys
    for t in (q, k, v):
        t[:starts[2]] = math.nan
    wq.wq_prompt_attention(q, k, v, torch.tensor([starts[2], starts[3] - 30], dtype=torch.int32).cuda(), o=o)
    assert torch.equal(o[starts[2]:starts[3] - 30], want[starts[2]:starts[3] - 30])


def test_strides_and_given_output():
    M, Hq, H, D = 300, 8, 2, 128
    q, k, v = qkv(M, Hq, H, D, 10)
    st = torch.tensor([0, 120, 300], dtype=torch.int32).cuda()
    want = wq.wq_prompt_attention(q, k, v, st)
    assert torch.equal(wq.wq_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), st), want)
    wide = torch.zeros(M, Hq + 3, D, dtype=torch.bfloat16, device="cuda")
    o = wide[:, 1:1 + Hq]
    assert wq.wq_prompt_attention(q, k, v, st, o=o) is o
    assert torch.equal(o, want) and (wide[:, 0] == 0).all() and (wide[:, 1 + Hq:] == 0).all()


def test_repeatable():
    a = run([333, 1000, 90], 16, 2, 128, 11)
    assert torch.equal(a, run([333, 1000, 90], 16, 2, 128, 11))


def test_offsets_beyond_32_bits():
    """Rows 2^18 values apart: the last sequence begins past 2^31 values (4.3 GB)."""
    M, ld = 8300, 1 << 18
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    rows = buf.view(M, ld)[:, :6 * 64].unflatten(1, (6, 64))
    rows.copy_(torch.randn(M, 6, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)))
    q, k, v = rows.split([4, 1, 1], dim=1)
    st = torch.tensor([0, 100, 8200, 8300], dtype=torch.int32).cuda()
    o = wq.wq_prompt_attention(q, k, v, st)
    want = wq.wq_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), st)
    assert torch.equal(o, want)
    check(o[8200:], q[8200:], k[8200:], v[8200:], [0, 100])


def test_bad_bounds_stay_inside():
    """`starts` that run outside 0 .. M or backwards are clamped: what they ask for is unspecified, every access stays
    inside the tensors (they are the middle of a larger buffer here) and nothing beyond the rows is written."""
    M, guard = 200, 300
    whole = torch.randn(M + 2 * guard, 6, 64, device="cuda").to(torch.bfloat16)
    q, k, v = whole[guard:guard + M].split([4, 1, 1], dim=1)
    out = torch.full((M + 2 * guard, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for st in ([-50, 100, 260], [0, 150, 20, 200], [300, 400], [-2**31, 2**31 - 1], [2**31 - 1, -2**31]):
        wq.wq_prompt_attention(q, k, v, torch.tensor(st, dtype=torch.int64).to(torch.int32).cuda(), o=out[guard:guard + M])
        torch.cuda.synchronize()
        assert (out[:guard] == 3).all() and (out[guard + M:] == 3).all()


def test_refusals():
    q, k, v = qkv(20, 4, 2, 128, 12)
    st = torch.tensor([0, 20], dtype=torch.int32).cuda()
    for args, kw, err in (((q.float(), k, v, st), {}, TypeError), ((q, k[:10], v, st), {}, ValueError),
                          ((q, k, v[:, :1], st), {}, ValueError), ((q, k, v, st.long()), {}, TypeError),
                          ((q, k, v, st[:1]), {}, ValueError), ((q, k, v, st.cpu()), {}, TypeError),
                          ((q[:, :3], k, v, st), {}, wq.WQError), ((q[..., :32], k[..., :32], v[..., :32], st), {}, ValueError),
                          ((q, k, v, st), dict(o=q), wq.WQError), ((q, k, v, st), dict(o=q[:10]), ValueError),
                          ((q[:0], k[:0], v[:0], st), {}, wq.WQError)):
        with pytest.raises(err):
            wq.wq_prompt_attention(*args, **kw)


def test_captured_and_replayed_with_other_bounds():
    q, k, v = qkv(256, 8, 2, 128, 13)
    st = torch.tensor([0, 100, 256], dtype=torch.int32).cuda()
    o = wq.wq_prompt_attention(q, k, v, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_prompt_attention(q, k, v, st, o=o)
    for starts in ([0, 256, 256], [3, 50, 200]):
        st.copy_(torch.tensor(starts, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(o, q, k, v, starts)


def test_two_streams_at_once():
    cases = [qkv(700, 8, 2, 128, s) for s in (14, 15)]
    st = torch.tensor([0, 300, 700], dtype=torch.int32).cuda()
    want = [wq.wq_prompt_attention(*c, st) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(wq.wq_prompt_attention(*cases[i % 2], st))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(got))
