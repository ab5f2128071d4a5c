"""A prompt and the decode steps after it through one attention block, as a server runs them: per-token INT8 and the
W8A8 matmul for the projections, norms and rotary positions, the store into the quantised cache, prompt attention,
then one token per sequence at a time through the same calls and the decode attention over the cache.

Every call is checked against binary64 on the inputs it was given (so no bound compounds another's), and the decode
step's attention also against the attention over the prompt's own keys and values, off by the cache's quantisation
alone."""
import math

import pytest
import torch

import group_wise_weight_b200 as wq
from group_wise_weight_b200 import build as wqbuild

pytestmark = pytest.mark.gpu
B, T, H, HQ, D, WIDTH = 5, 160, 2, 8, 128, 1024
LENGTHS = [1, 70, 130, 33, 128]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    wqbuild.build()
    wq.lib()
    torch.cuda.init()


class Block:
    def __init__(self, form):
        g = torch.Generator().manual_seed(21)
        w = (torch.randn((HQ + 2 * H) * D, WIDTH, generator=g) * 0.03).to(torch.bfloat16).cuda()
        self.w, self.ws = wq.wq_quantize_int8(w)
        wo = (torch.randn(WIDTH, HQ * D, generator=g) * 0.03).to(torch.bfloat16).cuda()
        self.wo, self.wos = wq.wq_quantize_int8(wo)
        self.qn, self.kn = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
        self.freq = (10000.0 ** (-2 * torch.arange(D // 2).double() / D)).float().cuda()
        self.form = form
        self.k_codes, self.v_codes = (torch.zeros(B, T, H, D // 2 if form == "int4" else D, dtype=torch.uint8).cuda()
                                      for _ in range(2))
        if form == "int4":
            self.par = [torch.zeros(B, T, H, dtype=torch.bfloat16).cuda() for _ in range(4)]
        else:
            self.k_scale, self.v_scale = torch.full((1,), 0.02).cuda(), torch.full((1,), 0.02).cuda()

    def linear(self, x, w, ws):
        xq, xs = wq.wq_quantize_int8_tokens(x)
        y = wq.wq_gemm_w8a8_int8(xq, xs, w, ws)
        acc = xq.double() @ w.double().t()
        ref = (acc.float() * (xs[:, None] * ws.float().view(1, -1))).to(torch.bfloat16)
        assert torch.equal(y, ref)
        return y

    def project(self, x, positions, slots):
        """q, k (normed and turned, in place) and v of the tokens, stored into the cache."""
        fused = self.linear(x, self.w, self.ws).view(-1, HQ + 2 * H, D)
        q, k, v = fused.split([HQ, H, H], dim=1)
        wq.wq_qk_norm_rope(q, k, positions, self.freq, self.qn, self.kn, q_out=q, k_out=k)
        if self.form == "int4":
            wq.wq_kv_store_int4(k, v, slots, self.k_codes, self.par[0], self.par[1], self.v_codes, self.par[2], self.par[3])
        else:
            wq.wq_kv_store_fp8(k, v, slots, self.k_codes, self.k_scale, self.v_codes, self.v_scale)
        return q, k, v

    def cached(self, b, n):
        """Keys and values of sequence b's first n places as the cache holds them, binary64."""
        found = []
        for i, codes in enumerate((self.k_codes, self.v_codes)):
            c = codes[b, :n]
            if self.form == "int4":
                s, z = (t[b, :n].double()[..., None] for t in self.par[2 * i:2 * i + 2])
                found.append(s * (torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).double() - z))
            else:
                found.append(c.view(torch.float8_e4m3fn).double() * float((self.k_scale, self.v_scale)[i]))
        return found

    def decode(self, q, lengths):
        if self.form == "int4":
            return wq.wq_decode_attention_int4(q.contiguous(), self.k_codes, self.par[0], self.par[1], self.v_codes,
                                               self.par[2], self.par[3], lengths)
        return wq.wq_decode_attention_fp8(q.contiguous(), self.k_codes, self.k_scale, self.v_codes, self.v_scale, lengths)


def attend(q, k, v):
    """(o, sum p |v|) of one query token [HQ][D] over keys and values [n][H][D], binary64."""
    kd, vd = (t.double().repeat_interleave(HQ // H, dim=1) for t in (k, v))
    p = torch.softmax(torch.einsum("hd,nhd->hn", q.double(), kd) / math.sqrt(D), dim=1)
    return torch.einsum("hn,nhd->hd", p, vd), torch.einsum("hn,nhd->hd", p, vd.abs())


@pytest.mark.parametrize("form", ["int4", "fp8"])
def test_prompt_then_decode(form):
    block = Block(form)
    g = torch.Generator().manual_seed(22)
    starts = torch.tensor([0] + LENGTHS).cumsum(0)
    M = int(starts[-1])
    x = torch.randn(M, WIDTH, generator=g).to(torch.bfloat16).cuda()
    positions = torch.cat([torch.arange(n) for n in LENGTHS]).int().cuda()
    slots = torch.cat([b * T + torch.arange(n) for b, n in enumerate(LENGTHS)]).cuda()
    q, k, v = block.project(x, positions, slots)
    o = wq.wq_prompt_attention(q, k, v, starts.int().cuda())
    block.linear(o.view(M, HQ * D), block.wo, block.wos)
    keys = [k[starts[b]:starts[b + 1]].clone() for b in range(B)]
    values = [v[starts[b]:starts[b + 1]].clone() for b in range(B)]
    for b in range(B):
        last = int(starts[b + 1]) - 1
        ref, size = attend(q[last], keys[b], values[b])
        assert ((o[last].double() - ref).abs() <= (2 ** -8 + 2 ** -10) * size + 2 ** -8 * ref.abs()).all()

    lengths = torch.tensor(LENGTHS, dtype=torch.int32).cuda()
    for step in range(3):
        x = torch.randn(B, WIDTH, generator=g).to(torch.bfloat16).cuda()
        slots = (torch.arange(B).cuda() * T + lengths).long()
        q, k, v = block.project(x, lengths.clone(), slots)
        lengths += 1
        o = block.decode(q, lengths)
        for b in range(B):
            n = int(lengths[b])
            keys[b], values[b] = torch.cat([keys[b], k[b:b + 1]]), torch.cat([values[b], v[b:b + 1]])
            kc, vc = block.cached(b, n)
            for full, cache in ((keys[b], kc), (values[b], vc)):  # within half a step of what was stored
                f = full.double()
                step_of = ((f.amax(-1) - f.amin(-1)) / 15 * 0.51 + f.abs().amax(-1) * 2 ** -8 if form == "int4"
                           else f.abs().amax(-1) * 2 ** -4 + 0.02 * 2 ** -9)
                assert ((f - cache).abs().amax(-1) <= step_of).all()
            ref, size = attend(q[b], kc, vc)
            assert ((o[b].double() - ref).abs() <= 4e-3 * size).all()


def test_decode_step_captured():
    """The decode step's calls as one CUDA graph, replayed with new inputs."""
    block, eager = Block("int4"), Block("int4")
    g = torch.Generator().manual_seed(23)
    x = torch.randn(B, WIDTH, generator=g).to(torch.bfloat16).cuda()
    lengths = torch.zeros(B, dtype=torch.int32).cuda()
    space = torch.zeros(wq.wq_gemm_w8a8_int8_workspace_bytes(B, (HQ + 2 * H) * D, WIDTH), dtype=torch.uint8).cuda()
    base = torch.arange(B).cuda() * T

    def step(block, x, lengths):
        xq, xs = wq.wq_quantize_int8_tokens(x)
        fused = wq.wq_gemm_w8a8_int8(xq, xs, block.w, block.ws, workspace=space).view(B, HQ + 2 * H, D)
        q, k, v = fused.split([HQ, H, H], dim=1)
        wq.wq_qk_norm_rope(q, k, lengths, block.freq, block.qn, block.kn, q_out=q, k_out=k)
        wq.wq_kv_store_int4(k, v, base + lengths, block.k_codes, block.par[0], block.par[1], block.v_codes,
                            block.par[2], block.par[3])
        return block.decode(q, lengths + 1)

    step(block, x, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(block, x, lengths)
    for n in range(4):
        x.copy_(torch.randn(B, WIDTH, generator=g).to(torch.bfloat16))
        lengths.fill_(n)
        graph.replay()
        want = step(eager, x, lengths)
        torch.cuda.synchronize()
        assert torch.equal(o, want)
