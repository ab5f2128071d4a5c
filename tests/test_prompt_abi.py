"""Host-side refusals of the prompt-side entry points (no call here reaches a launch) and the rules of their
overlap checks.  Addresses are fake and never dereferenced."""
import pytest
import torch

import group_wise_weight_b200 as wq
from group_wise_weight_b200 import build as wqbuild


@pytest.fixture(scope="module")
def L():
    wqbuild.build()
    return wq.lib()


def _bufs(n):
    return [(1 << 33) + i * (1 << 28) for i in range(n)]


X, Q, S, W, Y, Z, R, T = _bufs(8)
ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = (wq.WQ_ERR_ARG, wq.WQ_ERR_SHAPE, wq.WQ_ERR_ALIGN, wq.WQ_ERR_UNSUPPORTED,
                                             wq.WQ_ERR_WORKSPACE)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG), (dict(M=0), ARG), (dict(K=0), ARG),
    (dict(ldx=-8), ARG), (dict(xt=2), UNSUPPORTED), (dict(K=48), SHAPE), (dict(ldx=224), SHAPE),
    (dict(ldx=260), ALIGN), (dict(x=X + 8), ALIGN), (dict(q=Q + 4), ALIGN), (dict(s=S + 2), ALIGN),
    (dict(q=X + 16), ARG), (dict(s=X + 4), ARG), (dict(s=Q + 1020), ARG), (dict(M=1 << 31), SHAPE),
])
def test_quantize_int8_tokens_rejects(L, kw, code):
    a = dict(x=X, xt=wq.WQ_BF16, M=4, K=256, ldx=256, q=Q, s=S)
    a.update(kw)
    assert L.wq_quantize_int8_tokens(a["x"], a["xt"], a["M"], a["K"], a["ldx"], a["q"], a["s"], None) == code
    assert wq.wq_last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(xs=None), ARG), (dict(w=None), ARG), (dict(s=None), ARG), (dict(y=None), ARG),
    (dict(M=0), ARG), (dict(N=-1), ARG), (dict(K=40), SHAPE), (dict(K=131072), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(x=X + 8), ALIGN), (dict(xs=S + 2), ALIGN), (dict(w=W + 4), ALIGN), (dict(y=Y + 2), ALIGN),
    (dict(y=X + 512), ARG), (dict(y=W + 1024), ARG), (dict(y=Z), ARG), (dict(y=S), ARG),
    (dict(ws=None), WORKSPACE), (dict(wsb=1024), WORKSPACE), (dict(ws=R + 8), WORKSPACE), (dict(ws=Y), ARG),
])
def test_gemm_w8a8_int8_rejects(L, kw, code):
    a = dict(x=X, xs=S, M=1, N=1000, K=28672, w=W, s=Z, y=Y, ws=R, wsb=1 << 27)
    a.update(kw)
    assert L.wq_gemm_w8a8_int8(a["x"], a["xs"], a["M"], a["N"], a["K"], a["w"], a["s"], a["y"], a["ws"], a["wsb"],
                               None) == code
    assert wq.wq_last_error() != ""


def test_gemm_w8a8_int8_workspace_holds_the_counters(L):
    assert wq.wq_gemm_w8a8_int8_workspace_bytes(0, 16, 64) == 0
    assert wq.wq_gemm_w8a8_int8_workspace_bytes(1, 1000, 28672) > 65536  # tiles split between CTAs
    assert wq.wq_gemm_w8a8_int8_workspace_bytes(4096, 10240, 8192) == 0  # none split
    for M in (1, 5, 16, 17, 64, 100, 128, 129, 1000):
        for N, K in ((1, 32), (130, 28672), (512, 512), (8192, 8192), (57344, 1024), (10240, 131040)):
            need = wq.wq_gemm_w8a8_int8_workspace_bytes(M, N, K)
            assert need == 0 or need > 65536


def _rope(L, **kw):
    a = dict(q=X, ldq=1024, k=Q, ldk=256, qw=None, kw=None, eps=1e-6, pos=S, f=W, rot=128, il=0, M=4, Hq=8, H=2, D=128,
             qo=Y, ldqo=1024, ko=Z, ldko=256)
    a.update(kw)
    return L.wq_qk_norm_rope(a["q"], a["ldq"], a["k"], a["ldk"], a["qw"], a["kw"], a["eps"], a["pos"], a["f"],
                             a["rot"], a["il"], a["M"], a["Hq"], a["H"], a["D"], a["qo"], a["ldqo"], a["ko"],
                             a["ldko"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(pos=None), ARG), (dict(f=None), ARG), (dict(qo=None), ARG),
    (dict(ko=None), ARG), (dict(qw=R), ARG), (dict(kw=R), ARG), (dict(qw=R, kw=T, eps=-1.0), ARG),
    (dict(qw=R, kw=T, eps=float("nan")), ARG), (dict(M=0), ARG), (dict(H=0), ARG), (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED), (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE),
    (dict(D=64, rot=80), SHAPE), (dict(ldq=1016), SHAPE), (dict(ldk=248), SHAPE), (dict(ldqo=1023), SHAPE),
    (dict(ldq=1028), ALIGN), (dict(q=X + 8), ALIGN), (dict(ko=Z + 2), ALIGN), (dict(qw=R + 8, kw=T), ALIGN),
    (dict(pos=S + 2), ALIGN), (dict(f=W + 1), ALIGN),
    (dict(qo=X + 16), ARG), (dict(qo=X, ldqo=1032), ARG), (dict(qo=Q), ARG), (dict(ko=X), ARG), (dict(ko=Y + 2048), ARG),
    (dict(ko=S), ARG), (dict(qo=W), ARG), (dict(qw=Y + 64, kw=T), ARG), (dict(qw=R, kw=Z + 16), ARG),
])
def test_qk_norm_rope_rejects(L, kw, code):
    assert _rope(L, **kw) == code
    assert wq.wq_last_error() != ""


def _store(L, fp8=False, **kw):
    a = dict(k=X, ldk=256, v=Q, ldv=256, slots=S, M=4, S=64, H=2, D=128, kc=W, ks=Y, kz=Y + (1 << 20), vc=Z, vs=R,
             vz=R + (1 << 20))
    a.update(kw)
    if fp8:
        return L.wq_kv_store_fp8(a["k"], a["ldk"], a["v"], a["ldv"], a["slots"], a["M"], a["S"], a["H"], a["D"],
                                 a["kc"], a["ks"], a["vc"], a["vs"], None)
    return L.wq_kv_store_int4(a["k"], a["ldk"], a["v"], a["ldv"], a["slots"], a["M"], a["S"], a["H"], a["D"], a["kc"],
                              a["ks"], a["kz"], a["vc"], a["vs"], a["vz"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(kc=None), ARG), (dict(ks=None), ARG),
    (dict(vs=None), ARG), (dict(M=0), ARG), (dict(S=0), ARG), (dict(H=-2), ARG), (dict(D=64), UNSUPPORTED),
    (dict(ldk=248), SHAPE), (dict(ldv=128), SHAPE), (dict(M=1 << 29), SHAPE), (dict(S=1 << 41), SHAPE),
    (dict(ldk=260), ALIGN), (dict(k=X + 8), ALIGN), (dict(slots=S + 4), ALIGN), (dict(kc=W + 8), ALIGN), (dict(ks=Y + 2), ALIGN),
    (dict(kc=X + 64), ARG), (dict(vc=W + 4096), ARG), (dict(vc=S), ARG), (dict(vc=Q), ARG),
])
def test_kv_store_rejects(L, fp8, kw, code):
    assert _store(L, fp8, **kw) == code
    assert wq.wq_last_error() != ""


def test_kv_store_int4_rejects_overlapping_parts(L):
    assert _store(L, kz=None) == ARG
    assert _store(L, kz=Y + 16) == ARG
    assert _store(L, vs=Z + 128) == ARG


def _attn(L, **kw):
    a = dict(q=X, ldq=1024, k=Q, ldk=256, v=W, ldv=256, st=S, B=3, M=100, Hq=8, H=2, D=128, o=Y, ldo=1024)
    a.update(kw)
    return L.wq_prompt_attention(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["st"], a["B"], a["M"],
                                 a["Hq"], a["H"], a["D"], a["o"], a["ldo"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(st=None), ARG), (dict(o=None), ARG),
    (dict(B=0), ARG), (dict(M=0), ARG), (dict(H=0), ARG), (dict(D=80), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(H=3, ldk=384, ldv=384), UNSUPPORTED), (dict(Hq=130, H=2, ldq=130 * 128, ldo=130 * 128), UNSUPPORTED),
    (dict(M=1 << 31), SHAPE), (dict(M=(1 << 25) + 1), SHAPE), (dict(B=(1 << 20) + 1), SHAPE),
    (dict(B=1 << 20, Hq=60000, H=60000, ldq=60000 * 128, ldk=60000 * 128, ldv=60000 * 128, ldo=60000 * 128), SHAPE),
    (dict(ldq=1000), SHAPE), (dict(ldo=1016), SHAPE), (dict(ldv=100), SHAPE),
    (dict(ldk=260), ALIGN), (dict(q=X + 8), ALIGN), (dict(o=Y + 4), ALIGN), (dict(st=S + 2), ALIGN),
    (dict(o=X), ARG), (dict(o=Q + 16), ARG), (dict(o=W + 256 * 99 * 2), ARG), (dict(o=S), ARG),
])
def test_prompt_attention_rejects(L, kw, code):
    assert _attn(L, **kw) == code
    assert wq.wq_last_error() != ""


def test_columns_of_one_buffer_are_apart(L):
    # q, k, v as columns of a fused buffer of 12 heads: an output in the same buffer's other columns is refused only
    # where it shares columns; what passes the overlap checks ends at a later refusal (a misaligned `starts`, checked
    # before them, would hide this: the status of the overlapping call names the difference)
    ld = 20 * 128
    fused = dict(q=X, ldq=ld, k=X + 8 * 256, ldk=ld, v=X + 10 * 256, ldv=ld, ldo=ld)
    assert _attn(L, **fused, o=X + 11 * 256) == ARG          # shares v's second head
    assert _attn(L, **fused, o=X + 19 * 256) == ARG          # runs into the next row's first heads
    assert "overlaps" in wq.wq_last_error()
    assert _rope(L, q=X, ldq=ld, k=X + 8 * 256, ldk=ld, qo=X + 9 * 256, ldqo=ld, ko=X + 8 * 256, ldko=ld) == ARG


def test_binding_refuses_cpu_tensors_and_wrong_types(L):
    bf = torch.bfloat16
    with pytest.raises(TypeError):
        wq.wq_quantize_int8_tokens(torch.zeros(4, 256, dtype=bf))
    with pytest.raises(TypeError):
        wq.wq_gemm_w8a8_int8(torch.zeros(4, 64, dtype=torch.int8), torch.ones(4), torch.zeros(8, 64, dtype=torch.int8),
                             torch.ones(8, dtype=bf))
    q, k = torch.zeros(4, 8, 128, dtype=bf), torch.zeros(4, 2, 128, dtype=bf)
    with pytest.raises(TypeError):
        wq.wq_qk_norm_rope(q, k, torch.zeros(4, dtype=torch.int32), torch.zeros(64))
    with pytest.raises(TypeError):
        wq.wq_kv_store_fp8(k, k, torch.zeros(4, dtype=torch.int64), torch.zeros(2, 4, 2, 128, dtype=torch.uint8),
                           torch.ones(1), torch.zeros(2, 4, 2, 128, dtype=torch.uint8), torch.ones(1))
    with pytest.raises(TypeError):
        wq.wq_prompt_attention(q, k, k, torch.tensor([0, 4], dtype=torch.int32))
