"""What the routing and 8-bit entry points refuse before anything is enqueued, through the C ABI
and through the binding.  CPU only."""

import ctypes

import pytest
import torch

import token_dispatch_expert_gb300 as tde
from token_dispatch_expert_gb300 import _ActC, _Fp8GemmC, _Fp8WgradC, _QuantC

P = 4096   # a non-null, 16-byte aligned stand-in for a device address: never dereferenced
INVALID, UNSUPPORTED, OK = 1, 2, 0


@pytest.fixture(scope="module")
def L():
    tde.build()
    return tde.lib()


def cfg(**kw):
    base = dict(T=64, d=128, E=32, k=4, ffn=128)
    base.update(kw)
    return tde.make_config(**base)


def test_binding_states_the_header_constant():
    src = open(tde.__file__.replace("token_dispatch_expert_gb300/__init__.py", "include/moe.h")).read()
    assert f"#define MOE_FP8_WS_BYTES {tde.FP8_WS_BYTES}" in src


@pytest.mark.parametrize("kw,status", [
    (dict(score=2), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID),
    (dict(groups=8, top_groups=9), INVALID), (dict(groups=8, top_groups=0), INVALID),
    (dict(groups=16, top_groups=1), INVALID),        # 2 experts stay for k = 4
    (dict(groups=8, top_groups=4, group_top=3), INVALID),
    (dict(groups=32, top_groups=8, group_top=2), INVALID),   # groups of one expert
    (dict(renorm=2), INVALID), (dict(bias=4097), INVALID)])
def test_router_refusals(L, kw, status):
    c, r = cfg(), tde.make_router(**kw)
    args = [ctypes.byref(c), ctypes.byref(r)]
    assert L.moe_route_groups(*args, *[P] * 11, None) == status
    assert L.moe_route_groups_bwd(*args, *[P] * 5, None) == status


def test_router_refuses_other_routing_variants_sizes_and_pointers(L):
    r = tde.make_router()
    for kw in (dict(drop_negative=True), dict(drop_by_score=True, capacity=4),
               dict(select_bias=P)):
        c = cfg(**kw)
        assert L.moe_route_groups(ctypes.byref(c), ctypes.byref(r), *[P] * 11, None) == INVALID
    c = cfg()
    for n in range(11):
        for bad in (None, P + 4):
            ptrs = [P] * 11
            ptrs[n] = bad
            assert L.moe_route_groups(ctypes.byref(c), ctypes.byref(r), *ptrs, None) == INVALID
    assert L.moe_route_groups(ctypes.byref(c), None, *[P] * 11, None) == INVALID
    big = cfg(E=256)
    many = tde.make_router(groups=64, top_groups=8)
    assert L.moe_route_groups(ctypes.byref(big), ctypes.byref(many), *[P] * 11,
                              None) == UNSUPPORTED
    assert L.moe_route_groups(ctypes.byref(cfg(k=9)), ctypes.byref(r), *[P] * 11,
                              None) == UNSUPPORTED
    for n in range(7):
        ptrs = [P] * 7
        ptrs[n] = None
        assert L.moe_combine_bwd_dw(ctypes.byref(c), *ptrs, None) == INVALID


def test_token_blocks(L):
    assert tde.moe_fp8_token_blocks(0, 3) == 3
    assert tde.moe_fp8_token_blocks(129, 1) == 3
    assert tde.moe_fp8_token_blocks(-1, 1) == -1 and tde.moe_fp8_token_blocks(5, 0) == -1


QUANT = dict(rows=10, src_rows=10, G=2, C=100, ldx=100, ld=112, pow2=0)
QPTRS = dict(x=P, src_tok=None, offsets=P, codes=P, scales=P, codes_t=P, scales_t=P, ws=P)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(G=0), INVALID), (dict(C=0), INVALID), (dict(ldx=99), INVALID),
    (dict(ld=96), INVALID), (dict(ld=104), INVALID), (dict(pow2=2), INVALID),
    (dict(G=257), UNSUPPORTED), (dict(C=1 << 24), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(offsets=None), INVALID),
    (dict(offsets=P + 4), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(codes=P + 8), INVALID), (dict(codes_t=None), INVALID), (dict(scales_t=P + 4), INVALID),
    (dict(ws=None), INVALID), (dict(src_tok=P + 4), INVALID),
    (dict(src_tok=P, src_rows=0), INVALID),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), INVALID),
    (dict(rows=0, codes=None, scales=None), OK)])
def test_quantize_refusals(L, change, status):
    q = _QuantC(*[{**QUANT, **change}[n] for n in QUANT])
    p = [{**QPTRS, **change}[n] for n in QPTRS]
    assert L.moe_fp8_quantize(ctypes.byref(q), *p, None) == status
    assert L.moe_fp8_quantize(None, *p, None) == INVALID


@pytest.mark.parametrize("args,status", [
    ((P, 0, 8, 8, P, 16, P, None, 0, None, 0), INVALID),
    ((P, 1, 0, 8, P, 16, P, None, 0, None, 0), INVALID),
    ((P, 1, 8, 0, P, 16, P, None, 0, None, 0), INVALID),
    ((P, 1, 8, 17, P, 16, P, None, 0, None, 0), INVALID),
    ((P, 1, 8, 8, P, 16, P, P, 16, None, 0), INVALID),
    ((P, 1, 8, 8, P, 16, P, P, 8, P, 0), INVALID),
    ((P, 1, 8, 8, None, 16, P, None, 0, None, 0), INVALID),
    ((P + 1, 1, 8, 8, P, 16, P, None, 0, None, 0), INVALID),
    ((P, 1, 8, 8, P, 16, P, None, 0, None, 3), INVALID),
    ((P, 257, 8, 8, P, 16, P, None, 0, None, 0), UNSUPPORTED),
    ((P, 1, 1 << 24, 8, P, 16, P, None, 0, None, 0), UNSUPPORTED)])
def test_quantize_weights_refusals(L, args, status):
    assert L.moe_fp8_quantize_weights(*args, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(f=0), INVALID), (dict(ld=96), INVALID), (dict(pow2=-1), INVALID),
    (dict(G=300), UNSUPPORTED), (dict(f=1 << 24), UNSUPPORTED)])
def test_swiglu_refusals(L, change, status):
    base = dict(rows=10, G=2, f=100, ld=208, pow2=0)
    a = _ActC(*[{**base, **change}[n] for n in base])
    assert L.moe_fp8_swiglu(ctypes.byref(a), *[P] * 7, None) == status
    assert L.moe_fp8_swiglu_bwd(ctypes.byref(a), *[P] * 10, None) == status


def test_swiglu_pointer_refusals(L):
    a = _ActC(10, 2, 100, 208, 0)
    for n in (0, 2, 3, 6):
        p = [P] * 7
        p[n] = None
        assert L.moe_fp8_swiglu(ctypes.byref(a), *p, None) == INVALID
    for n in (0, 1, 3, 4, 5, 6, 7, 8, 9):
        p = [P] * 10
        p[n] = P + 4
        assert L.moe_fp8_swiglu_bwd(ctypes.byref(a), *p, None) == INVALID
    # h along the tokens only with the gradients along the tokens
    p = [P, P, P, P, P, None, None, P, P, P]
    assert L.moe_fp8_swiglu_bwd(ctypes.byref(a), *p, None) == INVALID


GEMM = dict(rows=10, G=2, N=100, K=200, lda=208, ldb=208, ldo=100, out_type=0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(G=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(lda=192), INVALID), (dict(lda=200), INVALID), (dict(ldb=201), INVALID),
    (dict(ldo=99), INVALID), (dict(out_type=2), INVALID), (dict(G=257), UNSUPPORTED),
    (dict(N=1 << 24, ldo=1 << 24), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(rows=0), OK)])
def test_gemm_refusals(L, change, status):
    g = _Fp8GemmC(*[{**GEMM, **change}[n] for n in GEMM])
    p = [None] * 7 if change == dict(rows=0) else [P] * 7
    if change == dict(rows=0):
        p[4] = P
    assert L.moe_fp8_gemm(ctypes.byref(g), *p, None) == status


def test_gemm_and_wgrad_pointer_refusals(L):
    g = _Fp8GemmC(*GEMM.values())
    w = _Fp8WgradC(10, 2, 64, 64, 0)
    for n in range(7):
        p = [P] * 7
        p[n] = None
        assert L.moe_fp8_gemm(ctypes.byref(g), *p, None) == INVALID
        assert L.moe_fp8_wgrad(ctypes.byref(w), *p, None) == INVALID
    p = [P] * 7
    p[5] = P + 1
    assert L.moe_fp8_gemm(ctypes.byref(g), *p, None) == INVALID
    for bad, status in (((-1, 2, 64, 64, 0), INVALID), ((10, 2, 0, 64, 0), INVALID),
                        ((10, 2, 64, 0, 0), INVALID), ((10, 2, 64, 64, 5), INVALID),
                        ((10, 257, 64, 64, 0), UNSUPPORTED), ((10, 2, 1 << 24, 64, 0), UNSUPPORTED)):
        assert L.moe_fp8_wgrad(ctypes.byref(_Fp8WgradC(*bad)), *[P] * 7, None) == status


def test_binding_refuses_host_tensors_wrong_types_and_shapes():
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    x = torch.zeros((4, 128), dtype=bf)
    ws = torch.zeros(256, dtype=u8)
    with pytest.raises(ValueError):
        tde.moe_fp8_quantize(x, torch.zeros((4, 128), dtype=u8), torch.zeros((4, 1)), ws=ws)
    with pytest.raises(ValueError):
        tde.moe_fp8_gemm(torch.zeros((4, 128), dtype=u8), torch.zeros((4, 2)),
                         torch.zeros((1, 8, 128), dtype=u8), torch.zeros((1, 1, 1)),
                         torch.zeros((4, 8), dtype=f32), 128, ws=ws)
    with pytest.raises(ValueError):
        tde.moe_fp8_wgrad(torch.zeros((8, 256), dtype=u8), torch.zeros((2, 8)),
                          torch.zeros((8, 256), dtype=u8), torch.zeros((2, 8)),
                          torch.zeros((1, 8, 8), dtype=torch.float16), ws=ws)
    with pytest.raises(ValueError):
        tde.make_router(bias=torch.zeros(8, dtype=f32))      # a host tensor
    with pytest.raises(ValueError):
        tde.make_router(bias=torch.zeros(8, dtype=torch.float64))
