"""The routing entry points of the binding refuse buffers of another type and buffers that are too
small: a kernel would read int64 indices as int32, or write fp32 values past a bf16 tensor's end.
CPU only: a refusal comes before the device is asked for, and the other buffers are addresses."""

import pytest
import torch

import token_dispatch_expert_gb300 as tde

# Stands for a device address: never dereferenced, and off 16 bytes, so that the library refuses a
# call that the binding lets pass.
P = 4100
T, E, K, D = 6, 16, 4, 64
I32, F32, BF = torch.int32, torch.float32, torch.bfloat16

ROUTE = [("logits", T * E, F32), ("topk_idx", T * K, I32), ("topk_w", T * K, F32),
         ("counts", E, I32), ("kept", E, I32), ("offsets", E + 1, I32), ("dest_row", T * K, I32),
         ("src_tok", T * K, I32), ("src_slot", T * K, I32), ("drop_mask", T * K, torch.uint8)]
ROUTE_BWD = [("logits", T * E, F32), ("topk_idx", T * K, I32), ("dw", T * K, F32),
             ("dlogits", T * E, F32)]
COMBINE = [("dy", T * D, BF), ("yp", None, BF), ("topk_w", T * K, F32), ("dest_row", T * K, I32),
           ("dyp", None, BF), ("dw", T * K, F32)]


def calls():
    cfg, router = tde.make_config(T, D, E, K, 64), tde.make_router()
    return [(lambda *a: tde.moe_route_groups(cfg, router, *a, P, stream=P), ROUTE),
            (lambda *a: tde.moe_route_groups_bwd(cfg, router, *a, P, stream=P), ROUTE_BWD),
            (lambda *a: tde.moe_combine_bwd_dw(cfg, *a, P, stream=P), COMBINE)]


def cases():
    for i, spec in enumerate((ROUTE, ROUTE_BWD, COMBINE)):
        for j, (name, n, dtype) in enumerate(spec):
            wrong = {I32: (torch.int64, F32, torch.int16), F32: (BF, torch.float64, I32),
                     BF: (torch.float16, F32), torch.uint8: (I32, torch.int16)}[dtype]
            for w in wrong:
                yield pytest.param(i, j, torch.zeros(n or 8, dtype=w), id=f"{i}-{name}-{w}")
            if n is not None:
                yield pytest.param(i, j, torch.zeros(n - 1, dtype=dtype), id=f"{i}-{name}-short")


@pytest.mark.parametrize("i,j,tensor", list(cases()))
def test_refuses_types_and_sizes(i, j, tensor):
    call, spec = calls()[i]
    args = [P] * len(spec)
    args[j] = tensor
    with pytest.raises(ValueError, match=f"^{spec[j][0]}: expected"):
        call(*args)


@pytest.mark.parametrize("i", [0, 1, 2])
def test_the_right_types_get_as_far_as_the_device(i):
    """Any shape of enough elements; the next thing asked of a host tensor is its device."""
    call, spec = calls()[i]
    for j, (name, n, dtype) in enumerate(spec):
        for extra in (0, 5):
            args = [P] * len(spec)
            args[j] = torch.zeros((n or 8) + extra, dtype=dtype)
            with pytest.raises(ValueError, match="expected a CUDA tensor"):
                call(*args)
    if i == 0:
        args = [P] * len(spec)
        args[-1] = torch.zeros(T * K, dtype=torch.bool)
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            call(*args)


def test_refuses_a_short_bias():
    router = tde.make_router(bias=P)
    router._keep = torch.zeros(E - 1)
    cfg = tde.make_config(T, D, E, K, 64)
    with pytest.raises(ValueError, match="^bias: expected 16 elements, got 15"):
        tde.moe_route_groups(cfg, router, *[P] * 11, stream=P)
