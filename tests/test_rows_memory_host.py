"""What the norms and the layers that keep 8-bit checkpoints hold, counted from their tensors.  CPU only:
the buffers are made on the meta device."""

import ctypes

import pytest
import torch

import token_dispatch_expert_gb300 as tde


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    tde.build()
    monkeypatch.setattr(tde, "moe_ws_init", lambda ws, stream=None: None)


def tensors(o):
    if isinstance(o, torch.Tensor):
        return [o]
    if isinstance(o, dict):
        o = o.values()
    elif not isinstance(o, (tuple, list)):
        return []
    return [t for v in o for t in tensors(v)]


def held(o, *shared):
    """Bytes of an object's own tensors: those that `shared` objects have too are theirs."""
    theirs = {id(t) for s in shared for t in tensors(vars(s))}
    own = {id(t): t for t in tensors(vars(o)) if id(t) not in theirs}
    return sum(t.numel() * t.element_size() for t in own.values())


def cfg(T=4096, d=4096, E=8, k=2, f=1408):
    return tde.make_config(T, d, E, k, f)


@pytest.mark.parametrize("T,d", [(1, 64), (256, 1024), (2048, 1024), (4096, 4096), (4096, 7168)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_norm_in_8_bits_holds_less_than_its_rows(T, d, fmt):
    """Codes, a scale for 128 of them and the statistics: no workspace of its own beside a shared one."""
    scratch = tde.MoEScratch(cfg(T, d, 8, 2, 64), device="meta")
    norms = [tde.MoENorm(T, d, checkpoint=fmt, device="meta", ws=scratch.ws) for _ in range(2)]
    for n in norms:
        assert n.ws is scratch.ws
        assert held(n, scratch) == T * d + T * -(-d // 128) * 4 + T * 8 < 2 * T * d


def test_workspaces_serve_the_norms():
    for T, d, k, f in ((1, 64, 1, 64), (3, 8192, 1, 64), (4096, 512, 2, 128)):
        c = cfg(T, d, 8, k, f)
        for ws in (tde.MoEScratch(c, device="meta").ws, tde.Fp8MoELayer(c, tde.make_router(), device="meta").ws):
            assert tde.MoENorm(T, d, device="meta", ws=ws).ws is ws
    with pytest.raises(ValueError, match="^ws: expected"):
        tde.MoENorm(4, 64, device="meta", ws=torch.empty(256, dtype=torch.uint8, device="meta"))
    # without one it has its own, as large as its gradient needs
    n = tde.MoENorm(4, 64, device="meta")
    assert n.ws.numel() == tde.moe_norm_ws_size(4, 64)


def up(n):
    return (n + 255) // 256 * 256


def test_stage_workspace_size():
    """The word of errors, the routing's scratch and the segments' maps; the rest of the whole layer's
    workspace is its intermediates."""
    for kw in ({}, dict(capacity=900, drop_by_score=True), dict(gate="sigmoid", drop_negative=True)):
        for T, d, E, k, f in ((1, 64, 1, 1, 64), (4096, 4096, 8, 2, 1408), (8192, 2048, 128, 8, 768)):
            c, R = tde.make_config(T, d, E, k, f, **kw), T * k
            stage, whole = tde.moe_stage_workspace_size(c), tde.moe_workspace_size(c)[0]
            assert stage + 2 * up(2 * R * d) + up(4 * R * f) == whole
            assert stage >= 256 + up(4 * E) + 256 * E + (4 * R if kw.get("drop_by_score") else 0)
    L, n = tde.lib(), ctypes.c_size_t(7)
    bad = tde.make_config(4, 100, 8, 2, 64)
    assert L.moe_stage_workspace_size(ctypes.byref(bad), ctypes.byref(n)) == 2 and n.value == 7
    assert L.moe_stage_workspace_size(None, ctypes.byref(n)) == 1
    assert L.moe_stage_workspace_size(ctypes.byref(cfg()), None) == 1


def test_scratch_holds_each_buffer_once():
    """[a | b] and its gradient, h, rows of the experts' outputs (then of their gradient) and of the
    inputs' gradient, dw, and a workspace without room for a second copy of any of them."""
    for T, d, E, k, f in ((256, 128, 8, 2, 256), (4096, 4096, 8, 2, 14336), (8192, 2048, 128, 8, 768)):
        c, R = tde.make_config(T, d, E, k, f), T * k
        s = tde.MoEScratch(c, device="meta")
        ws = max(tde.moe_stage_workspace_size(c), tde.moe_norm_ws_size(T, d))
        assert held(s) == R * (2 * 4 * f + 2 * f + 2 * 2 * d) + 4 * R + ws


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_borrowing_layer_allocates_what_it_keeps(monkeypatch, fmt):
    """The routing and two checkpoints, also while it is made; the lender the full-size buffers once."""
    T, d, E, k, f = 4096, 4096, 8, 2, 1408
    c, r, R, made = cfg(T, d, E, k, f), tde.make_router(), T * k, []
    empty = torch.empty

    def counted(*a, **kw):
        t = empty(*a, **kw)
        made.append(t.numel() * t.element_size())
        return t
    monkeypatch.setattr(torch, "empty", counted)
    lender = tde.Fp8MoELayer(c, r, device="meta", checkpoint=fmt)
    total = sum(made)
    assert total == held(lender)
    made.clear()
    borrower = tde.Fp8MoELayer(c, r, device="meta", checkpoint=fmt, scratch=lender)
    routing = 4 * (5 * R + 3 * E + 1) + R
    checkpoints = R * (2 * f + d) + R * 4 * (-(-2 * f // 128) + d // 128)
    assert sum(made) == held(borrower, lender) == routing + checkpoints
    # full-size: bf16 [a | b], h, dh, rows of d three times; codes of x, h, dy, dab both ways
    B = tde.moe_fp8_token_blocks(R, E)
    bf16 = 2 * R * (2 * f + f + f + 3 * d) + 4 * R
    codes = R * (2 * d + 3 * f) + 4 * R * (2 * (d // 128) + f // 128 + 2 * f // 128)
    codes_t = 128 * B * (2 * d + 3 * f) + 4 * B * (2 * d + 3 * f)
    ws = max(tde.moe_stage_workspace_size(c), tde.moe_norm_ws_size(T, d))
    assert total == routing + checkpoints + bf16 + codes + codes_t + ws
