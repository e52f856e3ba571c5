"""Layers that lend and borrow their full-size buffers: forward and backward of both in the order of a
training step give bit by bit what layers with buffers of their own give; and what they write of their workspace."""

import pytest
import torch

import token_dispatch_expert_gb300 as tde

pytestmark = pytest.mark.gpu


def both_ways(layers, batches, weights):
    """Forward of all, backward of all in reverse."""
    ys = [m.forward(lg, x, *w) for m, (lg, x, _), w in zip(layers, batches, weights)]
    gs = [None] * len(layers)
    for i in reversed(range(len(layers))):
        lg, x, dy = batches[i]
        gs[i] = layers[i].backward(lg, x, dy, *weights[i])
    assert all(m.status() == (0, 0) for m in layers)
    return ys, gs


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_layers_that_share_scratch(kind, fmt):
    T, d, E, k, f = 230, 256, 8, 2, 192
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    cfg, router = tde.make_config(T, d, E, k, f), tde.make_router("softmax")

    def new(lender):
        if kind == "fp8":
            return tde.Fp8MoELayer(cfg, router, checkpoint=fmt, scratch=lender)
        return tde.CheckpointedMoELayer(tde.MoEScratch(cfg) if lender is None else lender.scratch, fmt)
    owners = [new(None) for _ in range(3)]
    sharing = [new(None)]
    sharing += [new(sharing[0]) for _ in range(2)]
    weights = [(0.2 * rand(E, 2 * f, d)).bfloat16() for _ in owners], [(0.2 * rand(E, d, f)).bfloat16() for _ in owners]
    weights = list(zip(*weights))
    if kind == "fp8":
        weights = [(owners[0].quantize_weights(*w),) for w in weights]
    batches = [(rand(T, E), rand(T, d).bfloat16(), rand(T, d).bfloat16()) for _ in owners]
    (ys, gs), (yo, go) = both_ways(sharing, batches, weights), both_ways(owners, batches, weights)
    for i in range(3):
        assert torch.equal(ys[i], yo[i]) and bool(ys[i].any())
        assert set(gs[i]) == {"dx", "dW1", "dW2", "dlogits"}
        for n in gs[i]:
            assert torch.equal(gs[i][n], go[i][n]) and bool(gs[i][n].any()), (i, n)


@pytest.mark.parametrize("T,E,k,kw", [(300, 8, 2, {}), (1, 4, 1, {}), (257, 64, 6, dict(capacity=20, drop_by_score=True)),
                                      (513, 256, 8, dict(gate="sigmoid", drop_negative=True))])
def test_stages_stay_in_their_workspace(T, E, k, kw):
    """Nothing is written behind moe_stage_workspace_size, and the layer is right whatever it holds."""
    d, f = 128, 64
    c = tde.make_config(T, d, E, k, f, **kw)
    n, room = tde.moe_stage_workspace_size(c), 1 << 20
    rand = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    lg, x, dy = rand(T, E), rand(T, d).bfloat16(), rand(T, d).bfloat16()
    W1, W2 = (0.2 * rand(E, 2 * f, d)).bfloat16(), (0.2 * rand(E, d, f)).bfloat16()
    out = []
    for fill in (0xa5, 0x3c):
        scratch = tde.MoEScratch(c)
        buf = torch.full((n + room,), fill, dtype=torch.uint8, device="cuda")
        scratch.ws = buf[:n]
        tde.moe_ws_init(scratch.ws)
        m = tde.CheckpointedMoELayer(scratch)
        y = m.forward(lg, x, W1, W2)
        g = m.backward(lg, x, dy, W1, W2)
        assert m.status() == (0, 0)
        assert (buf[n:] == fill).all()
        out.append([y, *g.values()])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_status_of_a_norm():
    """The word of errors of its workspace, read and cleared, whose ever the workspace is."""
    scratch = tde.MoEScratch(tde.make_config(16, 64, 4, 1, 64))
    for n in (tde.MoENorm(16, 64), tde.MoENorm(16, 64, ws=scratch.ws)):
        assert n.status() == (0, 0)
        n.ws[:4].view(torch.int32).fill_(tde.DEVERR["TIMEOUT"])
        status, flags = n.status()
        assert tde.moe_status_string(status) == "MOE_ERR_TIMEOUT" and flags == tde.DEVERR["TIMEOUT"]
        assert n.status() == (0, 0)
