"""What the normalisation and the 8-bit checkpoints refuse before anything is enqueued, through the
C ABI and through the binding.  CPU only."""

import ctypes

import pytest
import torch

import token_dispatch_expert_gb300 as tde
from token_dispatch_expert_gb300 import _CkptC, _NormC

P = 4096   # a non-null, 16-byte aligned stand-in for a device address: never dereferenced
INVALID, UNSUPPORTED, OK = 1, 2, 0


@pytest.fixture(scope="module")
def L():
    tde.build()
    return tde.lib()


NORM = dict(rows=10, C=100, kind=0, eps=1e-5, x_type=0, y_type=0, p_type=1, g_type=1, format=0,
            ldx=100, ld_add=100, ld_y=100, ld_out=100, ld_codes=112)


def norm(**kw):
    return _NormC(*{**NORM, **kw}.values())


def call_norm(L, p, **kw):
    a = dict(x=P, residual=P, gamma=P, beta=P, y=P, total=P, mean=P, rstd=P, codes=P, scales=P)
    a.update(kw)
    return L.moe_norm(ctypes.addressof(p) if p else None, *a.values(), None)


def call_bwd(L, p, **kw):
    a = dict(dy=P, x=P, x_scales=P, mean=P, rstd=P, gamma=P, add=P, dx=P, dgamma=P, dbeta=P, ws=P)
    a.update(kw)
    return L.moe_norm_bwd(ctypes.addressof(p) if p else None, *a.values(), None)


def call_restore(L, p, **kw):
    a = dict(codes=P, scales=P, mean=P, rstd=P, gamma=P, beta=P, y=P)
    a.update(kw)
    return L.moe_ckpt_norm(ctypes.addressof(p) if p else None, *a.values(), None)


SIZES = [(dict(rows=-1), INVALID), (dict(C=0), INVALID), (dict(C=1 << 24), UNSUPPORTED),
         (dict(rows=2**31), UNSUPPORTED), (dict(kind=2), INVALID), (dict(kind=-1), INVALID),
         (dict(x_type=2), INVALID), (dict(y_type=-1), INVALID), (dict(p_type=3), INVALID),
         (dict(g_type=2), INVALID), (dict(format=2), INVALID), (dict(ld_codes=96), INVALID),
         (dict(ld_codes=104), INVALID), (dict(ld_y=99), INVALID)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(ldx=99), INVALID), (dict(ld_add=99), INVALID), (dict(ld_out=99), INVALID)])
def test_norm_sizes(L, kw, status):
    assert call_norm(L, norm(**kw)) == status


@pytest.mark.parametrize("kw,status", SIZES + [(dict(ld_add=99), INVALID), (dict(ld_out=99), INVALID)])
def test_norm_bwd_sizes(L, kw, status):
    assert call_bwd(L, norm(**kw)) == status


@pytest.mark.parametrize("kw,status", SIZES)
def test_ckpt_norm_sizes(L, kw, status):
    assert call_restore(L, norm(**kw)) == status


def test_norm_pointers(L):
    assert call_norm(L, None) == call_bwd(L, None) == call_restore(L, None) == INVALID
    for kw in (dict(x=None), dict(x=P + 1), dict(y=None), dict(y=P + 1), dict(residual=None),
               dict(residual=P + 1), dict(total=P + 1), dict(gamma=P + 4), dict(beta=P + 8),
               dict(mean=P + 4), dict(rstd=P + 4), dict(codes=None), dict(scales=None),
               dict(codes=P + 8), dict(scales=P + 4)):
        assert call_norm(L, norm(), **kw) == INVALID, kw
    # fp32 rows need four bytes
    assert call_norm(L, norm(x_type=1), x=P + 2) == INVALID
    assert call_norm(L, norm(y_type=1), y=P + 2) == INVALID
    assert call_norm(L, norm(kind=1)) == INVALID              # the RMS norm has no mean
    for kw in (dict(dy=None), dict(dy=P + 1), dict(x=None), dict(x=P + 8), dict(x_scales=P + 4),
               dict(mean=None), dict(mean=P + 4), dict(rstd=None), dict(rstd=P + 4), dict(gamma=P + 4),
               dict(add=P + 1), dict(dx=None), dict(dx=P + 1), dict(dgamma=P + 4), dict(dbeta=P + 4),
               dict(ws=None), dict(ws=P + 4), dict(x=P + 1, x_scales=None), dict(x=None, x_scales=None)):
        assert call_bwd(L, norm(), **kw) == INVALID, kw
    assert call_bwd(L, norm(kind=1)) == INVALID
    assert call_bwd(L, norm(ldx=99), x_scales=None) == INVALID
    for kw in (dict(codes=None), dict(codes=P + 8), dict(scales=None), dict(mean=None),
               dict(rstd=None), dict(gamma=P + 4), dict(beta=P + 4), dict(y=None), dict(y=P + 1)):
        assert call_restore(L, norm(), **kw) == INVALID, kw
    assert call_restore(L, norm(kind=1)) == INVALID


def test_no_rows(L):
    """Empty buffers may have no address; nothing is enqueued (there is no device here)."""
    none = dict.fromkeys(("x", "residual", "gamma", "beta", "y", "total", "mean", "rstd", "codes",
                          "scales"))
    assert call_norm(L, norm(rows=0), **none) == OK
    none = dict.fromkeys(("dy", "x", "x_scales", "mean", "rstd", "gamma", "add", "dx", "dgamma",
                          "dbeta", "ws"))
    assert call_bwd(L, norm(rows=0), **none) == OK
    none = dict.fromkeys(("codes", "scales", "mean", "rstd", "gamma", "beta", "y"))
    assert call_restore(L, norm(rows=0), **none) == OK


def test_workspace_size():
    assert tde.moe_norm_ws_size(1, 1) == 256 + 2 * 64 * 4
    assert tde.moe_norm_ws_size(10**6, 4096) == 256 + 608 * 2 * 4096 * 4
    assert tde.moe_norm_ws_size(0, 4096) == 256
    for bad in ((-1, 4), (4, 0), (4, 1 << 24), (1 << 31, 4)):
        assert tde.moe_norm_ws_size(*bad) == -1


CKPT = dict(rows=10, C=100, format=0, x_type=0, ldx=100, ld=112)


def ckpt(**kw):
    return _CkptC(*{**CKPT, **kw}.values())


CALLS = {"moe_ckpt_save": dict(x=P, live=P, codes=P, scales=P, ws=P),
         "moe_ckpt_load": dict(codes=P, scales=P, live=P, x=P, ws=P),
         "moe_ckpt_swiglu": dict(codes=P, scales=P, live=P, ab=P, h=P, ws=P),
         "moe_ckpt_swiglu_bwd": dict(dh=P, codes=P, scales=P, live=P, dab=P, h=P, ws=P)}


def call(L, name, p, **kw):
    return getattr(L, name)(ctypes.addressof(p) if p else None, *{**CALLS[name], **kw}.values(), None)


@pytest.mark.parametrize("name", CALLS)
def test_ckpt_refusals(L, name):
    assert call(L, name, None) == INVALID
    for kw, status in ((dict(rows=-1), INVALID), (dict(C=0), INVALID), (dict(C=1 << 24), UNSUPPORTED),
                       (dict(rows=2**31), UNSUPPORTED), (dict(format=2), INVALID),
                       (dict(x_type=2), INVALID), (dict(ld=96), INVALID), (dict(ld=104), INVALID)):
        assert call(L, name, ckpt(**kw)) == status, kw
    for arg in CALLS[name]:
        bad = (P + 2,) if arg == "live" else (P + 1,) if arg == "x" else (P + 4,)
        if arg not in ("live", "ab", "h"):
            bad += (None,)
        for b in bad:
            assert call(L, name, ckpt(), **{arg: b}) == INVALID, (arg, b)
    if "x" in CALLS[name]:
        assert call(L, name, ckpt(ldx=99)) == INVALID
        assert call(L, name, ckpt(x_type=1), x=P + 2) == INVALID
    else:
        assert call(L, name, ckpt(C=101, ldx=101)) == INVALID
    if name == "moe_ckpt_swiglu":
        assert call(L, name, ckpt(), ab=None, h=None) == INVALID
    none = dict.fromkeys(CALLS[name])
    assert call(L, name, ckpt(rows=0), **none) == OK


def test_combine_bwd_refusals(L):
    c = tde.make_config(64, 128, 32, 4, 128)

    def run(cfg=c, ld=128, fmt=0, **kw):
        a = dict(dy=P, codes=P, ld=ld, scales=P, fmt=fmt, topk_w=P, dest_row=P, dyp=P, dw=P, ws=P)
        a.update(kw)
        return L.moe_ckpt_combine_bwd(ctypes.addressof(cfg) if cfg else None, *a.values(), None)
    assert run(cfg=None) == run(ld=112) == run(ld=136) == run(fmt=2) == INVALID
    assert run(cfg=tde.make_config(64, 100, 32, 4, 128)) == UNSUPPORTED
    for arg in ("dy", "codes", "scales", "topk_w", "dest_row", "dyp", "dw", "ws"):
        assert run(**{arg: None}) == run(**{arg: P + 4}) == INVALID


# ------------------------------------------------------------------ the binding, on host tensors
F, B, I8 = torch.float32, torch.bfloat16, torch.int8


def z(*s, dt=B):
    return torch.zeros(s, dtype=dt)


@pytest.mark.parametrize("kw,message", [
    (dict(x=z(4, 8, dt=torch.float16)), "x: expected bfloat16 or float32"),
    (dict(x=z(8)), "x: expected a matrix"),
    (dict(x=z(8, 4).t()), "x: expected a matrix with adjacent"),
    (dict(), "expected a CUDA tensor")])
def test_norm_binding(kw, message):
    a = {**dict(x=z(4, 8), y=z(4, 8)), **kw}
    with pytest.raises(ValueError, match=message):
        tde.moe_norm(a["x"], a["y"])


class Dev(torch.Tensor):
    """A host tensor that says it is on the device: what a call refuses after asking for it."""
    is_cuda = True


def d(*s, dt=B):
    return z(*s, dt=dt).as_subclass(Dev)


@pytest.mark.parametrize("kw,message", [
    (dict(residual=d(4, 8, dt=F)), "residual: expected bfloat16"), (dict(residual=d(3, 8)), "residual: expected shape"),
    (dict(residual=d(4, 8), total=d(4, 8, dt=F)), "total: expected bfloat16"),
    (dict(gamma=d(7, dt=F)), "gamma: expected 8 elements"), (dict(gamma=d(8, dt=torch.float16)), "gamma: expected bfloat16 or"),
    (dict(gamma=d(8, dt=F), beta=d(8)), "beta: expected torch.float32"),
    (dict(mean=d(3, dt=F)), "mean: expected 4 elements"), (dict(rstd=d(4)), "rstd: expected float32"),
    (dict(kind="batch"), "kind: expected"), (dict(scales=d(4, 1, dt=F)), "scales: given without codes"),
    (dict(codes=d(4, 16, dt=torch.uint8), scales=d(4, 1, dt=F)), "codes: expected int8 or"),
    (dict(codes=d(5, 16, dt=I8), scales=d(4, 1, dt=F)), "codes: expected shape"),
    (dict(codes=d(4, 16, dt=I8), scales=d(4, 2, dt=F)), "scales: expected shape"),
    (dict(codes=d(4, 16, dt=I8), scales=d(4, 1)), "scales: expected float32")])
def test_norm_binding_types(kw, message):
    with pytest.raises(ValueError, match=message):
        tde.moe_norm(d(4, 8), d(4, 8), **kw)


def test_bwd_binding():
    v = d(4, dt=F)
    ok = dict(dy=d(4, 8), x=d(4, 8), mean=v, rstd=v, dx=d(4, 8), ws=d(4096, dt=torch.uint8))
    for kw, message in ((dict(x=d(4, 8, dt=F)), "x: expected bfloat16"), (dict(dx=d(4, 7)), "dx: expected shape"),
                        (dict(add=d(4, 8, dt=F)), "add: expected bfloat16"),
                        (dict(dgamma=d(7, dt=F)), "dgamma: expected 8"),
                        (dict(dgamma=d(8, dt=F), dbeta=d(8)), "dbeta: expected torch.float32"),
                        (dict(dgamma=d(8, dt=F), ws=d(256, dt=torch.uint8)), "ws: expected"),
                        (dict(scales=d(4, 1, dt=F)), "codes: expected int8")):
        with pytest.raises(ValueError, match=message):
            tde.moe_norm_bwd(**{**ok, **kw})


def test_ckpt_binding():
    c, s, ws = d(4, 16, dt=I8), d(4, 1, dt=F), d(256, dt=torch.uint8)
    for f, message in (
            (lambda: tde.moe_ckpt_save(d(4), c, s, ws=ws), "x: expected a matrix"),
            (lambda: tde.moe_ckpt_save(d(4, 16, dt=torch.float16), c, s, ws=ws), "x: expected bfloat16 or"),
            (lambda: tde.moe_ckpt_load(c, s, d(5, 16), ws=ws), "codes: expected shape"),
            (lambda: tde.moe_ckpt_save(d(4, 16), c, s, offsets=d(3, dt=torch.int64), ws=ws), "offsets: expected int32"),
            (lambda: tde.moe_ckpt_save(d(4, 16), c, s, offsets=d(0, dt=torch.int32), ws=ws), "offsets: expected at least"),
            (lambda: tde.moe_ckpt_swiglu(c, s, ws=ws), "ab, h: expected"),
            (lambda: tde.moe_ckpt_swiglu(c, s, d(4, 15), ws=ws), "ab: expected an even"),
            (lambda: tde.moe_ckpt_swiglu(c, s, d(4, 16), d(4, 16), ws=ws), "h: expected shape"),
            (lambda: tde.moe_ckpt_swiglu(c, s, d(4, 16, dt=F), ws=ws), "ab: expected bfloat16"),
            (lambda: tde.moe_ckpt_swiglu_bwd(d(4, 8), c, s, d(4, 8), ws=ws), "dab: expected shape"),
            (lambda: tde.moe_ckpt_swiglu_bwd(d(4, 8, dt=F), c, s, d(4, 16), ws=ws), "dh: expected bfloat16"),
            (lambda: tde.moe_ckpt_norm(c, s, d(4, dt=F), d(3, dt=F), d(4, 16)), "rstd: expected 4")):
        with pytest.raises(ValueError, match=message):
            f()
    cfg = tde.make_config(4, 64, 8, 1, 64)
    c, s, w = d(4, 64, dt=I8), d(4, 1, dt=F), d(4, dt=F)
    with pytest.raises(ValueError, match="dest_row: expected"):
        tde.moe_ckpt_combine_bwd(cfg, d(4, 64), c, s, w, d(4, dt=torch.int64), d(4, 64), w, ws)
    with pytest.raises(ValueError, match="dyp: expected 256 elements"):
        tde.moe_ckpt_combine_bwd(cfg, d(4, 64), c, s, w, d(4, dt=torch.int32), d(3, 64), w, ws)
