"""Refusals of the layer operators on the host, before any CUDA call, and the
binding's own argument checks."""
import ctypes
import math

import pytest
import torch

import entropy_logits_bf16_gb300 as rlk

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    rlk.build()
    return rlk.load()


@pytest.fixture
def armed(lib):
    """A launch would return the injected CUDA error (4): refusals come first."""
    lib.rlk_debug_inject_launch_failures(1000)
    yield
    lib.rlk_debug_inject_launch_failures(0)


def ckpt(codes=0x10000, scales=0x10000, ldc=112, lds=4):
    return ctypes.byref(rlk.CheckpointBuffers(codes, scales, ldc, lds))


def pack(lib, **kw):
    a = dict(x=FAKE, dtype=0, T=4, H=100, ldx=100, ck=ckpt())
    a.update(kw)
    return lib.rlk_checkpoint_pack(a["x"], a["dtype"], a["T"], a["H"], a["ldx"], a["ck"], None, None)


def unpack(lib, **kw):
    a = dict(x=FAKE, dtype=0, T=4, H=100, ldx=100, ck=ckpt())
    a.update(kw)
    return lib.rlk_checkpoint_unpack(a["ck"], a["T"], a["H"], a["x"], a["dtype"], a["ldx"], None)


CKPT_BAD = [dict(T=-1), dict(H=0), dict(H=(1 << 20) + 1, ldx=1 << 21), dict(ldx=99), dict(dtype=2), dict(x=None),
            dict(x=ODD), dict(ck=None), dict(ck=ckpt(codes=None)), dict(ck=ckpt(scales=None)),
            dict(ck=ckpt(codes=0x10008)), dict(ck=ckpt(ldc=96)), dict(ck=ckpt(ldc=104)), dict(ck=ckpt(lds=3))]


@pytest.mark.parametrize("kw", CKPT_BAD)
def test_checkpoint_rejects(lib, armed, kw):
    assert pack(lib, **kw) == 1 and unpack(lib, **kw) == 1


def test_checkpoint_accepts(lib, armed):
    assert pack(lib) == 4 and unpack(lib) == 4
    assert pack(lib, T=0, x=None, ck=None) == 0 and unpack(lib, T=0, x=None, ck=None) == 0


def norm_fwd(lib, **kw):
    a = dict(x=FAKE, dtype=0, T=4, H=100, ldx=100, w=FAKE, b=FAKE, pd=1, kind=0, eps=1e-5, y=FAKE, yd=0, ldy=100,
             mean=FAKE, rstd=FAKE, ck=None)
    a.update(kw)
    return lib.rlk_norm_fwd(a["x"], a["dtype"], a["T"], a["H"], a["ldx"], a["w"], a["b"], a["pd"], a["kind"], a["eps"],
                            a["y"], a["yd"], a["ldy"], a["mean"], a["rstd"], a["ck"], None, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(H=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21), dict(ldx=99), dict(ldy=99), dict(dtype=2),
    dict(pd=3), dict(yd=-1), dict(kind=2), dict(eps=-1e-5), dict(eps=math.nan), dict(eps=math.inf), dict(x=None),
    dict(y=None), dict(x=ODD), dict(y=ODD), dict(w=ctypes.c_void_p(0x10002)), dict(b=ODD), dict(ck=ckpt(ldc=96))])
def test_norm_fwd_rejects(lib, armed, kw):
    assert norm_fwd(lib, **kw) == 1


def test_norm_fwd_accepts(lib, armed):
    assert norm_fwd(lib) == 4
    assert norm_fwd(lib, w=None, b=None, mean=None, rstd=None, ck=ckpt()) == 4
    assert norm_fwd(lib, T=0, x=None, y=None) == 0


def norm_bwd(lib, **kw):
    a = dict(dy=FAKE, dd=1, lddy=100, x=FAKE, dtype=0, ldx=100, ck=None, T=4, H=100, w=FAKE, pd=1, kind=0, mean=FAKE,
             rstd=FAKE, dx=FAKE, gd=0, ldg=100, dw=FAKE, db=FAKE, acc=0, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.rlk_norm_bwd(a["dy"], a["dd"], a["lddy"], a["x"], a["dtype"], a["ldx"], a["ck"], a["T"], a["H"], a["w"],
                            a["pd"], a["kind"], a["mean"], a["rstd"], a["dx"], a["gd"], a["ldg"], a["dw"], a["db"],
                            a["acc"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(lddy=99), dict(ldx=99), dict(ldg=99), dict(dd=2), dict(dtype=2), dict(gd=2), dict(pd=2),
    dict(kind=5), dict(dy=None), dict(dx=None), dict(rstd=None), dict(mean=None), dict(x=None), dict(ck=ckpt()),
    dict(x=None, ck=ckpt(ldc=96)), dict(dy=ctypes.c_void_p(0x10002)), dict(dx=ODD), dict(x=ODD), dict(dw=ODD)])
def test_norm_bwd_rejects(lib, armed, kw):
    assert norm_bwd(lib, **kw) == 1


def test_norm_bwd_workspace_and_accepts(lib, armed):
    need = lib.rlk_workspace_size(rlk.OP_NORM_BWD, 4, 100, 0)
    assert need >= 4 * 2 * 100 * 4 and need % 256 == 0
    assert norm_bwd(lib, ws=None) == 3 and norm_bwd(lib, wsb=need - 1) == 3 and norm_bwd(lib, ws=ctypes.c_void_p(0x10008)) == 3
    assert norm_bwd(lib, wsb=need) == 4
    assert norm_bwd(lib, kind=1, mean=None, x=None, ldx=0, ck=ckpt(), w=None) == 4
    assert norm_bwd(lib, dw=None, db=None, ws=None, wsb=0) == 4
    assert norm_bwd(lib, T=0, dw=None, db=None, ws=None, wsb=0) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(4, 64)
    for call in (lambda: rlk.norm(x), lambda: rlk.checkpoint_pack(x), lambda: rlk.norm_backward(x, x, None, None, None),
                 lambda: rlk.new_checkpoint(4, 64, "cpu")):
        with pytest.raises(ValueError):
            call()


def pref(lib, n_pairs=2, n_tok=50, cfg=(0, 0.1, 0.0, 0.0, 0), lp=FAKE, ref=FAKE, off=FAKE, loss=FAKE, grad=FAKE,
         reward=FAKE, ws=FAKE, wsb=1 << 20):
    c = None if cfg is None else ctypes.byref(rlk.PrefConfig(*cfg))
    return lib.rlk_preference_loss(lp, ref, None, off, n_pairs, n_tok, c, loss, grad, reward, None, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(cfg=None), dict(cfg=(3, 0.1, 0, 0, 0)), dict(cfg=(0, 0.0, 0, 0, 0)), dict(cfg=(0, math.nan, 0, 0, 0)),
    dict(cfg=(0, 0.1, 0.5, 0, 0)), dict(cfg=(0, 0.1, -0.1, 0, 0)), dict(cfg=(1, 0.1, 0.1, 0, 0)),
    dict(cfg=(0, 0.1, 0, math.inf, 0)), dict(n_pairs=-1), dict(n_pairs=(1 << 24) + 1), dict(n_tok=-1), dict(n_tok=1 << 31),
    dict(lp=None), dict(off=None), dict(loss=None), dict(lp=ODD), dict(ref=ODD), dict(grad=ODD), dict(off=ODD)])
def test_preference_rejects(lib, armed, kw):
    assert pref(lib, **kw) == 1


def test_preference_workspace_and_accepts(lib, armed):
    need = lib.rlk_workspace_size(rlk.OP_PREFERENCE_LOSS, 50, 2, 0)
    assert need % 256 == 0 and need > 0
    assert pref(lib, ws=None) == 3 and pref(lib, wsb=need - 1) == 3 and pref(lib, ws=ctypes.c_void_p(0x10008)) == 3
    assert pref(lib, wsb=need) == 4 and pref(lib, ref=None, grad=None, reward=None) == 4 and pref(lib, n_tok=0, lp=None) == 4


def test_preference_binding_refuses():
    x = torch.zeros(4)
    with pytest.raises(ValueError):
        rlk.preference_loss(x, None, torch.zeros(3, dtype=torch.int32))


def lin(lib, **kw):
    a = dict(x=FAKE, ldx=64, w=FAKE, ldw=64, b=FAKE, bd=1, r=FAKE, ldr=32, M=5, N=32, K=64, act=1, y=FAKE, yd=0, ldy=32,
             z=FAKE, ldz=32, ws=None, wsb=0)
    a.update(kw)
    return lib.rlk_linear_fwd(a["x"], a["ldx"], a["w"], a["ldw"], a["b"], a["bd"], a["r"], a["ldr"], a["M"], a["N"], a["K"],
                              a["act"], a["y"], a["yd"], a["ldy"], a["z"], a["ldz"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(M=1 << 31), dict(N=0), dict(K=0), dict(N=(1 << 24) + 1, ldy=1 << 25, ldr=1 << 25, ldz=1 << 25),
    dict(K=(1 << 24) + 1, ldx=1 << 25, ldw=1 << 25), dict(act=4), dict(act=-1), dict(bd=2), dict(yd=2), dict(ldx=63), dict(ldw=63),
    dict(ldy=31), dict(ldr=31), dict(ldz=31), dict(x=None), dict(w=None), dict(y=None), dict(x=ODD), dict(w=ODD), dict(y=ODD),
    dict(z=ODD), dict(r=ODD), dict(b=ctypes.c_void_p(0x10002)), dict(y=ctypes.c_void_p(0x10002), yd=1)])
def test_linear_rejects(lib, armed, kw):
    assert lin(lib, **kw) == 1


def test_linear_workspace_and_accepts(lib, armed):
    assert lin(lib) == 4 and lin(lib, b=None, r=None, z=None, ldr=0, ldz=0) == 4 and lin(lib, M=0, x=None, w=None, y=None) == 0
    need = lib.rlk_workspace_size(rlk.OP_LINEAR, 5, 32, 64)
    for odd in (dict(x=ctypes.c_void_p(0x10002)), dict(ldx=65), dict(ldw=66)):
        assert lin(lib, **odd) == 3 and lin(lib, **odd, ws=FAKE, wsb=need) == 4
        assert lin(lib, **odd, ws=ctypes.c_void_p(0x10008), wsb=need) == 3 and lin(lib, **odd, ws=FAKE, wsb=16) == 3


def lin_bwd(lib, **kw):
    a = dict(dy=FAKE, lddy=32, x=FAKE, ldx=64, ck=None, w=FAKE, ldw=64, z=FAKE, ldz=32, M=4, N=32, K=64, act=1, dx=FAKE, xd=0,
             ldgx=64, dw=FAKE, wd=1, ldgw=64, db=FAKE, acc=0, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.rlk_linear_bwd(a["dy"], a["lddy"], a["x"], a["ldx"], a["ck"], a["w"], a["ldw"], a["z"], a["ldz"], a["M"], a["N"],
                              a["K"], a["act"], a["dx"], a["xd"], a["ldgx"], a["dw"], a["wd"], a["ldgw"], a["db"], a["acc"],
                              a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=0), dict(K=0), dict(act=9), dict(xd=2), dict(wd=2), dict(lddy=31), dict(ldx=63), dict(ldw=63),
    dict(ldz=31), dict(ldgx=63), dict(ldgw=63), dict(dy=None), dict(x=None), dict(ck=ckpt()), dict(x=None, ck=ckpt(ldc=48)),
    dict(w=None), dict(z=None), dict(dy=ODD), dict(x=ODD), dict(w=ODD), dict(z=ODD), dict(dx=ODD), dict(dw=ODD), dict(db=ODD)])
def test_linear_bwd_rejects(lib, armed, kw):
    assert lin_bwd(lib, **kw) == 1


def test_linear_bwd_workspace_and_accepts(lib, armed):
    need = lib.rlk_workspace_size(rlk.OP_LINEAR_BWD, 4, 32, 64)
    assert need % 256 == 0 and lin_bwd(lib, wsb=need) == 4
    assert lin_bwd(lib, ws=None) == 3 and lin_bwd(lib, wsb=256) == 3 and lin_bwd(lib, ws=ctypes.c_void_p(0x10008)) == 3
    assert lin_bwd(lib, act=0, z=None, db=None, ws=None, wsb=0) == 4            # no copies, no partial sums
    assert lin_bwd(lib, x=None, ldx=0, ck=ckpt(), acc=1) == 4
    assert lin_bwd(lib, dw=None, x=None, ldx=0) == 4 and lin_bwd(lib, dx=None, w=None) == 4
    assert lin_bwd(lib, acc=1, wd=0) == 2
    assert lin_bwd(lib, dx=None, dw=None, db=None) == 0 and lin_bwd(lib, M=0, dy=None, dw=None, db=None) == 0
