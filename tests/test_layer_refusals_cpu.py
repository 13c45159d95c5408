"""What the layers' entry points accept, on the host: a misaligned pointer to what the
kernels read or write four bytes at a time is an invalid argument, and a linear
layer's backward needs the workspace that it uses and no more."""
import ctypes

import pytest

import entropy_logits_bf16_gb300 as rlk

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)   # never dereferenced: a launch is made to fail


@pytest.fixture
def lib():
    """A launch would return the injected CUDA error (4): refusals come first."""
    rlk.build()
    lib = rlk.load()
    lib.rlk_debug_inject_launch_failures(1000)
    yield lib
    lib.rlk_debug_inject_launch_failures(0)


def ckpt():
    return ctypes.byref(rlk.CheckpointBuffers(0x10000, 0x10000, 112, 4))


@pytest.mark.parametrize("at", [None, "status"])
def test_checkpoint_pack(lib, at):
    p = {"status": FAKE, at: ODD}
    assert lib.rlk_checkpoint_pack(FAKE, 0, 4, 100, 100, ckpt(), p["status"], None) == (1 if at else 4)


@pytest.mark.parametrize("at", [None, "mean", "rstd", "status"])
def test_norm_fwd(lib, at):
    p = {"mean": FAKE, "rstd": FAKE, "status": FAKE, at: ODD}
    assert lib.rlk_norm_fwd(FAKE, 0, 4, 100, 100, FAKE, FAKE, 1, 0, 1e-5, FAKE, 0, 100, p["mean"], p["rstd"], None,
                            p["status"], None) == (1 if at else 4)


@pytest.mark.parametrize("at", [None, "mean", "rstd", "dw", "db"])
def test_norm_bwd(lib, at):
    p = {"mean": FAKE, "rstd": FAKE, "dw": FAKE, "db": FAKE, at: ODD}
    assert lib.rlk_norm_bwd(FAKE, 1, 100, FAKE, 0, 100, None, 4, 100, FAKE, 1, 0, p["mean"], p["rstd"], FAKE, 0, 100,
                            p["dw"], p["db"], 0, FAKE, 1 << 20, None) == (1 if at else 4)


@pytest.mark.parametrize("at", [None, "loss", "grad", "reward", "stats"])
def test_preference_loss(lib, at):
    p = {"loss": FAKE, "grad": FAKE, "reward": FAKE, "stats": FAKE, at: ODD}
    config = ctypes.byref(rlk.PrefConfig(0, 0.1, 0.0, 0.0, 0))
    assert lib.rlk_preference_loss(FAKE, FAKE, None, FAKE, 2, 50, config, p["loss"], p["grad"], p["reward"], p["stats"],
                                   FAKE, 1 << 20, None) == (1 if at else 4)


def linear_bwd(lib, M, N, K, ws_bytes, dx=FAKE, dw=FAKE, db=FAKE):
    """Aligned operands, no activation: nothing is copied."""
    pad = (N + 7) // 8 * 8, (K + 7) // 8 * 8
    return lib.rlk_linear_bwd(FAKE, pad[0], FAKE, pad[1], None, FAKE, pad[1], None, 0, M, N, K, 0, dx, 0, pad[1], dw, 1,
                              pad[1], db, 0, FAKE, ws_bytes, None)


@pytest.mark.parametrize("M,N", [(1, 64), (5, 1 << 20), (64, 4099), (1215, 4096), (1216, 4096), (1217, 4096), (16384, 4096)])
def test_the_bias_gradients_partial_sums_take_rows_into_account(lib, M, N):
    """A partial sum covers four rows or more, and there are 304 at most."""
    most = min(304, -(-M // 4)) * ((N + 7) // 8 * 8) * 4
    need = -(-most // 256) * 256
    assert linear_bwd(lib, M, N, 64, need) == 4 and linear_bwd(lib, M, N, 64, need - 1) == 3
    copies = sum(-(-rows * ((cols + 7) // 8 * 8) * 2 // 256) * 256 for rows, cols in ((M, N), (M, 64), (N, 64)))
    assert lib.rlk_workspace_size(rlk.OP_LINEAR_BWD, M, N, 64) == copies + need
