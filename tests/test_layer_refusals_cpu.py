"""Refusals of pointers that the layer operators' kernels read or write four bytes
at a time: a misaligned one is an invalid argument, on the host."""
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
