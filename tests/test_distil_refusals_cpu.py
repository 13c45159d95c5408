"""What the entry points of a distillation step's operators refuse, before any launch."""
import ctypes

import pytest

import entropy_logits_bf16_gb300 as rlk

OK, BAD = 0, 1
P = 1 << 20   # a pointer that is never looked at: every call here is refused, or has nothing to do


@pytest.fixture(scope="module")
def lib():
    rlk.build()
    return rlk.load()


FWD = dict(logits=P, dtype=0, T=2, V=100, ld=100, ids=P, n=3, temperature=1.0, top=4, lp=P, ent=P, ti=P, tl=P, state=P, status=P)
BWD = dict(logits=P, dtype=0, T=2, V=100, ld=100, ids=P, n=3, temperature=1.0, state=P, glp=P, gh=P, ti=P, top=4, gt=P, out=P, gd=0, ldg=100, status=P)
SIZES = [dict(T=-1), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25), dict(ld=99), dict(n=-1), dict(n=1025), dict(top=-1), dict(top=129), dict(temperature=0.0),
         dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=float("nan")), dict(temperature=1e-39), dict(dtype=2), dict(logits=0), dict(logits=P + 1),
         dict(dtype=1, logits=P + 2), dict(ids=0), dict(ids=P + 2), dict(status=P + 1), dict(state=P + 8)]


@pytest.mark.parametrize("change", SIZES + [dict(lp=0), dict(lp=P + 2), dict(ent=P + 1), dict(ti=0), dict(ti=P + 2), dict(tl=0), dict(tl=P + 2)], ids=str)
def test_token_logprobs_refuses(lib, change):
    a = {**FWD, **change}
    assert lib.rlk_token_logprobs_fwd(*a.values(), None) == BAD


@pytest.mark.parametrize("change", SIZES + [dict(state=0), dict(glp=P + 2), dict(gh=P + 1), dict(ti=0), dict(ti=P + 2), dict(gt=0), dict(gt=P + 2), dict(out=0), dict(out=P + 1),
                                            dict(gd=1, out=P + 2), dict(gd=3), dict(ldg=99)], ids=str)
def test_token_logprobs_backward_refuses(lib, change):
    a = {**BWD, **change}
    assert lib.rlk_token_logprobs_bwd(*a.values(), None) == BAD


def test_no_rows(lib):
    assert lib.rlk_token_logprobs_fwd(*{**FWD, "T": 0, "logits": 0}.values(), None) == OK
    assert lib.rlk_token_logprobs_bwd(*{**BWD, "T": 0, "logits": 0}.values(), None) == OK


def test_injected_failures(lib):
    for call, args in ((lib.rlk_token_logprobs_fwd, FWD), (lib.rlk_token_logprobs_bwd, BWD)):
        rlk.inject_launch_failures(1)
        assert call(*args.values(), None) == 4
    assert rlk.inject_launch_failures(0) == 0


def test_constants():
    header = open(rlk.LIB_PATH.rsplit("/", 2)[0] + "/include/rlk.h").read()
    assert f"#define RLK_MAX_TOKENS {rlk.MAX_TOKENS} " in header and f"#define RLK_MAX_ALTERNATIVES {rlk.MAX_ALTERNATIVES} " in header
    assert ctypes.sizeof(ctypes.c_float) * 4 == 16
