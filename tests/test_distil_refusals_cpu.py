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
BWD = dict(logits=P, dtype=0, T=2, V=100, ld=100, ids=P, n=3, temperature=1.0, state=P, glp=P, gh=P, ti=P, top=4, gt=P, out=P + 4096, gd=0, ldg=100, status=P)
SIZES = [dict(T=-1), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25), dict(ld=99), dict(n=-1), dict(n=1025), dict(top=-1), dict(top=129), dict(temperature=0.0),
         dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=float("nan")), dict(temperature=1e-39), dict(dtype=2), dict(logits=0), dict(logits=P + 1),
         dict(dtype=1, logits=P + 2), dict(ids=0), dict(ids=P + 2), dict(status=P + 1), dict(state=P + 8)]


@pytest.mark.parametrize("change", SIZES + [dict(lp=0), dict(lp=P + 2), dict(ent=P + 1), dict(ti=0), dict(ti=P + 2), dict(tl=0), dict(tl=P + 2)], ids=str)
def test_token_logprobs_refuses(lib, change):
    a = {**FWD, **change}
    assert lib.rlk_token_logprobs_fwd(*a.values(), None) == BAD


@pytest.mark.parametrize("change", SIZES + [dict(state=0), dict(glp=P + 2), dict(gh=P + 1), dict(ti=0), dict(ti=P + 2), dict(gt=0), dict(gt=P + 2), dict(out=0), dict(out=P), dict(out=P + 1),
                                            dict(gd=1, out=P + 2), dict(gd=3), dict(ldg=99)], ids=str)
def test_token_logprobs_backward_refuses(lib, change):
    a = {**BWD, **change}
    assert lib.rlk_token_logprobs_bwd(*a.values(), None) == BAD


GATED = dict(x=P, ldx=64, wg=P, ldwg=64, wu=P, ldwu=64, bg=P, bu=P, bdt=1, M=8, N=32, K=64, act=2, y=P, ydt=0, ldy=32, g=P, u=P, ldz=32, ws=0, wsb=0)
GATED_BWD = dict(dy=P, lddy=32, x=P, ldx=64, ck=None, wg=P, ldwg=64, wu=P, ldwu=64, g=P, ldg=32, u=P, ldu=32, M=8, N=32, K=64, act=2, dx=P, dxt=0, ldgx=64,
                 dwg=P, ldgwg=64, dwu=P, ldgwu=64, dwt=1, dbg=P, dbu=P, acc=0, ws=P, wsb=1 << 30)


@pytest.mark.parametrize("change", [dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=(1 << 24) + 1, ldy=1 << 25, ldz=1 << 25), dict(K=0), dict(ldx=63), dict(ldwg=63), dict(ldwu=63),
                                    dict(ldy=31), dict(ldz=31), dict(act=4), dict(act=-1), dict(bdt=2), dict(ydt=2), dict(x=0), dict(wg=0), dict(wu=0), dict(y=0), dict(x=P + 1),
                                    dict(wg=P + 1), dict(wu=P + 1), dict(bg=P + 2), dict(bu=P + 2), dict(y=P + 1), dict(ydt=1, y=P + 2), dict(g=0), dict(u=0), dict(g=P + 1),
                                    dict(u=P + 1)], ids=str)
def test_gated_linear_refuses(lib, change):
    assert lib.rlk_gated_linear_fwd(*{**GATED, **change}.values(), None) == BAD


def test_gated_linear_workspace(lib):
    for change in (dict(x=P + 2), dict(ldx=65), dict(wg=P + 2), dict(ldwg=66), dict(wu=P + 2), dict(ldwu=67)):
        assert lib.rlk_gated_linear_fwd(*{**GATED, **change}.values(), None) == 3
        assert lib.rlk_gated_linear_fwd(*{**GATED, **change, "ws": P + 8, "wsb": 1 << 30}.values(), None) == 3
    assert lib.rlk_gated_linear_bwd(*{**GATED_BWD, "ws": 0}.values(), None) == 3
    assert lib.rlk_gated_linear_bwd(*{**GATED_BWD, "wsb": 1000}.values(), None) == 3
    need = lib.rlk_workspace_size(rlk.OP_GATED_LINEAR, 8, 32, 64)
    assert need == 256 * ((8 * 64 * 2 + 255) // 256) + 2 * 32 * 64 * 2
    assert lib.rlk_workspace_size(rlk.OP_GATED_LINEAR, -1, 32, 64) == 0


@pytest.mark.parametrize("change", [dict(M=-1), dict(N=0), dict(K=0), dict(act=4), dict(lddy=31), dict(ldx=63), dict(ldwg=63), dict(ldwu=63), dict(ldg=31), dict(ldu=31),
                                    dict(ldgx=63), dict(ldgwg=63), dict(ldgwu=63), dict(dxt=2), dict(dwt=2), dict(dy=0), dict(x=0), dict(wg=0), dict(wu=0), dict(g=0), dict(u=0),
                                    dict(dy=P + 1), dict(x=P + 1), dict(wg=P + 1), dict(wu=P + 1), dict(g=P + 1), dict(u=P + 1), dict(dx=P + 1), dict(dwg=P + 2), dict(dwu=P + 2),
                                    dict(dwg=0), dict(dwu=0), dict(dbg=0), dict(dbu=0), dict(dbg=P + 2), dict(dbu=P + 2)], ids=str)
def test_gated_linear_backward_refuses(lib, change):
    assert lib.rlk_gated_linear_bwd(*{**GATED_BWD, **change}.values(), None) == BAD


def test_gated_linear_backward_accumulates_in_fp32_only(lib):
    assert lib.rlk_gated_linear_bwd(*{**GATED_BWD, "acc": 1, "dwt": 0}.values(), None) == 2


COEF = (ctypes.c_float * 3)(3.4445, -4.7750, 2.0315)
ORTH = dict(g=P, dtype=0, B=2, m=8, n=16, ldg=16, stride=128, steps=5, coef=COEF, eps=1e-7, out=P, ldo=16, ostride=128, status=P, ws=P, wsb=1 << 30)


@pytest.mark.parametrize("change", [dict(dtype=2), dict(B=-1), dict(B=65536), dict(m=0), dict(m=65537), dict(n=0), dict(n=65537, ldg=70000, ldo=70000), dict(ldg=15), dict(ldo=15),
                                    dict(stride=-1), dict(ostride=127), dict(steps=0), dict(steps=65), dict(coef=None), dict(coef=(ctypes.c_float * 3)(1, 17, 0)),
                                    dict(coef=(ctypes.c_float * 3)(float("nan"), 0, 0)), dict(eps=-1.0), dict(eps=float("nan")), dict(g=0), dict(out=0), dict(g=P + 1),
                                    dict(dtype=1, g=P + 2), dict(out=P + 1), dict(status=P + 2)], ids=lambda c: "-".join(c))
def test_orthogonalise_refuses(lib, change):
    assert lib.rlk_orthogonalise(*{**ORTH, **change}.values(), None) == BAD


def test_orthogonalise_workspace(lib):
    need = lib.rlk_workspace_size(rlk.OP_ORTHOGONALISE, 2, 8, 16)
    assert need >= 2 * (4 * 8 * 16 * 2 + 2 * 8 * 8 * 2)
    for change in (dict(ws=0), dict(ws=P + 8), dict(wsb=need - 1)):
        assert lib.rlk_orthogonalise(*{**ORTH, **change}.values(), None) == 3
    assert lib.rlk_workspace_size(rlk.OP_ORTHOGONALISE, 70000, 8, 16) == 0


def test_nothing_to_do(lib):
    assert lib.rlk_orthogonalise(*{**ORTH, "B": 0, "g": 0, "ws": 0}.values(), None) == OK
    assert lib.rlk_gated_linear_fwd(*{**GATED, "M": 0, "x": 0}.values(), None) == OK
    assert lib.rlk_gated_linear_bwd(*{**GATED_BWD, "M": 0, "dwg": 0, "dwu": 0, "dbg": 0, "dbu": 0}.values(), None) == OK
    assert lib.rlk_token_logprobs_fwd(*{**FWD, "T": 0, "logits": 0}.values(), None) == OK
    assert lib.rlk_token_logprobs_bwd(*{**BWD, "T": 0, "logits": 0}.values(), None) == OK


def test_injected_failures(lib):
    for call, args in ((lib.rlk_token_logprobs_fwd, FWD), (lib.rlk_token_logprobs_bwd, BWD), (lib.rlk_gated_linear_fwd, GATED),
                       (lib.rlk_gated_linear_bwd, GATED_BWD), (lib.rlk_orthogonalise, ORTH)):
        rlk.inject_launch_failures(1)
        assert call(*args.values(), None) == 4
    assert rlk.inject_launch_failures(0) == 0


def test_constants():
    header = open(rlk.LIB_PATH.rsplit("/", 2)[0] + "/include/rlk.h").read()
    assert f"#define RLK_MAX_TOKENS {rlk.MAX_TOKENS} " in header and f"#define RLK_MAX_ALTERNATIVES {rlk.MAX_ALTERNATIVES} " in header
    assert ctypes.sizeof(ctypes.c_float) * 4 == 16
