"""Log-probabilities of given tokens, entropy and top alternatives against 64 bits."""
import math

import pytest
import torch

from _distil import EPS32, HALF_ULP, tokens64, tokens_grad64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def logits(T, V, dtype, seed, kind="peaked"):
    g = torch.Generator().manual_seed(seed)
    z = 3.0 * torch.randn(T, V, generator=g)
    if kind == "peaked":
        z[torch.arange(T), torch.randint(0, V, (T,), generator=g)] += 9.0
    elif kind == "levels":
        z = torch.randint(-2, 3, (T, V), generator=g).float()        # long ties, zeros of both signs
        z[:, ::7] *= -1.0
    elif kind == "flat":
        z = torch.full((T, V), -1.25)
    elif kind == "up":
        z = torch.sort(z, dim=1)[0]
    elif kind == "down":
        z = torch.sort(z, dim=1, descending=True)[0]
    elif kind == "masked":
        z[torch.rand(T, V, generator=g) < 0.3] = -math.inf
    elif kind == "lowest":
        z[torch.rand(T, V, generator=g) < 0.3] = torch.finfo(dtype).min
    elif kind == "few":
        keep = torch.rand(T, V, generator=g) < 3.0 / V
        keep[:, V // 2] = True
        z[~keep] = -math.inf
    elif kind == "wide":
        z *= 1e4
    return z.to(dtype).cuda()


def given(T, V, C, seed):
    g = torch.Generator().manual_seed(seed + 1)
    ids = torch.randint(0, V, (T, C), generator=g, dtype=torch.int32)
    if C > 2:
        ids[:, 1] = ids[:, 0]                                        # a token given twice
        ids[torch.rand(T, C, generator=g) < 0.1] = -1
    return ids.cuda()


def odd_layout(z, lead=1):
    """The same rows in a wider buffer, off 16-byte boundaries."""
    T, V = z.shape
    buf = torch.full((T, V + 5), float("nan"), dtype=z.dtype, device=z.device)
    buf[:, lead:lead + V] = z
    return buf[:, lead:lead + V]


def check(rlk, z, ids, T, top):
    V = z.shape[1]
    lp, h, ti, tl, p, _ = tokens64(z, ids, T, top)
    got_lp, got_h, got_ti, got_tl = rlk.token_logprobs(z, ids, T, n_top=top)
    # Largest relative error of S: a sum of V / 1024 terms a lane and 40 joins and moves of the
    # reference, ex2's 2^-22, and the exponents' three roundings, E|d| <= H + ln V of them;
    # ln S and the difference add their own roundings.
    zf = z.double().cpu()
    spread = ((zf.max(1, keepdim=True)[0] - zf) / T)
    spread = torch.where(torch.isfinite(spread), spread, torch.zeros_like(spread))
    d_mean = (p * spread).sum(1)
    chain = V / 1024 + 40
    S = (chain + 4 + 4 * d_mean) * EPS32
    lnV = math.log(V) + 1

    def close(got, want, d):
        got = got.double().cpu()
        assert torch.equal(torch.isfinite(got), torch.isfinite(want)) and torch.equal(got == -math.inf, want == -math.inf)
        fin = torch.isfinite(want)
        tol = S[:, None] + (4 * d + 3 * lnV + 2 * want.abs().nan_to_num(posinf=0.0)) * EPS32
        assert ((got - want).abs() <= tol)[fin].all(), ((got - want).abs() / tol)[fin].max()

    if ids is not None:
        ii = ids.reshape(len(h), -1).cpu().long()
        close(got_lp.reshape(len(h), -1), lp, torch.gather(spread, 1, ii.clamp_min(0)))
    # E d: the same chain on terms w |d|, then two roundings more
    tol = S + (2 * chain * d_mean + 8 * d_mean * d_mean.clamp_min(1) + 3 * lnV + 4 * h) * EPS32
    assert ((got_h.double().cpu() - h).abs() <= tol).all(), ((got_h.double().cpu() - h).abs() / tol).max()
    if top:
        assert torch.equal(got_ti.cpu().long(), ti)
        close(got_tl, tl, torch.gather(spread, 1, ti.clamp_min(0)))


SHAPES = [(1, 1, 1, 1), (2, 3, 2, 3), (1, 8, 1, 0), (3, 33, 5, 33), (1, 1000, 1, 128), (5, 1023, 3, 20), (1, 151936, 1, 20), (37, 8193, 4, 5),
          (40, 20011, 1, 50), (90, 4099, 2, 128), (330, 2050, 1, 1)]


@pytest.mark.parametrize("T,V,C,top", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("odd", [False, True], ids=["aligned", "odd"])
def test_shapes(cuda_lib, T, V, C, top, dtype, odd):
    z = logits(T, V, dtype, V + T)
    check(cuda_lib, odd_layout(z) if odd else z, given(T, V, C, V), 1.0 if T % 2 else 0.7, top)


@pytest.mark.parametrize("kind", ["levels", "flat", "up", "down", "masked", "lowest", "few", "wide"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,top", [(1, 30011, 20), (2, 9000, 128), (50, 5000, 128), (170, 12345, 64), (310, 3001, 128)])
def test_kinds(cuda_lib, kind, dtype, T, V, top):
    z = logits(T, V, dtype, V, kind)
    keep = torch.arange(0, T, max(1, T // 6))                        # the 64-bit form row by row: six rows of the batch
    ids = given(T, V, 3, 5)
    lp, h, ti, tl = cuda_lib.token_logprobs(z, ids, 1.3, n_top=top)
    check(cuda_lib, z[keep], ids[keep], 1.3, top)
    part = cuda_lib.token_logprobs(z[keep], ids[keep], 1.3, n_top=top)
    for a, b in zip((lp, h, ti, tl), part):                          # and the batch's own rows are those, bit for bit
        assert torch.equal(a[keep].view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_one_row_one_set_of_bits(cuda_lib, dtype):
    V = 70001
    z = logits(1, V, dtype, 3).repeat(700, 1)
    ids = given(1, V, 5, 3).repeat(700, 1)
    want = cuda_lib.token_logprobs(z[:1], ids[:1], 0.9, n_top=9)
    bits = lambda t: t.view(torch.int32)
    for rows in (2, 19, 37, 38, 39, 76, 77, 152, 153, 700):
        for lead in (0, 1, 2, 3, 4):
            zz = odd_layout(z[:rows], lead) if lead else z[:rows]
            for a, b in zip(want, cuda_lib.token_logprobs(zz, ids[:rows], 0.9, n_top=9)):
                assert torch.equal(bits(a).expand(rows, *a.shape[1:]), bits(b)), (rows, lead)
    # nor on the other arguments
    lp, h, _, _ = cuda_lib.token_logprobs(z[:2], ids[:2, 1].contiguous(), 0.9)
    assert torch.equal(lp, want[0][:, 1].expand(2)) and torch.equal(h, want[1].expand(2))
    none, h, ti, tl = cuda_lib.token_logprobs(z[:2], None, 0.9, n_top=9)
    assert none is None and torch.equal(h, want[1].expand(2)) and torch.equal(ti, want[2].expand(2, 9)) and torch.equal(tl, want[3].expand(2, 9))


def test_bad_rows(cuda_lib):
    rlk = cuda_lib
    z = logits(6, 5001, F32, 1)
    z[1, 77] = float("nan")
    z[2, 4000] = math.inf
    z[3] = -math.inf
    ids = given(6, 5001, 4, 2).clamp_min(0)
    ids[:, 3] = -1
    ids[4, 0], ids[5, 1] = 5001, -2
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    state = rlk.new_token_state(6, "cuda")
    lp, h, ti, tl = rlk.token_logprobs(z, ids, 1.0, n_top=4, state=state, status_word=word)
    assert word.item() == rlk.STATUS_NONFINITE | rlk.STATUS_BAD_TOKEN_ID
    assert torch.isnan(h).tolist() == [False, True, True, True, False, False]
    assert torch.isnan(lp[1:4, :3]).all() and (lp[:, 3] == 0).all()
    assert torch.isnan(lp[4]).tolist() == [True, False, False, False] and torch.isnan(lp[5]).tolist() == [False, True, False, False]
    assert (ti[1:4] == -1).all() and torch.isnan(tl[1:4]).all() and torch.isfinite(tl[[0, 4, 5]]).all()
    word.zero_()
    g = rlk.token_logprobs_backward(z, ids, 1.0, state, torch.ones_like(lp), status_word=word)
    assert word.item() == rlk.STATUS_BAD_TOKEN_ID
    assert torch.isnan(g[1:]).all() and torch.isfinite(g[0]).all()
    word.zero_()
    g = rlk.token_logprobs_backward(z[:1], ids[:1], 1.1, state[:1], status_word=word)   # another temperature than the state's
    assert word.item() == rlk.STATUS_BAD_PARAM and torch.isnan(g).all()


@pytest.mark.parametrize("T,V,C,top", [(1, 1, 1, 1), (2, 9, 3, 4), (3, 1000, 1, 0), (5, 4099, 64, 20), (20, 40001, 7, 128), (4, 33000, 1024, 0), (300, 2049, 2, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gdt", [BF16, F32], ids=["to_bf16", "to_f32"])
@pytest.mark.parametrize("kind", ["peaked", "masked"])
def test_backward(cuda_lib, T, V, C, top, dtype, gdt, kind):
    rlk, temp = cuda_lib, 0.8
    if kind == "masked" and V < 100:
        kind = "levels"
    g = torch.Generator().manual_seed(V)
    for lead, lead_out in ((0, 0), (1, 1), (3, 0)):
        z = logits(T, V, dtype, V + C, kind)
        z = odd_layout(z, lead) if lead else z
        ids = given(T, V, C, C)
        ids[0, 0] = -1                                               # a row that may have nothing in its list
        state = rlk.new_token_state(T, "cuda")
        ti = rlk.token_logprobs(z, ids, temp, n_top=top, state=state)[2]
        glp, gh = torch.randn(T, C, generator=g).cuda(), torch.randn(T, generator=g).cuda()
        gt = torch.randn(T, top, generator=g).cuda() if top else None
        out = torch.full((T, V + 9), 7.0, dtype=gdt, device="cuda")
        view = out[:, lead_out:lead_out + V]
        assert rlk.token_logprobs_backward(z, ids, temp, state, glp, gh, top_ids=ti, grad_top=gt, out=view) is view
        want, terms = tokens_grad64(z, ids, temp, glp, gh, ti, gt)
        # p's relative error: the state's log2 S (as ln S above, 2^-23 of up to 18 on top) and the exponent's
        # roundings (|d| <= 60 where p counts); the products and the sum over C + top gradients add the rest
        rel = (V / 1024 + 40 + 4 * 60 + 24 + 2 * (C + top)) * EPS32
        tol = terms * rel + want.abs() * HALF_ULP[gdt] * 1.01 + 1e-37
        err = (view.double().cpu() - want).abs()
        assert (err <= tol).all(), (err / tol).max()
        rest = torch.ones(V + 9, dtype=torch.bool)
        rest[lead_out:lead_out + V] = False
        assert (out[:, rest.cuda()] == 7.0).all()                    # nothing beside the rows


def test_backward_only_some_gradients(cuda_lib):
    rlk = cuda_lib
    z = logits(3, 777, F32, 1)
    ids = given(3, 777, 1, 1)[:, 0].contiguous()
    state = rlk.new_token_state(3, "cuda")
    lp, h, ti, _ = rlk.token_logprobs(z, ids, 1.0, n_top=5, state=state)
    for glp, gh, gt in ((torch.ones_like(lp), None, None), (None, torch.ones_like(h), None), (None, None, torch.ones(3, 5, device="cuda")), (None, None, None)):
        got = rlk.token_logprobs_backward(z, ids, 1.0, state, glp, gh, top_ids=ti, grad_top=gt)
        want, terms = tokens_grad64(z, ids[:, None], 1.0, None if glp is None else glp[:, None], gh, ti, gt)
        assert ((got.double().cpu() - want).abs() <= terms * 400 * EPS32 + want.abs() * EPS32 * 2).all()
    got = rlk.token_logprobs_backward(z, None, 1.0, state, None, torch.ones_like(h))
    want, terms = tokens_grad64(z, None, 1.0, None, torch.ones_like(h), None, None)
    assert ((got.double().cpu() - want).abs() <= terms * 400 * EPS32 + want.abs() * EPS32 * 2).all()


def test_autograd_against_differences(cuda_lib):
    """The gradient against central differences of the 64-bit forward."""
    rlk, V, temp = cuda_lib, 61, 0.9
    z = logits(2, V, F32, 4)
    ids = torch.tensor([[3, 3, -1], [60, 0, 5]], dtype=torch.int32, device="cuda")
    w = torch.randn(2, 3, generator=torch.Generator().manual_seed(1)).double()
    wt = torch.randn(2, 4, generator=torch.Generator().manual_seed(2)).double()

    def loss64(zz):
        lp, h, ti, tl, _, _ = tokens64(zz, ids, temp, 4)
        return float((w * lp).sum() + 0.3 * h.sum() + (wt * tl).sum())

    x = z.clone().requires_grad_()
    lp, h, ti, tl = rlk.token_logprobs_autograd(x, ids, temp, n_top=4)
    ((w.cuda() * lp).sum() + 0.3 * h.sum() + (wt.cuda() * tl).sum()).backward()
    z64, e = z.double().cpu(), 1e-5
    for r in range(2):
        for i in range(V):
            a, b = z64.clone(), z64.clone()
            a[r, i] += e
            b[r, i] -= e
            # third derivatives are below 10 (sums of weights) / T^3, so the difference is off by 10 e^2 and 1e-16 / e
            assert abs((loss64(a) - loss64(b)) / (2 * e) - x.grad[r, i].item()) < 1e-5
    assert not ti.requires_grad
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(rlk.token_logprobs_autograd(x, ids)[0].sum(), x, create_graph=True)[0].sum(), x)


def test_streams_graph_and_repeat(cuda_lib):
    rlk = cuda_lib
    z, ids = logits(9, 30000, BF16, 2), given(9, 30000, 6, 2)
    g = torch.randn(9, 6, device="cuda")
    state = rlk.new_token_state(9, "cuda")
    run = lambda: (*rlk.token_logprobs(z, ids, 0.7, n_top=11, state=state), rlk.token_logprobs_backward(z, ids, 0.7, state, g))
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
        graph = torch.cuda.CUDAGraph()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    with torch.cuda.graph(graph):
        kept = run()
    z.copy_(logits(9, 30000, BF16, 8, "masked"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, run()))


def test_no_rows(cuda_lib):
    rlk = cuda_lib
    z = torch.empty(0, 100, device="cuda")
    lp, h, ti, tl = rlk.token_logprobs(z, torch.empty(0, 3, dtype=torch.int32, device="cuda"), n_top=2)
    assert lp.shape == (0, 3) and h.shape == (0,) and ti.shape == (0, 2) and tl.shape == (0, 2)


def test_offsets_past_32_bits(cuda_lib):
    """The last rows of logits with more than 2^32 bytes, and their gradient."""
    rlk, V, T = cuda_lib, 151937, 15000                              # 4.56 GB, rows off 16-byte boundaries
    z = torch.zeros(T, V, dtype=BF16, device="cuda")
    z[-3:] = logits(3, V, BF16, 1)
    ids = given(T, V, 2, 1)
    state = rlk.new_token_state(T, "cuda")
    lp, h, ti, tl = rlk.token_logprobs(z, ids, 1.0, n_top=3, state=state)
    check(rlk, z[-3:], ids[-3:], 1.0, 3)
    part = rlk.token_logprobs(z[-3:], ids[-3:], 1.0, n_top=3)
    assert all(torch.equal(a[-3:], b) for a, b in zip((lp, h, ti, tl), part))
    g = torch.ones(T, 2, device="cuda")
    dz = rlk.token_logprobs_backward(z, ids, 1.0, state, g)
    assert torch.equal(dz[-3:], rlk.token_logprobs_backward(z[-3:], ids[-3:], 1.0, state[-3:].contiguous(), g[-3:]))


@pytest.mark.parametrize("stage", [0, 2])
@pytest.mark.parametrize("V", [40001, 70001])
def test_waits_that_run_out(cuda_lib, stage, V):
    """Many long rows off 16-byte boundaries come through a ring of copies: a debug setting makes the first CTA wait for
    an arrival that never comes.  Its rows are NaN, the others keep their bits, the next call is clean."""
    rlk, T = cuda_lib, 500
    z = logits(2, V, BF16, 1).repeat(T // 2, 1)
    ids = given(T, V, 3, 1)
    want = rlk.token_logprobs(z, ids, 1.0, n_top=5)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    rlk.set_wait_limit(2_000_000)   # about a millisecond
    try:
        rlk.withhold_copy(stage)
        got = rlk.token_logprobs(z, ids, 1.0, n_top=5, status_word=word)
        torch.cuda.synchronize()
    finally:
        rlk.withhold_copy(-1)
        rlk.set_wait_limit(0)
    bad = torch.isnan(got[1])
    assert word.item() & rlk.STATUS_TIMEOUT and bad[0] and 0 < int(bad.sum()) < T
    assert torch.isnan(got[0][bad][ids[bad] >= 0]).all() and torch.isnan(got[3][bad]).all() and (got[2][bad] == -1).all()
    assert all(torch.equal(a[~bad], b[~bad]) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(rlk.token_logprobs(z, ids, 1.0, n_top=5), want))


def test_rows_of_one_call_through_the_ring(cuda_lib):
    """Every row of a batch that goes through the ring is what it is alone."""
    for dtype, V, lead in ((BF16, 33001, 1), (F32, 9002, 3), (BF16, 16385, 0)):
        z = logits(500, V, dtype, 3, "masked")
        z = odd_layout(z, lead) if lead else z
        ids = given(500, V, 2, 1)
        all_ = cuda_lib.token_logprobs(z, ids, 0.8, n_top=7)
        for r in (0, 1, 170, 455, 456, 457, 499):
            for a, b in zip(all_, cuda_lib.token_logprobs(z[r:r + 1], ids[r:r + 1], 0.8, n_top=7)):
                assert torch.equal(a[r:r + 1].view(torch.int32), b.view(torch.int32)), (dtype, V, r)


@pytest.mark.parametrize("V,top", [(1, 128), (7, 20), (100, 128), (127, 128)])
@pytest.mark.parametrize("T", [1, 30, 400])
def test_more_alternatives_than_tokens(cuda_lib, V, top, T):
    z = logits(T, V, BF16, V)
    ids = given(T, V, 2, 1)
    keep = torch.arange(0, T, max(1, T // 5))
    got = cuda_lib.token_logprobs(z, ids, 1.0, n_top=top)
    assert (got[2][:, V:] == -1).all() and (got[3][:, V:] == -math.inf).all() and (got[2][:, :V].sort(1)[0] == torch.arange(V, device="cuda")).all()
    check(cuda_lib, z[keep], ids[keep], 1.0, top)


def test_python_refusals(cuda_lib):
    rlk = cuda_lib
    z, ids = torch.randn(4, 50, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    state = rlk.new_token_state(4, "cuda")
    _, _, ti, _ = rlk.token_logprobs(z, ids, 1.0, n_top=3, state=state)
    g = torch.ones(4, 3, device="cuda")
    for bad in (lambda: rlk.token_logprobs(z.half(), ids), lambda: rlk.token_logprobs(z.cpu(), ids), lambda: rlk.token_logprobs(z, ids.cpu()), lambda: rlk.token_logprobs(z, ids.long()),
                lambda: rlk.token_logprobs(z, ids[:3]), lambda: rlk.token_logprobs(z, ids.t()), lambda: rlk.token_logprobs(z.t(), ids), lambda: rlk.token_logprobs(z[0], ids),
                lambda: rlk.token_logprobs(z, ids, n_top=129), lambda: rlk.token_logprobs(z, ids, n_top=-1), lambda: rlk.token_logprobs(z, ids, state=state[:3]),
                lambda: rlk.token_logprobs(z, torch.zeros(4, 1025, dtype=torch.int32, device="cuda")),
                lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, torch.ones(4, device="cuda")), lambda: rlk.token_logprobs_backward(z, None, 1.0, state, torch.ones(4, 2, device="cuda")),
                lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, grad_top=g), lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, top_ids=ti, grad_top=g[:, :2]),
                lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, out=torch.empty(4, 49, device="cuda")),
                lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, out=torch.empty(4, 50, device="cuda"), grad_dtype=BF16),
                lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, None, torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: rlk.token_logprobs(z, ids, 0.0), lambda: rlk.token_logprobs(z, ids, float("nan")), lambda: rlk.token_logprobs(z[:1].expand(4, 50), ids),
                lambda: rlk.token_logprobs_backward(z, ids, 1.0, state, out=z)):
        with pytest.raises(rlk.RlkError):
            bad()


@pytest.mark.parametrize("temp", [1e-30, 1e-4, 1e4, 1e30, 3e38])
def test_temperatures(cuda_lib, temp):
    z = logits(3, 3000, F32, 2)
    got = cuda_lib.token_logprobs(z, given(3, 3000, 3, 1), temp, n_top=3)
    x = z.double().cpu() / temp
    lp = torch.log_softmax(x, 1)
    h = -(lp.exp() * lp).nan_to_num(0.0).sum(1)
    # d = (z - M) / T to three roundings of it, S to 50 e; the entropy's terms w d likewise
    assert ((got[1].double().cpu() - h).abs() <= 2 ** -24 * (100 + 8 * h + 3000 / 512 * (1 + h))).all()
    best = lp.max(1)[0]
    assert torch.allclose(got[3][:, 0].double().cpu(), best, atol=2 ** -24 * 80, rtol=2 ** -21)
