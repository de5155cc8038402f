"""Linear attention with a head decay where little or nothing is there: batches of
empty sequences, decays that are not numbers, results that are not wanted; and its
gradients against differences.  Tolerances as in test_gpu_linear.py, which has the
arithmetic: `rel32` of a magnitude for the fp32 forms, 2 * 2^-8 of it where X and P
enter as bf16, and half a step of the type a result is stored in."""
import pytest
import torch

import linear_ref as R
from gated_deltanet_recurrence_rule_b200 import api
from test_gpu_linear import DEV, DT, dev, make, rel32

pytestmark = pytest.mark.gpu


def empty_batch(N, Hqk, Hv, Dk, Dv, dtype):
    z = lambda *s: torch.zeros(*s, dtype=DT[dtype], device=DEV)  # noqa: E731
    return (z(0, Hqk, Dk), z(0, Hqk, Dk), z(0, Hv, Dv), -torch.ones(Hv, device=DEV)), \
        torch.zeros(N + 1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype,odtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("sdtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [1, 3])
def test_prefill_of_empty_sequences(N, sdtype, dtype, odtype):
    """Their final states are their initial states, zeros without any."""
    args, cut = empty_batch(N, 2, 6, 128, 64, dtype)
    gen = torch.Generator().manual_seed(3)
    s0 = torch.randn(N, 6, 64, 128, generator=gen).to(DT[sdtype]).to(DEV)
    ws = torch.zeros(api.linear_prefill_workspace_size(N, 0, 2, 6, 128, 64, DT[dtype]), dtype=torch.uint8, device=DEV)
    for init in (s0, None):
        f = torch.full_like(s0, float("nan"))
        o, f2 = api.linear_prefill(*args, cu_seqlens=cut, initial_state=init, final_state=f, o_dtype=DT[odtype],
                                   workspace=ws)
        torch.cuda.synchronize()
        assert o.shape == (0, 6, 64) and f2 is f
        assert torch.equal(f, torch.zeros_like(s0) if init is None else s0)
    same = s0.clone()
    api.linear_prefill(*args, cu_seqlens=cut, initial_state=same, final_state=same, o_dtype=DT[odtype], workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(same, s0) and api.get_device_status(ws) == api.GDN_OK


def backward_of_empty(N, Hqk, Hv, dtype):
    args, cut = empty_batch(N, Hqk, Hv, 64, 128, dtype)
    gen = torch.Generator().manual_seed(5)
    dsf = torch.randn(N, Hv, 128, 64, generator=gen).to(DEV)
    do = torch.zeros(0, Hv, 128, dtype=DT[dtype], device=DEV)
    for d in (dsf, None):
        freed = [torch.full_like(dsf, float("nan")) for _ in range(4)]  # what fresh memory then holds
        del freed
        dq, dk, dv, ds0 = api.linear_prefill_backward(*args, do, cu_seqlens=cut, initial_state=dsf, d_final_state=d)
        torch.cuda.synchronize()
        assert dq.shape == dk.shape == (0, Hqk, 64) and dv.shape == (0, Hv, 128)
        assert torch.equal(ds0, torch.zeros_like(dsf) if d is None else dsf)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 3])
def test_backward_of_empty_sequences(N, dtype):
    backward_of_empty(N, 3, 3, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 3])
def test_backward_of_empty_sequences_with_shared_heads(N, dtype):
    backward_of_empty(N, 2, 6, dtype)


LENS = {"whole": [150, 0, 70], "cut": [2300, 0, 70]}  # (cut: in segments, in both forms)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", sorted(LENS))
def test_a_decay_that_is_no_number(dtype, lens):
    """A NaN in g makes everything of its head NaN that a token has reached, and
    nothing else: the other heads' bits are those without it."""
    L, Hqk, Hv, bad = LENS[lens], 2, 4, 1
    x, cu, S0, r = make(L, Hqk, Hv, 128, 64, dtype, seed=71)
    do, dsf = r(sum(L), Hv, 64).to(DT[dtype]), r(len(L), Hv, 64, 128)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    q, k, v, g, do, s0, dsf = dev(x["q"], x["k"], x["v"], x["g"], do, S0, dsf)
    gn = g.clone()
    gn[bad] = float("nan")

    def calls(g):
        o, f = api.linear_prefill(q, k, v, g, cu_seqlens=cut, initial_state=s0, o_dtype=DT[dtype])
        return o, f, *api.linear_prefill_backward(q, k, v, g, do, cu_seqlens=cut, initial_state=s0, d_final_state=dsf)

    want, got = calls(g), calls(gn)
    torch.cuda.synchronize()
    heads = lambda n: [h for h in range(n) if h != (bad if n == Hv else bad // (Hv // Hqk))]  # noqa: E731
    for name, a, b in zip(("o", "final_state", "dq", "dk", "dv", "d_initial_state"), want, got):
        assert torch.isfinite(a).all()
        rest = heads(a.shape[1])
        mine = [h for h in range(a.shape[1]) if h not in rest]
        assert torch.equal(a[:, rest], b[:, rest]), name
        if "state" in name:
            assert torch.isnan(b[[0, 2]][:, mine]).all() and torch.equal(a[1], b[1]), name  # (1 is empty)
        else:
            assert torch.isnan(b[:, mine]).all(), name


@pytest.mark.parametrize("Tn", [1, 5])
def test_a_decay_that_is_no_number_in_decode_and_trees(Tn):
    """The same for the tokens of a decode call, the nodes of a tree and its commit;
    where no node is accepted, the state is copied whatever its decay."""
    B, Hv, bad = 3, 4, 2
    gen = torch.Generator().manual_seed(73)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    q, k, v, g = r(B, Tn, 2, 64), r(B, Tn, 2, 64), r(B, Tn, Hv, 128), -torch.rand(Hv, generator=gen).to(DEV)
    pool = r(B, Hv, 128, 64)
    parent = torch.tensor([[i // 2 - (i == 0) for i in range(Tn)]] * B, dtype=torch.int32, device=DEV)
    accept = torch.tensor([Tn - 1, -1, 0], dtype=torch.int32, device=DEV)
    gn = g.clone()
    gn[bad] = float("nan")

    def calls(g):
        decoded, committed = torch.zeros_like(pool), torch.zeros_like(pool)
        o = api.linear_decode_tokens(q, k, v, g, pool, decoded)
        t = api.decode_tree(q, k, v, g, None, parent, pool)
        api.tree_commit(k, v, g, None, parent, accept, pool, committed)
        return o.movedim(2, 0), t.movedim(2, 0), decoded.movedim(1, 0), committed.movedim(1, 0)

    want, got = calls(g), calls(gn)
    torch.cuda.synchronize()
    rest = [h for h in range(Hv) if h != bad]
    for name, a, b in zip(("decode o", "tree o", "decoded state", "committed state"), want, got):
        assert torch.isfinite(a).all() and torch.equal(a[rest], b[rest]), name
        assert torch.isnan(b[bad][[0, 2]]).all(), name
        assert torch.equal(b[bad][1], pool[1, bad]) if name == "committed state" else torch.isnan(b[bad][1]).all(), name


def test_backward_from_transposed_states_repeats():
    """One segment of several chunks a sequence, on every multiprocessor: the starting
    states of dq and dk are transposed through the place of a later chunk's tiles.  The
    same bits each time, whatever ran between, and the formula's values."""
    L, Hv = [300] * 8, 24
    x, cu, S0, r = make(L, 8, Hv, 128, 128, "bf16", seed=81)
    do, dsf = r(sum(L), Hv, 128).to(torch.bfloat16), r(len(L), Hv, 128, 128)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    a = dev(x["q"], x["k"], x["v"], x["g"], do)
    s0, d = dev(S0, dsf)
    call = lambda s0, d: api.linear_prefill_backward(*a, cu_seqlens=cut, initial_state=s0, d_final_state=d)  # noqa: E731
    want = call(s0, d)
    for _ in range(20):
        call(-3.0 * s0, None)
        got = call(s0, d)
        for name, u, w in zip(("dq", "dk", "dv", "d_initial_state"), want, got):
            assert torch.equal(u, w), name
    refs, mags = R.scan_grads(x["q"][:300], x["k"][:300], x["v"][:300], x["g"], [0, 300], S0[:1], do[:300], dsf[:1])
    for name, u, ref, mag in zip(("dq", "dk", "dv"), want, refs, mags):
        R.check(u[:300], ref, mag, 2 * R.UB16, name, R.UB16)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 64)])
def test_gradients_against_aligned_differences(Dk, Dv):
    """Central differences of the kernels' own forward (fp32) along the sign of each
    gradient, so that nothing cancels in the derivative: the loss is linear in q, k, v
    and the initial state one at a time, so a step of any length gives it up to rounding.
    That is rel32 of every element's magnitude, weighted by the element's gradient; it
    stays below a hundredth of the derivative, so a gradient that is zero, scaled by
    1.02 or of the wrong sign is found."""
    L, Hqk, Hv = [70, 3, 131], 2, 4
    x, cu, S0, r = make(L, Hqk, Hv, Dk, Dv, "fp32", seed=77)
    do, dsf = r(sum(L), Hv, Dv), r(len(L), Hv, Dv, Dk)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    vals = [x["q"], x["k"], x["v"], S0]
    grads = api.linear_prefill_backward(*dev(*vals[:3], x["g"], do), cu_seqlens=cut, initial_state=S0.to(DEV),
                                        d_final_state=dsf.to(DEV), scale=0.5)
    refs, _ = R.scan_grads(*vals[:3], x["g"], cu, S0, do, dsf, 0.5)

    def loss(q, k, v, s0):
        """The loss of the kernels' forward, and how far its roundings may move it."""
        o, f = api.linear_prefill(*dev(q, k, v, x["g"]), cu_seqlens=cut, initial_state=s0.to(DEV), scale=0.5)
        ref, om, F, Fm = R.scan(q, k, v, x["g"], cu, s0, 0.5)
        tol = rel32(L, Dk)
        off = (R.d64(do).abs() * (tol * om + R.U32 * ref.abs())).sum() + (R.d64(dsf).abs() * (tol * Fm + R.U32 * F.abs())).sum()
        return float((R.d64(o) * R.d64(do)).sum() + (R.d64(f) * R.d64(dsf)).sum()), float(off)

    for i, (name, grad, ref) in enumerate(zip(("q", "k", "v", "initial state"), grads, refs)):
        # a step exact in fp32, and sums with it that round once
        d = (0.25 * ref.sign()).float()
        ends = [[t + s * d if j == i else t for j, t in enumerate(vals)] for s in (1.0, -1.0)]
        (a, ea), (b, eb) = (loss(*e) for e in ends)
        d = (R.d64(ends[0][i]) - R.d64(ends[1][i])) / 2  # the step as it was taken
        want, allowed = float((ref * d).sum()), (ea + eb) / 2
        assert allowed <= 0.01 * want, (name, allowed, want)
        assert abs((a - b) / 2 - want) <= allowed, (name, (a - b) / 2, want, allowed)
        got = float((R.d64(grad) * d).sum())
        assert abs((a - b) / 2 - got) <= 2 * allowed, (name, (a - b) / 2, got, allowed)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", sorted(LENS))
def test_states_that_are_not_wanted(dtype, lens):
    """Without a final state, and without the gradient of the initial one, the rest is
    the definition's (bf16: w C enters in two terms then, so o and dv may differ in
    rounding from those of a call that returns the state)."""
    L = LENS[lens]
    x, cu, S0, r = make(L, 2, 4, 128, 64, dtype, seed=91)
    do, dsf = r(sum(L), 4, 64).to(DT[dtype]), r(len(L), 4, 64, 128)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    a, (do_, s0, d) = dev(x["q"], x["k"], x["v"], x["g"]), dev(do, S0, dsf)
    o, f = api.linear_prefill(*a, cu_seqlens=cut, initial_state=s0, output_final_state=False, o_dtype=DT[dtype])
    *grads, ds0 = api.linear_prefill_backward(*a, do_, cu_seqlens=cut, initial_state=s0, d_final_state=d,
                                              want_d_initial_state=False)
    torch.cuda.synchronize()
    assert f is None and ds0 is None
    tol, stored = (2 * R.UB16, R.UB16) if dtype == "bf16" else (rel32(L, 128) + 2 * R.U32, R.U32)
    ref, om, _, _ = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0)
    R.check(o, ref, om, tol, "o", stored)
    refs, mags = R.scan_grads(x["q"], x["k"], x["v"], x["g"], cu, S0, do, dsf)
    for name, got, ref, mag in zip(("dq", "dk", "dv"), grads, refs, mags):
        R.check(got, ref, mag, tol, name, stored)


@pytest.mark.parametrize("dtype,odtype,chunk", [("bf16", "bf16", 128), ("bf16", "fp32", 64), ("fp32", "fp32", 64)])
@pytest.mark.parametrize("Hv", [4, 160])
def test_long_memories(dtype, odtype, chunk, Hv):
    """Decays whose power over a chunk falls half way between two fp32 numbers, carried
    over a hundred chunks and more, in segments (4 heads) and in one (160).  Relative rms
    error of a head's state: a chunk's sum takes at most 24 tensor-core additions, which
    cut by up to 2^-23 of a sum that grows from nothing, 6 * 2^-23 in the mean; the carry is
    off by two half steps, 2^-23, at most; additions of chunks round at random.  7 * 2^-23 <
    2^-20.  (A power rounded to fp32 is off by 2^-25 each time: 2^-18 over 128 chunks.)"""
    T, D = 16000, 64
    x, cu, _, _ = make([T], 1, Hv, D, D, dtype, seed=95, init=False)
    # of many decays those that rounding a chunk's power moves most
    g = -torch.exp(torch.linspace(-11.5, -9.0, 4001, dtype=torch.float64)).float()
    p = (g.double() * chunk).exp()
    g = g[((p.float().double() - p).abs()).argsort(descending=True)[:4]]
    x["g"][:4] = g
    o, f = api.linear_prefill(*dev(x["q"], x["k"], x["v"], x["g"]), o_dtype=DT[odtype])
    torch.cuda.synchronize()
    ref, _, F, _ = R.scan(x["q"], x["k"], x["v"][:, :4], g, cu)
    for h in range(4):
        err = float((R.d64(f[0, h]) - F[0, h]).norm() / F[0, h].norm())
        assert err <= 2.0 ** -20, f"state of head {h}: {err:.2e}"
