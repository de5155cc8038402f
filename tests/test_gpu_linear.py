"""Linear attention with a head decay (gdn_linear_prefill, its backward) on the GPU
against the fp64 definition.

Tolerances.  fp32 inputs or outputs: split tf32 products and fp32 sums, so an
element is off by at most (additions in a row) * 2 * 2^-24 times its magnitude
(tests/linear_ref.py), plus half a step of its type.  A chunk adds Dk + 64 or 128
terms and its state is carried over `chunks` chunks; the powers of the decay carry
|exponent| * 2^-24, at most 2^-24 * 88 where they do not vanish.  bf16 inputs and
outputs: the state and the token x token products are rounded to bf16 once as
operands, 2^-8 of the magnitude each in the worst case; the errors are random, so
the root mean square error is held to 2^-8 of the root mean square value (three
roundings of at most 2^-9 on average, sqrt(3) 2^-9 < 2^-8).
"""
import pytest
import torch

import linear_ref as R
from gated_deltanet_recurrence_rule_b200 import api

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(lens, Hqk, Hv, Dk, Dv, dtype, seed=0, init=True, slow=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    T, N = sum(lens), len(lens)
    x = dict(q=unit(r(T, Hqk, Dk)).to(DT[dtype]), k=unit(r(T, Hqk, Dk)).to(DT[dtype]), v=r(T, Hv, Dv).to(DT[dtype]),
             g=-torch.exp(torch.rand(Hv, generator=gen) * 9 - 9))
    if slow:
        x["g"] = x["g"] * 1e-3
    cu = [sum(lens[:i]) for i in range(N + 1)]
    return x, cu, (r(N, Hv, Dv, Dk) * 0.5 if init else None), r


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def rel32(lens, D):
    """Relative bound of the fp32 forms: the roundings of a chunk's sums, once for
    each chunk the state goes through, and those of the powers."""
    chunks = max(lens) // 64 + 2
    return 2.0 ** -24 * (2 * (D + 64) + 2 * chunks + 2 * 88 + 32)


def rms_close(x, ref, what, bound=R.UB16):
    x = R.d64(x)
    assert torch.isfinite(x).all(), f"{what}: not finite"
    if ref.numel() and float(ref.norm()) > 0:
        e = float((x - ref).norm() / ref.norm())
        assert e <= bound, f"{what}: relative rms error {e:.3e}"


LENS = {"one": [1], "short": [63, 0, 64, 65, 1], "ragged": [130, 0, 257, 1, 90], "long": [1500, 700, 0, 1]}


@pytest.mark.parametrize("dtype,odtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", sorted(LENS))
def test_prefill(dtype, odtype, Dk, Dv, lens):
    L = LENS[lens]
    x, cu, S0, _ = make(L, 2, 6, Dk, Dv, dtype, seed=len(L) + Dk, init=lens != "one")
    o, f = api.linear_prefill(*dev(x["q"], x["k"], x["v"], x["g"]), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                              initial_state=None if S0 is None else S0.to(DEV), scale=0.5, o_dtype=DT[odtype])
    torch.cuda.synchronize()
    ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0, 0.5)
    R.check(f, F, Fm, rel32(L, Dk), "final state", R.U32)
    if dtype == "bf16" and odtype == "bf16":
        rms_close(o, ref, "o")
        R.check(o, ref, om, 2 * R.UB16, "o", R.UB16)
    else:
        R.check(o, ref, om, rel32(L, Dk), "o", R.UB16 if odtype == "bf16" else R.U32)


def grads_ref(x, cu, S0, do, dsf, scale):
    """dq, dk, dv, dS0 from the formulas, token by token, and their magnitudes."""
    q, k, v, g, do, S0, dsf = (R.d64(t) for t in (x["q"], x["k"], x["v"], x["g"], do, S0, dsf))
    T, Hv, Dv = v.shape
    Hqk, Dk = q.shape[1:]
    rep = torch.arange(Hv) // (Hv // Hqk)
    q, k = q[:, rep], k[:, rep]
    lam = g.clamp_min(-30.0).exp()[:, None, None]
    N = len(cu) - 1
    z = torch.zeros(Hv, Dv, Dk, dtype=torch.float64)
    out = []
    for mag in (False, True):
        f = (lambda t: t.abs()) if mag else (lambda t: t)
        dq, dk, dv = (torch.zeros(T, Hv, d, dtype=torch.float64) for d in (Dk, Dk, Dv))
        dS0 = torch.zeros(N, Hv, Dv, Dk, dtype=torch.float64)
        for n in range(N):
            S = f(z if S0 is None else S0[n])
            for t in range(cu[n], cu[n + 1]):
                S = lam * S + f(v[t])[:, :, None] * f(k[t])[:, None, :]
                dq[t] = scale * torch.einsum("hvd,hv->hd", S, f(do[t]))
            D = f(z if dsf is None else dsf[n])
            for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
                D = D + scale * f(do[t])[:, :, None] * f(q[t])[:, None, :]
                dk[t] = torch.einsum("hvd,hv->hd", D, f(v[t]))
                dv[t] = torch.einsum("hvd,hd->hv", D, f(k[t]))
                D = lam * D
            dS0[n] = D
        fold = lambda y: y.unflatten(1, (Hqk, Hv // Hqk)).sum(2)  # noqa: E731
        out.append((fold(dq), fold(dk), dv, dS0))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("Hqk,Hv", [(2, 6), (3, 3)])
@pytest.mark.parametrize("lens", sorted(LENS))
def test_backward(dtype, Dk, Dv, Hqk, Hv, lens):
    L = LENS[lens]
    x, cu, S0, r = make(L, Hqk, Hv, Dk, Dv, dtype, seed=3 + len(L) + Dk, init=lens != "one")
    do = r(sum(L), Hv, Dv).to(DT[dtype])
    dsf = None if S0 is None else r(*S0.shape)
    g = api.linear_prefill_backward(*dev(x["q"], x["k"], x["v"], x["g"], do),
                                    cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                                    initial_state=dev(S0)[0], d_final_state=dev(dsf)[0], scale=0.5)
    torch.cuda.synchronize()
    refs, mags = grads_ref(x, cu, S0, do, dsf, 0.5)
    tol = rel32(L, max(Dk, Dv)) + (Hv // Hqk) * R.U32
    for name, a, ref, mag in zip(("dq", "dk", "dv", "d_initial_state"), g, refs, mags):
        if name == "d_initial_state" or dtype == "fp32":
            R.check(a, ref, mag, tol, name, R.U32)
        else:
            assert a.dtype == torch.bfloat16
            rms_close(a, ref, name)
            R.check(a, ref, mag, 2 * R.UB16, name, R.UB16)


def test_gradients_against_differences():
    """Central differences of the kernels' own forward (fp32): the loss is linear in
    o and the final state, and each input enters it linearly, so a difference of any
    step is the derivative up to rounding."""
    L = [70, 3, 131]
    x, cu, S0, r = make(L, 2, 4, 64, 64, "fp32", seed=77)
    T = sum(L)
    do, dsf = r(T, 4, 64), r(3, 4, 64, 64)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    g = api.linear_prefill_backward(*dev(x["q"], x["k"], x["v"], x["g"], do), cu_seqlens=cut, initial_state=S0.to(DEV),
                                    d_final_state=dsf.to(DEV), scale=0.5)

    def loss(q, k, v, s0):
        o, f = api.linear_prefill(*dev(q, k, v, x["g"]), cu_seqlens=cut, initial_state=s0.to(DEV), scale=0.5)
        return float((R.d64(o) * R.d64(do)).sum() + (R.d64(f) * R.d64(dsf)).sum()), \
            float((R.d64(o) * R.d64(do)).abs().sum() + (R.d64(f) * R.d64(dsf)).abs().sum())

    names, vals = ("q", "k", "v", "s0"), [x["q"], x["k"], x["v"], S0]
    for i, (name, grad) in enumerate(zip(names, g)):
        d = r(*vals[i].shape)
        up = [t + d if j == i else t for j, t in enumerate(vals)]
        down = [t - d if j == i else t for j, t in enumerate(vals)]
        (a, am), (b, bm) = loss(*up), loss(*down)
        want = float((R.d64(grad) * R.d64(d)).sum())
        # every o and f is off by at most rel32 of a magnitude no larger than 64 x itself on the sum
        assert abs((a - b) / 2 - want) <= 64 * rel32(L, 64) * (am + bm), name


def test_bf16_states_and_in_place():
    """bf16 states at rest are the fp32 ones rounded once; the final state may
    overwrite the initial one, in one segment and in several."""
    for L in ([300, 0, 70], [3000, 5, 0]):
        for odt in (torch.bfloat16, torch.float32):
            x, cu, S0, _ = make(L, 1, 2, 128, 128, "bf16", seed=5)
            cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
            S0 = S0.to(torch.bfloat16)
            args = dev(x["q"], x["k"], x["v"], x["g"])
            o, f = api.linear_prefill(*args, cu_seqlens=cut, initial_state=S0.float().to(DEV), o_dtype=odt)
            S = S0.to(DEV)
            o2, f2 = api.linear_prefill(*args, cu_seqlens=cut, initial_state=S, final_state=S, o_dtype=odt)
            S32 = S0.float().to(DEV)
            o3, f3 = api.linear_prefill(*args, cu_seqlens=cut, initial_state=S32, final_state=S32, o_dtype=odt)
            torch.cuda.synchronize()
            assert f2 is S and torch.equal(o, o2) and torch.equal(o, o3)
            assert torch.equal(f.to(torch.bfloat16), f2) and torch.equal(f, f3)


@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
def test_prefill_then_decode(odt):
    """A prompt in two calls, and its last tokens by the decode kernel, continue one
    another; and a sequence's results do not depend on its neighbours (whose values
    are not finite)."""
    x, cu, _, _ = make([700], 2, 6, 128, 128, "bf16", seed=9)
    args = dev(x["q"], x["k"], x["v"], x["g"])
    q, k, v, g = args
    o, f = api.linear_prefill(q, k, v, g, o_dtype=odt)
    o1, f1 = api.linear_prefill(q[:333], k[:333], v[:333], g, o_dtype=odt)
    o2, f2 = api.linear_prefill(q[333:690], k[333:690], v[333:690], g, initial_state=f1, o_dtype=odt)
    o3 = api.linear_decode_tokens(q[None, 690:], k[None, 690:], v[None, 690:], g, f2)
    ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu)
    tol = rel32([700], 128) if odt == torch.float32 else 2 * R.UB16
    stored = R.UB16 if odt == torch.bfloat16 else R.U32
    R.check(torch.cat([o1, o2]), ref[:690], om[:690], tol, "parts", stored)
    R.check(o3[0], ref[690:], om[690:], 3 * rel32([700], 128), "decode", R.U32)
    R.check(f2, F, Fm, 3 * rel32([700], 128), "state", R.U32)
    big = [torch.cat([torch.full_like(t[:77], float("nan")), t, torch.full_like(t[:200], float("inf"))]) for t in (q, k, v)]
    cut = torch.tensor([0, 77, 777, 977], dtype=torch.int32, device=DEV)
    ob, fb = api.linear_prefill(*big, g, cu_seqlens=cut, o_dtype=odt)
    torch.cuda.synchronize()
    assert torch.equal(ob[77:777], o) and torch.equal(fb[1], f[0])


def test_long_slow_decay():
    """Many segments, a memory longer than the sequence: the state and outputs of
    6,000 tokens at decays down to e^-1e-7."""
    L = [6000]
    for dtype, odt in (("bf16", "bf16"), ("fp32", "fp32")):
        x, cu, S0, _ = make(L, 1, 3, 128, 128, dtype, seed=15, slow=True)
        x["g"][0] = 0.0
        o, f = api.linear_prefill(*dev(x["q"], x["k"], x["v"], x["g"]), initial_state=S0.to(DEV), o_dtype=DT[odt])
        torch.cuda.synchronize()
        ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0)
        R.check(f, F, Fm, rel32(L, 128), "final state", R.U32)
        e = float((R.d64(f) - F).norm() / F.norm())
        assert e <= 2e-6, f"state relative error {e:.2e}"
        if odt == "fp32":
            R.check(o, ref, om, rel32(L, 128), "o", R.U32)
        else:
            rms_close(o, ref, "o")


def test_decay_limits():
    """lam = 0 (g = -inf), lam = 1 and strong decays."""
    for dtype, odt in (("bf16", torch.bfloat16), ("fp32", torch.float32)):
        x, cu, S0, _ = make([200, 40], 1, 4, 128, 128, dtype, seed=19)
        x["g"] = torch.tensor([float("-inf"), 0.0, -8.0, -0.7])
        cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o, f = api.linear_prefill(*dev(x["q"], x["k"], x["v"], x["g"]), cu_seqlens=cut, initial_state=S0.to(DEV), o_dtype=odt)
        torch.cuda.synchronize()
        ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0)
        R.check(f, F, Fm, rel32([200], 128), "final state", R.U32)
        R.check(o, ref, om, 2 * R.UB16 if dtype == "bf16" else rel32([200], 128), "o",
                R.UB16 if dtype == "bf16" else R.U32)


def test_bad_cu_seqlens():
    """Inconsistent offsets are recorded in the workspace and nothing is run on them."""
    for T, bad in ((300, [0, 200, 100, 300]), (300, [0, 100, 299]), (3000, [5, 3000]), (3000, [0, 3001]),
                   (3000, [0, 2000, 1000, 3000])):
        x, _, _, r = make([T], 1, 1, 64, 64, "fp32", seed=1)
        for backward in (False, True):
            ws = torch.zeros(api.linear_prefill_workspace_size(len(bad) - 1, T, 1, 1, 64, 64, torch.float32, backward),
                             dtype=torch.uint8, device=DEV)
            cut = torch.tensor(bad, dtype=torch.int32, device=DEV)
            args = dev(x["q"], x["k"], x["v"], x["g"])
            if backward:
                api.linear_prefill_backward(*args, args[2], cu_seqlens=cut, workspace=ws)
            else:
                api.linear_prefill(*args, cu_seqlens=cut, workspace=ws)
            assert api.get_device_status(ws) == api.GDN_ERR_BAD_SEQLENS
            assert api.get_device_status(ws) == api.GDN_OK


def test_many_sequences():
    """More sequences than the plan's sorted table and than one pass of its scan."""
    gen = torch.Generator().manual_seed(4)
    L = torch.randint(0, 9, (1300,), generator=gen).tolist() + [1100]
    x, cu, S0, _ = make(L, 1, 1, 64, 64, "bf16", seed=21)
    x["v"] = x["v"].contiguous()
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, f = api.linear_prefill(*dev(x["q"], x["k"], x["v"], x["g"]), cu_seqlens=cut, initial_state=S0.to(DEV))
    torch.cuda.synchronize()
    ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0)
    R.check(o, ref, om, rel32(L, 64), "o", R.U32)
    R.check(f, F, Fm, rel32(L, 64), "final state", R.U32)


@pytest.mark.parametrize("D", [64, 128])
def test_graph_and_streams(D):
    """Forward, backward and decode on a side stream and from a graph with its own
    workspaces, while eager calls use others: the same bits."""
    L = [2100, 33, 0, 450]
    x, cu, S0, r = make(L, 2, 4, D, D, "bf16", seed=23)
    T, N = sum(L), len(L)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    do = r(T, 4, D).to(torch.bfloat16).to(DEV)
    q, k, v, g = dev(x["q"], x["k"], x["v"], x["g"])
    s0 = S0.to(DEV)
    size = lambda b: api.linear_prefill_workspace_size(N, T, 2, 4, D, D, torch.bfloat16, b)  # noqa: E731

    def calls(ws, wb):
        o, f = api.linear_prefill(q, k, v, g, cu_seqlens=cut, initial_state=s0, o_dtype=torch.bfloat16, workspace=ws)
        grads = api.linear_prefill_backward(q, k, v, g, do, cu_seqlens=cut, initial_state=s0, d_final_state=s0, workspace=wb)
        o1 = api.linear_decode_tokens(q[None, :N].transpose(0, 1).contiguous(), k[None, :N].transpose(0, 1).contiguous(),
                                      v[None, :N].transpose(0, 1).contiguous(), g, f)
        return [o, f, o1, *grads]

    spaces = lambda: [torch.zeros(size(b), dtype=torch.uint8, device=DEV) for b in (False, True)]  # noqa: E731
    eager_ws, graph_ws = spaces(), spaces()
    eager = calls(*eager_ws)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        aside = calls(*graph_ws)
    torch.cuda.current_stream(DEV).wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed = calls(*graph_ws)
    graph.replay()
    again = calls(*eager_ws)
    torch.cuda.synchronize()
    for a, b, c, d in zip(eager, aside, graphed, again):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)


@pytest.mark.parametrize("Hqk,Hv", [(1, 3), (2, 2)])
@pytest.mark.parametrize("n", [700, 2300])
def test_gradients_of_a_sequence_do_not_depend_on_its_neighbours(Hqk, Hv, n):
    """The values of the sequences before and after are not finite; bit for bit."""
    x, _, S0, r = make([n], Hqk, Hv, 128, 128, "bf16", seed=33)
    do, dsf = r(n, Hv, 128).to(torch.bfloat16), r(1, Hv, 128, 128)
    one = api.linear_prefill_backward(*dev(x["q"], x["k"], x["v"], x["g"], do), initial_state=S0.to(DEV),
                                      d_final_state=dsf.to(DEV))
    wide = [torch.cat([torch.full_like(t[:77], float("nan")), t, torch.full_like(t[:200], float("inf"))])
            for t in (x["q"], x["k"], x["v"], do)]
    cut = torch.tensor([0, 77, 77 + n, 277 + n], dtype=torch.int32, device=DEV)
    three = lambda t: t.expand(3, *t.shape[1:]).contiguous()  # noqa: E731
    # (as many tokens as cut the sequence the same way: its share of a multiprocessor is rounded to chunks)
    many = api.linear_prefill_backward(*dev(*wide[:3], x["g"], wide[3]), cu_seqlens=cut,
                                       initial_state=three(S0).to(DEV), d_final_state=three(dsf).to(DEV))
    torch.cuda.synchronize()
    for name, a, b in zip(("dq", "dk", "dv"), one, many):
        b = b[77:77 + n]
        assert torch.isfinite(b).all(), name
        if n < 1000:
            assert torch.equal(a, b), name
        else:  # cut at other places: the roundings of the operands differ
            assert float((a.float() - b.float()).norm() / a.float().norm()) <= R.UB16, name
    assert torch.isfinite(many[3][1]).all()


def test_largest_pool_offsets():
    """A slot whose byte offset passes 32 bits (fp32 pool of 2,200 slots of 2 MB)."""
    Hv, D, slots = 32, 128, 2200
    x, _, _, r = make([2], 1, Hv, D, D, "bf16", seed=35)
    pool = torch.zeros(slots, Hv, D, D, device=DEV)
    last = r(Hv, D, D)
    pool[-1].copy_(last.to(DEV))
    src = torch.tensor([slots - 1], dtype=torch.int32, device=DEV)
    q, k, v, g = dev(x["q"], x["k"], x["v"], x["g"])
    par = torch.tensor([[-1, 0]], dtype=torch.int32, device=DEV)
    ot = api.decode_tree(q[None], k[None], v[None], g, None, par, pool, src_slot=src)
    o = api.linear_decode_tokens(q[None], k[None], v[None], g, pool, src_slot=src)
    torch.cuda.synchronize()
    ref, om, S, Sm, _ = R.tree(x["q"], x["k"], x["v"], x["g"], None, [-1, 0], last)
    R.check(ot[0], ref, om, R.gamma(D, 2, 2.0 ** -22, 18), "tree", R.U32)
    R.check(o[0], ref, om, R.gamma(D, 2), "decode", R.U32)
    R.check(pool[-1], S[1], Sm[1], R.gamma(1, 2), "state", R.U32)
    assert not pool[:-1].any()


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace and outputs."""
    L = [2500, 40]
    x, cu, S0, r = make(L, 4, 8, 128, 128, "bf16", seed=37)
    do = r(sum(L), 8, 128).to(torch.bfloat16).to(DEV)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    a, s0 = dev(x["q"], x["k"], x["v"], x["g"]), S0.to(DEV)
    size = lambda b: api.linear_prefill_workspace_size(2, sum(L), 4, 8, 128, 128, torch.bfloat16, b)  # noqa: E731

    def calls(ws, wb):
        return [*api.linear_prefill(*a, cu_seqlens=cut, initial_state=s0, o_dtype=torch.bfloat16, workspace=ws),
                *api.linear_prefill_backward(*a, do, cu_seqlens=cut, initial_state=s0, d_final_state=s0, workspace=wb)]

    spaces = [[torch.zeros(size(b), dtype=torch.uint8, device=DEV) for b in (False, True)] for _ in range(2)]
    want = calls(*spaces[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for _ in range(4):
        got = []
        for st, sp in zip(streams, spaces):
            with torch.cuda.stream(st):
                got.append(calls(*sp))
        torch.cuda.synchronize()
        for g in got:
            for u, v in zip(want, g):
                assert torch.equal(u, v)
    assert all(api.get_device_status(w) == api.GDN_OK for sp in spaces for w in sp)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_cut_sequences_among_many(dtype):
    """Over a thousand sequences, a few of them long enough to be cut into segments:
    outputs, final states, and the gradients that pass through the states."""
    L = [i % 4 for i in range(1200)]
    for i, n in ((10, 900), (500, 1700), (501, 700), (1030, 333), (1199, 1100)):
        L[i] = n
    x, cu, S0, r = make(L, 1, 2, 64, 64, dtype, seed=43)
    do, dsf = r(sum(L), 2, 64).to(DT[dtype]), r(len(L), 2, 64, 64) * 0.5
    args = dev(x["q"], x["k"], x["v"], x["g"])
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, f = api.linear_prefill(*args, cu_seqlens=cut, initial_state=S0.to(DEV), o_dtype=DT[dtype])
    dq, dk, dv, ds0 = api.linear_prefill_backward(*args, do.to(DEV), cu_seqlens=cut, initial_state=S0.to(DEV),
                                                  d_final_state=dsf.to(DEV))
    torch.cuda.synchronize()
    ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0)
    R.check(f, F, Fm, rel32(L, 64), "final state", R.U32)
    stored = R.UB16 if dtype == "bf16" else R.U32
    R.check(o, ref, om, 2 * R.UB16 if dtype == "bf16" else rel32(L, 64), "o", stored)
    tol = rel32(L, 64) + 2 * R.U32
    for got, w, m, name in zip((dq, dk, dv, ds0), *grads_ref(x, cu, S0, do, dsf, 1.0), ("dq", "dk", "dv", "dS0")):
        exact = dtype == "fp32" or name == "dS0"
        R.check(got, w, m, tol if exact else 2 * R.UB16, name, R.U32 if exact else R.UB16)


def test_workspace_of_a_larger_call():
    """A workspace made for more tokens serves fewer, which are cut more finely."""
    x, _, _, r = make([19200], 1, 1, 64, 64, "bf16", seed=51)
    do = r(19200, 1, 64).to(torch.bfloat16).to(DEV)
    a = dev(x["q"], x["k"], x["v"])
    g = x["g"].to(DEV)
    ws = [torch.zeros(api.linear_prefill_workspace_size(1, 19200, 1, 1, 64, 64, torch.bfloat16, b), dtype=torch.uint8,
                      device=DEV) for b in (False, True)]
    for T in (19200, 18944, 9000, 300, 1):
        part = [t[:T] for t in a]
        for odt in (torch.bfloat16, torch.float32):
            got = api.linear_prefill(*part, g, o_dtype=odt, workspace=ws[0])
            want = api.linear_prefill(*part, g, o_dtype=odt)
            assert all(torch.equal(u, v) for u, v in zip(got, want))
        got = api.linear_prefill_backward(*part, g, do[:T], workspace=ws[1])
        want = api.linear_prefill_backward(*part, g, do[:T])
        assert all(torch.equal(u, v) for u, v in zip(got, want) if u is not None)
    assert all(api.get_device_status(w) == api.GDN_OK for w in ws)
