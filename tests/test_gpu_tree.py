"""Trees of drafted tokens over cached states (gdn_decode_tree, gdn_tree_commit)
and linear decode (gdn_linear_decode_tokens) on the GPU against the fp64
definitions, element by element.

Tolerances (tests/linear_ref.py): the error bound of the arithmetic times the
value's magnitude.  ``split`` is what an operand loses when it enters a tensor-core
product as bf16 terms: 2^-24 with three terms, 2^-16 with two (bf16 inputs and o).
"""
import pytest
import torch

import linear_ref as R
from gated_deltanet_recurrence_rule_b200 import api

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(B, M, Hqk, Hv, Dk, Dv, dtype="bf16", sdtype="fp32", rule="delta", shape="random", seed=0, slots=None,
         raw=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=r(B, M, Hqk, Dk), k=r(B, M, Hqk, Dk), v=r(B, M, Hv, Dv).to(DT[dtype]))
    for n in ("q", "k"):
        x[n] = (x[n] if raw else unit(x[n])).to(DT[dtype])
    if rule == "delta":
        x["g"] = r(B, M, Hv) if raw else -torch.nn.functional.softplus(r(B, M, Hv))
        x["beta"] = r(B, M, Hv) if raw else torch.sigmoid(r(B, M, Hv))
    else:
        x["g"], x["beta"] = -torch.exp(r(Hv) - 2), None
    par = torch.empty(B, M, dtype=torch.int32)
    for b in range(B):
        for i in range(M):
            par[b, i] = {"chain": i - 1, "star": -1}.get(shape, int(torch.randint(-1, i, (1,), generator=gen)) if i else -1)
    pool = (r(slots or B, Hv, Dv, Dk) * 0.5).to(DT[sdtype])
    return x, par, pool


def gpu(x):
    return {n: (None if t is None else t.to(DEV)) for n, t in x.items()}


def split_of(dtype, odtype, sdtype):
    if dtype == "bf16" and odtype == "bf16":
        return 2.0 ** -16 if sdtype == "fp32" else 0.0
    return 2.0 ** -22  # three terms (2^-24) and the dropped products of their rests


def check_tree(o, x, par, pool, src, odtype, dtype, sdtype, scale=1.0, raw=False, what=""):
    Dk = x["k"].shape[3]
    for b in range(par.shape[0]):
        gate = (x["g"], None) if x["beta"] is None else (x["g"][b], x["beta"][b])
        ref, mag, _, _, depth = R.tree(x["q"][b], x["k"][b], x["v"][b], *gate, par[b].tolist(), pool[src[b]],
                                       scale, raw)
        rel = R.gamma(Dk, max(depth.values()), split_of(dtype, odtype, sdtype), extra=16 + par.shape[1])
        R.check(o[b], ref, mag, rel, f"{what} sequence {b}", R.UB16 if odtype == "bf16" else R.U32)


@pytest.mark.parametrize("dtype,odtype,sdtype", [("bf16", "bf16", "fp32"), ("bf16", "fp32", "fp32"),
                                                 ("bf16", "bf16", "bf16"), ("bf16", "fp32", "bf16"),
                                                 ("fp32", "fp32", "fp32"), ("fp32", "bf16", "bf16")])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("M,shape", [(1, "random"), (7, "random"), (16, "chain"), (33, "random")])
def test_tree_types_and_dims(dtype, odtype, sdtype, Dk, Dv, M, shape):
    x, par, pool = make(2, M, 2, 6, Dk, Dv, dtype, sdtype, shape=shape, seed=M + Dk + 2 * Dv, slots=5)
    src = [4, 1]
    o = api.decode_tree(**gpu(x), parent=par.to(DEV), state=pool.to(DEV), scale=0.5, o_dtype=DT[odtype],
                        src_slot=torch.tensor(src, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    check_tree(o, x, par, pool, src, odtype, dtype, sdtype, 0.5)


@pytest.mark.parametrize("rule", ["delta", "linear"])
@pytest.mark.parametrize("shape", ["random", "chain", "star"])
@pytest.mark.parametrize("M", [2, 8, 17, 32, 64])
def test_tree_shapes(rule, shape, M):
    x, par, pool = make(3, M, 1, 4, 128, 128, rule=rule, shape=shape, seed=100 + M)
    o = api.decode_tree(**gpu(x), parent=par.to(DEV), state=pool.to(DEV))
    torch.cuda.synchronize()
    check_tree(o, x, par, pool, [0, 1, 2], "fp32", "bf16", "fp32", what=f"{rule} {shape}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tree_raw_inputs(dtype):
    x, par, pool = make(2, 12, 2, 4, 128, 64, dtype, seed=7, raw=True)
    x["k"][0, 3] = 0  # a zero row stays zero
    o = api.decode_tree(**gpu(x), parent=par.to(DEV), state=pool.to(DEV), raw_inputs=True)
    torch.cuda.synchronize()
    check_tree(o, x, par, pool, [0, 1], "fp32", dtype, "fp32", raw=True)


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_padding_and_other_branches(rule):
    """Padding nodes and sequences are neither read nor written, and a NaN or an
    infinity stays on its branch."""
    B, M, Hv = 3, 20, 4
    x, par, pool = make(B, M, 2, Hv, 128, 128, rule=rule, seed=11, slots=6)
    par[0] = torch.tensor([-1, 0, -1, 2, 2, -1, 5, 6, 1, 1, 9, -7, -2, 9, 3, 3, 15, -1, 17, -2])
    pad = (par[0] < -1).nonzero().flatten().tolist()
    bad = [5, 6, 7]          # node 5 and what follows it
    clean = {n: (None if t is None else t.clone()) for n, t in x.items()}
    for i in pad:
        for n in ("q", "k", "v"):
            x[n][0, i] = float("nan")
    x["k"][0, 5] = float("inf")
    x["v"][0, 5] = float("nan")
    src = torch.tensor([2, -1, 5], dtype=torch.int32)
    o = torch.full((B, M, Hv, 128), 7.0, device=DEV)
    pg = pool.to(DEV)
    api.decode_tree(**gpu(x), parent=par.to(DEV), state=pg, src_slot=src.to(DEV), o=o)
    torch.cuda.synchronize()
    assert torch.equal(pg.cpu(), pool)
    assert (o[0, pad] == 7).all() and (o[1] == 7).all()
    good = [i for i in range(M) if i not in pad and i not in bad]
    gate = (clean["g"], None) if rule == "linear" else (clean["g"][0], clean["beta"][0])
    ref, mag, _, _, depth = R.tree(clean["q"][0], clean["k"][0], clean["v"][0], *gate, par[0].tolist(), pool[2])
    R.check(o[0, good], ref[good], mag[good], R.gamma(128, max(depth.values()), 2.0 ** -22, 16 + M), "clean branches")
    assert torch.isnan(o[0, bad]).all()


def test_zero_decay_and_extreme_gates():
    """alpha = 0 (g = -inf) forgets the path before it; beta = 0 and 1."""
    x, par, pool = make(2, 24, 2, 6, 64, 64, seed=13)
    x["g"][:, ::5] = float("-inf")
    x["g"][:, 1::5] = 0.0
    x["beta"][:, ::3] = 1.0
    x["beta"][:, 1::3] = 0.0
    o = api.decode_tree(**gpu(x), parent=par.to(DEV), state=pool.to(DEV))
    torch.cuda.synchronize()
    assert torch.isfinite(o).all()
    check_tree(o, x, par, pool, [0, 1], "fp32", "bf16", "fp32")


def test_bad_parents_and_slots_are_reported():
    x, par, pool = make(4, 6, 1, 2, 64, 64, seed=17, slots=4)
    par[0, 2] = 2                      # itself
    par[1, 1], par[1, 3] = -2, 1       # a padding node
    src = torch.tensor([0, 1, 9, 3], dtype=torch.int32, device=DEV)
    for only in (0, 1, 2):
        sl = src.clone()
        sl[[i for i in (0, 1, 2) if i != only]] = -1
        o = torch.full((4, 6, 2, 64), 7.0, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        api.decode_tree(**gpu(x), parent=par.to(DEV), state=pool.to(DEV), src_slot=sl, o=o, device_status=st)
        torch.cuda.synchronize()
        assert int(st) == api.GDN_ERR_INVALID_ARG
        assert (o[:3] == 7).all() and (o[3] != 7).any()


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("rule,raw", [("delta", False), ("delta", True), ("linear", False)])
@pytest.mark.parametrize("sdtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dtype,Dk,Dv,M,shape", [("bf16", 128, 128, 32, "random"), ("bf16", 64, 128, 9, "chain"),
                                                 ("fp32", 128, 64, 64, "chain"), ("fp32", 64, 64, 1, "chain")])
def test_commit(rule, raw, sdtype, dtype, Dk, Dv, M, shape):
    B = 4
    x, par, pool = make(B, M, 2, 6, Dk, Dv, dtype, sdtype, rule, shape, seed=200 + M, slots=9, raw=raw)
    src, dst, acc = [7, 0, -1, 3], [1, 0, 4, 5], [M - 1, -1, 0, M // 2]
    pin, pout = pool.to(DEV), torch.full_like(pool, float("nan")).to(DEV)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device=DEV)  # noqa: E731
    g = gpu(x)
    st = i32([0])
    api.tree_commit(g["k"], g["v"], g["g"], g["beta"], par.to(DEV), i32(acc), pin, pout, src_slot=i32(src),
                    dst_slot=i32(dst), raw_inputs=raw, device_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(pin.cpu(), pool)
    written = [dst[b] for b in range(B) if src[b] >= 0]
    assert torch.isnan(pout[[s for s in range(9) if s not in written]]).all()
    for b in range(B):
        if src[b] < 0:
            continue
        gate = (x["g"], None) if rule == "linear" else (x["g"][b], x["beta"][b])
        _, _, S, Sm, depth = R.tree(x["q"][b], x["k"][b], x["v"][b], *gate, par[b].tolist(), pool[src[b]], raw=raw)
        a = acc[b]
        R.check(pout[dst[b]], S[a], Sm[a], R.gamma(Dk, depth[a]) if a >= 0 else 0.0, f"sequence {b}",
                R.UB16 if sdtype == "bf16" else R.U32)
        if a < 0:
            assert torch.equal(pout[dst[b]].cpu(), pool[src[b]])


def test_commit_refuses_bad_paths():
    x, par, pool = make(4, 6, 1, 2, 64, 64, seed=31)
    par[0, 1] = -2                      # accept names a padding node
    par[1, 3], par[1, 5] = 5, 3         # a path that would go round
    acc = torch.tensor([1, 5, 6, 2], dtype=torch.int32, device=DEV)  # 6: no node
    for only in (0, 1, 2):
        sl = torch.tensor([i if i in (only, 3) else -1 for i in range(4)], dtype=torch.int32, device=DEV)
        out = torch.full_like(pool, 7.0).to(DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        g = gpu(x)
        api.tree_commit(g["k"], g["v"], g["g"], g["beta"], par.to(DEV), acc, pool.to(DEV), out, src_slot=sl,
                        device_status=st)
        torch.cuda.synchronize()
        assert int(st) == api.GDN_ERR_INVALID_ARG
        assert (out[:3] == 7).all() and (out[3] != 7).any()


def test_serving_loop():
    """Tree, acceptance, commit in place, and the next token by decode_tokens, on
    a side stream and replayed from a graph: the same bits as eager calls, and
    the definition's values."""
    B, M, Hqk, Hv, D = 5, 13, 2, 6, 128
    x, par, pool = make(B, M, Hqk, Hv, D, D, seed=41)
    nxt, _, _ = make(B, 1, Hqk, Hv, D, D, seed=42)
    acc = torch.tensor([12, 3, -1, 0, 7], dtype=torch.int32)
    g, n, pg, ag = gpu(x), gpu(nxt), par.to(DEV), acc.to(DEV)

    def calls(state, o, o1):
        api.decode_tree(**g, parent=pg, state=state, o=o)
        api.tree_commit(g["k"], g["v"], g["g"], g["beta"], pg, ag, state)
        api.decode_tokens(n["q"], n["k"], n["v"], n["g"], n["beta"], state, o=o1)

    def buffers():
        return pool.to(DEV), torch.zeros(B, M, Hv, D, device=DEV), torch.zeros(B, 1, Hv, D, device=DEV)

    eager, graphed = buffers(), buffers()
    calls(*eager)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        calls(*graphed)
    torch.cuda.current_stream(DEV).wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(eager, graphed):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(*graphed)
    graphed[0].copy_(pool)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, graphed):
        assert torch.equal(a, b)
    for b in range(B):
        _, _, S, Sm, depth = R.tree(x["q"][b], x["k"][b], x["v"][b], x["g"][b], x["beta"][b], par[b].tolist(), pool[b])
        a = int(acc[b])
        ref, mag, _, _, _ = R.tree(nxt["q"][b], nxt["k"][b], nxt["v"][b], nxt["g"][b], nxt["beta"][b], [-1], S[a])
        _, mag, _, _, _ = R.tree(nxt["q"][b], nxt["k"][b], nxt["v"][b], nxt["g"][b], nxt["beta"][b], [-1], Sm[a])
        R.check(eager[2][b], ref, mag, R.gamma(D, depth[a] + 1), f"next token of {b}", R.U32)


# ---------------------------------------------------------------- linear decode
@pytest.mark.parametrize("dtype,odtype,sdtype", [("bf16", "bf16", "fp32"), ("bf16", "fp32", "bf16"),
                                                 ("fp32", "fp32", "fp32"), ("fp32", "bf16", "bf16")])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("Tn", [1, 2, 5, 16])
def test_linear_decode(dtype, odtype, sdtype, Dk, Dv, Tn):
    B, Hqk, Hv = 4, 2, 6
    x, _, pool = make(B, Tn, Hqk, Hv, Dk, Dv, dtype, sdtype, "linear", seed=300 + Tn, slots=9)
    x["g"][0], x["g"][1], x["g"][2] = 0.0, -1e-5, -5.0
    src, dst = [7, 0, -1, 3], [1, 0, 4, 5]
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device=DEV)  # noqa: E731
    pin, pout = pool.to(DEV), torch.full_like(pool, float("nan")).to(DEV)
    o = torch.full((B, Tn, Hv, Dv), 7.0, dtype=DT[odtype], device=DEV)
    g = gpu(x)
    api.linear_decode_tokens(g["q"], g["k"], g["v"], g["g"], pin, pout, src_slot=i32(src), dst_slot=i32(dst), o=o,
                             scale=0.25)
    torch.cuda.synchronize()
    assert (o[2] == 7).all() and torch.equal(pin.cpu(), pool)
    assert torch.isnan(pout[[2, 3, 4, 6, 7, 8]]).all()
    for b in (0, 1, 3):
        ref, mag, S, Sm, _ = R.tree(x["q"][b], x["k"][b], x["v"][b], x["g"], None, list(range(-1, Tn - 1)),
                                    pool[src[b]], 0.25)
        R.check(o[b], ref, mag, R.gamma(Dk, Tn), "o", R.UB16 if odtype == "bf16" else R.U32)
        R.check(pout[dst[b]], S[Tn - 1], Sm[Tn - 1], R.gamma(1, Tn), "state", R.UB16 if sdtype == "bf16" else R.U32)


def test_linear_decode_in_place_bad_slots_and_zero_decay():
    B, Tn, Hv, D = 4, 3, 4, 128
    x, _, pool = make(B, Tn, 1, Hv, D, D, rule="linear", seed=51, slots=6)
    x["g"][0] = float("-inf")  # forgets at once: o_t = scale (k_t . q_t) v_t
    g, state = gpu(x), pool.to(DEV)
    o = torch.full((B, Tn, Hv, D), 7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    src = torch.tensor([5, 6, -3, 0], dtype=torch.int32, device=DEV)
    api.linear_decode_tokens(g["q"], g["k"], g["v"], g["g"], state, src_slot=src, o=o, device_status=st)
    torch.cuda.synchronize()
    assert int(st) == api.GDN_ERR_INVALID_ARG
    assert (o[1:3] == 7).all() and torch.equal(state[1:5].cpu(), pool[1:5])
    x["g"][0] = -30.0
    for b, s in ((0, 5), (3, 0)):
        ref, mag, S, Sm, _ = R.tree(x["q"][b], x["k"][b], x["v"][b], x["g"], None, [-1, 0, 1], pool[s])
        R.check(o[b], ref, mag, R.gamma(D, Tn), "o", R.U32)
        R.check(state[s], S[Tn - 1], Sm[Tn - 1], R.gamma(1, Tn), "state", R.U32)
