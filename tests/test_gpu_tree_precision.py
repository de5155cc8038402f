"""fp32 trees keep fp32's precision in the root mean square, not only in the worst case.

Bound.  A product of S0 or k with a key or query of 128 elements is summed in 8 steps of
16.  Tensor cores cut a step's sum by at most 2^-23 of its own size; steps are 1 / sqrt(8)
of the whole and independent, so together 2 * 2^-24 of it.  Their additions round by at
most 2^-24, 2^-24 / sqrt(3) in rms: sqrt(8 / 3) * 2^-24.  A path of at most 32 nodes adds
sqrt(32 / 3) * 2^-24.  2 + 1.7 + 3.3 < 8: at most 2^-21 of the rms value, with the
products left out (3 * 2^-27).  (Cut after every one of 48 products instead, as sums in
one accumulator are, outputs were off by 2^-20.)"""
import pytest
import torch

import linear_ref as R
from gated_deltanet_recurrence_rule_b200 import api
from test_gpu_tree import DEV, gpu, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sdtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rule,shape,M", [("linear", "random", 27), ("delta", "random", 32), ("delta", "chain", 16),
                                          ("delta", "star", 5), ("linear", "chain", 32)])
@pytest.mark.parametrize("Dv", [64, 128])
def test_rms_error_of_fp32_trees(rule, shape, M, sdtype, Dv):
    x, par, pool = make(2, M, 2, 4, 128, Dv, "fp32", sdtype, rule, shape, seed=400 + M)
    o = api.decode_tree(**gpu(x), parent=par.to(DEV), state=pool.to(DEV), o_dtype=torch.float32)
    torch.cuda.synchronize()
    for b in range(2):
        gate = (x["g"], None) if rule == "linear" else (x["g"][b], x["beta"][b])
        ref, _, _, _, _ = R.tree(x["q"][b], x["k"][b], x["v"][b], *gate, par[b].tolist(), pool[b])
        err = float((R.d64(o[b]) - ref).norm() / ref.norm())
        assert err <= 2.0 ** -21, f"sequence {b}: relative rms error {err:.2e}"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_chains_of_one_decay(dtype):
    """The linear rule along 64 nodes from a large state, at decays that fall half way
    between two fp32 numbers: outputs of the last nodes and the committed state.  A power
    is off by 2^-23 at most, the sums along the path by sqrt(64 / 3) * 2^-24 in rms, the
    products as above or (bf16) by 24 cuts of 2^-24 in the mean where the state enters in
    three terms: below 2^-20 for the state and fp32, 2^-19 for bf16.  (64 factors, each off by
    2^-25, are off by 2^-19.)"""
    M, Hv = 64, 4
    x, par, pool = make(2, M, 1, Hv, 128, 64, dtype, "fp32", "linear", "chain", seed=500)
    pool = pool * 16
    g = -torch.exp(torch.linspace(-11.0, -6.0, 20001, dtype=torch.float64)).float()
    p = g.double().exp()
    x["g"] = g[(p.float().double() - p).abs().argsort(descending=True)[:Hv]].contiguous()
    d = gpu(x)
    o = api.decode_tree(**d, parent=par.to(DEV), state=pool.to(DEV), o_dtype=torch.float32)
    out = torch.zeros_like(pool, device=DEV)
    api.tree_commit(d["k"], d["v"], d["g"], None, par.to(DEV), torch.full((2,), M - 1, dtype=torch.int32, device=DEV),
                    pool.to(DEV), out)
    torch.cuda.synchronize()
    for b in range(2):
        ref, _, S, _, _ = R.tree(x["q"][b], x["k"][b], x["v"][b], x["g"], None, par[b].tolist(), pool[b])
        err = float((R.d64(o[b, -8:]) - ref[-8:]).norm() / ref[-8:].norm())
        assert err <= (2.0 ** -20 if dtype == "fp32" else 2.0 ** -19), f"o of {b}: {err:.2e}"
        err = float((R.d64(out[b]) - S[M - 1]).norm() / S[M - 1].norm())
        assert err <= 2.0 ** -20, f"state of {b}: {err:.2e}"
