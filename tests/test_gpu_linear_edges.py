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
