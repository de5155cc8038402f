"""The bounded-wait path of the linear-attention tensor-core kernels, made to run out
on purpose without faulting or hanging anything.  With 144 CTAs that each ask for 96 KB
at once and nothing of it in L2 (14 MB: 2 us at 7 TB/s, and the latency), a limit of
1 us in the workspace header is shorter than some wait; the kernels record
GDN_ERR_DEVICE_TIMEOUT, let their own copies and MMAs finish, free their tensor memory
and return, and the next ordinary call with the same workspace is right."""
import pytest
import torch

import linear_ref as R
from gated_deltanet_recurrence_rule_b200 import api

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def set_limit(ws, us):
    ws[4:8].copy_(torch.tensor([us], dtype=torch.int32).view(torch.uint8).to(DEV))


@pytest.mark.parametrize("lens", [[300, 130, 77], [9000, 3, 400]])
@pytest.mark.parametrize("backward", [False, True])
def test_limit_runs_out_then_next_call_is_right(lens, backward):
    T, N = sum(lens), len(lens)
    gen = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(r(T, 16, 128)).bfloat16(), k=unit(r(T, 16, 128)).bfloat16(), v=r(T, 48, 128).bfloat16(),
             g=-torch.rand(48, generator=gen))
    S0 = r(N, 48, 128, 128)
    cu = [sum(lens[:i]) for i in range(N + 1)]
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    a = [t.to(DEV) for t in x.values()]
    ws = torch.zeros(api.linear_prefill_workspace_size(N, T, 16, 48, 128, 128, torch.bfloat16, backward),
                     dtype=torch.uint8, device=DEV)

    def call():
        if backward:
            return api.linear_prefill_backward(*a, a[2], cu_seqlens=cut, initial_state=S0.to(DEV), workspace=ws)
        return api.linear_prefill(*a, cu_seqlens=cut, initial_state=S0.to(DEV), o_dtype=torch.bfloat16, workspace=ws)

    want = call()
    assert api.get_device_status(ws) == api.GDN_OK
    set_limit(ws, 1)
    torch.zeros(1 << 29, dtype=torch.uint8, device=DEV)  # the inputs leave L2
    call()
    assert api.get_device_status(ws) == api.GDN_ERR_DEVICE_TIMEOUT
    set_limit(ws, 0)
    got = call()
    assert api.get_device_status(ws) == api.GDN_OK
    for u, v in zip(want, got):
        assert torch.equal(u, v)
    if not backward and T < 1000:
        ref, om, F, Fm = R.scan(x["q"], x["k"], x["v"], x["g"], cu, S0)
        R.check(got[0], ref, om, 2 * R.UB16, "o", R.UB16)
        R.check(got[1], F, Fm, 2.0 ** -15, "final state", R.U32)
