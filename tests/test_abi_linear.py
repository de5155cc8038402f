"""Host-side refusals of the linear-attention and token-tree entry points (no GPU
needed, no kernel launched; the fake addresses are never dereferenced)."""
import pytest
import torch

from gated_deltanet_recurrence_rule_b200 import api

BAD, UNSUP, OK = api.GDN_ERR_INVALID_ARG, api.GDN_ERR_UNSUPPORTED, api.GDN_OK


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_recurrence_rule_b200 import build

    build.build()
    return api.load()


P = 1 << 12
DIMS = dict(Hqk=2, Hv=6, Dk=64, Dv=64)


def decode(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, si=P, so=P, src=None, dst=None, slots=4, o=P, B=2, Tn=3, dt=0, odt=1, sdt=1,
             status=None, **DIMS)
    a.update(kw)
    return lib.gdn_linear_decode_tokens(a["q"], a["k"], a["v"], a["g"], a["si"], a["so"], a["src"], a["dst"],
                                        a["slots"], a["o"], a["B"], a["Tn"], a["Hqk"], a["Hv"], a["Dk"], a["Dv"],
                                        a["dt"], a["odt"], a["sdt"], 1.0, a["status"], None)


def tree(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, par=P, s=P, src=None, slots=4, o=P, B=2, M=3, dt=0, odt=1, sdt=1, form=0,
             status=None, **DIMS)
    a.update(kw)
    return lib.gdn_decode_tree(a["q"], a["k"], a["v"], a["g"], a["beta"], a["par"], a["s"], a["src"], a["slots"],
                               a["o"], a["B"], a["M"], a["Hqk"], a["Hv"], a["Dk"], a["Dv"], a["dt"], a["odt"],
                               a["sdt"], a["form"], 1.0, a["status"], None)


def commit(lib, **kw):
    a = dict(k=P, v=P, g=P, beta=P, par=P, acc=P, si=P, so=P, src=None, dst=None, slots=4, B=2, M=3, dt=0, sdt=1,
             form=0, status=None, **DIMS)
    a.update(kw)
    return lib.gdn_tree_commit(a["k"], a["v"], a["g"], a["beta"], a["par"], a["acc"], a["si"], a["so"], a["src"],
                               a["dst"], a["slots"], a["B"], a["M"], a["Hqk"], a["Hv"], a["Dk"], a["Dv"], a["dt"],
                               a["sdt"], a["form"], a["status"], None)


def prefill(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, cu=P, N=1, T=16, dt=0, odt=1, sdt=1, scale=1.0, s0=None, sf=None, o=P, ws=P,
             wsb=1 << 20, **DIMS)
    a.update(kw)
    return lib.gdn_linear_prefill(a["q"], a["k"], a["v"], a["g"], a["cu"], a["N"], a["T"], a["Hqk"], a["Hv"], a["Dk"],
                                  a["Dv"], a["dt"], a["odt"], a["sdt"], a["scale"], a["s0"], a["sf"], a["o"], a["ws"],
                                  a["wsb"], None)


def backward(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, cu=P, N=1, T=16, dt=0, scale=1.0, s0=None, do=P, dsf=None, dq=P, dk=P, dv=P, ds0=None,
             ws=P, wsb=1 << 20, **DIMS)
    a.update(kw)
    return lib.gdn_linear_prefill_backward(a["q"], a["k"], a["v"], a["g"], a["cu"], a["N"], a["T"], a["Hqk"], a["Hv"],
                                           a["Dk"], a["Dv"], a["dt"], a["scale"], a["s0"], a["do"], a["dsf"], a["dq"],
                                           a["dk"], a["dv"], a["ds0"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [prefill, backward])
def test_packed_refusals(lib, call):
    assert call(lib, Hv=5) == BAD and call(lib, Hqk=0) == BAD and call(lib, dt=2) == BAD
    assert call(lib, Dk=96) == UNSUP and call(lib, Dv=256) == UNSUP and call(lib, Dv=0) == BAD
    assert call(lib, N=-1) == BAD and call(lib, T=-1) == BAD and call(lib, T=2 ** 31) == BAD
    assert call(lib, N=0, T=0) == OK and call(lib, N=0, T=5) == BAD
    assert call(lib, N=2 ** 30, T=16) == UNSUP         # more CTAs than a grid takes
    for name in ("q", "k", "v", "g", "cu"):
        assert call(lib, **{name: None}) == BAD
    for name in ("q", "k", "v"):
        assert call(lib, **{name: P + 8}) == BAD       # bases are 16-byte aligned
    assert call(lib, g=P + 2) == BAD and call(lib, cu=P + 2) == BAD and call(lib, s0=P + 8) == BAD
    assert call(lib, ws=None) == api.GDN_ERR_WORKSPACE and call(lib, ws=P + 16) == api.GDN_ERR_WORKSPACE
    assert call(lib, wsb=255) == api.GDN_ERR_WORKSPACE
    need = lib.gdn_linear_prefill_workspace_size(3, 9000, 2, 6, 64, 64, 0, int(call is backward))
    assert need > 256
    assert call(lib, N=3, T=9000, wsb=need - 1) == api.GDN_ERR_WORKSPACE


def test_prefill_and_backward_outputs_are_checked(lib):
    assert prefill(lib, o=None) == BAD and prefill(lib, o=P + 8) == BAD and prefill(lib, sf=P + 8) == BAD
    assert prefill(lib, odt=2) == BAD and prefill(lib, sdt=2) == BAD
    for name in ("do", "dq", "dk", "dv"):
        assert backward(lib, **{name: None}) == BAD and backward(lib, **{name: P + 8}) == BAD
    assert backward(lib, dsf=P + 8) == BAD and backward(lib, ds0=P + 8) == BAD


def test_workspace_sizes(lib):
    size = lib.gdn_linear_prefill_workspace_size
    assert size(1, 16, 2, 6, 64, 64, 0, 0) >= 256
    assert size(1, 8192, 16, 48, 128, 128, 0, 1) > size(1, 8192, 16, 48, 128, 128, 0, 0) > 256
    assert size(1, 8192, 16, 48, 96, 128, 0, 0) == 0 and size(-1, 8, 2, 6, 64, 64, 0, 0) == 0
    assert size(1, 8, 2, 5, 64, 64, 0, 0) == 0 and size(1, 8, 2, 6, 64, 64, 7, 0) == 0


@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (2, 8), (16, 48), (25, 75), (100, 200)])
@pytest.mark.parametrize("backward", [0, 1])
def test_workspace_serves_smaller_calls(lib, Hqk, Hv, backward):
    last = 0
    for T in [*range(0, 6000, 64), 18944, 19200, 19300, 40000, 262144, 2 ** 31 - 1]:
        sizes = [lib.gdn_linear_prefill_workspace_size(N, T, Hqk, Hv, 128, 128, 0, backward) for N in (1, 2, 70, 1000)]
        assert sizes == sorted(sizes) and sizes[0] >= last
        last = sizes[0]


@pytest.mark.parametrize("call", [decode, tree, commit])
def test_common_refusals(lib, call):
    assert call(lib, Hv=5) == BAD and call(lib, Hqk=0) == BAD and call(lib, Hv=-6) == BAD
    assert call(lib, dt=2) == BAD and call(lib, sdt=2) == BAD
    assert call(lib, Dk=96) == UNSUP and call(lib, Dv=256) == UNSUP and call(lib, Dk=0) == BAD
    assert call(lib, B=-1) == BAD and call(lib, slots=-1) == BAD
    assert call(lib, B=5) == BAD                       # no slot map: needs batch <= slots
    assert call(lib, B=2 ** 30, slots=2 ** 30) == UNSUP  # more CTAs than a grid takes
    for name in ("k", "v", "g"):
        assert call(lib, **{name: None}) == BAD
        assert call(lib, **{name: P + 2}) == BAD       # misaligned
    assert call(lib, src=P + 1) == BAD and call(lib, status=P + 2) == BAD
    assert call(lib, B=0) == OK


def test_decode_refusals(lib):
    assert decode(lib, Tn=17) == UNSUP and decode(lib, Tn=-1) == BAD and decode(lib, Tn=0) == OK
    assert decode(lib, odt=7) == BAD
    for name in ("q", "si", "so", "o"):
        assert decode(lib, **{name: None}) == BAD
    for name in ("q", "si", "so", "o"):
        assert decode(lib, **{name: P + 8}) == BAD


def test_tree_refusals(lib):
    assert tree(lib, M=65) == UNSUP and tree(lib, M=-1) == BAD and tree(lib, M=0) == OK
    assert tree(lib, form=5) == BAD and tree(lib, odt=7) == BAD
    assert tree(lib, beta=None, form=1) == BAD         # the linear rule has no gates to map
    for name in ("q", "par", "s", "o"):
        assert tree(lib, **{name: None}) == BAD
    assert tree(lib, par=P + 2) == BAD and tree(lib, s=P + 8) == BAD and tree(lib, beta=P + 2) == BAD


def test_commit_refusals(lib):
    assert commit(lib, M=65) == UNSUP and commit(lib, M=0) == OK
    assert commit(lib, form=5) == BAD and commit(lib, beta=None, form=1) == BAD
    for name in ("par", "acc", "si", "so"):
        assert commit(lib, **{name: None}) == BAD
    assert commit(lib, acc=P + 2) == BAD and commit(lib, so=P + 8) == BAD and commit(lib, dst=P + 1) == BAD


def test_python_refuses_cpu_tensors(lib):
    x = torch.zeros(1, 2, 2, 64)
    v = torch.zeros(1, 2, 6, 64)
    s = torch.zeros(1, 6, 64, 64)
    g = torch.zeros(6)
    p = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_decode_tokens(x, x, v, g, s)
    with pytest.raises(ValueError, match="CUDA"):
        api.decode_tree(x, x, v, g, None, p, s)
    with pytest.raises(ValueError, match="CUDA"):
        api.tree_commit(x, v, g, None, p, p[:, 0], s)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_prefill(x[0], x[0], v[0], g)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_prefill_backward(x[0], x[0], v[0], g, v[0])
