"""Linear attention with a decay for each head, and verification of drafted token
trees against cached recurrent states: cases, plain forms and exact values.

Five operators, all over a state S (Dv x Dk, fp32) of each (sequence, value head),
value head h reading query/key head h / (Hv / Hqk):

  prefill   S_t = lam_h S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t  over packed sequences,
            lam_h = e^{g_h} a constant of the head
  backward  dq, dk, dv and dS_initial of that, given do and dS_final
  decode    the same rule for 1 to 16 new tokens of each sequence, states in a slot pool
  tree      o of every node of a tree of drafted tokens over the cached states, which stay as
            they are; rule "delta" is S_i = a_i S_p (I - b_i k_i k_i^T) + b_i v_i k_i^T, a_i =
            e^{g_i}, p the node's parent, and rule "linear" the one above
  commit    the state after the accepted node of each tree, written to its slot

``own`` selects the framework's kernels in ``run``; without it ``run`` is the plain form.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt: a chat turn, where the launches are what is paid for
        dict(name="prefill_short", op="prefill", lens="77", Hqk=16, Hv=48, Dk=128, Dv=128, dtype="bf16",
             odtype="bf16", init=False, scale=1.0),
        # one 8192-token prompt at the framework's benchmark head layout, continued from a state
        dict(name="prefill_8k", op="prefill", lens="8192", Hqk=16, Hv=48, Dk=128, Dv=128, dtype="bf16",
             odtype="bf16", init=True, scale=1.0),
        # a packed batch of prompts of very different lengths, odd ones, an empty one and a single token
        dict(name="prefill_packed", op="prefill",
             lens="9001,1,0,4097,16384,777,63,64,65,2500,130,12000,5555,31,8191,6200", Hqk=16, Hv=48,
             Dk=128, Dv=128, dtype="bf16", odtype="bf16", init=True, scale=1.0),
        # fp32 inputs and narrow heads, as the small fp32 workloads have them
        dict(name="prefill_fp32", op="prefill", lens="1000,1,0,2049", Hqk=2, Hv=6, Dk=64, Dv=64,
             dtype="fp32", odtype="fp32", init=True, scale=0.125),
        # one training step of the 8192-token layer
        dict(name="backward_8k", op="backward", lens="8192", Hqk=16, Hv=48, Dk=128, Dv=128, dtype="bf16",
             init=True, scale=1.0),
        # training on short ragged samples in fp32
        dict(name="backward_fp32", op="backward", lens="300,1,0,1025,77", Hqk=2, Hv=6, Dk=64, Dv=64,
             dtype="fp32", init=True, scale=0.125),
        # the decode step of a served batch, states in fp32
        dict(name="decode_64", op="decode", B=64, M=1, Hqk=16, Hv=48, Dk=128, Dv=128, dtype="bf16",
             odtype="bf16", sdtype="fp32", scale=1.0),
        # one user's few verified tokens, states at rest in bf16
        dict(name="decode_1x4", op="decode", B=1, M=4, Hqk=16, Hv=48, Dk=128, Dv=128, dtype="bf16",
             odtype="bf16", sdtype="bf16", scale=1.0),
        # a served batch verifies 32 drafted tokens of each sequence, gated delta rule
        dict(name="tree_64x32", op="tree", rule="delta", shape="random", B=64, M=32, Hqk=16, Hv=48, Dk=128,
             Dv=128, dtype="bf16", odtype="bf16", sdtype="fp32", scale=1.0),
        # two users, small trees, linear rule, fp32 outputs
        dict(name="tree_2x7", op="tree", rule="linear", shape="random", B=2, M=7, Hqk=16, Hv=48, Dk=128,
             Dv=128, dtype="bf16", odtype="fp32", sdtype="fp32", scale=1.0),
        # what the served batch accepted goes into its states
        dict(name="commit_64x32", op="commit", rule="delta", shape="random", B=64, M=32, Hqk=16, Hv=48,
             Dk=128, Dv=128, dtype="bf16", sdtype="fp32"),
        # one user's accepted chain of drafted tokens, state at rest in bf16
        dict(name="commit_1x16", op="commit", rule="delta", shape="chain", B=1, M=16, Hqk=16, Hv=48, Dk=128,
             Dv=128, dtype="bf16", sdtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "backward", "decode", "tree", "commit"])
    Hqk = rng.choice([1, 2, 4, 8, 16])
    Hv = Hqk * rng.choice([1, 2, 3, 4])
    Dk, Dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    case = dict(op=op, Hqk=Hqk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype)
    odtype = "bf16" if dtype == "bf16" and rng.random() < 0.75 else "fp32"
    scale = rng.choice([1.0, 0.125, 0.5])
    if op in ("prefill", "backward"):
        most = 65536 if op == "prefill" else 8192
        if dtype == "fp32":
            most = 8192 if op == "prefill" else 2048
        total = _log_int(rng, 1, max(1, min(most, most * 48 // Hv)))
        n = _log_int(rng, 1, min(24, total + 1))
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        case.update(lens=",".join(map(str, lens)), init=rng.random() < 0.6, scale=scale)
        if op == "prefill":
            case.update(odtype=odtype)
        return case
    case.update(B=_log_int(rng, 1, 64), sdtype=rng.choice(["fp32", "fp32", "bf16"]))
    if op == "decode":
        case.update(M=_log_int(rng, 1, 16), odtype=odtype, scale=scale)
        return case
    case.update(rule=rng.choice(["delta", "delta", "linear"]), shape=rng.choice(["random", "random", "chain"]),
                M=_log_int(rng, 1, 64 if op == "tree" and case["B"] <= 16 else 32))
    if op == "tree":
        case.update(odtype=odtype, scale=scale)
    return case


# ---------------------------------------------------------------- inputs
def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    rng = random.Random(int(seed) * 104729 + 5)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    dt, Hqk, Hv, Dk, Dv = DT[case["dtype"]], case["Hqk"], case["Hv"], case["Dk"], case["Dv"]
    s = dict(case=dict(case), op=case["op"])
    # decays of the heads from slow (a memory of 10^4 tokens) to fast (about one token)
    decay = -torch.exp(rand(Hv) * math.log(1e4) + math.log(1e-4))
    if case["op"] in ("prefill", "backward"):
        lens = _lens(case)
        T, N = sum(lens), len(lens)
        s.update(q=_unit(randn(T, Hqk, Dk)).to(dt), k=_unit(randn(T, Hqk, Dk)).to(dt), v=randn(T, Hv, Dv).to(dt),
                 g=decay, lens=lens, cu=ints([sum(lens[:i]) for i in range(N + 1)]),
                 S0=randn(N, Hv, Dv, Dk) * 0.3 if case["init"] else None)
        if case["op"] == "backward":
            s.update(do=randn(T, Hv, Dv).to(dt), dSf=randn(N, Hv, Dv, Dk) * 0.3 if case["init"] else None)
        return s
    B, M, sdt = case["B"], case["M"], DT[case["sdtype"]]
    slots = B + 3
    order = list(range(slots))
    rng.shuffle(order)
    src, dst = order[:B], order[::-1][:B]
    if B >= 4:  # a padding entry, as a batch rounded up to a fixed size has them
        src[rng.randrange(B)] = -1
    s.update(q=_unit(randn(B, M, Hqk, Dk)).to(dt), k=_unit(randn(B, M, Hqk, Dk)).to(dt), v=randn(B, M, Hv, Dv).to(dt),
             pool=(randn(slots, Hv, Dv, Dk) * 0.3).to(sdt), src=ints(src))
    if case["op"] in ("decode", "tree"):
        s["o"] = torch.zeros(B, M, Hv, Dv, dtype=DT[case["odtype"]], device=dev)
    if case["op"] in ("decode", "commit"):
        s.update(dst=ints(dst), pool_out=torch.zeros(slots, Hv, Dv, Dk, dtype=sdt, device=dev))
    if case["op"] == "decode":
        s["g"], s["beta"] = decay, None
        return s
    if case["rule"] == "delta":
        s.update(g=-torch.nn.functional.softplus(randn(B, M, Hv)), beta=torch.sigmoid(randn(B, M, Hv)))
    else:
        s.update(g=decay, beta=None)
    parent, accept = [], []
    for _ in range(B):
        n = M if M == 1 or rng.random() < 0.5 else rng.randint(1, M)  # nodes of this tree; the rest is padding
        parent.append([(i - 1 if case["shape"] == "chain" else rng.randint(-1, i - 1)) if i < n else -2 for i in range(M)])
        accept.append(rng.choice([n - 1, rng.randint(-1, n - 1)]))  # -1: no drafted token was accepted
    s.update(parent=ints(parent), accept=ints(accept))
    return s


# ---------------------------------------------------------------- the plain form
def _heads(x, Hv):
    """fp32, query/key heads repeated to the value heads that read them (dim -2)."""
    return x.float().repeat_interleave(Hv // x.shape[-2], dim=-2)


class _Chunks:
    """Packed sequences cut into chunks of C tokens: gather indices [nc, C] and their mask."""

    def __init__(self, cu, lens, C):
        dev = cu.device
        nch = (cu[1:] - cu[:-1] + C - 1) // C
        last = nch.cumsum(0)
        self.nc = sum((n + C - 1) // C for n in lens)
        c = torch.arange(self.nc, device=dev)
        self.seq = torch.searchsorted(last, c, right=True)
        self.start = cu[self.seq] + (c - (last - nch)[self.seq]) * C
        pos = self.start[:, None] + torch.arange(C, device=dev)
        self.mask = pos < cu[self.seq + 1][:, None]
        self.idx = torch.where(self.mask, pos, 0).long()
        self.len = self.mask.sum(1)
        self.from_start = self.start - cu[self.seq]
        self.to_end = cu[self.seq + 1] - self.start - self.len


def _pow(g, n):
    """e^{g n} with the exponent in 64 bits, as fp32."""
    return torch.exp(g.double() * n.double()).float()


def _scan(a, b, c, g, cu, lens, X0, back, first):
    """out_t = sum_{s <= t} lam^{t-s} (a_t . b_s) c_s + lam^{t+1} X0 a_t for each head and sequence, and the
    state after the last token; ``back``: from the last token to the first; ``first``: lam^t X0 a_t instead.
    a, b [T, H, Da], c [T, H, Dc], X0 [N, H, Dc, Da] or None."""
    C = 64
    ch = _Chunks(cu, lens, C)
    T, H, Da = a.shape
    Dc, dev = c.shape[-1], a.device
    off = 0 if first else 1
    N = len(lens)
    n = (cu[1:] - cu[:-1]).to(dev)
    end = torch.zeros(N, H, Dc, Da, device=dev)
    if X0 is not None:
        end = _pow(g[None, :], (n[:, None] - 1 + off).clamp(min=0))[:, :, None, None] * X0
    if ch.nc == 0:
        return torch.zeros(T, H, Dc, device=dev), end
    m = ch.mask[:, :, None, None]
    A, B, V = (torch.where(m, x[ch.idx], 0).transpose(1, 2) for x in (a, b, c))  # [nc, H, C, D]
    i = torch.arange(C, device=dev)
    d = (i[None, :] - i[:, None]) if back else (i[:, None] - i[None, :])          # [t, s]
    E = torch.where(d >= 0, _pow(g[:, None, None], d.clamp(min=0)), 0)            # [H, C, C]
    O = ((A @ B.transpose(-1, -2)) * E) @ V
    # each chunk's own contribution to the state at its end, [nc, H, Dc, Da]
    rest = (i[None, :].expand(ch.nc, C) if back else (ch.len[:, None] - 1 - i[None, :])).clamp(min=0)
    w = _pow(g[None, :, None], rest[:, None, :])
    X = (V * w[..., None]).transpose(-1, -2) @ B
    # the state each chunk starts from, over all earlier chunks of its sequence; p: tokens of the chunk before t
    p = ((ch.len[:, None] - 1 - i[None, :]).clamp(min=0) if back else i[None, :].expand(ch.nc, C))
    s0, s1 = ch.start, ch.start + ch.len
    gap = (s0[None, :] - s1[:, None]) if back else (s0[:, None] - s1[None, :])    # tokens between, [c, c']
    same = (ch.seq[:, None] == ch.seq[None, :]) & (gap >= 0)
    W = torch.where(same, _pow(g[:, None, None], gap.clamp(min=0)), 0)            # [H, nc, nc]
    Xs = (W @ X.transpose(0, 1).reshape(H, ch.nc, -1)).reshape(H, ch.nc, Dc, Da).transpose(0, 1)
    O = O + _pow(g[None, :, None], p[:, None, :] + 1)[..., None] * (A @ Xs.transpose(-1, -2))
    if X0 is not None:
        pos = (ch.to_end if back else ch.from_start)[:, None] + p
        w0 = _pow(g[None, :, None], pos[:, None, :] + off)
        O = O + w0[..., None] * (A @ X0[ch.seq].transpose(-1, -2))
    tail = ch.from_start if back else ch.to_end
    end = end.index_add(0, ch.seq, _pow(g[None, :], tail[:, None])[:, :, None, None] * X)
    out = torch.zeros(T, H, Dc, device=dev)
    out[ch.idx[ch.mask]] = O.transpose(1, 2)[ch.mask]
    return out, end


def _tree(s):
    """u of every node, E (decay from a node to its descendants), E0 (from the cached state), fp32."""
    case = s["case"]
    Hv = case["Hv"]
    q, k, v = _heads(s["q"], Hv).transpose(1, 2), _heads(s["k"], Hv).transpose(1, 2), s["v"].float().transpose(1, 2)
    B, H, M, _ = k.shape
    par = s["parent"].long()
    real = par >= -1
    g = s["g"][None, None, :].expand(B, M, Hv) if s["beta"] is None else s["g"]
    alpha = torch.exp(g).transpose(1, 2)                                            # [B, H, M]
    link = (par[:, :, None] == torch.arange(M, device=par.device)) & real[:, :, None]
    n = torch.where(link[:, None], alpha[..., None], 0)                             # alpha_i at [i, parent]
    E = torch.eye(M, device=par.device) + n
    for _ in range(max(1, M - 1).bit_length()):                                     # sum of all powers of n
        n = n @ n
        E = E + n @ E
    anc = E != 0
    root = torch.where((par == -1)[:, None], alpha, 0)
    E0 = (E @ root[..., None])[..., 0]                                              # decay from the cached state
    pool = s["pool"].float()
    S0 = pool[s["src"].long().clamp(min=0)]                                         # [B, H, Dv, Dk]
    u = v
    if s["beta"] is not None:
        beta = s["beta"].transpose(1, 2)[..., None]
        A = beta * torch.where(anc, E, 0).tril(-1) * (k @ k.transpose(-1, -2))
        u = beta * (v - E0[..., None] * (k @ S0.transpose(-1, -2)))
        p = -A
        u = u + p @ u
        for _ in range(max(1, M - 1).bit_length() - 1):                             # (I + A)^-1 by squaring
            p = p @ p
            u = u + p @ u
    return q, k, u, E, E0, S0, real


def run(state):
    s, op = state, state["op"]
    case = s["case"]
    Hqk, Hv = case["Hqk"], case["Hv"]
    if own:
        return _run_own(s)
    if op == "prefill":
        q, k, v = _heads(s["q"], Hv), _heads(s["k"], Hv), s["v"].float()
        o, f = _scan(q, k, v, s["g"], s["cu"], s["lens"], s["S0"], False, False)
        return dict(o=(case["scale"] * o).to(DT[case["odtype"]]), final_state=f)
    if op == "backward":
        q, k, v = _heads(s["q"], Hv), _heads(s["k"], Hv), s["v"].float()
        do = case["scale"] * s["do"].float()
        T, dt = q.shape[0], DT[case["dtype"]]
        S0T = None if s["S0"] is None else s["S0"].transpose(-1, -2)
        dSf = s["dSf"]
        dq, _ = _scan(do, v, k, s["g"], s["cu"], s["lens"], S0T, False, False)
        dv, D = _scan(k, q, do, s["g"], s["cu"], s["lens"], dSf, True, True)
        dk, _ = _scan(v, do, q, s["g"], s["cu"], s["lens"], None if dSf is None else dSf.transpose(-1, -2), True, True)
        n = (s["cu"][1:] - s["cu"][:-1])[:, None, None, None]
        dS0 = torch.where(n > 0, torch.exp(s["g"])[None, :, None, None] * D, 0 if dSf is None else dSf)
        group = lambda x: x.reshape(T, Hqk, Hv // Hqk, -1).sum(2).to(dt)  # noqa: E731
        return dict(dq=group(dq), dk=group(dk), dv=dv.to(dt), d_initial_state=dS0)
    live = (s["src"] >= 0)
    if op == "decode":
        M = case["M"]
        q, k, v = _heads(s["q"], Hv).transpose(1, 2), _heads(s["k"], Hv).transpose(1, 2), s["v"].float().transpose(1, 2)
        i = torch.arange(M, device=q.device)
        d = i[:, None] - i[None, :]
        E = torch.where(d >= 0, _pow(s["g"][:, None, None], d.clamp(min=0)), 0)
        S0 = s["pool"].float()[s["src"].long().clamp(min=0)]
        o = ((q @ k.transpose(-1, -2)) * E) @ v + _pow(s["g"][:, None], i + 1)[..., None] * (q @ S0.transpose(-1, -2))
        S = _pow(s["g"], torch.tensor(float(M)))[:, None, None] * S0 + (v * E[:, -1, :, None]).transpose(-1, -2) @ k
        o = torch.where(live[:, None, None, None], (case["scale"] * o).transpose(1, 2), s["o"].float())
        return dict(o=o.to(s["o"].dtype), state=_put(s, S, live))
    q, k, u, E, E0, S0, real = _tree(s)
    if op == "tree":
        o = (E * (q @ k.transpose(-1, -2))) @ u + E0[..., None] * (q @ S0.transpose(-1, -2))
        keep = live[:, None] & real
        return dict(o=torch.where(keep[:, :, None, None], (case["scale"] * o).transpose(1, 2), s["o"].float()).to(s["o"].dtype))
    at = s["accept"].long()
    some = (at >= 0)[:, None, None]
    pick = at.clamp(min=0)[:, None, None].expand(-1, E.shape[1], 1)
    e0 = torch.where(some, E0.gather(2, pick), 1)
    e = torch.where(some, E.gather(2, pick[..., None].expand(-1, -1, 1, E.shape[-1]))[:, :, 0], 0)
    return dict(state=_put(s, e0[..., None] * S0 + (u * e[..., None]).transpose(-1, -2) @ k, live))


def _put(s, S, live):
    """The states of the live sequences in their slots of the output pool; its other slots stay."""
    slot = s["dst"].long()
    old = s["pool_out"][slot]
    s["pool_out"][slot] = torch.where(live[:, None, None, None], S.to(old.dtype), old)
    return s["pool_out"]


def _run_own(s):
    from gated_deltanet_recurrence_rule_b200 import api
    case, op = s["case"], s["op"]
    if op in ("prefill", "backward") and "workspace" not in s:  # kept from call to call, as a program does
        T, Hqk, Dk = s["q"].shape
        Hv, Dv = s["v"].shape[1:]
        s["workspace"] = torch.zeros(api.linear_prefill_workspace_size(len(s["lens"]), T, Hqk, Hv, Dk, Dv, s["q"].dtype,
                                                                       backward=op == "backward"),
                                     dtype=torch.uint8, device=s["q"].device)
    if op == "prefill":
        o, f = api.linear_prefill(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"], initial_state=s["S0"],
                                  scale=case["scale"], o_dtype=DT[case["odtype"]], workspace=s["workspace"])
        return dict(o=o, final_state=f)
    if op == "backward":
        dq, dk, dv, dS0 = api.linear_prefill_backward(s["q"], s["k"], s["v"], s["g"], s["do"], cu_seqlens=s["cu"],
                                                      initial_state=s["S0"], d_final_state=s["dSf"],
                                                      scale=case["scale"], workspace=s["workspace"])
        return dict(dq=dq, dk=dk, dv=dv, d_initial_state=dS0)
    if op == "decode":
        api.linear_decode_tokens(s["q"], s["k"], s["v"], s["g"], s["pool"], s["pool_out"], src_slot=s["src"],
                                 dst_slot=s["dst"], o=s["o"], scale=case["scale"])
        return dict(o=s["o"], state=s["pool_out"])
    if op == "tree":
        api.decode_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parent"], s["pool"], src_slot=s["src"],
                        o=s["o"], scale=case["scale"])
        return dict(o=s["o"])
    api.tree_commit(s["k"], s["v"], s["g"], s["beta"], s["parent"], s["accept"], s["pool"], s["pool_out"],
                    src_slot=s["src"], dst_slot=s["dst"])
    return dict(state=s["pool_out"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    Hqk, Hv, Dk, Dv = case["Hqk"], case["Hv"], case["Dk"], case["Dv"]
    e = 2 if case["dtype"] == "bf16" else 4
    S = Hv * Dk * Dv
    if case["op"] in ("prefill", "backward"):
        lens = _lens(case)
        T, N = sum(lens), len(lens)
        qk, vv = T * Hqk * Dk * e, T * Hv * Dv
        if case["op"] == "prefill":
            eo = 2 if case["odtype"] == "bf16" else 4
            return dict(bytes=2 * qk + vv * (e + eo) + N * S * 4 * (2 if case["init"] else 1),
                        flops=4 * T * S)  # one update of S and one product with it a token
        return dict(bytes=4 * qk + 3 * vv * e + N * S * 4 * (3 if case["init"] else 1), flops=12 * T * S)
    B, M = case["B"], case["M"]
    es = 2 if case["sdtype"] == "bf16" else 4
    if case["op"] == "decode":
        eo = 2 if case["odtype"] == "bf16" else 4
        return dict(bytes=B * (M * (2 * Hqk * Dk * e + Hv * Dv * (e + eo)) + 2 * S * es), flops=4 * B * M * S)
    gates = 8 * M * Hv if case["rule"] == "delta" else 0
    products = 4 if case["rule"] == "delta" else 2
    if case["op"] == "tree":
        eo = 2 if case["odtype"] == "bf16" else 4
        return dict(bytes=B * (M * (2 * Hqk * Dk * e + Hv * Dv * (e + eo) + 4) + S * es + gates),
                    flops=products * B * M * S)
    # only the accepted path is needed; its length is the drafts', at least one node
    return dict(bytes=B * (2 * S * es + Hqk * Dk * e + Hv * Dv * e + 4 * M), flops=products * B * S)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """Token by token in fp64 from the definitions, all sequences side by side."""
    if case["op"] in ("prefill", "backward") and max(_lens(case)) * len(_lens(case)) * case["Hv"] > 20_000_000:
        return None
    s = prepare(case, seed)
    Hqk, Hv, Dk, Dv = case["Hqk"], case["Hv"], case["Dk"], case["Dv"]
    rep = [h // (Hv // Hqk) for h in range(Hv)]
    if case["op"] in ("prefill", "backward"):
        lens, lam = s["lens"], s["g"].double().exp()[None, :, None, None]
        N, T = len(lens), sum(lens)
        at = [sum(lens[:i]) for i in range(N)]
        q, k, v = s["q"].double()[:, rep], s["k"].double()[:, rep], s["v"].double()
        order = sorted(range(N), key=lambda i: -lens[i])  # the sequences still running are a prefix
        rank = torch.tensor(order, device=q.device)
        base = torch.tensor([at[i] for i in order], device=q.device)
        first = torch.zeros(N, Hv, Dv, Dk, dtype=torch.float64, device=q.device)
        S = first.clone() if s["S0"] is None else s["S0"].double()[rank]
        rows = lambda S, x: (S @ x.unsqueeze(-1)).squeeze(-1)  # noqa: E731
        outer = lambda x, y: x.unsqueeze(-1) * y.unsqueeze(-2)  # noqa: E731
        o = torch.zeros(T, Hv, Dv, dtype=torch.float64, device=q.device)
        back = case["op"] == "backward"
        if back:
            do = case["scale"] * s["do"].double()
            dq = torch.zeros(T, Hv, Dk, dtype=torch.float64, device=q.device)
        for t in range(max(lens)):
            n = sum(x > t for x in lens)
            j = base[:n] + t
            S[:n] = lam * S[:n] + outer(v[j], k[j])
            if back:
                dq[j] = rows(S[:n].transpose(-1, -2), do[j])
            else:
                o[j] = case["scale"] * rows(S[:n], q[j])
        undo = torch.empty_like(rank)
        undo[rank] = torch.arange(N, device=q.device)
        if not back:
            return dict(o=o, final_state=S[undo])
        D = first.clone() if s["dSf"] is None else s["dSf"].double()[rank]  # dL/dS after the last token
        dk, dv = torch.zeros_like(dq), torch.zeros_like(o)
        for t in range(max(lens) - 1, -1, -1):
            n = sum(x > t for x in lens)
            j = base[:n] + t
            D[:n] = D[:n] + outer(do[j], q[j])
            dk[j] = rows(D[:n].transpose(-1, -2), v[j])
            dv[j] = rows(D[:n], k[j])
            D[:n] = lam * D[:n]
        group = lambda x: x.unflatten(1, (Hqk, Hv // Hqk)).sum(2)  # noqa: E731
        return dict(dq=group(dq), dk=group(dk), dv=dv, d_initial_state=D[undo])
    B, M = case["B"], case["M"]
    out = s["pool_out"].double() if "pool_out" in s else None
    o = s["o"].double() if "o" in s else None
    src, par, acc = s["src"].tolist(), None, None
    if case["op"] != "decode":
        par, acc = s["parent"].tolist(), s["accept"].tolist()
    for b in range(B):
        if src[b] < 0:
            continue
        S0 = s["pool"][src[b]].double()
        states = {-1: S0}
        for i in range(M):
            p = i - 1 if par is None else par[b][i]
            if p < -1:
                continue
            q, k, v = s["q"][b, i].double()[rep], s["k"][b, i].double()[rep], s["v"][b, i].double()
            a = (s["g"] if s["beta"] is None else s["g"][b, i]).double().exp()
            S = a[:, None, None] * states[p]
            w = v
            if s["beta"] is not None:
                w = s["beta"][b, i].double()[:, None] * (v - torch.einsum("hvd,hd->hv", S, k))
            states[i] = S + w[:, :, None] * k[:, None, :]
            if o is not None:
                o[b, i] = case["scale"] * torch.einsum("hvd,hd->hv", states[i], q)
        if out is not None:
            out[int(s["dst"][b])] = states[M - 1 if acc is None else acc[b]]
    if case["op"] == "decode":
        return dict(o=o, state=out)
    return dict(o=o) if case["op"] == "tree" else dict(state=out)
