"""Measured cases of the decayed linear attention (prefill, decode, gradients)
and of the norms around a block fused with its gate and residual scale
(forward, gradients).

With ``own`` false ``run`` computes an operator in its plain form (elementary
torch operations in 32 bits, prefix sums of the decays in 64); with ``own``
true it makes the library calls a user makes.

Decayed linear attention, per sequence and value head (S is d_v x d_k):

    S_t = e^(g_t) S_(t-1) + v_t k_t^T,   o_t = S_t q_t

with one log-decay per token and value head, or one per value head.  The
block norms, per row:

    h = rho r + c s * act(z) * post(x),   y = pre(h)

with post and pre RMS norms with their scales.
"""
import math
import random

import torch

own = False

CHUNK = 128
FLOOR = -20.0
EPS = 1e-6
RHO, BRANCH = 0.875, 0.5  # residual scale and branch scale of the block-norm cases


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # a prompt batch of the library's main workload: 4 x 4096 tokens, 16 q/k and 32 value heads
        dict(name="prefill_4x4096", op="prefill", dtype="bf16", n=4, tokens=16384, ragged=0, hk=16, hv=32, dk=128,
             dv=128, per_token=True),
        # one long document, 65,536 tokens, 48 value heads: fewer chains than SMs, so the sequence is split
        dict(name="prefill_long", op="prefill", dtype="bf16", n=1, tokens=65536, ragged=0, hk=16, hv=48, dk=128,
             dv=128, per_token=True),
        # a packed batch of ragged sequences in fp32, fixed decays, unequal head sizes
        dict(name="prefill_ragged_f32", op="prefill", dtype="f32", n=7, tokens=5003, ragged=3, hk=4, hv=8, dk=64,
             dv=96, per_token=False),
        # a single short prompt: the latency of the call
        dict(name="prefill_short", op="prefill", dtype="bf16", n=1, tokens=101, ragged=0, hk=8, hv=8, dk=128, dv=128,
             per_token=True),
        # serving: one token for each of 256 sequences, 512 MiB of state
        dict(name="decode_256", op="decode", dtype="bf16", n=256, tokens=256, ragged=0, hk=16, hv=32, dk=128, dv=128,
             per_token=True),
        # one sequence in fp32 with small odd-sized heads: the latency of a decode step
        dict(name="decode_1_f32", op="decode", dtype="f32", n=1, tokens=1, ragged=0, hk=3, hv=6, dk=80, dv=72,
             per_token=False),
        # training on the main workload, with the gradients of the decays
        dict(name="backward_4x4096", op="backward", dtype="bf16", n=4, tokens=16384, ragged=0, hk=16, hv=32, dk=128,
             dv=128, per_token=True),
        # training on a packed ragged batch in fp32 with fixed (learned) decays
        dict(name="backward_ragged_f32", op="backward", dtype="f32", n=5, tokens=2039, ragged=5, hk=2, hv=4, dk=64,
             dv=64, per_token=False),
        # the residual stream of the main workload (32 heads x 128) after a mixer: gate, both norms, scale
        dict(name="norm_16384x4096", op="norm", dtype="bf16", rows=16384, width=4096, gate=True, post=True,
             wide_residual=False),
        # the same for eight decoded tokens, with a 32-bit residual stream
        dict(name="norm_8x2048", op="norm", dtype="bf16", rows=8, width=2048, gate=True, post=True,
             wide_residual=True),
        # its gradients
        dict(name="norm_bwd_16384x4096", op="norm_bwd", dtype="bf16", rows=16384, width=4096, gate=True, post=True,
             wide_residual=False),
        # an odd width in fp32 without a gate
        dict(name="norm_bwd_odd_f32", op="norm_bwd", dtype="f32", rows=1031, width=1371, gate=False, post=True,
             wide_residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "decode", "backward", "norm", "norm_bwd"])
    if op in ("norm", "norm_bwd"):
        width = _log(rng, 256, 8192)
        if rng.random() < 0.6:
            width = max(256, width // 64 * 64)  # widths of real models; the others stay odd
        rows = _log(rng, 1, min(32768, (1 << 26) // width))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, width=width,
                    gate=rng.random() < 0.6, post=rng.random() < 0.7, wide_residual=rng.random() < 0.3)
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 1, 2, 3])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dk, dv = (128, 128) if rng.random() < 0.5 else (8 * rng.randint(4, 16), 8 * rng.randint(4, 16))
    if op == "decode":
        n = _log(rng, 1, max(2, 8192 // hv))
        return dict(op=op, dtype=dtype, n=n, tokens=n, ragged=0, hk=hk, hv=hv, dk=dk, dv=dv,
                    per_token=rng.random() < 0.7)
    most = 24576 if dtype == "bf16" else 4096
    if op == "backward":
        most //= 2
    tokens, n, ragged = _log(rng, 1, most), rng.randint(1, 6), rng.randint(1, 9999)
    if rng.random() < 0.5:  # equal lengths
        tokens, ragged = max(1, tokens // n) * n, 0
    return dict(op=op, dtype=dtype, n=n, tokens=tokens, ragged=ragged, hk=hk, hv=hv, dk=dk, dv=dv,
                per_token=rng.random() < 0.7)


def _lengths(case):
    """Lengths of the sequences: equal, or cut at places that ``ragged`` gives (some may be empty)."""
    n, tokens = case["n"], case["tokens"]
    if not case["ragged"]:
        return [tokens // n] * n
    r = random.Random(case["ragged"])
    cuts = [0] + sorted(r.randint(0, tokens) for _ in range(n - 1)) + [tokens]
    return [b - a for a, b in zip(cuts, cuts[1:])]


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] in ("norm", "norm_bwd"):
        rows, d = case["rows"], case["width"]
        rt = torch.float32 if case["wide_residual"] else dt
        s = dict(case=case, x=(0.7 * normal(rows, d)).to(dt), residual=(2.0 * normal(rows, d)).to(rt),
                 gate=normal(rows, d).to(dt) if case["gate"] else None,
                 post_weight=1 + 0.1 * normal(d) if case["post"] else None,
                 scale=1 + 0.2 * normal(d), pre_weight=1 + 0.1 * normal(d))
        if case["op"] == "norm_bwd":
            s["d_y"] = normal(rows, d).to(dt)
            s["d_h"] = normal(rows, d).to(rt)
        return s
    n, tokens, hk, hv, dk, dv = (case[k] for k in ("n", "tokens", "hk", "hv", "dk", "dv"))
    decode = case["op"] == "decode"
    q, k, v = normal(tokens, hk, dk), normal(tokens, hk, dk), normal(tokens, hv, dv)
    q = (q / q.norm(dim=-1, keepdim=True)).to(dt)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    v = v.to(dt)
    if case["per_token"]:  # softplus-shaped log-decays, heads from slow to quick
        rate = torch.exp2(-torch.linspace(0.0, 7.0, hv, device=dev))
        g = -torch.nn.functional.softplus(normal(tokens, hv)) * rate
    else:  # one fixed decay a head
        g = -torch.exp2(-8.0 * torch.arange(1, hv + 1, device=dev) / hv) * (1 + 0.1 * torch.rand(
            hv, generator=gen, device=dev))
    s = dict(case=case, g=g.float().contiguous())
    if decode:
        return dict(s, q=q, k=k, v=v, state=0.3 * normal(n, hv, dv, dk))
    lens = _lengths(case)
    s["state0"] = 0.3 * normal(n, hv, dv, dk)
    s["cu"] = None
    lead = (n, tokens // n)
    if case["ragged"]:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
        lead = (tokens,)
    if g.dim() == 2:
        s["g"] = s["g"].view(*lead, hv)
    s.update(q=q.view(*lead, hk, dk), k=k.view(*lead, hk, dk), v=v.view(*lead, hv, dv))
    # the padded layout of the plain form: token of each (sequence, position), and whether there is one
    width = max(CHUNK, -(-max(lens) // CHUNK) * CHUNK)
    pos = torch.arange(width, device=dev)[None, :]
    ln = torch.tensor(lens, device=dev)[:, None]
    start = torch.tensor([sum(lens[:i]) for i in range(n)], device=dev)[:, None]
    s["valid"] = pos < ln
    s["rows"] = torch.where(s["valid"], start + pos, torch.zeros_like(pos)).clamp(max=max(tokens - 1, 0))
    if case["op"] == "backward":
        s["d_o"] = normal(*lead, hv, dv).to(dt)
        s["d_final"] = 0.1 * normal(n, hv, dv, dk)
    return s


# -------------------------------------------------------------- the plain forms
def _padded(s, t, heads):
    """[tokens, h, d] -> fp32 [n, heads, width, d], absent tokens zero, heads of a group repeated."""
    t = t.reshape(-1, t.shape[-2], t.shape[-1]).float()
    t = t[s["rows"]] * s["valid"][..., None, None]
    return t.repeat_interleave(heads // t.shape[2], dim=2).transpose(1, 2)


def _decays(s, hv):
    """Floored log-decays in 64 bits, [n, hv, width]; zero at absent tokens."""
    g = s["g"]
    g = g.double().clamp(min=FLOOR)
    if g.dim() == 1:
        g = g[None, :].expand(s["case"]["tokens"], hv)
    g = g.reshape(-1, hv)[s["rows"]] * s["valid"][..., None]
    return g.transpose(1, 2)


def _mix(x, y, z, g, s0):
    """out_t = S_t x_t with S_t = e^(g_t) S_(t-1) + z_t y_t^T from S = s0, by chunks; returns (out, last S)."""
    n, h, width, _ = x.shape
    nc = width // CHUNK
    x, y, z = (t.reshape(n, h, nc, CHUNK, -1) for t in (x, y, z))
    g = g.reshape(n, h, nc, CHUNK)
    cum = g.cumsum(-1)
    total = cum[..., -1]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    mask = torch.exp(torch.where(tri, cum[..., :, None] - cum[..., None, :], -math.inf)).float()
    intra = ((x @ y.transpose(-1, -2)) * mask) @ z
    local = (z * torch.exp(total[..., None] - cum).float()[..., None]).transpose(-1, -2) @ y  # [n, h, nc, dz, dy]
    # the state before each chunk: the local states of the chunks before it, decayed; s0 is chunk -1
    ends = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)  # decay up to each chunk's start
    before = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp(torch.where(before, ends[..., :, None] - ends[..., None, :], -math.inf)).float()
    src = torch.cat([s0[:, :, None], local], 2)
    states = (carry @ src.reshape(n, h, nc + 1, -1)).reshape(src.shape)
    inter = (x @ states[:, :, :-1].transpose(-1, -2)) * torch.exp(cum).float()[..., None]
    return (intra + inter).reshape(n, h, width, -1), states[:, :, -1]


def _rows_out(s, t, like, dtype):
    """[n, h, width, d] -> the tokens' rows, shaped like ``like``."""
    return t.transpose(1, 2)[s["valid"]].reshape(like.shape).to(dtype)


def _plain_prefill(s):
    hv = s["case"]["hv"]
    q, k, v = (_padded(s, s[n], hv) for n in "qkv")
    o, last = _mix(q, k, v, _decays(s, hv), s["state0"])
    return _rows_out(s, o, s["v"], s["v"].dtype), last


def _plain_decode(s):
    group = s["case"]["hv"] // s["case"]["hk"]
    q, k = (s[n].float().repeat_interleave(group, dim=1) for n in "qk")
    a = torch.exp(s["g"].clamp(min=FLOOR)).expand(s["case"]["n"], -1)
    s["state"].copy_(s["state"] * a[..., None, None] + s["v"].float()[..., :, None] * k[..., None, :])
    o = (s["state"] * q[..., None, :]).sum(-1)
    return o.to(s["v"].dtype), s["state"]


def _plain_backward(s):
    case = s["case"]
    hk, hv = case["hk"], case["hv"]
    q, k, v, do = (_padded(s, s[n], hv) for n in ("q", "k", "v", "d_o"))
    g = _decays(s, hv)
    s0, dsf = s["state0"], s["d_final"]
    dq, last = _mix(do, v, k, g, s0.transpose(-1, -2))
    # the state's gradient runs back in time; token t of it decays by the next token's g
    flip = lambda t: t.flip(2)  # noqa: E731
    back = torch.cat([torch.zeros_like(g[..., :1]), flip(g)[..., :-1]], -1)
    dv, ds = _mix(flip(k), flip(q), flip(do), back, dsf)
    dk, _ = _mix(flip(v), flip(do), flip(q), back, dsf.transpose(-1, -2))
    dk, dv = flip(dk), flip(dv)
    # <dS_t, S_t> seen from both sides: dg_t - dg_(t+1) = q_t . dq_t - k_t . dk_t
    end = (dsf.double() * last.transpose(-1, -2).double()).sum((-1, -2))
    step = (q * dq).double().sum(-1) - (k * dk).double().sum(-1)
    dg = step.flip(-1).cumsum(-1).flip(-1) + end[..., None]
    dg = dg * s["valid"][:, None, :]
    if s["g"].dim() == 1:
        dg = (dg.sum((0, 2)) * (s["g"] >= FLOOR)).float()
    else:
        dg = (dg.transpose(1, 2)[s["valid"]].reshape(s["g"].shape) * (s["g"] >= FLOOR)).float()
    group = hv // hk

    def heads(t):  # gradients of the value heads that share a q/k head are summed
        n, _, w, d = t.shape
        return t.reshape(n, hk, group, w, d).sum(2)

    ds0 = ds * torch.exp(g[..., 0]).float()[..., None, None]
    dt = s["q"].dtype
    return dict(dq=_rows_out(s, heads(dq), s["q"], dt), dk=_rows_out(s, heads(dk), s["k"], dt),
                dv=_rows_out(s, dv, s["v"], dt), dg=dg, d_initial_state=ds0)


def _plain_norm_parts(s):
    x, r = s["x"].float(), s["residual"].float()
    r1 = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) if s["post_weight"] is not None else None
    n1 = x if r1 is None else x * r1
    u = n1 if r1 is None else n1 * s["post_weight"]
    sg = 1 / (1 + torch.exp(-s["gate"].float())) if s["gate"] is not None else None
    b = u if sg is None else u * (s["gate"].float() * sg)
    h = RHO * r + BRANCH * s["scale"] * b
    r2 = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return r1, n1, u, sg, b, h, r2


def _plain_norm(s):
    _, _, _, _, _, h, r2 = _plain_norm_parts(s)
    return h.to(s["residual"].dtype), (h * r2 * s["pre_weight"]).to(s["x"].dtype)


def _plain_norm_bwd(s):
    r1, n1, u, sg, b, h, r2 = _plain_norm_parts(s)
    dy, n2 = s["d_y"].float(), h * r2
    dn2 = dy * s["pre_weight"]
    dh = s["d_h"].float() + r2 * (dn2 - n2 * (dn2 * n2).mean(-1, keepdim=True))
    out = dict(d_residual=(RHO * dh).to(s["residual"].dtype), d_pre_weight=(dy * n2).sum(0),
               d_scale=(BRANCH * dh * b).sum(0))
    db = BRANCH * s["scale"] * dh
    if sg is not None:
        z = s["gate"].float()
        out["d_gate"] = (db * u * sg * (1 + z * (1 - sg))).to(s["x"].dtype)
        db = db * (z * sg)
    if r1 is not None:
        out["d_post_weight"] = (db * n1).sum(0)
        dn1 = db * s["post_weight"]
        db = r1 * (dn1 - n1 * (dn1 * n1).mean(-1, keepdim=True))
    out["dx"] = db.to(s["x"].dtype)
    return out


# ------------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from linear_attention_sequence_sm_b200 import gdn
        if op == "prefill":
            return gdn.decay_forward(s["q"], s["k"], s["v"], s["g"], initial_state=s["state0"], cu_seqlens=s["cu"])
        if op == "decode":
            o = gdn.decay_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"])
            return o, s["state"]
        if op == "backward":
            return gdn.decay_backward(s["q"], s["k"], s["v"], s["g"], s["d_o"], d_final_state=s["d_final"],
                                      initial_state=s["state0"], cu_seqlens=s["cu"])
        norm = gdn.BlockNorm(post_weight=s["post_weight"], post_norm=s["post_weight"] is not None, scale=s["scale"],
                             pre_weight=s["pre_weight"], residual_scale=RHO, branch_scale=BRANCH, eps=EPS)
        if op == "norm":
            return gdn.block_norm_forward(s["x"], s["residual"], norm, gate=s["gate"])
        got = gdn.block_norm_backward(s["x"], s["residual"], norm, gate=s["gate"], d_y=s["d_y"], d_h=s["d_h"])
        return {k: t for k, t in got.items() if t is not None}
    return dict(prefill=_plain_prefill, decode=_plain_decode, backward=_plain_backward, norm=_plain_norm,
                norm_bwd=_plain_norm_bwd)[op](s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_bwd"):
        n, d = case["rows"] * case["width"], case["width"]
        re = 4 if case["wide_residual"] else e
        gate = e if case["gate"] else 0
        if case["op"] == "norm":  # x, gate, residual in; h, y out; the scales
            return dict(bytes=n * (2 * e + gate + 2 * re) + 12 * d, flops=14 * n)
        return dict(bytes=n * (3 * e + 2 * gate + 3 * re) + 24 * d, flops=40 * n)
    t, hk, hv, dk, dv = (case[k] for k in ("tokens", "hk", "hv", "dk", "dv"))
    gb = 4 * (t if case["per_token"] else 1) * hv
    states = 4 * case["n"] * hv * dk * dv
    qk, vo = t * hk * dk * e, t * hv * dv * e
    if case["op"] in ("prefill", "decode"):  # q, k, v, g and the state in, o and the state out
        return dict(bytes=2 * qk + 2 * vo + gb + 2 * states, flops=4 * t * hv * dk * dv)
    # q, k, v, d_o, g and two states in; dq, dk, dv, dg and a state out; two states carried, three gradients read
    return dict(bytes=4 * qk + 3 * vo + 2 * gb + 3 * states, flops=10 * t * hv * dk * dv)


# --------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(s)
    return _exact_mixer(s)


def _exact_mixer(s):
    """Token by token from the recurrence, all sequences and heads at once."""
    case = s["case"]
    op, hk, hv, n = case["op"], case["hk"], case["hv"], case["n"]
    head = torch.arange(hv, device="cuda") // (hv // hk)
    lens = [1] * n if op == "decode" else _lengths(case)
    starts = [sum(lens[:i]) for i in range(n)]
    q, k = (s[t].reshape(-1, hk, case["dk"]).double() for t in "qk")
    v = s["v"].reshape(-1, hv, case["dv"]).double()
    g = s["g"].double()
    g = g.reshape(-1, hv) if g.dim() > 1 else g[None].expand(case["tokens"], hv)
    alpha = torch.exp(torch.clamp(g, min=FLOOR))
    S = (s["state"] if op == "decode" else s["state0"]).double().clone()
    o = torch.zeros_like(v)
    steps = max(lens)
    # at step i, the sequences that have a token i, and that token's row
    live = [[j for j in range(n) if lens[j] > i] for i in range(steps)]
    same = all(x == lens[0] for x in lens)
    at = torch.tensor(starts, device="cuda")
    if op == "backward":
        do = s["d_o"].reshape(-1, hv, case["dv"]).double()
        dq = torch.zeros(case["tokens"], hv, case["dk"], dtype=torch.float64, device="cuda")
        dk, dv, dg = torch.zeros_like(dq), torch.zeros_like(v), torch.zeros_like(alpha)
    who = None
    for i in range(steps):
        if who is None or (not same and len(live[i]) != len(live[i - 1])):
            who = torch.tensor(live[i], device="cuda")
        rows = at[who] + i
        Si = S if same else S[who]
        Si = torch.baddbmm((Si * alpha[rows][..., None, None]).flatten(0, 1), v[rows].flatten(0, 1)[:, :, None],
                           k[rows][:, head].flatten(0, 1)[:, None, :]).view(Si.shape)
        if same:
            S = Si
        else:
            S[who] = Si
        if op == "backward":
            dq[rows] = torch.einsum("nhvk,nhv->nhk", Si, do[rows])
        else:
            o[rows] = torch.einsum("nhvk,nhk->nhv", Si, q[rows][:, head])
    if op != "backward":
        return [o.reshape(s["v"].shape), S]
    dS = s["d_final"].double().clone()
    edge = (dS * S).sum((-1, -2))  # <dS, S> past each sequence's last token
    who = None
    for i in reversed(range(steps)):
        if who is None or len(live[i]) != len(who):
            who = torch.tensor(live[i], device="cuda")
        rows = at[who] + i
        Di = dS[who]
        Di = Di + do[rows][..., :, None] * q[rows][:, head][..., None, :]
        dk[rows] = torch.einsum("nhvk,nhv->nhk", Di, v[rows])
        dv[rows] = torch.einsum("nhvk,nhk->nhv", Di, k[rows][:, head])
        # <dS_t, S_t> = <what follows> + d_o . o, of which v_t k_t^T's share is not the decay's
        edge[who] = edge[who] + (dq[rows] * q[rows][:, head]).sum(-1) - (dk[rows] * k[rows][:, head]).sum(-1)
        dg[rows] = edge[who]
        dS[who] = Di * alpha[rows][..., None, None]
    dg = torch.where(g >= FLOOR, dg, torch.zeros_like(dg))
    dg = dg.sum(0) if s["g"].dim() == 1 else dg.reshape(s["g"].shape)
    by_group = lambda t: torch.zeros(t.shape[0], hk, t.shape[2], dtype=t.dtype, device="cuda").index_add_(  # noqa: E731
        1, head, t)
    return dict(dq=by_group(dq).reshape(s["q"].shape), dk=by_group(dk).reshape(s["k"].shape),
                dv=dv.reshape(s["v"].shape), dg=dg, d_initial_state=dS)


def _exact_norm(s):
    """The definition in 64 bits; the gradients by differentiation of it."""
    wanted = s["case"]["op"] == "norm_bwd"
    names = [k for k in ("x", "residual", "gate", "post_weight", "scale", "pre_weight") if s[k] is not None]
    step = 2048  # rows at a time: the 64-bit graph of all of them would be large
    rows = s["x"].shape[0]
    parts, sums = {}, {}
    for a in range(0, rows, step):
        leaf = {}
        for k in names:
            t = s[k][a:a + step] if s[k].dim() == 2 else s[k]
            leaf[k] = t.double().requires_grad_(wanted)
        rms = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS)  # noqa: E731
        b = rms(leaf["x"]) * leaf["post_weight"] if "post_weight" in leaf else leaf["x"]
        if "gate" in leaf:
            b = b * leaf["gate"] * torch.sigmoid(leaf["gate"])
        h = RHO * leaf["residual"] + BRANCH * leaf["scale"] * b
        y = rms(h) * leaf["pre_weight"]
        if not wanted:
            parts.setdefault("h", []).append(h)
            parts.setdefault("y", []).append(y)
            continue
        loss = (y * s["d_y"][a:a + step].double()).sum() + (h * s["d_h"][a:a + step].double()).sum()
        for k, d in zip(names, torch.autograd.grad(loss, [leaf[k] for k in names])):
            if s[k].dim() == 2:
                parts.setdefault("dx" if k == "x" else "d_" + k, []).append(d)
            else:
                sums["d_" + k] = sums.get("d_" + k, 0) + d
    if not wanted:
        return [torch.cat(parts["h"]), torch.cat(parts["y"])]
    return {**{k: torch.cat(v) for k, v in parts.items()}, **sums}
