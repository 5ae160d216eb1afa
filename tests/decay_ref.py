"""Plain 64-bit references of the decayed linear attention and the block
norms (CPU, token by token), and seeded inputs."""
from __future__ import annotations

import torch

FLOOR = -20.0
U32 = 2.0 ** -24  # half a step of fp32


def lens_of(q, cu):
    if cu is None:
        return [q.shape[1]] * q.shape[0]
    c = cu.tolist()
    return [b - a for a, b in zip(c, c[1:])]


def _flat(t):
    return t.reshape(-1, t.shape[-2], t.shape[-1]).double().cpu()


def _alpha(g, tokens, hv):
    g = g.double().cpu()
    g = g.reshape(-1, hv) if g.dim() > 1 else g[None].expand(tokens, hv)
    return g, torch.exp(g.clamp(min=FLOOR))


def forward(q, k, v, g, s0=None, cu=None):
    """(o [tokens, hv, dv], final states [N, hv, dv, dk]) in 64 bits."""
    lens = lens_of(q, cu)
    qf, kf, vf = _flat(q), _flat(k), _flat(v)
    tokens, hv, dv = vf.shape
    head = torch.arange(hv) // (hv // qf.shape[1])
    _, a = _alpha(g, tokens, hv)
    S = torch.zeros(len(lens), hv, dv, qf.shape[-1], dtype=torch.float64) if s0 is None else s0.double().cpu().clone()
    o = torch.zeros_like(vf)
    t = 0
    for n, ln in enumerate(lens):
        for _ in range(ln):
            S[n] = a[t][:, None, None] * S[n] + vf[t][:, :, None] * kf[t, head][:, None, :]
            o[t] = (S[n] * qf[t, head][:, None, :]).sum(-1)
            t += 1
    return o, S


def backward(q, k, v, g, do, dsf=None, s0=None, cu=None):
    """Gradients by the reverse recurrence; dg_t = a_t <dS_t, S_(t-1)> directly."""
    lens = lens_of(q, cu)
    qf, kf, vf, of = _flat(q), _flat(k), _flat(v), _flat(do)
    tokens, hv, dv = vf.shape
    hk, dk = qf.shape[1], qf.shape[2]
    head = torch.arange(hv) // (hv // hk)
    gg, a = _alpha(g, tokens, hv)
    shape = (len(lens), hv, dv, dk)
    S0 = torch.zeros(shape, dtype=torch.float64) if s0 is None else s0.double().cpu()
    D0 = torch.zeros(shape, dtype=torch.float64) if dsf is None else dsf.double().cpu()
    dq, dk_, dv_ = torch.zeros_like(qf), torch.zeros_like(kf), torch.zeros_like(vf)
    dg, ds0 = torch.zeros(tokens, hv, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    start = 0
    for n, ln in enumerate(lens):
        hist = [S0[n]]
        for t in range(start, start + ln):
            hist.append(a[t][:, None, None] * hist[-1] + vf[t][:, :, None] * kf[t, head][:, None, :])
        D = D0[n].clone()
        for i in reversed(range(ln)):
            t = start + i
            D = D + of[t][:, :, None] * qf[t, head][:, None, :]
            dq.index_put_((torch.tensor([t]), head), (hist[i + 1] * of[t][:, :, None]).sum(1), accumulate=True)
            dk_.index_put_((torch.tensor([t]), head), (D * vf[t][:, :, None]).sum(1), accumulate=True)
            dv_[t] = (D * kf[t, head][:, None, :]).sum(-1)
            dg[t] = a[t] * (D * hist[i]).sum((-1, -2)) * (gg[t] >= FLOOR)
            D = a[t][:, None, None] * D
        ds0[n] = D
        start += ln
    return dict(dq=dq, dk=dk_, dv=dv_, dg=dg if g.dim() > 1 else dg.sum(0), d_initial_state=ds0)


def make(seed, hk, hv, dk, dv, dtype, batch=None, lens=None, per_token=True, rate=1.0, s0=True):
    """q, k (unit rows), v, g, initial state and cu_seqlens on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    lead = tuple(batch) if batch else (sum(lens),)
    n = batch[0] if batch else len(lens)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    g = -torch.nn.functional.softplus(r(*lead, hv)) * rate * torch.exp2(-torch.arange(hv) * 2.0) if per_token else \
        -rate * torch.exp2(-2.0 * torch.arange(hv))
    cu = None if batch else torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    return dict(q=unit(r(*lead, hk, dk)).to(dtype), k=unit(r(*lead, hk, dk)).to(dtype), v=r(*lead, hv, dv).to(dtype),
                g=g.float().contiguous(), s0=0.3 * r(n, hv, dv, dk) if s0 else None, cu=cu,
                do=r(*lead, hv, dv).to(dtype), dsf=0.2 * r(n, hv, dv, dk))


def cuda(d):
    return {k: (t.cuda() if t is not None else None) for k, t in d.items()}


def worst(x, ref, lens, token_axis):
    """The largest relative 2-norm error over (sequence, head) slices."""
    x, ref = x.detach().double().cpu().reshape(ref.shape), ref
    if not token_axis:
        num, den = (x - ref).flatten(2).norm(dim=-1), ref.flatten(2).norm(dim=-1)
        return float((num / den.clamp(min=1e-30)).max()) if num.numel() else 0.0
    out, t = 0.0, 0
    for ln in lens:
        if ln:
            a, b = x[t:t + ln], ref[t:t + ln]
            a, b = (a[..., None], b[..., None]) if a.dim() == 2 else (a, b)
            num, den = (a - b).norm(dim=(0, 2)), b.norm(dim=(0, 2))
            out = max(out, float((num / den.clamp(min=1e-30)).max()))
        t += ln
    return out


def block_norm(x, residual, gate, w1, scale, w2, post=True, pre=True, eps=1e-6, rho=1.0, branch=1.0,
               activation="silu", zero_centred=False):
    """(h, y) in 64 bits; differentiable."""
    one = 1.0 if zero_centred else 0.0
    rms = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)  # noqa: E731
    b = rms(x) if post else x
    if post and w1 is not None:
        b = b * (one + w1)
    if gate is not None:
        b = b * torch.sigmoid(gate) * (gate if activation == "silu" else 1.0)
    b = branch * b if scale is None else branch * scale * b
    h = b if residual is None else rho * residual + b
    y = None
    if pre:
        y = rms(h) if w2 is None else rms(h) * (one + w2)
    return h, y
