"""The decayed linear attention and the block norms as a model runs them: a
residual stream normed into each mixer, whose input side is the short
convolution and whose output is normed per head, projected and joined to the
stream; prefill, single-token decoding behind it, and training.

Each operator's result is held against 64 bits on the inputs that it was
given, so its own tolerance applies (see the operators' own tests): fp32 sums
within 256 u, and with the per-head output norm two such errors of o and one of
its own sums: 4 * 256 u."""
import pytest
import torch

import decay_ref as R

pytestmark = pytest.mark.gpu

F32 = 256 * R.U32
NORM = 64 * R.U32 + 8 * 2.0 ** -20
HK, HV, D, LAYERS, TAPS = 1, 2, 32, 2, 4
WIDTH, CH = 96, 2 * HK * D + HV * D


def weights(device="cuda"):
    gen = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    w = []
    for _ in range(LAYERS):
        w.append(dict(into=r(WIDTH, CH) / WIDTH ** 0.5, conv=0.5 * r(CH, TAPS), gate=r(WIDTH, HV * D) / WIDTH ** 0.5,
                      decay=r(WIDTH, HV) / WIDTH ** 0.5, on=1 + 0.2 * r(D), out=r(HV * D, WIDTH) / (HV * D) ** 0.5,
                      post=1 + 0.2 * r(WIDTH), scale=0.5 + 0.1 * r(WIDTH), pre=1 + 0.2 * r(WIDTH)))
    return [{k: t.to(device) for k, t in x.items()} for x in w]


def split_heads(x):
    lead = x.shape[:-1]
    q, k, v = x.split([HK * D, HK * D, HV * D], dim=-1)
    unit = lambda t: (t / (t.norm(dim=-1, keepdim=True) + 1e-6)).contiguous()  # noqa: E731
    return unit(q.reshape(*lead, HK, D)), unit(k.reshape(*lead, HK, D)), v.reshape(*lead, HV, D).contiguous()


def norm(gdn, w):
    return gdn.BlockNorm(post_weight=w["post"], scale=w["scale"], pre_weight=w["pre"], eps=1e-5, branch_scale=0.8)


def close(x, ref, bar):
    x = x.detach().double().cpu().reshape(ref.shape)
    assert float((x - ref).norm() / ref.norm()) <= bar


def model(x, ws, states, cu=None, check=False):
    """The tokens' last pre-norms; ``states`` (conv, mixer) per layer are replaced by those after them."""
    from linear_attention_sequence_sm_b200 import gdn
    one = cu is None
    h, y = gdn.block_norm_forward(x, None, gdn.BlockNorm(post_norm=False, eps=1e-5))
    for i, w in enumerate(ws):
        p = (y @ w["into"])
        conv, conv_state = gdn.short_conv(p[:, None] if one else p, w["conv"], cu_seqlens=cu, state=states[i][0],
                                          silu=True)
        q, k, v = split_heads(conv[:, 0] if one else conv)
        g = -torch.nn.functional.softplus(y @ w["decay"])
        on = gdn.OutputNorm(weight=w["on"], gate=(y @ w["gate"]).reshape(v.shape), eps=1e-5)
        if one:
            state = states[i][1].clone()
            o = gdn.decay_decode_step(q, k, v, g, state, output_norm=on)
        else:
            o, state = gdn.decay_forward(q, k, v, g, initial_state=states[i][1], cu_seqlens=cu, output_norm=on)
        b = o.reshape(-1, HV * D) @ w["out"]
        h2, y2 = gdn.block_norm_forward(b, h, norm(gdn, w))
        if check:
            lift = (lambda t: t[:, None]) if one else (lambda t: t)
            ro, rs = R.forward(lift(q), lift(k), lift(v), lift(g), states[i][1], None if one else cu.cpu())
            z = on.gate.double().cpu().reshape(ro.shape)
            ref = ro / (ro.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w["on"].double().cpu() * z * torch.sigmoid(z)
            close(o, ref, 4 * F32)
            close(state, rs, F32)
            rh, ry = R.block_norm(*(t.double().cpu() for t in (b, h)), None,
                                  *(w[n].double().cpu() for n in ("post", "scale", "pre")), eps=1e-5, branch=0.8)
            close(h2, rh, NORM)
            close(y2, ry, NORM)
        states[i] = (conv_state, state)
        h, y = h2, y2
    return y


def fresh(n):
    return [(torch.zeros(n, CH, TAPS - 1, device="cuda"), torch.zeros(n, HV, D, D, device="cuda"))
            for _ in range(LAYERS)]


def test_prefill_then_decode():
    """Decoding behind a prefill gives what one prefill over all tokens gives: both are within their tolerances of
    the same numbers, and four layers' worth of operators stand between input and output."""
    ws, gen = weights(), torch.Generator().manual_seed(62)
    lens, more = [70, 1, 130], 3
    xs = [torch.randn(n + more, WIDTH, generator=gen).cuda() for n in lens]
    cum = lambda ls: torch.tensor([sum(ls[:i]) for i in range(len(ls) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    st = fresh(3)
    model(torch.cat([x[:n] for x, n in zip(xs, lens)]), ws, st, cum(lens), check=True)
    for t in range(more):
        y = model(torch.stack([x[n + t] for x, n in zip(xs, lens)]), ws, st, check=True)
    whole = fresh(3)
    full = [n + more for n in lens]
    yw = model(torch.cat(xs), ws, whole, cum(full))
    last = cum(full)[1:].long() - 1
    # Per layer the attention, its norm, the block norm and two matrix products (within 256 u each) differ between
    # the two runs, by 8 * 256 u of their results together; a layer's Jacobian at most doubles what came in
    # (normed rows, unit keys), so two layers give (2 + 1) * 8 * 256 u.
    close(y, yw[last].double().cpu(), 24 * F32)
    for (_, a), (_, b) in zip(st, whole):
        close(a, b.double().cpu(), 24 * F32)


def test_decoding_captured_in_a_graph():
    ws, gen = weights(), torch.Generator().manual_seed(63)
    x = torch.randn(5, WIDTH, generator=gen).cuda()
    st = fresh(5)
    run = lambda: model(x, ws, list(st))  # noqa: E731 (the states stay as they are)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, run())


def test_training_step_of_a_block():
    """Gradients of one block, mixer to block norm, against 64-bit differentiation of the recurrence."""
    from linear_attention_sequence_sm_b200 import gdn
    w, gen = weights()[0], torch.Generator().manual_seed(64)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    lens = [90, 37]
    T = sum(lens)
    cu = torch.tensor([0, 90, 127], dtype=torch.int32)
    x, h = r(T, CH), r(T, WIDTH)
    g = -torch.nn.functional.softplus(r(T, HV))
    dh, dy = r(T, WIDTH), r(T, WIDTH)
    q, k, v = split_heads(x)
    c = {n: t.cuda() for n, t in dict(q=q, k=k, v=v, g=g, h=h, dh=dh, dy=dy, cu=cu).items()}
    o, _ = gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], cu_seqlens=c["cu"])
    b = o.reshape(T, HV * D) @ w["out"]
    nb = gdn.block_norm_backward(b, c["h"], norm(gdn, w), d_h=c["dh"], d_y=c["dy"])
    d_o = (nb["dx"] @ w["out"].T).reshape(o.shape).contiguous()
    got = gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], d_o, cu_seqlens=c["cu"])
    got.update(h=nb["d_residual"], post=nb["d_post_weight"], scale=nb["d_scale"], pre=nb["d_pre_weight"],
               out=o.reshape(T, HV * D).T @ nb["dx"])

    leaf = {n: t.double().requires_grad_() for n, t in dict(q=q, k=k, v=v, g=g, h=h).items()}
    leaf.update({n: w[n].double().cpu().requires_grad_() for n in ("out", "post", "scale", "pre")})
    outs = []
    for s, e in zip(cu[:-1].tolist(), cu[1:].tolist()):
        S = torch.zeros(HV, D, D, dtype=torch.float64)
        for t in range(s, e):
            kk, qq = (leaf[n][t].repeat_interleave(HV // HK, 0) for n in "kq")
            S = leaf["g"][t].exp()[:, None, None] * S + leaf["v"][t][:, :, None] * kk[:, None, :]
            outs.append((S * qq[:, None, :]).sum(-1))
    rb = torch.stack(outs).reshape(T, HV * D) @ leaf["out"]
    rh, ry = R.block_norm(rb, leaf["h"], None, leaf["post"], leaf["scale"], leaf["pre"], eps=1e-5, branch=0.8)
    names = list(leaf)
    want = dict(zip(names, torch.autograd.grad((rh * dh.double()).sum() + (ry * dy.double()).sum(),
                                               [leaf[n] for n in names])))
    # Forward: o and b, 2 * 256 u; the norm's gradients move by at most three times that (two normed factors and the
    # norm's scale) beside their own; then a product and a pass more: 12 * 256 u.  Gradients of the decays: 32 times
    # an operator's own, as in its test.
    for n in ("q", "k", "v", "h", "out", "post", "scale", "pre"):
        close(got["d" + n if n in "qkv" else n], want[n], 12 * F32)
    close(got["dg"], want["g"], 44 * F32)
