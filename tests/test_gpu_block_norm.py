"""The block norms on the GPU against their definition in 64 bits, gradients
by differentiation of it and by differences.

Tolerances in half steps (fp32: u = 2^-24; bf16: 2^-8): a row's values pass
two norms whose sums of up to 16384 squares err by at most sqrt(n) u in the
norm-wise mean (pairwise over lanes and warps: far less), about 16 fp32
operations and, for bf16 rows, the sigmoid of the fast exponential, 2^-20
relative; bf16 results are rounded once, and sums over rows of fp32 terms err
by sqrt(rows) u."""
import pytest
import torch

import decay_ref as R

pytestmark = pytest.mark.gpu

F32 = 64 * R.U32
SIG = 8 * 2.0 ** -20  # the fast sigmoid passes through at most eight products
WIDTHS = [(1, 1), (3, 7), (5, 256), (129, 264), (64, 1000), (33, 1371), (4, 2048), (17, 4096), (6, 5000), (2, 8200),
          (3, 16384), (400, 512)]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]


def make(seed, rows, width, dt, rt, gate=True, residual=True, weights=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=(0.7 * r(rows, width)).to(dt), residual=(2 * r(rows, width)).to(rt) if residual else None,
                gate=r(rows, width).to(dt) if gate else None, w1=r(width) if weights else None,
                scale=1 + 0.3 * r(width) if weights else None, w2=r(width) if weights else None,
                d_h=r(rows, width).to(rt if residual else dt), d_y=r(rows, width).to(dt))


def reference(d, need_grad, use_dh=True, use_dy=True, **kw):
    names = ("x", "residual", "gate", "w1", "scale", "w2")
    leaf = {n: None if d[n] is None else d[n].double().requires_grad_(need_grad) for n in names}
    h, y = R.block_norm(*(leaf[n] for n in names), **kw)
    if not need_grad:
        return h, y
    loss = 0.0
    if use_dh:
        loss = loss + (h * d["d_h"].double()).sum()
    if use_dy:
        loss = loss + (y * d["d_y"].double()).sum()
    have = [n for n in names if leaf[n] is not None]
    g = torch.autograd.grad(loss, [leaf[n] for n in have], allow_unused=True)
    return {n: (torch.zeros_like(leaf[n]) if t is None else t) for n, t in zip(have, g)}


def norm_of(c, **kw):
    from linear_attention_sequence_sm_b200 import gdn
    return gdn.BlockNorm(post_weight=c["w1"] if kw.get("post", True) else None, post_norm=kw.get("post", True),
                         scale=c["scale"], pre_weight=c["w2"] if kw.get("pre", True) else None,
                         pre_norm=kw.get("pre", True), eps=kw.get("eps", 1e-6), residual_scale=kw.get("rho", 1.0),
                         branch_scale=kw.get("branch", 1.0), activation=kw.get("activation", "silu"),
                         zero_centred=kw.get("zero_centred", False))


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach()
    return float((a - b).norm() / b.norm().clamp(min=1e-30))


def bar(t):
    return (2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0) + F32 + SIG


VARIANTS = [dict(), dict(post=False), dict(rho=0.75, branch=0.5, zero_centred=True), dict(activation="sigmoid"),
            dict(eps=1e-2)]


@pytest.mark.parametrize("types", TYPES, ids=["bf16", "bf16_wide", "f32"])
@pytest.mark.parametrize("size", WIDTHS, ids=str)
@pytest.mark.parametrize("gate", [True, False])
def test_forward_and_backward(gate, size, types):
    from linear_attention_sequence_sm_b200 import gdn
    for i, kw in enumerate(VARIANTS):
        d = make(40 + i, *size, *types, gate=gate)
        if not kw.get("post", True):
            d["w1"] = None
        c = R.cuda(d)
        n = norm_of(c, **kw)
        h, y = gdn.block_norm_forward(c["x"], c["residual"], n, gate=c["gate"])
        got = gdn.block_norm_backward(c["x"], c["residual"], n, gate=c["gate"], d_h=c["d_h"], d_y=c["d_y"])
        torch.cuda.synchronize()
        rh, ry = reference(d, False, **kw)
        assert h.dtype == types[1] and y.dtype == types[0]
        assert rel(h, rh) <= bar(h) and rel(y, ry) <= bar(y), kw
        ref = reference(d, True, **kw)
        names = dict(x="dx", residual="d_residual", gate="d_gate", w1="d_post_weight", scale="d_scale",
                     w2="d_pre_weight")
        for k, name in names.items():
            if k not in ref:
                assert got[name] is None
                continue
            if size[1] == 1 and k == "x" and kw.get("post", True):
                continue  # x / |x| of one value: its gradient is eps-sized, all of it cancellation
            # the gradients subtract a mean from terms of their own size: twice the forward's error
            assert rel(got[name], ref[k]) <= 2 * bar(got[name]) + (1e-4 if size[1] < 8 else 0.0), (name, kw)


@pytest.mark.parametrize("types", TYPES, ids=["bf16", "bf16_wide", "f32"])
def test_parts_left_out(types):
    """No weights, no residual, no norm after; one upstream gradient at a time."""
    from linear_attention_sequence_sm_b200 import gdn
    d = make(50, 37, 1024, *types, residual=False, weights=False)
    c = R.cuda(d)
    n = norm_of(c)
    h, y = gdn.block_norm_forward(c["x"], None, n, gate=c["gate"])
    rh, ry = reference(d, False)
    assert h.dtype == types[0] and rel(h, rh) <= bar(h) and rel(y, ry) <= bar(y)
    d = make(51, 37, 1024, *types)
    c = R.cuda(d)
    bare = norm_of(c, pre=False)
    h, y = gdn.block_norm_forward(c["x"], c["residual"], bare, gate=c["gate"])
    assert y is None
    d0 = dict(d, w2=None)
    rh, _ = reference(d0, False, pre=False)
    assert rel(h, rh) <= bar(h)
    got = gdn.block_norm_backward(c["x"], c["residual"], bare, gate=c["gate"], d_h=c["d_h"])
    ref = reference(d0, True, use_dy=False, pre=False)
    assert rel(got["dx"], ref["x"]) <= 2 * bar(got["dx"]) and got["d_pre_weight"] is None
    full = norm_of(c)
    got = gdn.block_norm_backward(c["x"], c["residual"], full, gate=c["gate"], d_y=c["d_y"])
    ref = reference(d, True, use_dh=False)
    assert rel(got["d_residual"], ref["residual"]) <= 2 * bar(got["d_residual"])
    assert rel(got["d_gate"], ref["gate"]) <= 2 * bar(got["d_gate"])
    got = gdn.block_norm_backward(c["x"], c["residual"], full, gate=c["gate"], d_h=c["d_h"])
    assert bool((got["d_pre_weight"] == 0).all())


def test_in_place_and_empty():
    from linear_attention_sequence_sm_b200 import gdn
    d = make(52, 300, 4096, torch.bfloat16, torch.float32)
    c = R.cuda(d)
    n = norm_of(c)
    h, y = gdn.block_norm_forward(c["x"], c["residual"], n, gate=c["gate"])
    x, r = c["x"].clone(), c["residual"].clone()
    gdn.block_norm_forward(x, r, n, gate=c["gate"], h=r, y=x)
    torch.cuda.synchronize()
    assert torch.equal(r, h) and torch.equal(x, y)
    e = {k: (t[:0] if t is not None and t.dim() == 2 else t) for k, t in c.items()}
    h, y = gdn.block_norm_forward(e["x"], e["residual"], n, gate=e["gate"])
    got = gdn.block_norm_backward(e["x"], e["residual"], n, gate=e["gate"], d_h=e["d_h"], d_y=e["d_y"])
    torch.cuda.synchronize()
    assert h.shape == (0, 4096) and y.shape == (0, 4096)
    assert all(bool((got[k] == 0).all()) for k in ("d_post_weight", "d_scale", "d_pre_weight"))


def test_backward_against_differences():
    from linear_attention_sequence_sm_b200 import gdn
    d = make(53, 9, 300, torch.float32, torch.float32)
    c = R.cuda(d)
    kw = dict(rho=0.75, branch=0.5)
    got = gdn.block_norm_backward(c["x"], c["residual"], norm_of(c, **kw), gate=c["gate"], d_h=c["d_h"], d_y=c["d_y"])
    names = dict(x="dx", residual="d_residual", gate="d_gate", w1="d_post_weight", scale="d_scale", w2="d_pre_weight")

    def loss(x):
        h, y = R.block_norm(*(x[n] for n in names), **kw)
        return float((h * d["d_h"].double()).sum() + (y * d["d_y"].double()).sum())

    base = {k: d[k].double() for k in names}
    gen = torch.Generator().manual_seed(3)
    for k, name in names.items():
        step = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        diff = (loss({**base, k: base[k] + 1e-5 * step}) - loss({**base, k: base[k] - 1e-5 * step})) / 2e-5
        terms = got[name].double().cpu() * step
        assert abs(float(terms.sum()) - diff) <= 1e-4 * float(terms.norm()), k


def test_same_bits_and_graph():
    from linear_attention_sequence_sm_b200 import gdn
    d = make(54, 1000, 1024, torch.bfloat16, torch.bfloat16)
    c = R.cuda(d)
    n = norm_of(c)
    run = lambda: [*gdn.block_norm_forward(c["x"], c["residual"], n, gate=c["gate"]),  # noqa: E731
                   *gdn.block_norm_backward(c["x"], c["residual"], n, gate=c["gate"], d_h=c["d_h"],
                                            d_y=c["d_y"]).values()]
    a, b = run(), run()
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    c["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(outs, run()))


@pytest.mark.parametrize("types", TYPES, ids=["bf16", "bf16_wide", "f32"])
@pytest.mark.parametrize("size", [(1301, 4096), (2503, 2048), (2601, 1032), (9477, 264), (10003, 24)], ids=str)
def test_many_rows(size, types):
    """Rows enough for several groups a block, the last ones short; each part of the gradients wanted or not."""
    from linear_attention_sequence_sm_b200 import gdn
    names = dict(x="dx", residual="d_residual", gate="d_gate", w1="d_post_weight", scale="d_scale", w2="d_pre_weight")
    full = dict(rho=0.75, branch=0.5, zero_centred=True)
    for gate, use, kw in ((True, {}, full), (False, dict(use_dh=False), dict(activation="sigmoid")),
                          (True, {}, dict(activation="sigmoid", post=False)), (True, dict(use_dy=False), dict(pre=False)),
                          (False, {}, dict()), (False, {}, dict(post=False)), (True, {}, dict(post=False)),
                          (True, {}, dict(activation="sigmoid"))):
        d = make(57, *size, *types, gate=gate)
        for k, on in (("w1", kw.get("post", True)), ("w2", kw.get("pre", True))):
            if not on:
                d[k] = None
        c = R.cuda(d)
        up = {k: c[k] for k, flag in (("d_h", "use_dh"), ("d_y", "use_dy")) if use.get(flag, True)}
        got = gdn.block_norm_backward(c["x"], c["residual"], norm_of(c, **kw), gate=c["gate"], **up)
        torch.cuda.synchronize()
        ref = reference(d, True, **use, **kw)
        for k, name in names.items():
            if k not in ref:
                assert got[name] is None
                continue
            # twice the forward's error, as in test_forward_and_backward; column sums of `rows` fp32 terms each: a
            # chain of at most rows / 148 + 16 additions, (that + 296) u of terms that do not cancel in the norm
            bars = 2 * bar(got[name]) + (size[0] / 148 + 312) * R.U32
            assert rel(got[name], ref[k]) <= bars, (name, gate, kw)


@pytest.mark.parametrize("types", TYPES, ids=["bf16", "bf16_wide", "f32"])
@pytest.mark.parametrize("size", [(14_001, 264), (3_553, 1032), (1_801, 2048), (1_801, 4096), (601, 5128), (601, 8192),
                                  (453, 12_288)], ids=str)
@pytest.mark.parametrize("gate", [True, False])
def test_rows_enough_to_use_every_stage_again(gate, size, types):
    """A block's stages of rows are filled, read and filled again several times over, the last groups short; the
    forward and the gradients against their definition."""
    from linear_attention_sequence_sm_b200 import gdn
    kw = dict(rho=0.75, branch=0.5)
    d = make(58, *size, *types, gate=gate)
    c = R.cuda(d)
    n = norm_of(c, **kw)
    h, y = gdn.block_norm_forward(c["x"], c["residual"], n, gate=c["gate"])
    got = gdn.block_norm_backward(c["x"], c["residual"], n, gate=c["gate"], d_h=c["d_h"], d_y=c["d_y"])
    torch.cuda.synchronize()
    rh, ry = reference(d, False, **kw)
    ref = reference(d, True, **kw)
    worst = lambda a, b: float(((a.double().cpu() - b).norm(dim=-1) / b.norm(dim=-1)).max())  # noqa: E731
    # row by row, so that one row left out or taken twice shows
    assert worst(h, rh.detach()) <= bar(h) and worst(y, ry.detach()) <= bar(y)
    names = dict(x="dx", residual="d_residual", gate="d_gate", w1="d_post_weight", scale="d_scale", w2="d_pre_weight")
    for k, name in names.items():
        if k not in ref:
            continue
        # as in test_many_rows
        bars = 2 * bar(got[name]) + (size[0] / 148 + 312) * R.U32
        assert rel(got[name], ref[k]) <= bars, name
        if k in ("x", "residual", "gate"):
            # a row's gradients: three sums more than its values
            assert worst(got[name], ref[k].detach()) <= 4 * bar(got[name]), name
