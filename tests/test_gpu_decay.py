"""The decayed linear attention on the GPU against its recurrence in 64 bits.

Tolerances, relative 2-norms over (sequence, head) slices, counted in half
steps of the types (fp32: u = 2^-24; bf16: 2^-8).  A token's output sums at
most 64 + 128 products inside a chunk and a state that came through the
chunks before it (at most 24 here), each sum within u of its terms: 256 u.
bf16 outputs add their own rounding and, on the tensor cores, the rounding of
the masked products and of the state's copy: 3 half steps.  dg adds and takes
off the one-ended sums of up to 16 chunks on each side, each within 256 u of
sums no larger than the slice: 32 * 256 u."""
import pytest
import torch

import decay_ref as R
import streams

pytestmark = pytest.mark.gpu

F32 = 256 * R.U32
BF16 = 3 * 2.0 ** -8
DG = 32 * 256 * R.U32

SHAPES = [  # hk, hv, dk, dv
    (1, 1, 128, 128), (2, 4, 128, 128), (1, 3, 64, 64), (2, 2, 40, 72), (1, 2, 128, 64), (1, 2, 24, 128),
    (2, 2, 33, 17), (1, 1, 1, 1),
]
LENGTHS = [dict(batch=(1, 1)), dict(batch=(2, 64)), dict(batch=(1, 65)), dict(lens=[63, 0, 130, 1]),
           dict(lens=[0, 0]), dict(batch=(3, 191)), dict(lens=[700, 5])]


def dtypes(f):
    return pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])(f)


def run_forward(d, **kw):
    from linear_attention_sequence_sm_b200 import gdn
    c = R.cuda(d)
    out = gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=c["s0"], cu_seqlens=c["cu"], **kw)
    torch.cuda.synchronize()
    return out


def check_forward(d, o, sf):
    lens = R.lens_of(d["q"], d["cu"])
    ro, rs = R.forward(d["q"], d["k"], d["v"], d["g"], d["s0"], d["cu"])
    bar = BF16 if d["q"].dtype == torch.bfloat16 else F32
    assert R.worst(o, ro, lens, True) <= bar
    assert R.worst(sf, rs, lens, False) <= F32


@dtypes
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, lengths, dtype):
    d = R.make(3, *shape, dtype, **lengths)
    check_forward(d, *run_forward(d))


@dtypes
@pytest.mark.parametrize("shape", [(1, 2, 128, 128), (1, 1, 64, 40)], ids=str)
def test_forward_per_head_decays_and_no_state(shape, dtype):
    d = R.make(5, *shape, dtype, lens=[200, 31], per_token=False, s0=False)
    check_forward(d, *run_forward(d))


@dtypes
@pytest.mark.parametrize("tokens", [257, 512, 1500])
def test_forward_split_sequences(tokens, dtype):
    """Few chains: sequences are cut into segments (the first longer than 256)."""
    d = R.make(7, 1, 2, 128, 128, dtype, lens=[tokens, 100])
    check_forward(d, *run_forward(d))


@dtypes
def test_forward_simt_and_default_agree_with_strong_decays(dtype):
    """Decays of e^-1 to e^-20 a token, values below the floor among them, and none at all."""
    d = R.make(9, 1, 4, 128, 128, dtype, lens=[150, 64])
    d["g"][:, 0] = 0.0
    d["g"][:, 1] = -1.0
    d["g"][:, 2] = -20.0
    d["g"][::3, 3] = -40.0
    d["g"][1::7, 3] = float("-inf")
    for simt in (False, True):
        check_forward(d, *run_forward(d, force_simt=simt))


@dtypes
def test_decode_continues_prefill(dtype):
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(11, 2, 4, 128, 128, dtype, batch=(3, 70))
    _, rs = R.forward(d["q"], d["k"], d["v"], d["g"], d["s0"])
    ro, _ = R.forward(d["q"], d["k"], d["v"], d["g"], d["s0"])
    c = R.cuda(d)
    cut = {k: c[k][:, :66].contiguous() for k in ("q", "k", "v", "g")}
    _, state = gdn.decay_forward(cut["q"], cut["k"], cut["v"], cut["g"], initial_state=c["s0"])
    outs = []
    for t in range(66, 70):
        outs.append(gdn.decay_decode_step(c["q"][:, t].contiguous(), c["k"][:, t].contiguous(),
                                          c["v"][:, t].contiguous(), c["g"][:, t].contiguous(), state))
    torch.cuda.synchronize()
    ref = ro.reshape(3, 70, 4, 128)[:, 66:]
    got = torch.stack(outs, 1).double().cpu()
    rel = (got - ref).norm(dim=(1, 3)) / ref.norm(dim=(1, 3))
    # the decode step keeps everything in fp32 and rounds once
    assert float(rel.max()) <= (2.0 ** -8 + F32 if dtype == torch.bfloat16 else F32)
    assert R.worst(state, rs, None, False) <= F32


@dtypes
@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("shape", [(1, 1, 128, 128), (2, 6, 128, 100), (3, 6, 80, 72), (1, 2, 33, 5), (1, 1, 256, 64),
                                   (2, 2, 132, 130), (1, 2, 16, 1), (4, 8, 64, 64)], ids=str)
@pytest.mark.parametrize("n", [1, 5, 200])
def test_decode(n, shape, per_token, dtype):
    from linear_attention_sequence_sm_b200 import gdn
    hk, hv, dk, dv = shape
    d = R.make(13, hk, hv, dk, dv, dtype, batch=(n, 1), per_token=per_token)
    ro, rs = R.forward(d["q"], d["k"], d["v"], d["g"], d["s0"])
    c = R.cuda(d)
    state = c["s0"].clone()
    one = lambda t: t[:, 0].contiguous()  # noqa: E731
    o = gdn.decay_decode_step(one(c["q"]), one(c["k"]), one(c["v"]), one(c["g"]) if per_token else c["g"], state)
    torch.cuda.synchronize()
    # An output is one sum of d_k products, and where they cancel its own size bounds nothing: the error
    # of a sum of d_k products of fp32 values, each s = a s' + v k within 3 u of |a s'| + |v k| (a's own
    # error, the product's, the sum's), is at most (d_k + 4) u sum_j (|a s'_j| + |v k_j|) |q_j|.
    absd = {k: (t.abs() if k != "g" else t) for k, t in d.items() if k in ("q", "k", "v", "g", "s0")}
    size, _ = R.forward(absd["q"], absd["k"], absd["v"], absd["g"], absd["s0"])
    half = 2.0 ** -8 if dtype == torch.bfloat16 else R.U32
    err = (o.double().cpu() - ro).abs()
    assert bool((err <= (dk + 4) * R.U32 * size * (1 + half) + half * ro.abs()).all())
    assert R.worst(state, rs, None, False) <= 4 * R.U32


def grads(d, **kw):
    from linear_attention_sequence_sm_b200 import gdn
    c = R.cuda(d)
    out = gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], c["do"], d_final_state=c["dsf"], initial_state=c["s0"],
                             cu_seqlens=c["cu"], **kw)
    torch.cuda.synchronize()
    return out


def check_backward(d, got, dg_bar=DG):
    lens = R.lens_of(d["q"], d["cu"])
    ref = R.backward(d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"], d["s0"], d["cu"])
    bar = BF16 if d["q"].dtype == torch.bfloat16 else F32
    for name in ("dq", "dk", "dv"):
        assert got[name].dtype == d["q"].dtype
        assert R.worst(got[name], ref[name], lens, True) <= bar, name
    assert R.worst(got["d_initial_state"], ref["d_initial_state"], lens, False) <= F32
    if d["g"].dim() == 1:
        rel = (got["dg"].double().cpu() - ref["dg"]).norm() / ref["dg"].norm().clamp(min=1e-30)
        assert float(rel) <= dg_bar
    else:
        assert R.worst(got["dg"], ref["dg"], lens, True) <= dg_bar


@dtypes
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, lengths, dtype):
    d = R.make(17, *shape, dtype, **lengths)
    check_backward(d, grads(d))


@dtypes
@pytest.mark.parametrize("tokens", [300, 1500])
@pytest.mark.parametrize("per_token", [True, False])
def test_backward_split_sequences(per_token, tokens, dtype):
    d = R.make(19, 1, 2, 128, 128, dtype, lens=[64, tokens], per_token=per_token)
    check_backward(d, grads(d))


@dtypes
def test_backward_without_states(dtype):
    d = R.make(21, 2, 2, 128, 128, dtype, batch=(2, 130), s0=False)
    d["dsf"] = None
    got = grads(d)
    check_backward(d, got)
    lean = grads(d, want_dg=False, want_d_initial_state=False)
    assert lean["dg"] is None and lean["d_initial_state"] is None
    # without dg the state's copy is rounded once (with it, its products feed a 32-bit sum): the bars
    # of the formula hold either way, equal bits do not
    check_backward(d, dict(got, **{n: lean[n] for n in ("dq", "dk", "dv")}))


@dtypes
@pytest.mark.parametrize("simt", [False, True])
def test_backward_strong_decays(simt, dtype):
    """dg stays accurate where the decays are strong (small beside q . dq) and is zero below the floor."""
    d = R.make(23, 1, 4, 128, 128, dtype, lens=[150, 64])
    d["g"][:, 0] = 0.0
    d["g"][:, 1] = -3.0
    d["g"][:, 2] = -8.0
    d["g"][::3, 3] = -40.0
    got = grads(d, force_simt=simt)
    check_backward(d, got)
    assert bool((got["dg"][::3, 3] == 0).all())


def test_backward_against_differences():
    """Directional differences of the 64-bit forward against the kernels' gradients (fp32)."""
    d = R.make(25, 1, 2, 24, 16, torch.float32, lens=[70, 9])
    got = grads(d)

    def loss(x):
        o, S = R.forward(x["q"], x["k"], x["v"], x["g"], x["s0"], d["cu"])
        return float((o * d["do"].double().reshape(o.shape)).sum() + (S * d["dsf"].double()).sum())

    gen = torch.Generator().manual_seed(1)
    names = dict(q="dq", k="dk", v="dv", g="dg", s0="d_initial_state")
    base = {k: d[k].double() for k in names}
    for k, name in names.items():
        step = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        diff = (loss({**base, k: base[k] + h * step}) - loss({**base, k: base[k] - h * step})) / (2 * h)
        terms = got[name].double().cpu().reshape(step.shape) * step
        # the difference is off by h^2 times third derivatives and 1e-16 / h of the loss
        assert abs(float(terms.sum()) - diff) <= 1e-4 * float(terms.norm()), k


def test_same_call_same_bits():
    d = R.make(27, 2, 6, 128, 128, torch.bfloat16, lens=[300, 64, 77])
    a, b = grads(d), grads(d)
    assert all(torch.equal(a[k], b[k]) for k in a)
    x, y = run_forward(d), run_forward(d)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@dtypes
def test_output_side(dtype):
    """The output side over o: one more rounding of o (stored, then read again)."""
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(29, 1, 2, 128, 128, dtype, batch=(2, 70))
    gen = torch.Generator().manual_seed(2)
    w, z = torch.randn(128, generator=gen), torch.randn(2, 70, 2, 128, generator=gen).to(dtype)
    y, _ = run_forward(d, output_norm=gdn.OutputNorm(weight=w.cuda(), gate=z.cuda(), eps=1e-6))
    ro, _ = R.forward(d["q"], d["k"], d["v"], d["g"], d["s0"])
    zz = z.double().reshape(ro.shape)
    ref = ro / (ro.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double() * zz * torch.sigmoid(zz)
    # two relative errors of o (its own and its root mean square's) and the result's rounding
    bar = 2 * BF16 + 2.0 ** -8 if dtype == torch.bfloat16 else 4 * F32
    assert R.worst(y, ref, [70, 70], True) <= bar
    one = lambda t: t[:, 0].contiguous()  # noqa: E731
    c = R.cuda(d)
    y1 = gdn.decay_decode_step(one(c["q"]), one(c["k"]), one(c["v"]), one(c["g"]), c["s0"].clone(),
                               output_norm=gdn.OutputNorm(weight=w.cuda(), gate=one(z.cuda()), eps=1e-6))
    first = ref.reshape(2, 70, 2, 128)[:, 0]
    assert R.worst(y1, first, [1, 1], True) <= bar


def test_bad_cu_seqlens_leaves_outputs_and_says_so():
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(31, 1, 2, 128, 128, torch.bfloat16, lens=[40, 60])
    c = R.cuda(d)
    for bad in ([0, 101, 100], [1, 40, 100], [0, 40, 99], [0, 60, 40], [0, -1, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        shape = gdn.make_shape(c["q"], c["v"], cu, 64)
        ws = torch.empty(gdn.decay_workspace_size(shape, backward=True), dtype=torch.uint8, device="cuda")
        o, sf = torch.full_like(c["v"], 7.0), torch.full_like(c["s0"], 7.0)
        gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=c["s0"], cu_seqlens=cu, out=o, final_state=sf,
                          workspace=ws)
        assert gdn.read_device_status(ws) == gdn.GDN_ERR_DEVICE_CHECK
        assert bool((o == 7).all()) and bool((sf == 7).all())
        gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], c["do"], cu_seqlens=cu, workspace=ws)
        assert gdn.read_device_status(ws) == gdn.GDN_ERR_DEVICE_CHECK
    gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], cu_seqlens=c["cu"], workspace=ws)
    assert gdn.read_device_status(ws) == gdn.GDN_OK


def test_final_state_in_place_and_other_stream():
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(33, 1, 2, 128, 128, torch.bfloat16, batch=(1, 400))
    o, sf = run_forward(d)
    c = R.cuda(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = c["s0"].clone()
    side.wait_stream(torch.cuda.current_stream())
    o2, s2 = gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=state, final_state=state, stream=side)
    side.synchronize()
    assert s2 is state and torch.equal(o, o2) and torch.equal(sf, state)


def test_captured_and_replayed():
    """Prefill, decode and backward in one graph, replayed on new inputs."""
    from linear_attention_sequence_sm_b200 import gdn
    d, e = (R.make(s, 1, 2, 128, 128, torch.bfloat16, lens=[300, 50]) for s in (35, 36))
    c = R.cuda(d)
    state = c["s0"].clone()
    one = {k: c[k][:2].contiguous() for k in ("q", "k", "v", "g")}

    def step():
        state.copy_(c["s0"])
        o, sf = gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=state, cu_seqlens=c["cu"],
                                  final_state=state)
        t = gdn.decay_decode_step(one["q"], one["k"], one["v"], one["g"], state)
        gr = gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], c["do"], d_final_state=c["dsf"],
                                initial_state=c["s0"], cu_seqlens=c["cu"])
        return [o, t, state, *gr.values()]

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for src in (e, d):
        for k, t in R.cuda(src).items():
            c[k].copy_(t)
        for k in one:
            one[k].copy_(c[k][:2])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@dtypes
@pytest.mark.parametrize("simt", [False, True])
def test_nan_decay_stays_in_its_head_and_after_its_token(simt, dtype):
    """A NaN log-decay is not taken for the floor: its head is NaN from that token on, all else as without it."""
    d = R.make(37, 1, 2, 128, 128, dtype, lens=[100, 140, 30])
    o, sf = run_forward(d, force_simt=simt)
    d["g"][170, 1] = float("nan")  # sequence 1, its second chunk
    on, sn = run_forward(d, force_simt=simt)
    hit = torch.zeros(270, 2, dtype=torch.bool)
    hit[170:240, 1] = True
    on, o = on.cpu(), o.cpu()
    assert bool(on[hit].isnan().all()) and torch.equal(on[~hit], o[~hit])
    assert bool(sn[1, 1].isnan().all()) and torch.equal(sn[1, 0], sf[1, 0]) and torch.equal(sn[::2], sf[::2])
    from linear_attention_sequence_sm_b200 import gdn
    c = R.cuda(d)
    one = {k: c[k][169:171].clone() for k in ("q", "k", "v", "g")}
    t = gdn.decay_decode_step(one["q"], one["k"], one["v"], one["g"], c["s0"][:2].clone())
    assert bool(t[1, 1].isnan().all()) and not bool(t[0].isnan().any()) and not bool(t[1, 0].isnan().any())


@dtypes
@pytest.mark.parametrize("simt", [False, True])
def test_values_of_other_sequences_do_not_leak(simt, dtype):
    """Infinities and NaN in a sequence stay in it, with ends inside chunks on both sides."""
    d = R.make(39, 1, 2, 128, 128, dtype, lens=[70, 50, 90])
    o, sf = run_forward(d, force_simt=simt)
    base = grads(d, force_simt=simt)
    bad = {k: (t.clone() if t is not None else None) for k, t in d.items()}
    for k, x in (("q", float("nan")), ("k", float("inf")), ("v", float("-inf")), ("do", float("nan"))):
        bad[k][70:120] = x
    on, sn = run_forward(bad, force_simt=simt)
    got = grads(bad, force_simt=simt)
    keep = torch.ones(210, dtype=torch.bool)
    keep[70:120] = False
    assert torch.equal(on.cpu()[keep], o.cpu()[keep]) and torch.equal(sn[::2], sf[::2])
    for k in ("dq", "dk", "dv", "dg"):
        assert torch.equal(got[k].cpu()[keep], base[k].cpu()[keep]), k
    assert torch.equal(got["d_initial_state"][::2], base["d_initial_state"][::2])


def test_output_side_leaves_rejected_calls_alone():
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(31, 1, 2, 128, 128, torch.bfloat16, lens=[40, 60])
    c = R.cuda(d)
    cu = torch.tensor([0, 60, 40], dtype=torch.int32, device="cuda")
    o = torch.full_like(c["v"], 7.0)
    gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], cu_seqlens=cu, out=o, output_norm=gdn.OutputNorm(eps=1e-6))
    torch.cuda.synchronize()
    assert bool((o == 7).all())


def test_workspaces_belong_to_the_calls_stream():
    """A call queued on a side stream behind other work: memory that later work on the current stream takes and
    fills must not be the call's workspace."""
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(41, 1, 2, 128, 128, torch.bfloat16, lens=[700, 64])
    want, wf = grads(d), run_forward(d)
    c = R.cuda(d)
    sizes = [gdn.decay_workspace_size(gdn.make_shape(c["q"], c["v"], c["cu"], 64), backward=b) for b in (True, False)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
    got = gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], c["do"], d_final_state=c["dsf"], initial_state=c["s0"],
                             cu_seqlens=c["cu"], stream=side)
    o, sf = gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=c["s0"], cu_seqlens=c["cu"], stream=side)
    for n in sizes * 2:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert torch.equal(o, wf[0]) and torch.equal(sf, wf[1])


@dtypes
def test_many_sequences_and_checkpoints(dtype):
    """Gradients where cuts, checkpoints and sequence ends fall into one another: one long sequence among short ones."""
    d = R.make(43, 1, 2, 64, 64, dtype, lens=[1, 30, 1300, 2, 64, 257, 1])
    check_backward(d, grads(d))


@dtypes
@pytest.mark.parametrize("shape", [(1, 3, 33, 17), (2, 4, 7, 5), (1, 2, 12, 20)], ids=str)
@pytest.mark.parametrize("per_token", [True, False])
def test_backward_grouped_heads_of_odd_sizes(per_token, shape, dtype):
    d = R.make(45, *shape, dtype, lens=[70, 0, 33], per_token=per_token)
    check_backward(d, grads(d))


def test_two_calls_at_once():
    """Prefills and gradients on two streams side by side, each with its own workspace."""
    from linear_attention_sequence_sm_b200 import gdn
    ds = [R.make(s, 2, 4, 128, 128, torch.bfloat16, lens=ls) for s, ls in ((47, [900, 130, 64]), (48, [65] * 9))]
    want = [(run_forward(d), grads(d)) for d in ds]
    cs = [R.cuda(d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cs, streams)):
            f = gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=c["s0"], cu_seqlens=c["cu"], stream=s)
            b = gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], c["do"], d_final_state=c["dsf"],
                                   initial_state=c["s0"], cu_seqlens=c["cu"], stream=s)
            got[i].append((f, b))
    torch.cuda.synchronize()
    for (wf, wb), runs in zip(want, got):
        for f, b in runs:
            assert torch.equal(f[0], wf[0]) and torch.equal(f[1], wf[1])
            assert all(torch.equal(b[k], wb[k]) for k in wb)


def test_outputs_belong_to_the_calls_stream():
    from linear_attention_sequence_sm_b200 import gdn
    d = R.make(51, 1, 2, 128, 128, torch.bfloat16, lens=[300, 64])
    c = R.cuda(d)
    rows = c["v"].reshape(-1, 256).contiguous()
    one = {k: c[k][:2].contiguous() for k in ("q", "k", "v", "g")}
    norm, state = gdn.BlockNorm(), c["s0"].clone()

    def decode(s):
        with torch.cuda.stream(s):
            state.copy_(c["s0"])
        return [gdn.decay_decode_step(one["q"], one["k"], one["v"], one["g"], state, stream=s)]

    calls = [
        lambda s: gdn.decay_forward(c["q"], c["k"], c["v"], c["g"], initial_state=c["s0"], cu_seqlens=c["cu"], stream=s),
        decode,
        lambda s: list(gdn.decay_backward(c["q"], c["k"], c["v"], c["g"], c["do"], d_final_state=c["dsf"],
                                          initial_state=c["s0"], cu_seqlens=c["cu"], stream=s).values()),
        lambda s: gdn.block_norm_forward(rows, rows, norm, stream=s),
        lambda s: [t for t in gdn.block_norm_backward(rows, rows, norm, d_h=rows, d_y=rows, stream=s).values()
                   if t is not None],
    ]
    streams.check_outputs_belong_to_the_calls_stream(calls)


def dg_sizes(d):
    """a_t |dS_t| |S_(t-1)| (2-norms) per token and head, in 64 bits: what dg_t = a_t <dS_t, S_(t-1)> is a product of."""
    lens = R.lens_of(d["q"], d["cu"])
    q, k, v, do = (d[n].reshape(-1, *d[n].shape[-2:]).double() for n in ("q", "k", "v", "do"))
    hv = v.shape[1]
    head = torch.arange(hv) // (hv // q.shape[1])
    a = d["g"].double().reshape(-1, hv).clamp(min=R.FLOOR).exp()
    left, right, start = torch.zeros_like(a), torch.zeros_like(a), 0
    for n, ln in enumerate(lens):
        S, D = d["s0"][n].double(), d["dsf"][n].double()
        for t in range(start, start + ln):
            left[t] = S.flatten(1).norm(dim=-1)
            S = a[t][:, None, None] * S + v[t][:, :, None] * k[t, head][:, None, :]
        for t in reversed(range(start, start + ln)):
            D = D + do[t][:, :, None] * q[t, head][:, None, :]
            right[t] = D.flatten(1).norm(dim=-1)
            D = a[t][:, None, None] * D
        start += ln
    return a * left * right


@dtypes
@pytest.mark.parametrize("simt", [False, True])
def test_backward_lone_strong_decays_among_slow_ones(simt, dtype):
    """A token whose decay nearly ends what came before it: its dg is tiny beside its neighbours' and still right.
    dg_t is a product of the two states, put together from four parts (pairs inside the chunk, pairs with one end in
    it on either side, pairs across it), each within 256 u of the product of the norms it is made of; the parts of
    tokens drawn independently have norms of at most about the whole's, twice that for the bar."""
    d = R.make(49, 2, 4, 64, 64, dtype, lens=[1100, 130])
    d["g"].fill_(-0.01)
    for h, x in enumerate((-8.0, -12.0, -15.0, -19.0)):
        for t in (0, 1, 640, 700, 767, 1090, 1150):
            d["g"][t, h] = x
    got = grads(d, force_simt=simt)
    ref = R.backward(d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"], d["s0"], d["cu"])
    err = (got["dg"].double().cpu() - ref["dg"]).abs()
    assert float((err / dg_sizes(d)).max()) <= 8 * 256 * R.U32
    check_backward(d, got)


@pytest.mark.parametrize("where", [75, 154, 219], ids=["first chunk", "second chunk", "last token"])
@pytest.mark.parametrize("x", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("form", ["bf16", "bf16_simt", "f32"])
def test_one_infinity_or_nan_reaches_what_it_must_and_no_more(form, x, where):
    """An element that is not finite makes exactly those results not finite that the recurrence makes of it: nothing
    before its token (behind it, for the gradients that run backward in time), whatever the chunk it falls into.  All
    other results are what they are without it."""
    dtype, simt = (torch.float32 if form == "f32" else torch.bfloat16), form == "bf16_simt"
    d = R.make(53, 2, 4, 48, 72, dtype, lens=[70, 150, 20])
    o, sf = run_forward(d, force_simt=simt)
    base = dict(grads(d, force_simt=simt), o=o, sf=sf)
    for name, at in (("q", (where, 1, 5)), ("k", (where, 0, 40)), ("v", (where, 1, 70)), ("do", (where, 3, 11))):
        bad = dict(d, **{name: d[name].clone()})
        bad[name][at] = x
        ro, rs = R.forward(bad["q"], bad["k"], bad["v"], bad["g"], bad["s0"], bad["cu"])
        ref = dict(R.backward(bad["q"], bad["k"], bad["v"], bad["g"], bad["do"], bad["dsf"], bad["s0"], bad["cu"]), o=ro, sf=rs)
        o, sf = run_forward(bad, force_simt=simt)
        got = dict(grads(bad, force_simt=simt), o=o, sf=sf)
        for k, r in ref.items():
            g, b = got[k].cpu().reshape(r.shape), base[k].cpu().reshape(r.shape)
            hit = ~r.isfinite()
            if form == "bf16" and k in ("o", "dq", "dk", "dv"):
                # some of these come from other products than without the element: each within three half steps of
                # the formula (see above), here of the row's largest value
                scale = b.float().abs().amax(-1, keepdim=True).expand_as(b)
                assert bool(((g.float() - b.float()).abs() <= 2 * BF16 * scale)[~hit].all()), (name, k)
            else:
                assert torch.equal(g[~hit], b[~hit]), (name, k)
            assert not bool(g[hit].isfinite().any()), (name, k)


def test_no_tokens_and_a_rejected_cu_seqlens():
    """Without tokens a fixed decay's gradient is zero, and as it was where cu_seqlens is rejected."""
    import ctypes
    from linear_attention_sequence_sm_b200 import gdn
    q, v = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.full((2,), -0.5, device="cuda")
    for cus, want in (([0, 0, 0], 0.0), ([0, 5, 0], 7.0), ([1, 0, 0], 7.0)):
        cu = torch.tensor(cus, dtype=torch.int32, device="cuda")
        sh = gdn.make_shape(q, v, cu, 64)
        n = gdn.decay_workspace_size(sh, backward=True)
        ws, dg = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.full((2,), 7.0, device="cuda")
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        st = gdn.LIB.gdn_decay_backward(ctypes.byref(sh), p(q), p(q), p(v), p(g), gdn.GDN_DECAY_PER_HEAD, None, p(cu),
                                        p(v), None, p(q), p(q), p(v), p(dg), None, p(ws), n, None)
        assert st == gdn.GDN_OK
        assert gdn.read_device_status(ws) == (gdn.GDN_OK if want == 0 else gdn.GDN_ERR_DEVICE_CHECK)
        assert dg.tolist() == [want, want]


@pytest.mark.parametrize("form", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 4, 128, 128), (1, 2, 24, 40)], ids=str)
def test_more_units_than_blocks(shape, form):
    """Blocks take several (sequence, head) pairs one after the other, of unequal lengths, some empty: 148 blocks on
    the tensor cores, 1184 on the CUDA cores."""
    gen = torch.Generator().manual_seed(55)
    n = (2800 if form == "f32" else 400) // shape[1]
    pool = torch.tensor([0, 1, 2, 63, 64, 65] if form == "bf16" else [0, 1, 2, 5])
    lens = pool[torch.randint(len(pool), (n,), generator=gen)].tolist()
    lens[3::50] = [130] * len(lens[3::50])
    d = R.make(55, *shape, torch.float32 if form == "f32" else torch.bfloat16, lens=lens)
    check_forward(d, *run_forward(d))
    check_backward(d, grads(d))


@pytest.mark.parametrize("per_token", [True, False])
def test_more_cut_units_than_blocks(per_token):
    """Units of cut sequences, more of them than blocks, with local states, joins and start states for each."""
    d = R.make(56, 4, 12, 64, 64, torch.bfloat16, lens=[3900, 40, 1], per_token=per_token)
    check_forward(d, *run_forward(d))
    check_backward(d, grads(d))


def two_terms(x):
    """x as the sum of its two leading bf16 terms."""
    a = x.bfloat16().float()
    return a + (x - a).bfloat16().float()


def worst_for_two_terms(values):
    """The value whose two leading bf16 terms leave the most of it, and what they leave (relative)."""
    left = (two_terms(values) / values - 1).abs()
    i = int(left.argmax())
    return values[i], float(left[i])


def test_third_terms_are_there():
    """States and the dots of the decays' gradient are sums of three bf16 terms.  Inputs that are all alike, so that
    what a lost third term takes off adds up: about 2^-18, 64 half steps of fp32.  With sums of equal values, most of
    them exact, the results must be within 16."""
    bar = 16 * R.U32
    # The state after 64 tokens, z = y = 1: 63 e^g + 1 with one decay at the end; e^g, the weight of all tokens but the
    # last, is what is split (the exponential is within two units, four half steps, of the true one).
    gs = -torch.rand(20000, generator=torch.Generator().manual_seed(57)) * 0.5
    w, left = worst_for_two_terms(gs.exp())
    assert left > 3.5 * bar
    g = torch.zeros(1, 64, 1)
    g[0, -1, 0] = gs[int((gs.exp() == w).nonzero()[0])]
    one = torch.ones(1, 64, 1, 128, dtype=torch.bfloat16)
    d = dict(q=one, k=one, v=one, g=g, s0=torch.zeros(1, 1, 128, 128), cu=None, do=one, dsf=None)
    _, sf = run_forward(d)
    _, rs = R.forward(d["q"], d["k"], d["v"], d["g"], d["s0"])
    assert float((sf.double().cpu() / rs - 1).abs().max()) <= bar
    # dg without decays, from an initial state of one value: the dot of q with S0^T do, S0's copy in three terms
    s, left = worst_for_two_terms(1 + torch.rand(20000, generator=torch.Generator().manual_seed(58)))
    assert left > 3.5 * bar
    d.update(g=torch.zeros(1, 64, 1), v=torch.zeros_like(one), s0=torch.full((1, 1, 128, 128), float(s)))
    got = grads(d)
    ref = R.backward(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["s0"])
    rel = (got["dg"].double().cpu().reshape(ref["dg"].shape) / ref["dg"] - 1).abs()
    assert float(rel.max()) <= bar
