"""Refusals of the decayed linear attention and the block norms, before any
CUDA work (CPU): the binding's shape checks and the C entry points'."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def gdn():
    from linear_attention_sequence_sm_b200 import build
    build.build()
    from linear_attention_sequence_sm_b200 import gdn as mod
    return mod


B, T, HK, HV, DK, DV = 2, 10, 1, 2, 16, 8


def args(**over):
    x = dict(q=torch.zeros(B, T, HK, DK), k=torch.zeros(B, T, HK, DK), v=torch.zeros(B, T, HV, DV),
             g=torch.zeros(B, T, HV))
    x.update(over)
    return [x[n] for n in ("q", "k", "v", "g")]


def device_error(e):
    return "CUDA tensor" in str(e.value)


def test_good_shapes_reach_the_device_check(gdn):
    for g in (torch.zeros(B, T, HV), torch.zeros(HV)):
        for call in (lambda: gdn.decay_forward(*args(g=g), initial_state=torch.zeros(B, HV, DV, DK)),
                     lambda: gdn.decay_backward(*args(g=g), torch.zeros(B, T, HV, DV))):
            with pytest.raises(ValueError) as e:
                call()
            assert device_error(e)
    cu = torch.tensor([0, 4, 4, T], dtype=torch.int32)
    flat = args(q=torch.zeros(T, HK, DK), k=torch.zeros(T, HK, DK), v=torch.zeros(T, HV, DV), g=torch.zeros(T, HV))
    with pytest.raises(ValueError) as e:
        gdn.decay_forward(*flat, initial_state=torch.zeros(3, HV, DV, DK), cu_seqlens=cu)
    assert device_error(e)
    with pytest.raises(ValueError) as e:
        gdn.decay_decode_step(torch.zeros(3, HK, DK), torch.zeros(3, HK, DK), torch.zeros(3, HV, DV),
                              torch.zeros(HV), torch.zeros(3, HV, DV, DK))
    assert device_error(e)


@pytest.mark.parametrize("over,what", [
    (dict(g=torch.zeros(HV + 1)), "g"), (dict(g=torch.zeros(B, T)), "g"), (dict(g=torch.zeros(B, T, HV, 1)), "g"),
    (dict(k=torch.zeros(B, T, HK, DK + 1)), "k"), (dict(v=torch.zeros(B, T + 1, HV, DV)), "v"),
    (dict(q=torch.zeros(T, HK, DK), k=torch.zeros(T, HK, DK)), "q"),
])
def test_mis_shaped_inputs(gdn, over, what):
    for call in (lambda: gdn.decay_forward(*args(**over)),
                 lambda: gdn.decay_backward(*args(**over), torch.zeros(B, T, HV, DV))):
        with pytest.raises(ValueError) as e:
            call()
        assert what in str(e.value) and not device_error(e)


def test_mis_shaped_states_and_outputs(gdn):
    for kw in (dict(initial_state=torch.zeros(B, HV, DK, DV)), dict(out=torch.zeros(B, T, HV, DV + 1)),
               dict(final_state=torch.zeros(B, HV, DV + 1, DK))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            gdn.decay_forward(*args(), **kw)
    with pytest.raises(ValueError, match="d_o"):
        gdn.decay_backward(*args(), torch.zeros(B, T, HV, DV + 1))
    with pytest.raises(ValueError, match="d_final_state"):
        gdn.decay_backward(*args(), torch.zeros(B, T, HV, DV), d_final_state=torch.zeros(1, HV, DV, DK))
    with pytest.raises(ValueError, match="state"):
        gdn.decay_decode_step(torch.zeros(3, HK, DK), torch.zeros(3, HK, DK), torch.zeros(3, HV, DV),
                              torch.zeros(3, HV), torch.zeros(3, HV, DK, DV))
    with pytest.raises(ValueError, match="g"):
        gdn.decay_decode_step(torch.zeros(3, HK, DK), torch.zeros(3, HK, DK), torch.zeros(3, HV, DV),
                              torch.zeros(4, HV), torch.zeros(3, HV, DV, DK))


def shape(gdn, **kw):
    base = dict(batch=2, seq_len=64, num_seqs=2, num_qk_heads=2, num_v_heads=4, head_dim_k=128, head_dim_v=128,
                chunk_size=64, dtype=gdn.GDN_DTYPE_BF16, flags=0)
    base.update(kw)
    return gdn.Shape(**base)


P = 0x10000  # aligned, never read


def forward(gdn, s, q=P, k=P, v=P, g=P, layout=0, s0=0, cu=0, o=P, sf=0, ws=P, nbytes=1 << 40):
    return gdn.LIB.gdn_decay_forward(ctypes.byref(s), q, k, v, g, layout, s0, cu, None, o, sf, ws, nbytes, None)


def backward(gdn, s, q=P, k=P, v=P, g=P, layout=0, s0=0, cu=0, do=P, dsf=0, dq=P, dk=P, dv=P, dg=P, ds0=0, ws=P,
             nbytes=1 << 40):
    return gdn.LIB.gdn_decay_backward(ctypes.byref(s), q, k, v, g, layout, s0, cu, do, dsf, dq, dk, dv, dg, ds0, ws,
                                      nbytes, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_c_shape_refusals(gdn, call):
    inv, uns = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED
    for kw, want in ((dict(num_v_heads=5), inv), (dict(batch=3), inv), (dict(dtype=7), inv), (dict(head_dim_k=0), inv),
                     (dict(seq_len=-1), inv), (dict(flags=1 << 9), inv), (dict(flags=gdn.GDN_FLAG_QK_L2NORM), uns),
                     (dict(flags=gdn.GDN_FLAG_GATE_LOGITS), uns), (dict(flags=gdn.GDN_FLAG_SPLIT), uns),
                     (dict(chunk_size=32), uns), (dict(head_dim_v=129), uns),
                     (dict(num_qk_heads=1, num_v_heads=70000), uns),
                     (dict(batch=1, num_seqs=1, seq_len=2 ** 31 - 2048, num_v_heads=2, head_dim_k=8, head_dim_v=8), uns)):
        assert call(gdn, shape(gdn, **kw)) == want, kw
    assert call(gdn, shape(gdn), layout=2) == inv
    assert call(gdn, shape(gdn), cu=P) == inv  # batch 2 with cu_seqlens
    assert call(gdn, shape(gdn, batch=1, num_seqs=0), cu=P) == inv  # tokens without sequences


@pytest.mark.parametrize("call,names", [(forward, "q k v g o".split()), (backward, "q k v g do dq dk dv".split())])
def test_c_pointer_refusals(gdn, call, names):
    for n in names:
        assert call(gdn, shape(gdn), **{n: 0}) == gdn.GDN_ERR_INVALID_ARGUMENT, n
        assert call(gdn, shape(gdn), **{n: P + 8}) == gdn.GDN_ERR_MISALIGNED, n
    assert call(gdn, shape(gdn), s0=P + 4) == gdn.GDN_ERR_MISALIGNED
    assert call(gdn, shape(gdn), ws=0) == gdn.GDN_ERR_INVALID_ARGUMENT
    assert call(gdn, shape(gdn), ws=P + 16) == gdn.GDN_ERR_MISALIGNED
    need = gdn.decay_workspace_size(shape(gdn), backward=call is backward)
    assert call(gdn, shape(gdn), nbytes=need - 1) == gdn.GDN_ERR_WORKSPACE_TOO_SMALL


def test_c_decode_refusals(gdn):
    def call(n=1, hk=1, hv=2, dk=16, dv=16, dtype=1, q=P, k=P, v=P, g=P, layout=0, state=P, o=P):
        return gdn.LIB.gdn_decay_decode_step(n, hk, hv, dk, dv, dtype, q, k, v, g, layout, state, None, o, None)
    inv, uns = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(hk=0), dict(hv=3, hk=2), dict(dtype=2), dict(layout=-1), dict(q=0), dict(g=0),
               dict(state=0), dict(o=0)):
        assert call(**kw) == inv, kw
    for kw in (dict(dk=257), dict(dv=(1 << 20) + 1), dict(n=1 << 30, hv=4), dict(n=1 << 20, hv=1 << 10, dk=256)):
        assert call(**kw) == uns, kw
    assert call(state=P + 8) == gdn.GDN_ERR_MISALIGNED
    assert call(n=0, q=0) == gdn.GDN_OK


def test_c_decode_output_side_refused_before_the_state_moves(gdn):
    side = gdn.OutputSideC(0, 0, 1e-6, 0)
    assert gdn.LIB.gdn_decay_decode_step(1, 1, 1, 16, 129, 1, P, P, P, P, 0, P, ctypes.byref(side), P,
                                         None) == gdn.GDN_ERR_UNSUPPORTED


def test_workspace_of_many_short_sequences(gdn):
    """No state is kept for a sequence's first position: 4096 sequences of 16 tokens need little more than one of
    65,536."""
    many = gdn.decay_workspace_size(shape(gdn, batch=4096, num_seqs=4096, seq_len=16, num_v_heads=32), backward=True)
    one = gdn.decay_workspace_size(shape(gdn, batch=1, num_seqs=1, seq_len=65536, num_v_heads=32), backward=True)
    assert many < 1.1 * one


def test_workspace_grows_with_the_problem(gdn):
    small = gdn.decay_workspace_size(shape(gdn))
    assert small % 256 == 0
    assert gdn.decay_workspace_size(shape(gdn, batch=1, num_seqs=1, seq_len=65536)) > small
    assert gdn.decay_workspace_size(shape(gdn), backward=True) > small


def norm_struct(gdn, flags, eps=1e-6, rho=1.0, branch=1.0, w1=0, s=0, w2=0):
    return gdn.BlockNormC(w1, s, w2, eps, rho, branch, flags)


def test_block_norm_refusals(gdn):
    inv, uns = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED
    post, pre, silu, sig = (gdn.GDN_BLOCK_POST_NORM, gdn.GDN_BLOCK_PRE_NORM, gdn.GDN_BLOCK_GATE_SILU,
                            gdn.GDN_BLOCK_GATE_SIGMOID)

    def fwd(c, rows=4, width=64, dt=1, rt=1, x=P, r=P, z=0, h=P, y=P):
        return gdn.LIB.gdn_block_norm_forward(rows, width, dt, rt, x, r, z, ctypes.byref(c), h, y, None)

    def bwd(c, rows=4, width=64, dt=1, rt=1, x=P, r=P, z=0, dh=P, dy=P, dx=P, dr=P, dz=0, w=0, s=0, p=0, ws=P,
            nbytes=1 << 40):
        return gdn.LIB.gdn_block_norm_backward(rows, width, dt, rt, x, r, z, ctypes.byref(c), dh, dy, dx, dr, dz, w, s,
                                               p, ws, nbytes, None)
    ok = norm_struct(gdn, post | pre)
    for call in (fwd, bwd):
        for kw, want in ((dict(rows=-1), inv), (dict(width=0), inv), (dict(dt=3), inv), (dict(dt=0, rt=1), uns),
                         (dict(width=16385), uns), (dict(x=0), inv), (dict(x=P + 2), gdn.GDN_ERR_MISALIGNED),
                         (dict(z=P), inv), (dict(rows=1 << 31), uns)):
            assert call(ok, **kw) == want, kw
        for c in (norm_struct(gdn, post | pre, eps=0.0), norm_struct(gdn, post | pre, eps=float("nan")),
                  norm_struct(gdn, post | pre, rho=float("inf")), norm_struct(gdn, post | pre, branch=float("nan")),
                  norm_struct(gdn, post | pre | 64), norm_struct(gdn, post | pre | silu),
                  norm_struct(gdn, pre, w1=P)):
            assert call(c) == inv
        assert call(norm_struct(gdn, post | pre | silu | sig), z=P) == inv
        assert call(norm_struct(gdn, post | pre, w1=P + 4)) == gdn.GDN_ERR_MISALIGNED
    assert fwd(norm_struct(gdn, post)) == inv  # y without PRE_NORM
    assert fwd(ok, y=0) == inv
    assert fwd(norm_struct(gdn, post), h=0, y=0) == inv
    assert bwd(norm_struct(gdn, post)) == inv  # d_y without PRE_NORM
    assert bwd(ok, dh=0, dy=0) == inv
    assert bwd(ok, r=0) == inv and bwd(ok, dz=P) == inv
    assert bwd(norm_struct(gdn, pre), w=P) == inv
    assert bwd(ok, ws=0) == inv and bwd(ok, nbytes=16) == gdn.GDN_ERR_WORKSPACE_TOO_SMALL
    assert fwd(ok, rows=0, x=0, h=0, y=0) == gdn.GDN_OK


def test_block_norm_outputs_are_two_buffers(gdn):
    n = norm_struct(gdn, gdn.GDN_BLOCK_PRE_NORM)
    assert gdn.LIB.gdn_block_norm_forward(2, 64, 1, 1, P, P, 0, ctypes.byref(n), P, P, None) == gdn.GDN_ERR_INVALID_ARGUMENT


def test_block_norm_binding_refusals(gdn):
    x, r = torch.zeros(4, 32), torch.zeros(4, 32)
    n = gdn.BlockNorm()
    with pytest.raises(ValueError) as e:
        gdn.block_norm_forward(x, r, n)
    assert device_error(e)
    with pytest.raises(ValueError, match="residual"):
        gdn.block_norm_forward(x, r[:3], n)
    with pytest.raises(ValueError, match="gate"):
        gdn.block_norm_forward(x, r, n, gate=torch.zeros(4, 31))
    with pytest.raises(ValueError, match="scale"):
        gdn.block_norm_forward(x, r, gdn.BlockNorm(scale=torch.zeros(31)))
    with pytest.raises(TypeError, match="residual"):
        gdn.block_norm_forward(x, r.half(), n)
    with pytest.raises(ValueError, match="y needs pre_norm"):
        gdn.block_norm_forward(x, r, gdn.BlockNorm(pre_norm=False), y=x)
    with pytest.raises(ValueError, match="d_h or d_y"):
        gdn.block_norm_backward(x, r, n)
    with pytest.raises(ValueError, match="d_y needs pre_norm"):
        gdn.block_norm_backward(x, r, gdn.BlockNorm(pre_norm=False), d_y=x)
    for kw in (dict(activation="relu"), dict(post_norm=False, post_weight=x), dict(pre_norm=False, pre_weight=x)):
        with pytest.raises(ValueError):
            gdn.BlockNorm(**kw)


def refused_workspaces(gdn, nbytes):
    return [(torch.zeros(2 * nbytes, dtype=torch.uint8), "CUDA tensor"),
            (torch.zeros(1, dtype=torch.uint8).expand(2 * nbytes), "CUDA tensor|contiguous"),
            (torch.zeros(2 * nbytes, dtype=torch.uint8, device="meta"), "CUDA tensor")]


@pytest.mark.parametrize("name", ["decay_forward", "decay_backward", "block_norm_backward"])
def test_workspace_of_another_place(gdn, monkeypatch, name):
    """A workspace is checked like every tensor: the library would write its header through the bare pointer.  (The
    checks of the other tensors are left out, so that CPU tensors get as far as the workspace.)"""
    need = gdn._need
    monkeypatch.setattr(gdn, "_ready", lambda *a: True)
    monkeypatch.setattr(gdn, "_need", lambda t, n, *a: need(t, n, *a) if n == "workspace" else None)
    x = torch.zeros(4, 32)
    call = dict(decay_forward=lambda ws: gdn.decay_forward(*args(), workspace=ws),
                decay_backward=lambda ws: gdn.decay_backward(*args(), torch.zeros(B, T, HV, DV), workspace=ws),
                block_norm_backward=lambda ws: gdn.block_norm_backward(x, x, gdn.BlockNorm(), d_h=x, workspace=ws))[name]
    for ws, what in refused_workspaces(gdn, 1 << 22):
        with pytest.raises(ValueError, match=what):
            call(ws)


def test_small_workspace_is_refused_not_replaced(gdn, monkeypatch):
    """A workspace that the call does not use would hold no status of it."""
    monkeypatch.setattr(gdn, "_need", lambda *a: None)
    with pytest.raises(ValueError, match="workspace has 255 bytes, the call needs 256"):
        gdn._room(torch.zeros(255, dtype=torch.uint8), 256, torch.device("cpu"), None)
    ws = torch.zeros(256, dtype=torch.uint8)
    assert gdn._room(ws, 256, torch.device("cpu"), None) is ws
