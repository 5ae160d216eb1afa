"""The delta rule's, KDA's and the convolution's calls on another stream than
the current one: whose memory their outputs and workspaces are."""
import ctypes

import pytest
import torch

import streams

pytestmark = pytest.mark.gpu


def inputs():
    gen = torch.Generator(device="cuda").manual_seed(81)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    return dict(q=unit(r(2, 300, 4, 128)), k=unit(r(2, 300, 4, 128)), v=r(2, 300, 4, 128).bfloat16(),
                g=-torch.nn.functional.softplus(r(2, 300, 4)), beta=r(2, 300, 4).sigmoid(),
                gk=-torch.nn.functional.softplus(r(2, 300, 4, 128)), s0=0.1 * r(2, 4, 128, 128),
                do=r(2, 300, 4, 128).bfloat16(), w=0.5 * r(4, 128, 4))


def backward(c, s):
    """The gradients whose sums have one order (those of the gates are added by atomics)."""
    from linear_attention_sequence_sm_b200 import gdn
    out = gdn.chunk_backward(c["q"], c["k"], c["v"], c["g"], c["beta"], c["do"], initial_state=c["s0"], stream=s)
    return [out[n] for n in ("dq", "dk", "dv", "d_initial_state")]


def backward_bytes(c):
    from linear_attention_sequence_sm_b200 import gdn
    n = ctypes.c_size_t(0)
    sh = gdn.make_shape(c["q"], c["v"], None, 32)
    assert gdn.LIB.gdn_chunk_backward_workspace_size(ctypes.byref(sh), ctypes.byref(n)) == gdn.GDN_OK
    return n.value


def test_outputs_belong_to_the_calls_stream():
    from linear_attention_sequence_sm_b200 import gdn
    c = inputs()
    qkv, state = [c[n] for n in "qkv"], c["s0"].clone()
    one = {n: t[:, 0].contiguous() for n, t in c.items() if n not in ("s0", "w")}
    few = {n: t[:, :3].contiguous() for n, t in c.items() if n not in ("s0", "w")}

    def step(s, fn, g):
        with torch.cuda.stream(s):
            state.copy_(c["s0"])
        return [fn(one["q"], one["k"], one["v"], one[g], one["beta"], state, stream=s)]

    streams.check_outputs_belong_to_the_calls_stream([
        lambda s: gdn.chunk_forward(*qkv, c["g"], c["beta"], initial_state=c["s0"], stream=s),
        lambda s: gdn.chunk_forward(*qkv, c["g"], c["beta"], initial_state=c["s0"], stream=s, split=True),
        lambda s: gdn.chunk_forward_noalloc(*qkv, c["g"], c["beta"], initial_state=c["s0"], stream=s),
        lambda s: step(s, gdn.decode_step, "g"),
        lambda s: gdn.kda_forward(*qkv, c["gk"], c["beta"], initial_state=c["s0"], stream=s),
        lambda s: step(s, gdn.kda_decode_step, "gk"),
        lambda s: gdn.decode_multi(few["q"], few["k"], few["v"], few["g"], few["beta"], c["s0"], stream=s),
        lambda s: backward(c, s),
        lambda s: gdn.short_conv(c["v"], c["w"], stream=s),
    ])


def test_workspaces_belong_to_the_calls_stream():
    """A call queued on a side stream behind other work: memory that later work on the current stream takes and
    fills is not the call's workspace."""
    from linear_attention_sequence_sm_b200 import gdn
    c = inputs()
    qkv, more = [c[n] for n in "qkv"], dict(initial_state=c["s0"])
    sh = gdn.make_shape(c["q"], c["v"], None, 64, split=True)
    calls = [(gdn.workspace_size(sh), lambda s: gdn.chunk_forward(*qkv, c["g"], c["beta"], split=True, stream=s, **more)),
             (gdn.kda_workspace_size(gdn.make_shape(c["q"], c["v"], None, 64)),
              lambda s: gdn.kda_forward(*qkv, c["gk"], c["beta"], stream=s, **more)),
             (backward_bytes(c), lambda s: backward(c, s))]
    side = torch.cuda.Stream()
    for nbytes, call in calls:
        want = [t.clone() for t in call(None)]
        kept = [call(side), [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]]
        torch.cuda.synchronize()
        del kept  # (both streams have memory to give without asking the driver, which would wait for them)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(side)
        taken = [torch.empty(nbytes, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((t == 255).all()) for t in taken)
