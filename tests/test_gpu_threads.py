"""Calls from two host threads at a time, each on its own stream: every call
is taken and gives what it gives alone.  The binding lets go of the
interpreter's lock during a call, so the two run inside the library together;
whatever a call sets that belongs to a kernel (its shared-memory limit) must
suit every other call of that kernel."""
import ctypes
import threading

import pytest
import torch

import decay_ref as R

pytestmark = pytest.mark.gpu

CALLS = 20_000


def run_together(*calls, bar=0.0):
    """Each call (stream -> (entry point, its arguments, outputs)) CALLS times in a thread of its own: refused by
    none, and the outputs at the end what the call alone gives (to ``bar``, in the 2-norm).  The arguments are made before, so that the threads
    spend their time inside the library."""
    from linear_attention_sequence_sm_b200 import gdn
    jobs = []
    for call in calls:
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        fn, args, outs = call(s.cuda_stream)
        assert fn(*args) == gdn.GDN_OK
        s.synchronize()
        jobs.append((fn, args, outs, [t.clone() for t in outs]))
    start, refused = threading.Barrier(len(jobs)), []

    def work(fn, args, outs, want):
        start.wait()
        for _ in range(CALLS):
            st = fn(*args)
            if st:
                refused.append((st, gdn.LIB.gdn_last_error_message()))
                return

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    for _, _, outs, want in jobs:
        assert all(float((a - b).norm()) <= bar * float(b.norm()) for a, b in zip(outs, want))


def p(t):
    return ctypes.c_void_p(t.data_ptr() if t is not None else None)


def decay_call(shape, backward, dtype=torch.float32):
    from linear_attention_sequence_sm_b200 import gdn
    c = R.cuda(R.make(71, *shape, dtype, batch=(1, 3)))
    sh = gdn.make_shape(c["q"], c["v"], None, 64)
    nbytes = gdn.decay_workspace_size(sh, backward)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def call(stream):
        q, k, v, g, do, s0 = (c[n] for n in ("q", "k", "v", "g", "do", "s0"))
        ins = [ctypes.byref(sh), p(q), p(k), p(v), p(g), 0, p(s0), None]
        tail = [p(ws), nbytes, ctypes.c_void_p(stream)]
        if backward:
            outs = [torch.empty_like(t) for t in (q, k, v, g, s0)]
            return gdn.LIB.gdn_decay_backward, ins + [p(do), None, *map(p, outs), *tail], outs
        outs = [torch.empty_like(v), torch.empty_like(s0)]
        return gdn.LIB.gdn_decay_forward, ins + [None, *map(p, outs), *tail], outs
    return call


@pytest.mark.parametrize("backward", [False, True])
def test_decay_of_two_head_sizes(backward):
    run_together(decay_call((1, 1, 128, 128), backward), decay_call((1, 1, 33, 17), backward))


def norm_call(rows, width, gate, backward):
    from linear_attention_sequence_sm_b200 import gdn
    gen = torch.Generator(device="cuda").manual_seed(72)
    x, r, z, dh, dy = (torch.randn(rows, width, generator=gen, device="cuda") for _ in range(5))
    z = z if gate else None
    n = gdn.BlockNorm().c_struct(x, z)
    nbytes = gdn.block_norm_workspace_size(rows, width)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    f32 = gdn.GDN_DTYPE_F32

    def call(stream):
        outs = [torch.empty_like(x), torch.empty_like(x)]
        ins = [rows, width, f32, f32, p(x), p(r), p(z), ctypes.byref(n)]
        if backward:
            return gdn.LIB.gdn_block_norm_backward, [*ins, p(dh), p(dy), *map(p, outs), None, None, None, None, p(ws),
                                                     nbytes, ctypes.c_void_p(stream)], outs
        return gdn.LIB.gdn_block_norm_forward, [*ins, *map(p, outs), ctypes.c_void_p(stream)], outs
    call.keep = (x, r, z, dh, dy, n)
    return call


@pytest.mark.parametrize("backward", [False, True])
def test_block_norms_of_two_widths(backward):
    run_together(norm_call(3, 2048, True, backward), norm_call(3, 1800, False, backward))


def delta_call(kind, d, chunk=64):
    from linear_attention_sequence_sm_b200 import gdn
    gen = torch.Generator(device="cuda").manual_seed(73)
    r = lambda *s: 0.3 * torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = (r(1, 3, 1, d) for _ in range(4))
    g, beta = -r(1, 3, 1, d if kind == "kda" else 1).abs().reshape(1, 3, 1, -1), r(1, 3, 1).sigmoid()
    sh = gdn.make_shape(q, v, None, 32 if kind == "backward" else chunk, force_simt=True)
    size, fn = dict(chunk=(gdn.LIB.gdn_chunk_forward_workspace_size, gdn.LIB.gdn_chunk_forward),
                    kda=(gdn.LIB.gdn_kda_forward_workspace_size, gdn.LIB.gdn_kda_forward),
                    backward=(gdn.LIB.gdn_chunk_backward_workspace_size, gdn.LIB.gdn_chunk_backward))[kind]
    nbytes = ctypes.c_size_t(0)
    assert size(ctypes.byref(sh), ctypes.byref(nbytes)) == gdn.GDN_OK
    ws = torch.empty(nbytes.value, dtype=torch.uint8, device="cuda")

    def call(stream):
        ins = [ctypes.byref(sh), p(q), p(k), p(v), p(g), p(beta), None, None]
        tail = [p(ws), nbytes, ctypes.c_void_p(stream)]
        if kind == "backward":
            outs = [torch.empty_like(t) for t in (q, k, v, g, beta)]
            return fn, [*ins, p(do), None, *map(p, outs), None, *tail], outs
        outs = [torch.empty_like(v)]
        return fn, [*ins, *([None] if kind == "kda" else []), p(outs[0]), None, *tail], outs
    call.keep = (q, k, v, do, g, beta, sh, ws)
    return call


@pytest.mark.parametrize("kind", ["chunk", "kda", "backward"])
def test_delta_rule_of_two_head_sizes(kind):
    # (the delta rule's gradients add slices of the state by atomics, in any order: fp32 sums of a few hundred terms)
    run_together(delta_call(kind, 128), delta_call(kind, 32, 16 if kind == "chunk" else 64),
                 bar=256 * R.U32 if kind == "backward" else 0.0)
