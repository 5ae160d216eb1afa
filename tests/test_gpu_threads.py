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


def run_together(*calls):
    """Each call (stream -> (entry point, its arguments, outputs)) CALLS times in a thread of its own: refused by
    none, and the outputs at the end what the call alone gives.  The arguments are made before, so that the threads
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
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


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
