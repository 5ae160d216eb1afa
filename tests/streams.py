"""Whose memory a call's outputs are, checked on a GPU."""
import torch


def check_outputs_belong_to_the_calls_stream(calls):
    """``calls``: stream (None: the current one) -> new output tensors of one
    call queued there.  New outputs come from the memory of the call's stream.
    Dropped while that stream still has work on them, they are not given to the
    current stream's work; nor do they take what the current stream's work still
    uses; and where the current stream reads them behind the call, they are not
    given back to the call's stream too soon."""
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    busy = lambda: torch.cuda._sleep(20_000_000)  # noqa: E731 (about ten milliseconds)

    def fill(like):
        return [torch.empty_like(t).fill_(7) for t in like for _ in range(2)]

    for call in calls:
        want = [t.clone() for t in call(None)]
        # (both streams get all the memory they will need first: asking the driver for more would wait for them)
        with torch.cuda.stream(side):
            spare = [fill(want), fill(want)]
        spare.append([fill(want), fill(want)])
        torch.cuda.synchronize()
        del spare
        # the call's stream is behind: the dropped outputs' memory is still its own
        with torch.cuda.stream(side):
            busy()
        outs = call(side)
        with torch.cuda.stream(side):
            kept = [t.clone() for t in outs]
        del outs
        junk = fill(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        assert all(bool((t == 7).all()) for t in junk)
        del junk, kept
        # the current stream is behind: memory that its work was given is not an output's
        old = [torch.empty_like(t) for t in want]
        busy()
        for t in old:
            t.fill_(7)
        del old, t
        outs = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        # read by the current stream, then dropped: not yet the call's stream's memory again
        outs = call(side)
        here.wait_stream(side)
        busy()
        kept = [t.clone() for t in outs]
        del outs
        with torch.cuda.stream(side):
            junk = fill(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        del junk, kept
