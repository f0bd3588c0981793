"""That grouped products, the layer and adapters run on the stream that they are
given, and on no other: their results are there while the current stream is held
back, and are read on the stream itself."""
import numpy as np
import pytest
import torch

from test_gpu_grouped_paths import BUSY, _calls

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _held(times=4):
    """Holds the current stream back for some time; an event behind that."""
    torch.cuda._sleep(times * BUSY)
    event = torch.cuda.Event()
    event.record()
    return event


def _beside(work):
    """What work returns while the current stream is held back.  Longer, if a busy host
    took longer than that; never, if the work waits for the current stream."""
    for times in (4, 16, 64):
        torch.cuda.synchronize()
        held = _held(times)
        got = work()
        before = not held.query()
        torch.cuda.synchronize()
        if before:
            return got
    pytest.fail("the work was done only after the held stream's")


def _streams(n):
    """n streams that the held one does not hold back too, as it does those that share
    its hardware queue: found with a torch operation."""
    found, probe = [], torch.zeros(64, device=DEV)
    for _ in range(32):
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        held = _held()
        with torch.cuda.stream(stream):
            probe.add_(1)
        stream.synchronize()
        if not held.query():
            found.append(stream)
        torch.cuda.synchronize()
        if len(found) == n:
            return found
    pytest.fail("no streams beside the held one")


def _poison(stream, like):
    """What the stream's next tensors of these sizes are made of holds no result."""
    with torch.cuda.stream(stream):
        junk = [torch.empty_like(like).fill_(-7) for _ in range(6)]
        del junk
    stream.synchronize()


def _on(stream, y):
    with torch.cuda.stream(stream):
        return y.cpu()                   # waits for this stream alone


CALLS = ["group", "layer", "one launch", "few", "prompt"]        # each makes its own output


@pytest.mark.parametrize("name", CALLS)
def test_given_stream(name):
    print(f"[case] given stream {name}", flush=True)
    call = _calls(np.random.default_rng(41))[name]
    want = call().cpu()
    stream, = _streams(1)
    _poison(stream, call(stream=stream))
    assert torch.equal(_beside(lambda: _on(stream, call(stream=stream))), want)


@pytest.mark.parametrize("name", CALLS + ["products"])
def test_two_streams_at_once(name):
    """Calls in turn on two streams made the current one, a third held back: each is
    there when its own stream has run."""
    print(f"[case] two streams {name}", flush=True)
    call = _calls(np.random.default_rng(42))[name]
    want = call().cpu()
    streams = _streams(2)
    for s in streams:
        with torch.cuda.stream(s):
            like = call()
        _poison(s, like)

    def work():
        outs = []
        for i in range(6):
            with torch.cuda.stream(streams[i % 2]):
                outs.append(call())
        return [_on(streams[i % 2], y) for i, y in enumerate(outs)]

    assert all(torch.equal(y, want) for y in _beside(work))


def test_the_held_stream_holds():
    """What the tests above lean on: work queued behind the wait is not there yet."""
    print("[case] held stream", flush=True)
    ys = [torch.full((1000,), -7.0, device=DEV) for _ in range(3)]
    stream, = _streams(1)
    ys[0].add_(0).cpu()

    def work():
        y = ys.pop()
        y.add_(1)
        return y, _on(stream, y)

    y, seen = _beside(work)
    assert (seen == -7).all() and (y == -6).all()
