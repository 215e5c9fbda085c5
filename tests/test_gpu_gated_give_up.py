"""A wait of the gated recurrence or of its gradient that gives up: the call reports it once, what the wait would have given is
NaN, all else is right, and so is the next call."""
import pytest
import torch

import primitives_device_scan_amd as ds
from gpu_util import say

pytestmark = pytest.mark.gpu

TOKENS, DIM, OFFSETS = 12_000, 256, [0, 9000, 9100, 12_000]
TRIES = 40  # that a tile is asked for before it is there is a matter of a microsecond, in each of 90 waits a call


@pytest.fixture
def setting():
    g = torch.Generator().manual_seed(1)
    gate, x, dh = (torch.randn((TOKENS, DIM), generator=g).cuda() for _ in range(3))
    return gate, x, dh, torch.tensor(OFFSETS, dtype=torch.int32, device="cuda")


def calls(gate, x, dh, offsets):
    """The scan and the gradient, and their results where nothing gives up."""
    scan = lambda: ds.gated_scan(gate, x, offsets, mix=True)
    want = scan()
    grad = lambda: ds.gated_scan_grad(gate, want[0], dh, offsets, x=x, mix=True)
    return [(scan, want), (grad, grad())]


def holds(got, want, gave_up):
    bad = [torch.isnan(a) for a in got]
    assert all(bool((n | (a == b)).all()) for a, b, n in zip(got, want, bad)), "a value that is neither right nor NaN"
    assert gave_up == bool(torch.stack([n.any() for n in bad]).any()), "NaN without a report, or a report without NaN"


def test_reported_once(setting):
    pairs = calls(*setting)
    assert ds.query_timeout() is False
    for call, want in pairs:
        seen = 0
        ds.set_spin_limit(1)
        try:
            for _ in range(TRIES):
                got = call()
                gave_up = ds.query_timeout()
                holds(got, want, gave_up)
                seen += gave_up
        finally:
            ds.set_spin_limit(0)
        say("gave up in", seen, "of", TRIES)
        assert seen > 0
        got = call()
        assert ds.query_timeout() is False
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_recorded(setting):
    """A graph with scratch of its own, replayed on a stream that has no workspace."""
    pairs = calls(*setting)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call, want in pairs:
        graph = torch.cuda.CUDAGraph()
        ds.set_spin_limit(1)
        try:
            with torch.cuda.graph(graph, stream=side):
                got = call()
        finally:
            ds.set_spin_limit(0)
        seen = 0
        for _ in range(TRIES):
            with torch.cuda.stream(side):
                graph.replay()
            gave_up = ds.query_timeout(stream=side)
            holds(got, want, gave_up)
            seen += gave_up
            again = call()  # with the usual limit, beside it
            assert ds.query_timeout() is False and all(torch.equal(a, b) for a, b in zip(again, want))
        say("gave up in", seen, "of", TRIES)
        assert seen > 0
