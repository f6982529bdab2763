"""A ring whose store goes away: the process that keeps it may have ended well
while others are still at their last step."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from context_long_sequence_gb300 import transport as tr  # noqa: E402


class Store:
    """Answers `lasts` checks, then is gone."""

    def __init__(self, lasts, flag=b""):
        self.lasts, self.flag, self.checks = lasts, flag, 0

    def check(self, keys):
        self.checks += 1
        if self.checks > self.lasts:
            raise RuntimeError("Connection reset by peer")
        return bool(self.flag)

    def get(self, key):
        return self.flag


def comm_of(store):
    comm = object.__new__(tr.DistComm)
    comm.rank, comm.world, comm.store = 3, 4, store
    return comm


def test_lost_store_before_a_ring_is_an_error():
    with pytest.raises(tr.TransportError) as e:
        comm_of(Store(0)).check_abort(4)
    assert e.value.kind == "error" and e.value.step == 4 and "Connection reset" in e.value.detail


def test_lost_store_within_a_ring_is_left_to_the_waits():
    comm_of(Store(0)).check_abort(2, True)


@pytest.mark.parametrize("begun", [False, True])
def test_abort_is_raised_where_the_store_has_it(begun):
    with pytest.raises(tr.TransportError) as e:
        comm_of(Store(9, b"timeout on process 2")).check_abort(1, begun)
    assert e.value.kind == "peer_abort" and e.value.detail == "timeout on process 2"


class Kernels:
    """Counts the steps of a ring of one process."""

    def __init__(self):
        self.steps = []

    empty_like = staticmethod(torch.empty_like)

    def partial_buffers(self, q, R):
        return [None] * R, [None] * R

    def fwd_step(self, a, s, q, k, v, o, lse):
        self.steps.append((a, s))

    def merge(self, o_p, l_p, o, lse):
        self.steps.append("merged")


class Comm(tr.LocalComm):
    def __init__(self, store):
        super().__init__()
        self.of = comm_of(store)

    def check_abort(self, step, begun=False):
        self.of.check_abort(step, begun)


@pytest.mark.parametrize("lasts", [1, 2])
def test_ring_ends_without_its_store(lasts):
    R, k = 3, Kernels()
    kv = [(torch.zeros(1, 2), torch.zeros(1, 2)) for _ in range(R)]
    rings = [torch.zeros(1, 2) for _ in range(R)]
    place = tr.RingPlacement(R=R, U=1, world=1, rank=0)
    tr.ring_forward(Comm(Store(lasts)), k, place, rings, kv, rings, rings)
    assert len(k.steps) == R * R + R
    with pytest.raises(tr.TransportError):
        tr.ring_forward(Comm(Store(0)), k, place, rings, kv, rings, rings)
