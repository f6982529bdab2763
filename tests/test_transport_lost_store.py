"""What a ring makes of a store that does not answer: a lost connection ends
no ring that has begun, every other failure does."""
import multiprocessing as mp
import os
import socket
import sys
import time

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from context_long_sequence_gb300 import transport as tr  # noqa: E402


class Store:
    """Answers `lasts` checks, then raises `error`."""

    def __init__(self, lasts, error=None, get_error=None):
        self.lasts, self.error, self.get_error = lasts, error, get_error

    def check(self, keys):
        self.lasts -= 1
        if self.lasts < 0 and self.error is not None:
            raise self.error
        return self.get_error is not None

    def get(self, key):
        raise self.get_error


def comm_of(store):
    comm = object.__new__(tr.DistComm)
    comm.rank, comm.world, comm.store = 3, 4, store
    return comm


class Comm(tr.LocalComm):
    def __init__(self, store):
        super().__init__()
        self.of, self.steps = comm_of(store), []

    def check_abort(self, step, begun=False):
        self.steps.append(step)
        self.of.check_abort(step, begun)


class Kernels:
    empty_like = grad_buffer = staticmethod(torch.empty_like)

    def partial_buffers(self, q, R):
        return [None] * R, [None] * R

    def delta(self, o, do, lse):
        return None

    def fwd_step(self, a, s, q, k, v, o, lse):
        pass

    def bwd_step(self, a, s, q, do, stats, k, v, dq, dk, dv):
        for g in (dk, dv):
            g.copy_(g + 1 if s else torch.ones_like(g))

    def merge(self, o_p, l_p, o, lse):
        o.fill_(1)


def ring(way, comm, R=3):
    kv, x = ([(torch.zeros(1, 2), torch.zeros(1, 2)) for _ in range(R)] for _ in range(2))
    x = [torch.zeros(1, 2) for _ in range(R)]
    place = tr.RingPlacement(R=R, U=1, world=1, rank=0)
    if way == "forward":
        tr.ring_forward(comm, Kernels(), place, x, kv, x, x)
        assert all((o == 1).all() for o in x)
    else:
        got = tr.ring_backward(comm, Kernels(), place, x, kv, x, x, x, x)
        assert all((g == R).all() for pair in got for g in pair)
    assert comm.steps == list(range(R))


LOST = [RuntimeError("Connection reset by peer"), torch.distributed.DistNetworkError("failed to recv, got 0 bytes"),
        RuntimeError("sendBytes failed: Broken pipe"), ConnectionResetError("gone")]
OTHER = [RuntimeError("wait timeout after 1000 ms"), ValueError("a key of no store"), MemoryError()]


@pytest.mark.parametrize("way", ["forward", "backward"])
@pytest.mark.parametrize("error", LOST, ids=lambda e: type(e).__name__)
def test_lost_connection_ends_no_ring_that_has_begun(way, error):
    for lasts in (1, 2):
        comm = Comm(Store(lasts, error))
        ring(way, comm)
        assert f"at step {lasts}" in comm.of.lost
    with pytest.raises(tr.TransportError) as e:
        ring(way, Comm(Store(0, error)))
    assert e.value.kind == "error" and e.value.step == 0


@pytest.mark.parametrize("way", ["forward", "backward"])
@pytest.mark.parametrize("error", OTHER, ids=lambda e: type(e).__name__)
@pytest.mark.parametrize("lasts", [0, 1, 2])
def test_other_failures_of_the_store_end_the_ring(way, error, lasts):
    """They may hide another process's abort."""
    with pytest.raises(tr.TransportError) as e:
        ring(way, Comm(Store(lasts, error)))
    assert e.value.kind == "error" and e.value.step == lasts and "store" in e.value.detail
    with pytest.raises(tr.TransportError):
        comm_of(Store(0, error)).check_abort(2, True)


def test_a_wait_that_fails_later_names_the_lost_store():
    class Handle:
        def wait(self, timeout):
            raise RuntimeError("timed out")
    import datetime
    comm = comm_of(Store(0, LOST[0]))
    comm.timeout = datetime.timedelta(seconds=1)
    with pytest.raises(tr.TransportError) as e:
        comm.wait(Handle(), 1, 2)
    assert "store" not in e.value.detail
    comm.check_abort(1, True)
    with pytest.raises(tr.TransportError) as e:
        comm.wait(Handle(), 2, 2)
    assert e.value.kind == "timeout" and "store" in e.value.detail and "at step 1" in e.value.detail


def _member(rank, world, port, gone, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    import datetime

    import torch.distributed as dist
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=30))
    comm = tr.DistComm(timeout_s=30.0)

    class Late(Kernels):
        """Rank 2 is at its step 1 until rank 0, which keeps the store, has ended."""

        def fwd_step(self, a, s, *rest):
            if rank == 2 and s == 1:
                gone.wait(60)
    x, kv = [torch.zeros(1, 2)], [(torch.full((1, 2), float(rank)), torch.zeros(1, 2))]
    try:
        tr.ring_forward(comm, Late(), tr.RingPlacement(R=world, U=1, world=world, rank=rank), x, kv, x, x)
        out.put((rank, "ok", comm.lost))
    except Exception as e:
        out.put((rank, repr(e)[:300], comm.lost))
    out.close()
    out.join_thread()
    os._exit(0)


def test_the_keeper_of_the_store_may_end_steps_before_another():
    """Four processes: rank 0 has all its chunks while rank 2 is at step 1 of 0 .. 3,
    so that two checks of rank 2 find the store gone, the first of them not its last."""
    ctx = mp.get_context("spawn")
    out, gone = ctx.Queue(), ctx.Event()
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    procs = [ctx.Process(target=_member, args=(r, 4, port, gone, out)) for r in range(4)]
    for p in procs:
        p.start()
    procs[0].join(timeout=60)
    ended = not procs[0].is_alive()
    time.sleep(0.2)
    gone.set()
    got = dict((r, rest) for r, *rest in (out.get(timeout=60) for _ in procs))
    for p in procs:
        p.join(timeout=30)
        if p.is_alive():
            p.kill()
    assert ended and all(status == "ok" for status, _ in got.values()), got
    assert "at step 2" in got[2][1], got


@pytest.mark.parametrize("error", LOST + OTHER, ids=lambda e: type(e).__name__)
def test_abort_counts_without_its_reason(error):
    """The store may go between the check and the reading of the reason."""
    with pytest.raises(tr.TransportError) as e:
        comm_of(Store(9, get_error=error)).check_abort(1)
    assert e.value.kind == "peer_abort" and e.value.step == 1


@pytest.mark.parametrize("way", ["forward", "backward"])
@pytest.mark.parametrize("lasts", [1, 2, 9])
def test_a_communicator_that_takes_the_step_alone(way, lasts):
    """check_abort(step), as a user's own communicator has it."""
    class Own(Comm):
        def check_abort(self, step):
            super().check_abort(step)
    ring(way, Own(Store(lasts, LOST[0])))
    with pytest.raises(tr.TransportError):
        ring(way, Own(Store(0, LOST[0])))
