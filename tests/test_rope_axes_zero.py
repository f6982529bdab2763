"""rope_axes = 0 of a paged plan means one axis, in the C ABI and the binding alike."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

from paged_ref import Batch  # noqa: E402
from test_paged_host import cpa, make_plan  # noqa: E402, F401


@pytest.mark.parametrize("kw", [dict(), dict(rope_dim=64)])
def test_no_axes_are_one_axis(cpa, kw):  # noqa: F811
    assert make_plan(cpa, rope_axes=0, **kw).rope_axes == make_plan(cpa, **kw).rope_axes == 1


@pytest.mark.gpu
def test_append_under_a_plan_of_no_axes(cpa):  # noqa: F811
    """Positions of one axis are served, bit for bit as under a plan that says nothing of axes."""
    b = Batch(past=[3, 0, 21], new=[2, 1, 5], d=64, Hq=4, Hkv=2, seed=4, appended=False)
    positions, got = np.random.default_rng(4).integers(0, 2 ** 20, b.N), []
    for kw in (dict(rope_axes=0), dict()):
        cache, batch, q, k, v = b.to_gpu(cpa, positions)
        q_out = torch.empty(b.N, 4, 64, dtype=b.dtype, device="cuda")
        cpa.cp_cache_append(b.plan(cpa, rope_dim=64, **kw), cache, batch, q, k, v, q_out)
        got += [q_out, cache.k.view(torch.int16)]
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
