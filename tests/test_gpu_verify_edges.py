"""cp_verify_drafts at the edges of its documentation: batches without rows
whose arrays are null, and borders between the stretches of a row that its
warps share."""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

from test_gpu_paged_use import ints  # noqa: E402
from test_gpu_verify import cpa  # noqa: E402, F401


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("B", [1, 7, 300])
@pytest.mark.parametrize("lengths", [True, False])
def test_verify_without_rows(cpa, B, dtype, lengths):  # noqa: F811
    """Sequences, but no rows: every array but the sequences' own may be null,
    the random numbers too; each sequence has accepted 0 and its length."""
    plan = cpa.PagedPlan(8, 2, 128, page_size=16, dtype=torch.bfloat16, max_seqs=B, max_tokens=1, max_new=1, max_pages=4)
    start, kv = ints(np.zeros(B + 1)), ints(100 + np.arange(B))
    batch = cpa.cp_paged_batch_t(B, 0, start.data_ptr(), kv.data_ptr())
    accepted, out = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    v = cpa.cp_verify_t(128000, dtype, None, 128000, None, 0, None, None, None, accepted.data_ptr(), None, out.data_ptr() if lengths else None)
    stream = torch.cuda.current_stream().cuda_stream
    assert cpa._L().cp_verify_drafts(plan.handle, ctypes.addressof(batch), ctypes.addressof(v), stream) == 0
    assert (accepted == 0).all() and (torch.equal(out, kv) if lengths else (out == -7).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 4, 8, 16, 64])
@pytest.mark.parametrize("seed", [3, 4, 5])
def test_verify_borders_between_stretches(cpa, B, dtype, seed):  # noqa: F811
    """A row of 128 equal blocks of random weights, random numbers on the borders
    between them, r = j / 128.  V = 128000: a cluster of 16 or 8 CTAs has 128 or 64
    warps, each a stretch of one or two whole blocks, aligned alike.  Equal stretches
    have equal sums, so that the sum before stretch j is j times one
    number, exactly, and the token the first of stretch j; within a
    stretch (64 warps, odd j) the block's first or the one before it, as the two halves'
    sums round apart."""
    blocks, n = 128, 1000
    gen = torch.Generator().manual_seed(seed)
    block = torch.softmax(5 * torch.randn(n, generator=gen), 0) / blocks
    row = block.to(dtype).cuda().repeat(blocks)
    assert (row > 0).all()
    p = row.repeat(B, 1)
    plan = cpa.PagedPlan(8, 2, 128, page_size=16, dtype=torch.bfloat16, max_seqs=B, max_tokens=B, max_new=1, max_pages=4)
    batch = cpa.PagedBatch(ints(np.arange(B + 1)), ints(np.full(B, 10)), ints(np.zeros((B, 4))), n_tokens=B)
    tokens, u = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")
    per = 1 if B <= 8 else 2  # blocks of a warp
    for j0 in range(0, blocks, B):
        j = np.arange(j0, j0 + B)
        r = torch.from_numpy((j / blocks).astype(np.float32)).cuda()
        accepted, out = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        cpa.cp_verify_drafts(plan, batch, tokens, p, None, u, r, accepted, out)
        got = out.cpu().numpy()
        exact = j % per == 0
        assert np.array_equal(got[exact], n * j[exact]), (j[exact][got[exact] != n * j[exact]], got)
        assert ((got == n * j) | (got == n * j - 1)).all(), got
