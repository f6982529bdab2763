"""cp_verify_drafts at the edges of its documentation: batches without rows
whose arrays are null."""
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
