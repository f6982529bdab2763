"""Host-side refusals of the paged-cache ABI at the ends of its ranges (no GPU:
the checks come before any use of the addresses)."""
import ctypes
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

from test_paged_host import FAKE, c_args, cpa, make_plan  # noqa: E402, F401


@pytest.mark.parametrize("cache", [
    # Strides and counts whose span passes 2^63: (2^31 - 1) pages, 2^35 elements
    # apart, under tokens that lie 2^35 + 8 apart, overlap.
    dict(num_pages=2 ** 31 - 1, page_stride=1 << 35, token_stride=(1 << 35) + 8),
    dict(num_pages=2 ** 31 - 1, page_stride=(1 << 36) - 8, token_stride=(1 << 36) - 8),
    dict(num_pages=2 ** 31 - 1, page_stride=(1 << 36) - 8),
])
def test_cache_spans_that_overflow(cpa, cache):  # noqa: F811
    plan = make_plan(cpa, rope_dim=128)
    c, b = c_args(cpa, plan, cache)
    L, A = cpa._L(), ctypes.addressof
    assert L.cp_attn_paged(plan.handle, A(c), A(b), FAKE, 1024, FAKE, FAKE, FAKE, plan.workspace_size(), None) == -1
    assert L.cp_cache_append(plan.handle, A(c), A(b), FAKE, 1024, FAKE, 256, FAKE, 256, FAKE, 1024, None) == -1


@pytest.mark.parametrize("scale,ok", [(3e38, False), (2.4e38, False), (2.3e38, True), (1e-38, True)])
def test_softmax_scale_stays_a_number_in_base_2(cpa, scale, ok):  # noqa: F811
    """The kernels multiply by scale * log2(e) in fp32: one that is infinite
    makes 0 * inf of a score of 0."""
    if ok:
        make_plan(cpa, softmax_scale=scale)
        return
    with pytest.raises(cpa.CPError) as e:
        make_plan(cpa, softmax_scale=scale)
    assert e.value.code == -1


def test_plan_without_cuda_in_torch(cpa, monkeypatch):  # noqa: F811
    """A plan holds no device memory and is made wherever the library loads; a
    call on host tensors is refused there too."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    plan = make_plan(cpa)
    assert plan.workspace_size() > 0
    k = torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    b = cpa.PagedBatch(torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 100, **i32), n_tokens=1)
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(cpa.CPError, match="not the current device"):
        cpa.cp_attn_paged(plan, cpa.PagedCache(k, k.clone()), b, q, q.clone(), torch.zeros(8, 1))
