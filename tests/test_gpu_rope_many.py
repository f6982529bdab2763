"""cp_rope over as many tokens as an int32 counts, in place: 2^31 - 1 of one head of 16."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

from serving_ref import rotate  # noqa: E402
from test_gpu_rope import check, cpa, frequencies  # noqa: E402, F401


def test_rope_of_the_most_tokens(cpa):  # noqa: F811
    n, d, BF = 2 ** 31 - 1, 16, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("not enough memory")
    x = torch.zeros(n, 1, d, dtype=BF, device="cuda")           # 64 GiB
    positions = torch.zeros(n, dtype=torch.int32, device="cuda")
    spots = torch.tensor([0, 1, 4863, 4864, 2 ** 27, 2 ** 30 - 1, 2 ** 30, n - 4865, n - 2, n - 1], device="cuda")
    gen = torch.Generator().manual_seed(1)
    rows = torch.randn(len(spots), 1, d, generator=gen).to(BF)
    at = torch.randint(1, 2 ** 31 - 1, (len(spots),), generator=gen)
    x[spots], positions[spots] = rows.cuda(), at.to(torch.int32).cuda()
    cpa.cp_rope(cpa.RopePlan(d, d), positions, [x], [x])
    ref, size = rotate(rows.double().numpy(), at.numpy()[None], [0] * (d // 2), frequencies(d), False)
    check(x[spots], ref, size, BF)
    x[spots] = 0
    assert not x.view(torch.int64).any()                         # zeros stay zeros
