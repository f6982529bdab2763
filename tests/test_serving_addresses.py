"""cp_verify_drafts refuses arrays of one address, as its documentation says (no
GPU: the checks come before any use of the addresses)."""
import ctypes
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

from test_paged_host import FAKE, c_args, cpa, make_plan  # noqa: E402, F401

A = ctypes.addressof
ROWS = ("tokens", "accept_u", "p", "q")          # inputs of [n_tokens] rows
OUT = ("accepted", "out_tokens", "kv_len_out")


def call(cpa, n_tokens=10, **same):  # noqa: F811
    """Every array has an address of its own but for those in `same`."""
    plan = make_plan(cpa)
    names = ("q_start", "kv_len", "sample_u", *ROWS, *OUT)
    at = {name: FAKE + 4096 * (i + 1) for i, name in enumerate(names)}
    at.update({name: at[other] for name, other in same.items()})
    _, b = c_args(cpa, plan, None, dict(n_tokens=n_tokens, q_start=at["q_start"], kv_len=at["kv_len"]))
    v = cpa.cp_verify_t(1000, 2, at["p"], 1000, at["q"], 1000, *(at[k] for k in ("tokens", "accept_u", "sample_u", *OUT)))
    return cpa._L().cp_verify_drafts(plan.handle, A(b), A(v), None)


PAIRS = [(out, other) for out in OUT for other in ("q_start", "kv_len", "sample_u", *ROWS, *OUT) if out != other]
MAY = ("kv_len_out", "kv_len")


@pytest.mark.parametrize("out,other", [x for x in PAIRS if x != MAY])
def test_verify_outputs_are_no_other_array(cpa, out, other):  # noqa: F811
    assert call(cpa, **{out: other}) == cpa.CP_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are none: a call that is not refused would use them")
def test_verify_lengths_may_be_in_place(cpa):  # noqa: F811
    """And without rows the rows' arrays, which are not touched, may be anything."""
    assert call(cpa, kv_len_out="kv_len") != cpa.CP_ERR_INVALID_ARG
    assert call(cpa, n_tokens=0, out_tokens="accepted") != cpa.CP_ERR_INVALID_ARG
    assert call(cpa, n_tokens=0, accepted="kv_len_out") == cpa.CP_ERR_INVALID_ARG
