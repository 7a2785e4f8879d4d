"""The most requests of one kda_tree_verify: refused beyond, served at the
limit."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _build, _lib

import tree_testutil as tt

MOST = 1 << 24


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


A = 0x10000  # a 16-byte aligned stand-in address: never dereferenced below


@pytest.mark.parametrize("B,Q,code", [(MOST + 1, 5, _lib.KDA_ERR_ARG), (MOST + 1, 64, _lib.KDA_ERR_ARG),
                                      (2 ** 31 - 1, 9, _lib.KDA_ERR_ARG),
                                      # (far enough to be refused for another reason)
                                      (MOST + 1, 4, _lib.KDA_ERR_ALIGN), (MOST, 5, _lib.KDA_ERR_ALIGN)])
def test_requests_beyond_the_limit(lib, B, Q, code):
    assert lib.kda_tree_verify(A + 2, A, A, A, A, A, A, -5.0, 0.1, A, 0, 128 * 128, 4, A, A, A, 10, A,
                               A, A, A, 8 * 128, 8 * 256, B, 8, A, A, B, 1, Q, 0, None,
                               None) == code


@pytest.mark.gpu
def test_as_many_requests_as_there_may_be(lib):
    """16.8 million requests, the last alone live.  It gives what it gives alone."""
    import torch
    case = tt.tree_case([tt.comb(9)], 1, seed=1, pending=3)
    d, e = tt.on_device(case), tt.on_device(case)
    tt.call_verify(case, d)
    full = lambda n, v: torch.full((n,), v, dtype=torch.int32, device="cuda")
    last = lambda t, v: (t[-1:].copy_(torch.as_tensor(v)), t)[1]
    slot, row = int(case["state_slots"][0]), int(case["record_rows"][0])
    e["state_slots"] = last(full(MOST, 0), slot)
    e["record_rows"] = last(full(MOST, -1), row)
    e["query_start_loc"] = last(full(MOST + 1, 0), 9)
    tt.call_verify(case, e)
    for n in ("out", "node_corr", "state", "status"):
        assert torch.equal(d[n], e[n]), n
    assert int(d["status"].item()) == 0
