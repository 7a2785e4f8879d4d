"""Calls most of whose requests have no tokens, as a server's are whose slots
are mostly idle: right wherever the idle ones stand, and not slower for them."""
import numpy as np
import pytest

from prompt_testutil import call_rule, on_device, ragged_case
from test_gpu_prompt_maps import check_conv, conv_case, run_conv
from test_gpu_prompt_rule import ops, verify

pytestmark = pytest.mark.gpu

LENS = [0] * 50 + [30] + [0] * 100 + [5, 0, 70] + [0] * 300
BOUNDS = {50: 7, 153: 64}


def test_conv():
    case = conv_case(LENS, 2, seed=1, resume=(50, 153), boundary=BOUNDS, tail=3)
    check_conv(case, run_conv(case))


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_rule(op):
    case = ragged_case(lens=LENS, H=1, seed=2, resume=(50, 153), boundary=BOUNDS, tail=3)
    d = on_device(case)
    call_rule(ops()[op], case, d)
    verify(op, case, d)


def time_of(call):
    import torch
    for _ in range(3):
        call()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    for _ in range(10):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


def test_conv_takes_no_longer_for_idle_requests():
    """(Ten times as long would be a walk of every CTA through all of them.)"""
    times = []
    for idle in (0, 4000):
        case = conv_case([256], 8, seed=3)
        n = 1 + idle
        for name in ("sources", "destinations", "boundaries", "boundary_lens"):
            case[name] = np.concatenate([case[name], np.zeros(idle, np.int32)])
        case["query_start_loc"] = np.full(n + 1, 256, dtype=np.int32)
        case["query_start_loc"][0] = 0
        from prompt_testutil import to_torch
        d = {k: None if a is None else to_torch(a, "cuda") for k, a in case.items() if k != "Q"}
        times.append(time_of(lambda: run_conv(case, d)))
    assert times[1] <= 10 * times[0], times
