"""kda_prefill and kda_recurrent where sizes change along a prompt: values
that fall or rise from one chunk to the next, states that are forgotten,
single outlying tokens, write gates that are nearly closed.  What a chunk
leaves is compared with the FP64 recurrence relative to the largest entry of
what is left, head by head."""
import numpy as np
import pytest

from oracle import kda_oracle as ko
from oracle import prompt_oracle as po
from prompt_testutil import (OUT_REL_L2, QUERY, REL, call_rule, on_device, ragged_case, to_numpy)
from linear_attention_speculative_recoverssm_gb300 import synth

pytestmark = pytest.mark.gpu


def ops():
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill, kda_recurrent
    return {"prefill": kda_prefill, "recurrent": kda_recurrent}


def set_decay(case, log_decay, tokens=slice(None), seed=0):
    """The given log decay a token, times e^(0.3 N(0, 1)) by channel.  (A steep
    stretch is one by its raw gates, the channels' biases being those of the
    rest.)"""
    rng = np.random.default_rng(seed)
    H = case["A_log"].shape[0]
    lb = case["lower_bound"]
    logit = lambda share: np.log(share / (1 - share))
    share = np.clip(log_decay / lb * np.exp(0.3 * rng.standard_normal((H, 128))), 1e-6, 0.98)
    if tokens == slice(None):
        case["A_log"][:] = 0
        case["dt_bias"][:] = logit(share)
        case["raw_g"][:] = 0
    else:
        case["raw_g"][tokens] = synth.to_bf16_bits(
            (logit(share) - case["dt_bias"]).astype(np.float32))


def scale_values(case, tokens, by):
    case["v"][tokens] = synth.to_bf16_bits(
        (ko.bf16_to_f64(case["v"][tokens]) * by).astype(np.float32))


def run(op, case):
    d = on_device(case)
    call_rule(ops()[op], case, d)
    return to_numpy(d["out"]), to_numpy(d["state"]), int(d["status"][0])


def check(op, case):
    got, state, status = run(op, case)
    ref = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in case.items()}
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    assert po.rule(out_f64=f64, sizes=sizes, **ref) == 0 and status == 0
    slots = [s for n in ("destinations", "boundaries") for s in case[n] if s > 0]
    for s in slots:
        r = ref["state"][s].astype(np.float64)
        err = np.abs(state[s] - r).max(axis=(1, 2)) / np.abs(r).max(axis=(1, 2))
        assert np.all(err <= REL), f"slot {s}: {err}"
    out = ko.bf16_to_f64(got)
    # (the recurrence in FP32: its state's error, on every output)
    slack = (QUERY if op == "prefill" else REL) * sizes
    assert np.all(np.abs(out - f64) <= 2.0 ** -8 * np.abs(f64) + slack), "outputs"
    for b in range(len(case["destinations"])):
        t0, t1 = case["query_start_loc"][b:b + 2]
        for a in range(t0, t1, 64):
            part = slice(a, min(a + 64, t1))
            err = np.linalg.norm(out[part] - f64[part])
            assert err <= OUT_REL_L2 * np.linalg.norm(f64[part]), (b, a)


OPS = pytest.mark.parametrize("op", ["prefill", "recurrent"])


@OPS
@pytest.mark.parametrize("by", [1e-1, 1e-2, 1e-3, 1e3])
def test_values_that_fall(op, by):
    """Values of another size from a request's 65th token on."""
    case = ragged_case(lens=[128, 100], H=2, seed=3, boundary={0: 100})
    set_decay(case, -0.5)
    for a, b in ((64, 128), (192, 228)):
        scale_values(case, slice(a, b), by)
    check(op, case)


@OPS
@pytest.mark.parametrize("size", [1e2, 1e4])
def test_large_resumed_state(op, size):
    """A state of large entries, which the prompt forgets."""
    case = ragged_case(lens=[128, 100], H=2, seed=4, resume=(0, 1), boundary={0: 60})
    set_decay(case, -0.5)
    case["state"] *= np.float32(size)
    check(op, case)


@OPS
@pytest.mark.parametrize("size", [1e2, 1e3])
@pytest.mark.parametrize("steep", [False, True])
def test_outlying_token(op, size, steep):
    """One token's values far larger than all others; with `steep` the gates
    forget it before the chunk ends."""
    case = ragged_case(lens=[128, 100], H=2, seed=5)
    set_decay(case, -0.4)
    for t0 in (0, 128):
        scale_values(case, slice(t0 + 30, t0 + 31), size)
        if steep:
            set_decay(case, -4.0, slice(t0 + 31, t0 + 64), seed=6)
    check(op, case)


@OPS
@pytest.mark.parametrize("raw_beta", [-8.0, -12.0, -18.0, -40.0])
def test_closed_write_gates(op, raw_beta):
    """Write gates of sigmoid(raw_beta) throughout, from a fresh state: all of
    it is as small as they are."""
    case = ragged_case(lens=[128, 100, 41], H=2, seed=7, resume=(), boundary={0: 64})
    set_decay(case, -0.05)
    case["raw_beta"][:] = synth.to_bf16_bits(np.array([raw_beta], dtype=np.float32))
    check(op, case)
