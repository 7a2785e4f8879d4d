"""kda_prefill and kda_recurrent where sizes change along a prompt: values
that fall or rise from one chunk to the next, states that are forgotten,
single outlying tokens, write gates that are nearly closed.  What a chunk
leaves is compared with the FP64 recurrence relative to the largest entry of
what is left, head by head."""
import numpy as np
import pytest

from oracle import kda_oracle as ko
from oracle import prompt_oracle as po
from kda_testutil import bf16_ulp
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
        g, r = ko.state_to_f64(state[s]), ko.state_to_f64(ref["state"][s])
        step = bf16_ulp(r) if state.dtype == np.uint16 else 0.0
        err = np.maximum(np.abs(g - r) - step, 0).max(axis=(1, 2)) / np.abs(r).max(axis=(1, 2))
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
@pytest.mark.parametrize("by", [1e-1, 1e-2, 1e-3, 1e-5, 1e-7, 1e-12, 1e3, 1e7])
def test_values_that_fall(op, by):
    """Values of another size from a request's 65th token on."""
    case = ragged_case(lens=[128, 100], H=2, seed=3, boundary={0: 100})
    set_decay(case, -0.5)
    for a, b in ((64, 128), (192, 228)):
        scale_values(case, slice(a, b), by)
    check(op, case)


@OPS
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6, 1e8, 1e20])
def test_large_resumed_state(op, size):
    """A state of large entries, which the prompt forgets."""
    case = ragged_case(lens=[128, 100], H=2, seed=4, resume=(0, 1), boundary={0: 60})
    set_decay(case, -0.5)
    case["state"] *= np.float32(size)
    check(op, case)


@OPS
@pytest.mark.parametrize("size", [1e2, 1e3, 1e5, 1e8])
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


@OPS
@pytest.mark.parametrize("pool", ["f32", "bf16"])
def test_values_that_vanish(op, pool):
    """Values of 1e20, then none while everything is forgotten, then ordinary
    ones: three chunks, and a fourth that is cut short."""
    case = ragged_case(lens=[250, 100], H=2, seed=8, pool=pool, boundary={0: 192})
    set_decay(case, -4.0)
    scale_values(case, slice(0, 64), 1e20)
    scale_values(case, slice(64, 128), 0.0)
    check(op, case)


@OPS
def test_forgotten_in_a_long_prompt(op):
    """The same in prompts that go by segments, at places in and between
    them: whole states forgotten by nearly closed gates."""
    case = ragged_case(lens=[4200, 2100], H=2, seed=9, resume=(1,), boundary={0: 2049})
    set_decay(case, -2.0)
    for t0 in (0, 1000, 16 * 64 - 10, 3000, 4200 + 500):
        scale_values(case, slice(t0, t0 + 2), 1e6)
        case["raw_beta"][t0 + 40:t0 + 70] = synth.to_bf16_bits(np.array([-20.0], np.float32))
    check(op, case)


@OPS
@pytest.mark.parametrize("lens", [[130, 100, 70, 200], [4200, 2100, 64, 70]])
def test_forgotten_in_place(op, lens):
    """A forgotten state whose slot is also the destination's or the
    boundary's."""
    case = ragged_case(lens=lens, H=2, seed=11, resume=range(4), boundary={1: 70, 2: 64, 3: 65})
    set_decay(case, -0.5)
    case["state"] *= np.float32(1e8)
    s, d, bnd = case["sources"], case["destinations"], case["boundaries"]
    s[0], s[1], s[2], s[3] = d[0], bnd[1], bnd[2], d[3]
    check(op, case)


def test_many_forget():
    """More (request, head) items to do again than there are SMs."""
    lens = [80] * 40
    case = ragged_case(lens=lens, H=5, seed=12, resume=range(40), boundary={3: 70, 30: 2})
    set_decay(case, -0.5)
    case["state"] *= np.float32(1e8)
    check("prefill", case)


@OPS
def test_some_rows_only(op):
    """Value channels of one group of 32 forget what the others keep: each
    group is checked on its own, and so are its outputs."""
    case = ragged_case(lens=[200, 64, 65], H=2, seed=10)
    set_decay(case, -0.5)
    v = ko.bf16_to_f64(case["v"]).copy()
    v[:64, :, 40:70] *= 1e8
    v[:, :, 3] = 0
    case["v"] = synth.to_bf16_bits(v.astype(np.float32))
    got, state, status = run(op, case)
    ref = {k: x.copy() if isinstance(x, np.ndarray) else x for k, x in case.items()}
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    assert po.rule(out_f64=f64, sizes=sizes, **ref) == 0 and status == 0
    for s in case["destinations"]:
        r = ref["state"][s].astype(np.float64).reshape(2, 4, 32, 128)
        err = np.abs(state[s].reshape(r.shape) - r).max(axis=(2, 3))
        assert np.all(err <= REL * np.abs(r).max(axis=(2, 3))), f"slot {s}"
    out = ko.bf16_to_f64(got)
    slack = (QUERY if op == "prefill" else REL) * sizes
    assert np.all(np.abs(out - f64) <= 2.0 ** -8 * np.abs(f64) + slack), "outputs"


@OPS
@pytest.mark.parametrize("lens", [[64], [100, 64]])
def test_steep_half_block(op, lens):
    """Gates that forget e^-10 a token for eight tokens, then a slow decline
    behind closed write gates: the last of the eight is what is left."""
    case = ragged_case(lens=lens, H=2, seed=14, resume=(), lower_bound=-10.0)
    set_decay(case, -0.27)
    for t0 in case["query_start_loc"][:-1]:
        case["raw_g"][t0 + 24:t0 + 32] = synth.to_bf16_bits(np.array([30.0], np.float32))
        case["raw_beta"][t0 + 32:t0 + 64] = synth.to_bf16_bits(np.array([-30.0], np.float32))
    check(op, case)


def same_finite(got, want, name):
    np.testing.assert_array_equal(np.isfinite(got), np.isfinite(want), err_msg=name)


@pytest.mark.parametrize("at", [30, 100, 127, 128])
@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80, 0xFF80])
@pytest.mark.parametrize("name", ["q", "k", "v", "raw_g", "raw_beta"])
def test_not_finite(name, bits, at):
    """A NaN or an infinity of one token: the outputs before it are those
    without it, and from it on what the recurrence makes of it."""
    case = ragged_case(lens=[200, 150], H=2, seed=13, resume=(1,), boundary={0: at})
    clean = {k: x.copy() if isinstance(x, np.ndarray) else x for k, x in case.items()}
    for t in (at, 200 + at):  # (one channel of the first head, and all of its beta)
        case[name][(t, 0, 5) if case[name].ndim == 3 else (t, 0)] = bits
    got, state, status = run("prefill", case)
    want, left, _ = run("recurrent", case)
    assert status == 0
    got, want = ko.bf16_to_f64(got), ko.bf16_to_f64(want)
    same_finite(got, want, "outputs")
    same_finite(state, left, "states")
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    po.rule(out_f64=f64, sizes=sizes, **clean)
    close = np.abs(got - f64) <= 2.0 ** -8 * np.abs(f64) + QUERY * sizes
    for t0, t1, h in ((0, at, 0), (200, 200 + at, 0), (0, 350, 1)):
        assert np.all(close[t0:t1, h]), "outputs that it does not reach"
    s = case["boundaries"][0]
    assert np.abs(state[s] - clean["state"][s]).max() <= REL * np.abs(clean["state"][s]).max()
    fin = np.isfinite(want)
    rounded = 2 * 2.0 ** -8 * np.abs(want) + 2 * QUERY * np.nanmax(np.where(fin, np.abs(want), 0))
    assert np.all((np.abs(got[fin] - want[fin]) <= rounded[fin]))
    fin = np.isfinite(left)
    assert np.all(np.abs(state[fin] - left[fin]) <= 2 * REL * np.abs(left[fin]).max())


@pytest.mark.parametrize("pool", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[64, 41], [300, 130, 70], [2100]])
def test_outputs_as_good_as_token_by_token(pool, lens):
    """The chunked form's outputs before their rounding to BF16: off by what its
    operands' 22 bits leave of what they are sums of, 3 2^-22 for each of the two
    products (hi.lo and lo.hi rounded, lo.lo left out) and twice that for the
    operands of A, which are products themselves; so nearly all round to what
    the FP64 recurrence's round to."""
    case = ragged_case(lens=lens, H=3, seed=sum(lens), pool=pool, resume=range(1, len(lens)),
                       boundary={0: lens[0] // 2})
    got, _, status = run("prefill", case)
    ref = {k: x.copy() if isinstance(x, np.ndarray) else x for k, x in case.items()}
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    assert po.rule(out_f64=f64, sizes=sizes, **ref) == 0 and status == 0
    out = ko.bf16_to_f64(got)
    # (and the decays', REL's 2.5e-5 of a state, on what is left of a token)
    slack = (9 * 2.0 ** -22 + 2.5e-5) * sizes
    assert np.all(np.abs(out - f64) <= 2.0 ** -8 * np.abs(f64) + slack)
    assert np.mean(got == ref["out"]) >= 0.995


@OPS
@pytest.mark.parametrize("log_decay", [-0.1, -4.0])
def test_padding_rows(op, log_decay):
    """Tokens of zeros before a prompt, inside it and over whole chunks: zero
    keys and values write nothing, and the gates forget meanwhile."""
    case = ragged_case(lens=[300, 150, 70], H=2, seed=15, resume=(1,), boundary={0: 100})
    set_decay(case, log_decay)
    for a, b in ((0, 40), (90, 110), (128, 260), (300, 375), (450, 451)):
        for name in ("q", "k", "v"):
            case[name][a:b] = 0
    check(op, case)


def test_captured_and_at_once():
    """One captured call replayed on inputs that the parts hold, do not hold and
    hold again, beside eager calls of the other kind on another stream: bit for
    bit what each gives alone."""
    import torch
    cases = []
    for seed, size in ((16, 1.0), (17, 1e8), (18, 1.0)):
        case = ragged_case(lens=[130, 70, 200], H=3, seed=seed, resume=range(3),
                           boundary={0: 64, 2: 101})
        set_decay(case, -0.5)
        case["state"] *= np.float32(size)
        cases.append(case)
    for c in cases[1:]:
        for name in ("sources", "destinations", "boundaries"):
            c[name] = cases[0][name]
    alone = [run("prefill", c) for c in cases]
    d = on_device(cases[0])
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call_rule(ops()["prefill"], cases[0], d)
    for i, case in enumerate(cases):
        other = on_device(cases[(i + 1) % 3])
        for name, t in on_device(case).items():
            d[name].copy_(t)
        torch.cuda.synchronize()
        graph.replay()
        call_rule(ops()["prefill"], case, other, stream=side)
        torch.cuda.synchronize()
        for got, want in ((d, alone[i]), (other, alone[(i + 1) % 3])):
            np.testing.assert_array_equal(to_numpy(got["out"]), want[0])
            np.testing.assert_array_equal(to_numpy(got["state"]), want[1])
