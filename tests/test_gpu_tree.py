"""The tree operators on the GPU against the FP64 oracle: the convolution, the
delta rule, the accepted path's records and windows, and the four together.

Tolerances: an output is rounded to BF16 once (half a step, 2^-8 of its
value); before that, corrections and states are off by 1e-4 of the head's
largest value at most, the framework's bound for FP32 states (its parts are
derived in prompt_testutil: decays good to 2^-22, here over at most 16 tokens,
sums of 128 products, 128 2^-24, and of at most eight corrections).  The
products' operands hold 22 bits at least: 2 2^-22 of |S row| |x| <= 1e-6 of it.
"""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib, synth
from oracle import kda_oracle as ko
from oracle import tree_oracle as to

import tree_testutil as tt
from kda_testutil import copy_case
from prompt_testutil import REL, check_outputs, check_states

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import _build
    assert torch.cuda.is_available()
    _build.build()
    _lib.load()


# --------------------------------------------------------------------------
# the rule
# --------------------------------------------------------------------------

def run_verify(case, d=None, **over):
    d = tt.on_device(case) if d is None else d
    tt.call_verify(case, d, **over)
    return d


def check_verify(case, d, bad=0, qsl="query_start_loc"):
    """Everything that a call leaves, against the oracle's."""
    ref = tt.copy_case(case)
    f64 = np.zeros(case["out"].shape)
    live = np.zeros(len(f64), dtype=bool)
    before = case["state"].copy()
    n_bad = to.verify(**{n: ref[n] for n in tt.VERIFY}, Q=case["Q"], out_f64=f64,
                      lower_bound=case["lower_bound"], q_scale=case["q_scale"],
                      null_slot=case["null_slot"])
    assert n_bad == bad
    live = (ref["node_corr"] != 123.0).any(axis=(1, 2))
    e = {n: tt.to_numpy(d[n]) for n in ("out", "node_corr", "state", "status")}
    assert e["status"][0] == (_lib.KDA_ERR_ARG if bad else 0)
    check_outputs(e["out"], ref["out"], f64, live)
    np.testing.assert_array_equal(e["node_corr"][~live], ref["node_corr"][~live])
    if live.any():
        scale = np.abs(ref["node_corr"][live]).max(axis=(0, 2), keepdims=True)
        assert np.all(np.abs(e["node_corr"][live] - ref["node_corr"][live]) <= REL * scale)
    check_states(e["state"], ref["state"], before)
    for n in ("corr", "key_gate", "pending", "parents", "state_slots"):
        if case[n] is not None:
            np.testing.assert_array_equal(tt.to_numpy(d[n]), case[n])


RNG = np.random.default_rng(0)
SHAPES = {
    "one": [[-1]],
    "two": [[-1, 0]],
    "chains": [tt.chain(8), tt.chain(3), tt.chain(1), tt.chain(7)],
    "stars": [tt.star(64), tt.star(9), tt.star(2)],
    "combs": [tt.comb(64), tt.comb(31), tt.comb(33), tt.comb(17)],
    "random": [tt.random_tree(RNG, n) for n in (1, 5, 64, 15, 16, 17, 24, 32, 33, 48, 63)],
    "forests": [tt.random_tree(RNG, n, roots=r) for n, r in ((12, 3), (64, 64), (40, 2), (7, 7))],
    "small": [tt.random_tree(RNG, n) for n in (3, 6, 1, 5, 2, 4, 6, 6, 1, 3, 5, 4)],
    "empty": [[], tt.random_tree(RNG, 6), [], tt.chain(4), []],
}


@pytest.mark.parametrize("H", [1, 3, 40])
@pytest.mark.parametrize("shape", SHAPES)
def test_verify_shapes(shape, H):
    case = tt.tree_case(SHAPES[shape], H, seed=3, tail=2)
    check_verify(case, run_verify(case))


@pytest.mark.parametrize("H", [2, 41])
@pytest.mark.parametrize("pool,replay", [("f32", False), ("bf16", False)])
@pytest.mark.parametrize("shape", ["one", "small", "combs", "random", "forests"])
def test_verify_reads_the_pool(shape, pool, replay, H):
    case = tt.tree_case(SHAPES[shape], H, seed=4, pool=pool, replay=replay)
    check_verify(case, run_verify(case))


@pytest.mark.parametrize("B,H,n", [(6, 32, 12), (40, 8, 30), (3, 64, 64), (160, 1, 9), (9, 3, 6),
                                   (50, 7, 4)])
def test_verify_batches(B, H, n):
    """Few and many items to an SM: every launch shape."""
    rng = np.random.default_rng(B)
    trees = [tt.random_tree(rng, int(rng.integers(max(1, n // 2), n + 1))) for _ in range(B)]
    case = tt.tree_case(trees, H, seed=5, inert=(1,), rowless=(2,))
    check_verify(case, run_verify(case))


@pytest.mark.parametrize("B,H,n", [(3, 2, 11), (60, 4, 11), (3, 2, 5), (60, 4, 5), (5, 3, 40)])
@pytest.mark.parametrize("rq,pending", [(1, 1), (3, 9), (8, 8), (8, 0), (8, -4), (5, 3)])
def test_verify_pending(rq, pending, B, H, n):
    """Counts beyond the row are clamped; none leaves the page as it is."""
    trees = [tt.random_tree(RNG, n) for _ in range(B)]
    case = tt.tree_case(trees, H, seed=6, rq=rq, pending=pending)
    check_verify(case, run_verify(case))


@pytest.mark.parametrize("lower_bound", [-10.0, -0.01, 0.0, 3.0])
@pytest.mark.parametrize("B", [2, 80])
def test_verify_gates(lower_bound, B):
    """Gates that forget at once, hardly, not at all, and that grow."""
    trees = [tt.random_tree(RNG, 20) for _ in range(B)]
    case = tt.tree_case(trees, 2, seed=7, lower_bound=lower_bound, memory=2.0, pending=3)
    check_verify(case, run_verify(case))


@pytest.mark.parametrize("n", [6, 13])
@pytest.mark.parametrize("B", [5, 90])
def test_verify_inert_and_rowless(B, n):
    """Inert requests get zeros whatever their parents hold; without a record
    row nothing is replayed; rows behind the last request stay."""
    trees = [tt.random_tree(RNG, n) for _ in range(B)]
    case = tt.tree_case(trees, 2, seed=8, inert=(0, 3), rowless=(1,), tail=3)
    t0 = case["query_start_loc"][3]
    case["parents"][t0:t0 + 6] = [9, -7, 100, 2, 2, 1]
    d = run_verify(case)
    check_verify(case, d)
    assert not tt.to_numpy(d["out"])[t0:t0 + 6].any()
    assert (tt.to_numpy(d["out"])[-3:] == tt.MARK).all()


@pytest.mark.parametrize("B", [6, 100])
def test_verify_reports(B):
    """Bad windows, trees, slots and rows: reported, and nothing of the
    request touched; the others are served."""
    trees = [tt.random_tree(RNG, 10) for _ in range(B)]
    for what in ("self", "below", "ahead", "deep", "slot", "row", "window", "order"):
        case = tt.tree_case(trees, 2, seed=9)
        t0, bad = case["query_start_loc"][2], 1
        if what == "self":
            case["parents"][t0 + 4] = 4
        elif what == "below":
            case["parents"][t0 + 4] = -2
        elif what == "ahead":
            case["parents"][t0 + 4] = 2 ** 31 - 1
        elif what == "deep":
            case["parents"][t0:t0 + 9] = np.arange(-1, 8)
        elif what == "slot":
            case["state_slots"][2] = len(case["state"])
        elif what == "row":
            case["record_rows"][2] = len(case["corr"])
        elif what == "window":
            case["Q"] = 9
            bad = B
        else:
            # a window that ends before it begins, and the one that follows it
            case["query_start_loc"][3] = t0 - 1
            bad = 2
        if what == "window":
            # (n_tokens fits B windows of Q: only one request is longer)
            case = tt.tree_case([t[:9] for t in trees[:-1]] + [trees[-1]], 2, seed=9)
            case["Q"], bad = 9, 1
            over = {n: case[n][:-1] for n in ("q", "k", "v", "raw_g", "raw_beta", "parents",
                                              "node_corr", "out")}
            case.update({n: np.ascontiguousarray(a) for n, a in over.items()})
        if what == "order":
            case["parents"][:] = -1
        d = run_verify(case)
        check_verify(case, d, bad=bad)


def test_verify_null_slot_and_uniform():
    case = tt.tree_case([tt.random_tree(RNG, 13) for _ in range(5)], 2, seed=10)
    case["query_start_loc"] = None
    case["null_slot"] = -1
    case["state_slots"][4] = 0
    check_verify(case, run_verify(case))
    case = tt.tree_case([tt.chain(8)] * 4, 2, seed=11)
    case["parents"] = case["query_start_loc"] = None  # chains without parents
    check_verify(case, run_verify(case))


def test_verify_record_rows_by_default():
    case = tt.tree_case([tt.random_tree(RNG, 5) for _ in range(4)], 2, seed=12)
    case["record_rows"] = None
    check_verify(case, run_verify(case))


@pytest.mark.parametrize("B", [3, 70])
def test_verify_strides_and_far_slots(B):
    """Rows of pools and records apart from one another: views of larger
    tensors, whose other bytes stay."""
    import torch
    case = tt.tree_case([tt.random_tree(RNG, 12) for _ in range(B)], 2, seed=13)
    d = tt.on_device(case)
    for n, pad in (("state", 512), ("corr", 132), ("key_gate", 72)):
        x = d[n]
        wide = torch.full((x.shape[0], x[0].numel() + pad), 7.0, dtype=x.dtype, device="cuda")
        wide[:, :x[0].numel()] = x.reshape(x.shape[0], -1)
        d[n] = wide[:, :x[0].numel()].view(x.shape)
        d[n + "_rest"] = wide[:, x[0].numel():]
    run_verify(case, d)
    check_verify(case, d)
    for n in ("state", "corr", "key_gate"):
        assert (d[n + "_rest"] == 7).all()


def test_verify_slots_beyond_32_bits():
    """A pool of more than 2^32 bytes and more than 2^31 elements."""
    import torch
    case = tt.tree_case([tt.random_tree(RNG, 9) for _ in range(3)], 2, seed=14, extra_slots=0)
    d = tt.on_device(case)
    stride = 2 ** 29 + 4
    pool = torch.zeros(4 * stride + 2 * 128 * 128, device="cuda")
    far = pool.as_strided(d["state"].shape, (stride, 128 * 128, 128, 1))
    far.copy_(d["state"])
    d["state"] = far
    run_verify(case, d)
    check_verify(case, d)


@pytest.mark.parametrize("par", [[-1, 0, 0, 1, 2, 3, 4, 2, 0, 8], [-1, 0, 0, 1, 2, 0]])
@pytest.mark.parametrize("B,H", [(2, 2), (50, 4)])
def test_verify_other_branches_are_never_met(B, H, par):
    """NaNs and infinities in one branch (and behind the windows) reach that
    branch's nodes alone: the others hold the same bits as without them."""
    N = len(par)
    case = tt.tree_case([par] * B, H, seed=15, tail=2)
    clean = run_verify(case)
    hit = [2, 4, 6, 7] if N == 10 else [2, 4]  # the branch of node 2
    nan, inf = 0x7FC0, 0x7F80
    dirty = tt.copy_case(case)
    for b in range(B):
        t = case["query_start_loc"][b] + 2
        dirty["k"][t], dirty["q"][t], dirty["v"][t] = nan, inf, inf
        dirty["raw_g"][t], dirty["raw_beta"][t] = nan, nan
        t = case["query_start_loc"][b] + N - 1  # a leaf
        dirty["q"][t] = nan
    for n in ("q", "k", "v", "raw_g", "raw_beta"):
        dirty[n][-2:] = nan
    d = run_verify(dirty)
    own = np.ones(len(case["out"]), dtype=bool)
    leaf = np.zeros_like(own)
    for b in range(B):
        own[case["query_start_loc"][b] + np.array(hit)] = False
        leaf[case["query_start_loc"][b] + N - 1] = True
    for n in ("out", "node_corr"):
        got, want = tt.to_numpy(d[n]), tt.to_numpy(clean[n])
        keep = own & ~leaf if n == "out" else own
        np.testing.assert_array_equal(got[keep], want[keep])
    np.testing.assert_array_equal(tt.to_numpy(d["state"]), tt.to_numpy(clean["state"]))
    assert np.isnan(tt.to_numpy(d["node_corr"])[case["query_start_loc"][0] + np.array(hit)]).all()
    assert np.isnan(ko.bf16_to_f64(tt.to_numpy(d["out"])[leaf])).all()


@pytest.mark.parametrize("B", [2, 60])
def test_verify_zero_keys_and_large_states(B):
    """Keys and queries of zeros (their norm is the root of 1e-6 alone), states
    of 1e30 and of 1e-30."""
    for size in (1e30, 1e-30):
        case = tt.tree_case([tt.random_tree(RNG, 14) for _ in range(B)], 2, seed=16, pending=0)
        case["state"] *= np.float32(size)
        case["k"][3], case["q"][5] = 0, 0
        if size > 1:
            case["v"][:] = 0x7149  # some 1e30
        check_verify(case, run_verify(case))


def test_verify_on_another_stream_and_captured():
    """On a stream of its own, and captured: replays with other inputs in the
    same tensors give what eager calls give."""
    import torch
    cases = [tt.tree_case([tt.random_tree(np.random.default_rng(s), n) for n in (20, 9, 31)], 4,
                          seed=20 + s) for s in range(3)]
    side = torch.cuda.Stream()
    d = tt.on_device(cases[0])
    side.wait_stream(torch.cuda.current_stream())
    run_verify(cases[0], d, stream=side)
    side.synchronize()
    check_verify(cases[0], d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_verify(cases[0], d)
    for case in cases:
        fresh = tt.on_device(case)
        for n in tt.VERIFY:
            d[n].copy_(fresh[n])
        graph.replay()
        torch.cuda.synchronize()
        check_verify(case, d)


def test_verify_without_tokens_replays():
    case = tt.tree_case([[], [], []], 2, seed=17, pending=4)
    d = run_verify(case)
    check_verify(case, d)
    assert (tt.to_numpy(d["state"]) != case["state"]).any()


def test_verify_agrees_with_the_step_on_chains():
    """Both from the same checkpoints, records and windows."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_replay_verify
    B, H, Q = 7, 4, 8
    case = tt.tree_case([tt.chain(Q)] * B, H, seed=18)
    d, e = run_verify(case), tt.on_device(case)
    kda_replay_verify(e["q"], e["k"], e["v"], e["raw_g"], e["raw_beta"], e["A_log"], e["dt_bias"],
                      e["state"], e["state_slots"], e["record_rows"], e["pending"], e["corr"],
                      e["key_gate"], e["out"], Q=Q, lower_bound=-5.0, q_scale=case["q_scale"])
    torch.cuda.synchronize()
    rows = case["record_rows"]
    u = tt.to_numpy(d["node_corr"]).reshape(B, Q, H, 128).transpose(0, 2, 1, 3)
    want = tt.to_numpy(e["corr"])[rows]
    assert np.abs(u - want).max() <= 2 * REL * np.abs(want).max()
    s, want = tt.to_numpy(d["state"]), tt.to_numpy(e["state"])
    assert np.abs(s - want).max() <= 2 * REL * np.abs(want).max()


# --------------------------------------------------------------------------
# the convolution
# --------------------------------------------------------------------------

def run_conv(case, d=None, **over):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_tree_conv
    d = tt.on_device(case) if d is None else d
    for n in ("cq", "ck", "cv"):
        d[n] = torch.full_like(d["q"], 3.0)
    kw = dict(Q=case["Q"], record_rows=d["record_rows"], pending=d["pending"],
              query_start_loc=d["query_start_loc"], null_slot=case["null_slot"], status=d["status"])
    kw.update(over)
    kda_tree_conv(d["x"], d["conv_weight"], d["conv_bias"], d["conv_state"], d["state_slots"],
                  d["parents"], d["cq"], d["ck"], d["cv"], **kw)
    return d


def check_conv(case, d, bad=0):
    T, H = case["q"].shape[:2]
    q, k, v = (np.full((T, H, 128), 0x4040, dtype=np.uint16) for _ in range(3))  # 3.0
    f64 = np.full((T, 3, H, 128), np.nan)
    n_bad = to.conv(x=case["x"], conv_weight=case["conv_weight"], conv_bias=case["conv_bias"],
                    conv_state=case["conv_state"], state_slots=case["state_slots"],
                    parents=case["parents"], q=q, k=k, v=v, Q=case["Q"],
                    record_rows=case["record_rows"], pending=case["pending"],
                    query_start_loc=case["query_start_loc"], null_slot=case["null_slot"],
                    out_f64=f64)
    assert n_bad == bad and tt.to_numpy(d["status"])[0] == (_lib.KDA_ERR_ARG if bad else 0)
    live = ~np.isnan(f64).any(axis=(1, 2, 3))
    for i, (got, ref) in enumerate(zip((d["cq"], d["ck"], d["cv"]), (q, k, v))):
        got = tt.to_numpy(got)
        np.testing.assert_array_equal(got[~live], ref[~live])
        want = f64[live][:, i]
        # half a BF16 step; four products and the fast exponential and
        # reciprocal in FP32: 2^-20 of sums that are 32 at most in size
        assert np.all(np.abs(ko.bf16_to_f64(got[live]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15)
    np.testing.assert_array_equal(tt.to_numpy(d["conv_state"]), case["conv_state"])


@pytest.mark.parametrize("H", [1, 5])
@pytest.mark.parametrize("shape", SHAPES)
def test_conv_shapes(shape, H):
    case = tt.tree_case(SHAPES[shape], H, seed=30, tail=2)
    check_conv(case, run_conv(case))


@pytest.mark.parametrize("rq,pending", [(1, 1), (2, 2), (3, 7), (5, 4), (8, 8), (8, 0), (7, -1)])
def test_conv_windows(rq, pending):
    case = tt.tree_case([tt.random_tree(RNG, 7) for _ in range(4)], 2, seed=31, rq=rq,
                        pending=pending, inert=(2,), rowless=(1,))
    check_conv(case, run_conv(case))


def test_conv_without_bias_replay_or_offsets():
    case = tt.tree_case([tt.random_tree(RNG, 16) for _ in range(60)], 3, seed=32)
    case["conv_bias"] = case["pending"] = case["query_start_loc"] = None
    check_conv(case, run_conv(case))


def test_conv_reports():
    case = tt.tree_case([tt.random_tree(RNG, 8) for _ in range(5)], 2, seed=33)
    case["parents"][case["query_start_loc"][1] + 3] = 3
    case["state_slots"][2] = len(case["conv_state"])
    case["record_rows"][3] = len(case["pending"])
    check_conv(case, run_conv(case), bad=3)


def test_conv_equals_the_layer_prologue():
    """On chains it is the layer's convolution, bit for bit, pending windows
    included."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_layer_prologue
    B, H, Q = 6, 2, 8
    c = synth.layer_case(B=B, H=H, Q=Q, slots=16, seed=3)
    names = ("x", "conv_weight", "conv_bias", "conv_state", "f_a", "f_b", "state_slots",
             "record_rows", "pending")
    d = {n: tt.to_torch(c[n], "cuda") for n in names}
    outs = [torch.zeros((B * Q, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    case = dict(Q=Q, null_slot=0, q=np.zeros((B * Q, H, 128), dtype=np.uint16),
                parents=np.tile(np.arange(-1, Q - 1), B).astype(np.int32), query_start_loc=None,
                **{n: c[n] for n in names})
    e = run_conv(case)
    kda_layer_prologue(d["x"], d["conv_weight"], d["conv_bias"], d["conv_state"], d["f_a"],
                       d["f_b"], d["state_slots"], d["record_rows"], d["pending"], *outs, Q=Q)
    live = np.repeat(c["state_slots"] > 0, Q)
    for got, want in zip((e["cq"], e["ck"], e["cv"]), outs):
        np.testing.assert_array_equal(tt.to_numpy(got)[live], tt.to_numpy(want)[live])


# --------------------------------------------------------------------------
# the accepted path
# --------------------------------------------------------------------------

def select_case(trees, H, seed, **kw):
    case = tt.tree_case(trees, H, seed=seed, **kw)
    rng = np.random.default_rng(seed + 100)
    rq = case["corr"].shape[2]
    paths = np.full((len(trees), 8), -1, dtype=np.int32)
    counts = np.zeros(len(trees), dtype=np.int32)
    for b, par in enumerate(trees):
        path = [0] if par else []
        while path and len(path) < rq:
            children = [t for t, a in enumerate(par) if a == path[-1]]
            if not children or rng.random() < 0.2:
                break
            path.append(int(rng.choice(children)))
        paths[b, :len(path)], counts[b] = path, len(path)
    case.update(path=paths, accepted=counts, eager=None,
                node_corr=rng.standard_normal(case["node_corr"].shape).astype(np.float32))
    return case


def run_select(case, d=None, windows=True, **over):
    from linear_attention_speculative_recoverssm_gb300 import kda_tree_select
    d = tt.on_device(case) if d is None else d
    kw = dict(Q=case["Q"], query_start_loc=d["query_start_loc"], null_slot=case["null_slot"],
              status=d["status"], pending=d["pending"], eager=d["eager"])
    if windows:
        kw.update(x=d["x"], conv_state=d["conv_state"])
    kw.update(over)
    kda_tree_select(d["path"], d["accepted"], d["k"], d["raw_g"], d["node_corr"], d["state_slots"],
                    d["record_rows"], d["corr"], d["key_gate"], **kw)
    return d


def check_select(case, d, bad=0, windows=True):
    ref = tt.copy_case(case)
    n_bad = to.select(path=ref["path"], accepted=ref["accepted"], k=ref["k"], raw_g=ref["raw_g"],
                      node_corr=ref["node_corr"], state_slots=ref["state_slots"],
                      record_rows=ref["record_rows"], corr=ref["corr"], key_gate=ref["key_gate"],
                      Q=case["Q"], x=ref["x"] if windows else None,
                      conv_state=ref["conv_state"] if windows else None, pending=ref["pending"],
                      eager=ref["eager"], query_start_loc=ref["query_start_loc"], null_slot=case["null_slot"])
    assert n_bad == bad and tt.to_numpy(d["status"])[0] == (_lib.KDA_ERR_ARG if bad else 0)
    for n in ("corr", "key_gate", "conv_state", "pending", "path", "accepted", "node_corr", "x"):
        if ref[n] is not None:
            np.testing.assert_array_equal(tt.to_numpy(d[n]), ref[n], err_msg=n)


@pytest.mark.parametrize("windows", [True, False])
@pytest.mark.parametrize("H", [1, 3, 9])
@pytest.mark.parametrize("shape", SHAPES)
def test_select_shapes(shape, H, windows):
    case = select_case(SHAPES[shape], H, 40, tail=2)
    check_select(case, run_select(case, windows=windows), windows=windows)


@pytest.mark.parametrize("rq", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("pending", [0, 1, 2, 9, -1])
def test_select_windows(rq, pending):
    trees = [tt.chain(8), tt.star(3), tt.chain(2), [], tt.comb(12), tt.chain(3)]
    case = select_case(trees, 2, 41, rq=rq, pending=pending, inert=(1,), rowless=(2,))
    check_select(case, run_select(case))
    case["eager"] = np.array([1, 1, 1, 1, 0, 2], np.uint8)
    check_select(case, run_select(case))


def test_select_reports():
    trees = [tt.comb(12) for _ in range(7)]
    case = select_case(trees, 2, 42, rq=4)
    case["accepted"][:] = [1, 5, -1, 2, 2, 2, 2]
    case["path"][3, 1], case["path"][4, 0], case["path"][5, 1] = 12, -1, 2 ** 31 - 1
    case["path"][6, 1], case["path"][0, 1:] = 11, 500  # (behind the count: not looked at)
    check_select(case, run_select(case), bad=5)


def test_select_uniform_and_captured():
    import torch
    cases = [select_case([tt.random_tree(np.random.default_rng(s), 10) for _ in range(5)], 2, 43 + s)
             for s in range(2)]
    for case in cases:
        case["query_start_loc"] = None
    d = tt.on_device(cases[0])
    run_select(cases[0], d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_select(cases[0], d)
    for case in cases:
        fresh = tt.on_device(case)
        for n in fresh:
            if fresh[n] is not None:
                d[n].copy_(fresh[n])
        graph.replay()
        torch.cuda.synchronize()
        check_select(case, d)


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------

def test_decoding_with_trees_and_chains():
    """Steps of trees and of chains in turn through DeferredRecoverSSM, with
    the layer's convolution before each, eager rows (of trees: the layer's own
    window goes by the pending count) and a flush among them;
    against the plain recurrence over each request's accepted tokens."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import (DeferredRecoverSSM,
                                                               kda_draft_accept,
                                                               kda_layer_prologue, kda_tree_conv)
    H, B, rq, V = 2, 4, 8, 40
    D = H * 128
    rng = np.random.default_rng(50)
    bits = lambda *s, std=1.0: synth.to_bf16_bits((rng.standard_normal(s) * std).astype(np.float32))
    w, bias, f_b = bits(3, 4, D, std=0.5), bits(3 * D, std=0.1), bits(D, 128, std=0.1)
    A_log = rng.uniform(0, 1.5, H).astype(np.float32)
    dt = (rng.standard_normal((H, 128)) - 2).astype(np.float32)
    slots, rows = np.array([3, 1, 5, 2], np.int32), np.array([2, 0, 3, 1], np.int32)
    state0 = (rng.standard_normal((6, H, 128, 128)) * 0.1).astype(np.float32)
    conv0 = bits(6, 3 * D, rq + 2)
    dev = lambda a: tt.to_torch(a, "cuda")
    d = {n: dev(a) for n, a in dict(state=state0, conv=conv0, w=w, bias=bias, f_b=f_b, A=A_log,
                                    dt=dt, slots=slots, rows=rows,
                                    pending=np.zeros(4, np.int32),
                                    corr=np.zeros((4, H, rq, 128), np.float32),
                                    kg=np.zeros((4, H, rq, 256), np.uint16),
                                    status=np.zeros(1, np.int32)).items()}
    loop = DeferredRecoverSSM(d["state"], d["slots"], d["rows"], d["pending"], d["corr"], d["kg"],
                              d["A"], d["dt"], Q=rq, lower_bound=-5.0, q_scale=128 ** -0.5,
                              status=d["status"])
    history = [[conv0[s, :, i] for i in range(3)] for s in slots]  # inputs so far, per request
    states = [state0[s].astype(np.float64) for s in slots]
    to32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for step in range(7):
        tree = step % 3 != 1
        lens = [int(n) for n in rng.integers(1, 30, B)] if tree else [rq] * B
        trees = [tt.random_tree(rng, n) for n in lens] if tree else [tt.chain(rq)] * B
        T = sum(lens)
        x, f_a, beta = bits(T, 3 * D), bits(T, 128), bits(T, H)
        par, starts = tt.packed(trees), tt.starts_of(trees)
        q, k, v, g, out = (torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda")
                           for _ in range(5))
        node_corr = torch.zeros((T, H, 128), device="cuda")
        if step == 4:
            loop.flush()
        # the target likes the drafts: paths of some length
        tokens = rng.integers(0, V, T).astype(np.int32)
        target = rng.dirichlet(np.full(V, 0.3), T).astype(np.float32)
        for b in range(B):
            for t in range(1, lens[b]):
                target[starts[b] + trees[b][t], tokens[starts[b] + t]] += 1.0
        u, un = rng.random(T).astype(np.float32), rng.random(B).astype(np.float32)
        accepted, path, nxt = to32(B), to32(B, 8), to32(B)
        common = dict(Q=max(lens), query_start_loc=dev(starts))
        if tree:
            kda_tree_conv(dev(x), d["w"], d["bias"], d["conv"], d["slots"], dev(par), q, k, v,
                          record_rows=d["rows"], pending=d["pending"], status=d["status"], **common)
            g.copy_((dev(f_a).float() @ d["f_b"].float().t()).view(T, H, 128))
            loop.verify_tree(q, k, v, g, dev(beta), dev(par), node_corr, out, **common)
        else:
            kda_layer_prologue(dev(x), d["w"], d["bias"], d["conv"], dev(f_a), d["f_b"], d["slots"],
                               d["rows"], d["pending"], q, k, v, g, Q=rq, status=d["status"])
            loop.verify(q, k, v, g, dev(beta), out)
        kda_draft_accept(dev(target), dev(tokens), dev(u), dev(un), accepted, path, nxt,
                         parents=dev(par), status=d["status"], **common)
        count, way = tt.to_numpy(accepted).copy(), tt.to_numpy(path)
        ref = to.accept(target=target.astype(np.float64), tokens=tokens, accept_uniforms=u,
                        sample_uniforms=un, Q=max(lens), parents=par, query_start_loc=starts)
        for got, want in zip((count, way, tt.to_numpy(nxt)), ref):
            np.testing.assert_array_equal(got, want)
        eager = torch.tensor([0, 1, 0, int(step == 5)], dtype=torch.uint8, device="cuda")
        if tree:
            loop.accept_tree(path, accepted, k, g, node_corr, x=dev(x), conv_state=d["conv"],
                             eager=eager, **common)
        else:
            loop.accept(accepted)
        # the plain recurrence down every node's path
        kq, kk, kv, kgate = (ko.bf16_to_f64(tt.to_numpy(t)) for t in (q, k, v, g))
        got = ko.bf16_to_f64(tt.to_numpy(out))
        f = ko.bf16_to_f64(w).transpose(1, 0, 2).reshape(4, 3 * D)
        ref_out = np.zeros_like(got)
        for b in range(B):
            node_states, node_inputs = [], []
            for t, p in enumerate(trees[b]):
                i = starts[b] + t
                line = (history[b] if p < 0 else node_inputs[p]) + [x[i]]
                node_inputs.append(line)
                s = ko.bf16_to_f64(np.stack(line[-4:]))
                z = ko.bf16_to_f64(bias) + sum(f[j] * s[j] for j in range(4))
                y = (z * ko.sigmoid(z)).reshape(3, H, 128)
                for have, want in zip((kq[i], kk[i], kv[i]), y):
                    assert np.all(np.abs(have - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15)
                S = states[b] if p < 0 else node_states[p]
                dec = np.exp(-5.0 * ko.sigmoid(np.exp(A_log.astype(np.float64))[:, None]
                                               * (kgate[i] + dt)))
                kn, qn = ko.l2norm(kk[i]), ko.l2norm(kq[i]) * 128 ** -0.5
                S = S * dec[:, None]
                c = ko.sigmoid(ko.bf16_to_f64(beta[i]))[:, None] * (kv[i] - np.einsum("hvk,hk->hv", S, kn))
                S = S + c[..., None] * kn[:, None]
                node_states.append(S)
                ref_out[i] = np.einsum("hvk,hk->hv", S, qn)
            last = way[b, count[b] - 1]
            states[b], history[b] = node_states[last], node_inputs[last]
        scale = np.abs(ref_out).max()
        assert np.all(np.abs(got - ref_out) <= 2.0 ** -8 * np.abs(ref_out) + REL * scale), step
        assert tt.to_numpy(d["status"])[0] == 0
    loop.flush()
    for b in range(B):
        got = tt.to_numpy(d["state"])[slots[b]]
        assert np.abs(got - states[b]).max() <= REL * np.abs(states[b]).max()
