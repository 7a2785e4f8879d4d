"""kda_prefill and kda_recurrent against the FP64 recurrence: ragged lengths,
fresh and resumed states, boundaries, inert requests, both pools, every edge
of the chunks; then what is refused or reported, streams and graphs."""
import numpy as np
import pytest

from oracle import prompt_oracle as po
from prompt_testutil import (QUERY, call_rule, check_outputs, check_states, on_device, ragged_case,
                             to_numpy, to_torch)

pytestmark = pytest.mark.gpu


def ops():
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill, kda_recurrent
    return {"prefill": kda_prefill, "recurrent": kda_recurrent}


def run_and_check(op, case, **over):
    d = on_device(case)
    call_rule(ops()[op], case, d, **over)
    verify(op, case, d)
    return d


def verify(op, case, d, bad=0):
    ref = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in case.items()}
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    left_out = po.rule(out_f64=f64, sizes=sizes, **ref)
    assert left_out == bad
    got = to_numpy(d["out"])
    qsl, dst = case["query_start_loc"], case["destinations"]
    live = np.zeros(len(got), dtype=bool)
    touched = (ref["out"] != case["out"]).reshape(len(got), -1).any(axis=1)
    for b in range(len(dst)):
        if dst[b] > case["null_slot"] and 0 <= qsl[b] <= qsl[b + 1] <= len(got):
            live[qsl[b]:qsl[b + 1]] = True
    check_outputs(got, ref["out"], f64, live & touched,
                  QUERY * sizes if op == "prefill" else 0.0)
    check_states(to_numpy(d["state"]), ref["state"], case["state"])
    assert (int(d["status"][0]) != 0) == (bad > 0)


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
@pytest.mark.parametrize("pool", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2, 1, 1], [15, 16, 17], [63, 64, 65], [0, 5, 0, 33, 0],
                                  [127, 1, 128, 129, 200], [500]])
def test_ragged(op, pool, lens):
    H = 3
    boundary = {b: max(1, n // 2) for b, n in enumerate(lens) if n > 1 and b % 2 == 0}
    run_and_check(op, ragged_case(lens=lens, H=H, seed=sum(lens) + len(lens), pool=pool,
                                  boundary=boundary, tail=3))


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_boundary_anywhere(op):
    """Boundaries at the first token, at chunk edges, at the last token and
    beyond the window (then S_n)."""
    lens = [70, 130, 64, 65, 200, 90, 3]
    run_and_check(op, ragged_case(lens=lens, H=2, seed=5,
                                  boundary={0: 1, 1: 64, 2: 64, 3: 64, 4: 199, 5: 1000, 6: 2}))


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_inert_and_no_boundaries(op):
    case = ragged_case(lens=[20, 70, 5, 64], H=2, seed=8, inert=(1, 2))
    case["boundaries"] = case["boundary_lens"] = None
    run_and_check(op, case)


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_in_place_shared_and_own_boundary(op):
    """A request may leave its state in its source, or its boundary's; a
    source may serve several requests."""
    case = ragged_case(lens=[70, 30, 66, 128], H=2, seed=9, boundary={1: 10, 3: 100})
    s, d, bnd = case["sources"], case["destinations"], case["boundaries"]
    s[0] = d[0]
    s[1] = bnd[1]
    s[2] = s[3] = case["sources"][3]
    run_and_check(op, case)


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
@pytest.mark.parametrize("H", [1, 5, 16])
def test_heads(op, H):
    run_and_check(op, ragged_case(lens=[40, 100], H=H, seed=20 + H, pool="f32"))


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
@pytest.mark.parametrize("pool", ["f32", "bf16"])
@pytest.mark.parametrize("most", [1, 8, 40])
def test_more_items_than_fit(op, pool, most):
    """Hundreds of (request, head) items: empty, inert, fresh and resumed
    windows of one token, of a group of eight and of several, boundaries."""
    rng = np.random.default_rng(most)
    lens = [int(n) for n in rng.integers(0, most + 1, size=60)]
    lens[:6] = [most, 0, most, min(most, 17), 1, min(most, 16)]
    boundary = {b: max(1, n // 2) for b, n in enumerate(lens) if n > 1 and b % 5 == 0}
    resume = [b for b in range(60) if b % 7 != 3]
    run_and_check(op, ragged_case(lens=lens, H=11, seed=100 + most, pool=pool, boundary=boundary,
                                  inert=(2, 9, 30), resume=resume, tail=2))


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_uniform_windows(op):
    case = ragged_case(lens=[70] * 3, H=2, seed=31)
    d = on_device(case)
    d["query_start_loc"] = None
    call_rule(ops()[op], case, d)
    verify(op, case, d)


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
@pytest.mark.parametrize("null_slot", [-1, 4])
def test_other_null_slots(op, null_slot):
    """Slot 0 is a slot where the null slot is -1; slots up to it are none."""
    case = ragged_case(lens=[70, 3, 100, 20, 50], H=2, seed=25, boundary={2: 66}, resume=(0, 1, 3))
    case["null_slot"] = null_slot
    case["sources"][case["sources"] == 0] = null_slot  # (fresh, none reads slot 0 but its writer)
    case["destinations"][1] = case["sources"][1] = 0
    run_and_check(op, case)


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
@pytest.mark.parametrize("lower_bound", [-10.0, -0.5, 0.0])
def test_gate_bounds(op, lower_bound):
    """The steepest gates (every channel forgetting e^-10 a token), and none."""
    case = ragged_case(lens=[100, 64, 17], H=2, seed=33, lower_bound=lower_bound, memory=2.0)
    if lower_bound == -10.0:
        case["dt_bias"][0] = 4.0
    run_and_check(op, case)


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_mixed_magnitudes(op):
    """Zero keys and queries (normalised by the 1e-6 alone), values from
    1e-20 to 1e20 in different value channels, a state of large entries."""
    case = ragged_case(lens=[90, 64], H=2, seed=35, resume=(0, 1))
    from linear_attention_speculative_recoverssm_gb300 import synth
    case["k"][3] = 0
    case["q"][4] = 0
    f = np.ones(128, dtype=np.float32)
    f[:8] = [1e20, 1e-20, 1e10, 1e-10, 1e5, 1e-5, 7e4, 3e-8]
    from oracle import kda_oracle as ko
    case["v"] = synth.to_bf16_bits((ko.bf16_to_f64(case["v"]) * f).astype(np.float32))
    case["state"] *= f[:, None]
    d = on_device(case)
    call_rule(ops()[op], case, d)
    # a value channel at a time: each within the tolerance of its own scale
    ref = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in case.items()}
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    po.rule(out_f64=f64, sizes=sizes, **ref)
    slack = QUERY * sizes * (op == "prefill")
    got, gs = ko.bf16_to_f64(to_numpy(d["out"])), to_numpy(d["state"])
    for c in list(range(8)) + [100]:
        scale = np.abs(f64[:, :, c]).max()
        assert np.all(np.abs(got[:, :, c] - f64[:, :, c]) <=
                      2.0 ** -8 * np.abs(f64[:, :, c]) + 1e-4 * scale + slack[:, :, c]), c
        r = ref["state"][case["destinations"], :, c].astype(np.float64)
        assert np.all(np.abs(gs[case["destinations"], :, c] - r) <= 1e-4 * np.abs(r).max()), c


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_nan_stays_in_its_request(op):
    """NaN and infinities in one request, in rows behind the last, in an
    unused slot and in an inert request's slots reach no other request."""
    case = ragged_case(lens=[30, 40, 66, 20], H=2, seed=37, inert=(3,), tail=5, resume=(0, 2))
    clean = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in case.items()}
    for name, bits in (("q", 0x7FC0), ("k", 0x7F80), ("v", 0x7FC0), ("raw_g", 0x7FC0),
                       ("raw_beta", 0xFF80)):
        case[name][30:70] = bits   # request 1
        case[name][136:] = 0x7FC0  # the inert request and the tail
    unused = np.setdiff1d(np.arange(case["state"].shape[0]),
                          np.concatenate([case["sources"], case["destinations"]]))
    case["state"][unused] = np.nan
    case["state"][0] = np.nan  # the null slot
    d = on_device(case)
    call_rule(ops()[op], case, d)
    d2 = on_device(clean)
    call_rule(ops()[op], clean, d2)
    got, want = to_numpy(d["out"]), to_numpy(d2["out"])
    for a, b in ((0, 30), (70, 136), (136, 156), (156, 161)):
        np.testing.assert_array_equal(got[a:b], want[a:b])
    for b in (0, 2):
        s = case["destinations"][b]
        np.testing.assert_array_equal(to_numpy(d["state"])[s], to_numpy(d2["state"])[s])


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_reported_requests(op):
    """Windows outside the activations or too long, and slots outside the
    pool: reported, nothing of theirs touched, the others as ever."""
    case = ragged_case(lens=[70, 30, 20, 10], H=2, seed=41)
    case["Q"] = 69  # request 0 is too long
    case["destinations"][2] = case["state"].shape[0]
    case["sources"][3] = case["state"].shape[0] + 7
    d = on_device(case)
    call_rule(ops()[op], case, d)
    verify(op, case, d, bad=3)
    assert int(d["status"][0]) == -1
    case = ragged_case(lens=[10, 30], H=2, seed=42)
    case["query_start_loc"][2] = 41  # past the last token
    d = on_device(case)
    call_rule(ops()[op], case, d)
    verify(op, case, d, bad=1)


def test_prefill_and_recurrent_agree_when_continued():
    """A prompt in one call, and in three that go on from one another."""
    import torch
    case = ragged_case(lens=[300], H=2, seed=43, resume=())
    d = on_device(case)
    call_rule(ops()["prefill"], case, d)
    whole, whole_state = to_numpy(d["out"]), to_numpy(d["state"])[case["destinations"][0]]
    e = on_device(case)
    outs, at = [], 0
    for i, (n, op) in enumerate([(130, "prefill"), (1, "recurrent"), (169, "prefill")]):
        part = dict(e)
        for name in ("q", "k", "v", "raw_g", "raw_beta"):
            part[name] = e[name][at:at + n].contiguous()
        part["out"] = torch.zeros((n, 2, 128), dtype=torch.bfloat16, device="cuda")
        part["query_start_loc"] = to_torch(np.array([0, n], dtype=np.int32), "cuda")
        part["sources"] = e["sources"] if i == 0 else e["destinations"]
        call_rule(ops()[op], case, part)
        outs.append(to_numpy(part["out"]))
        at += n
    from oracle import kda_oracle as ko
    a, b = ko.bf16_to_f64(np.concatenate(outs)), ko.bf16_to_f64(whole)
    # two BF16 roundings of values that are REL and QUERY apart, each side
    f64, sizes = np.zeros(case["v"].shape), np.zeros(case["v"].shape)
    ref = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in case.items()}
    po.rule(out_f64=f64, sizes=sizes, **ref)
    assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 2e-4 * np.abs(b).max() +
                  2 * QUERY * sizes)
    got = to_numpy(e["state"])[case["destinations"][0]]
    assert np.abs(got - whole_state).max() <= 2e-4 * np.abs(whole_state).max()


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_graph_streams_and_repeats(op):
    """Captured and replayed on another stream with other inputs in the same
    buffers: bit for bit what eager calls give; the same call twice too."""
    import torch
    lens = [70, 1, 130]
    cases = [ragged_case(lens=lens, H=2, seed=s, boundary={0: 33}) for s in (51, 52)]
    for c in cases[1:]:
        for name in ("sources", "destinations", "boundaries"):
            c[name] = cases[0][name]
    eager = []
    for c in cases:
        d = on_device(c)
        call_rule(ops()[op], c, d)
        eager.append((to_numpy(d["out"]), to_numpy(d["state"])))
        d = on_device(c)
        call_rule(ops()[op], c, d)
        np.testing.assert_array_equal(eager[-1][0], to_numpy(d["out"]))
        np.testing.assert_array_equal(eager[-1][1], to_numpy(d["state"]))
    d = on_device(cases[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call_rule(ops()[op], cases[0], d)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call_rule(ops()[op], cases[0], d)
    for c, (out, state) in zip(cases, eager):
        fresh = on_device(c)
        for name in d:
            d[name].copy_(fresh[name])
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out, to_numpy(d["out"]))
        np.testing.assert_array_equal(state, to_numpy(d["state"]))


def test_two_prefills_at_once():
    """Two calls on two streams, each with its own workspace, at the same
    time: each as if alone."""
    import torch
    cases = [ragged_case(lens=[300, 200], H=4, seed=s) for s in (61, 62)]
    ds = [on_device(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for c, d, s in zip(cases, ds, streams):
            call_rule(ops()["prefill"], c, d, stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cases, ds):
        verify("prefill", c, d)


def test_strided_pool():
    """Slots further apart than their size, in a pool that is a part of a
    larger tensor."""
    import torch
    for op in ("prefill", "recurrent"):
        case = ragged_case(lens=[66, 5], H=2, seed=71)
        d = on_device(case)
        wide = torch.zeros((case["state"].shape[0], 3, 128, 128), device="cuda")
        wide[:, :2] = d["state"]
        d["state"] = wide[:, :2]
        call_rule(ops()[op], case, d)
        assert not bool(wide[:, 2].any())
        d["state"] = d["state"].contiguous()
        verify(op, case, d)


def long_case(lens, H, seed, pool="f32", **kw):
    # (what a state remembers stays under 50 tokens, as in the other cases)
    return ragged_case(lens=lens, H=H, seed=seed, pool=pool, **kw)


@pytest.mark.parametrize("pool", ["f32", "bf16"])
@pytest.mark.parametrize("lens,boundary", [
    ([4096], {}), ([4097], {0: 1}), ([4200], {0: 4199}), ([6000], {0: 2048}), ([6000], {0: 2049}),
    ([4500, 0, 9, 5, 130, 4096], {0: 64 * 35, 3: 2, 4: 100}), ([64 * 33, 64 * 65], {1: 64 * 32 + 1})])
def test_long_prompts(pool, lens, boundary):
    """Prompts of 64 chunks and more, few heads: the form that works by
    segments, boundaries in a segment and at its edges, short and empty
    requests beside the long ones."""
    run_and_check("prefill", long_case(lens, 2, seed=sum(lens), pool=pool, boundary=boundary,
                                       inert=(5,) if len(lens) > 5 and pool == "bf16" else (),
                                       resume=(0, 3, 4), tail=3))


def test_long_prompt_many_heads():
    """More (request, head) items than the segments' form takes."""
    run_and_check("prefill", long_case([4100], 77, seed=77, boundary={0: 70}))


@pytest.mark.parametrize("n", [1, 5, 8, 9, 40, 41, 64])
@pytest.mark.parametrize("most", [0, 5000])
@pytest.mark.parametrize("inert", [(), (0,)])
def test_one_request(n, most, inert):
    """A single request, its window far below the longest allowed too."""
    case = ragged_case(lens=[n], H=3, seed=n, inert=inert, boundary={0: max(1, n - 1)}, resume=(0,),
                       tail=50 if most else 0)
    case["Q"] = max(n, most)
    run_and_check("prefill", case)


def test_graphs_share_a_workspace():
    """Two captured calls of different shapes on one workspace, replayed in
    turn and again, beside eager calls on it: each as if alone."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill_workspace_bytes
    cases = [long_case([4300], 2, seed=81, boundary={0: 77}),
             ragged_case(lens=[70, 1, 130, 20], H=5, seed=82, boundary={2: 33})]
    need = max(kda_prefill_workspace_bytes(len(c["v"]), len(c["destinations"]), c["v"].shape[1])
               for c in cases)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    ds, graphs = [on_device(c) for c in cases], []
    for c, d in zip(cases, ds):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            call_rule(ops()["prefill"], c, d, workspace=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0):
        fresh = on_device(cases[i])
        for name in fresh:
            ds[i][name].copy_(fresh[name])
        graphs[i].replay()
        other = on_device(cases[1 - i])
        call_rule(ops()["prefill"], cases[1 - i], other, workspace=ws)
        torch.cuda.synchronize()
        verify("prefill", cases[i], ds[i])
        verify("prefill", cases[1 - i], other)


@pytest.mark.parametrize("again", [2, 40])
@pytest.mark.parametrize("n", [640, 4200])
def test_offsets_that_go_back(n, again):
    """Offsets 0, n, 0, n, ..: every second window is negative, and the others
    together ask for more chunks than the tokens have.  All that does not fit
    is reported and left out; nothing else is touched."""
    import torch
    B = 2 * again + 1
    case = ragged_case(lens=[n] + [0] * (B - 1), H=2, seed=n + again, resume=(0,), tail=3)
    case["query_start_loc"] = np.array([0, n] * (again + 1), dtype=np.int32)
    d = on_device(case)
    call_rule(ops()["prefill"], case, d)
    torch.cuda.synchronize()
    assert int(d["status"][0]) != 0
    state, dst = to_numpy(d["state"]), case["destinations"]
    spared = np.ones(len(state), dtype=bool)
    spared[dst[::2]] = False
    np.testing.assert_array_equal(state[spared], case["state"][spared])
    np.testing.assert_array_equal(to_numpy(d["out"])[n:], case["out"][n:])
    if n == 640:  # one segment: the first request is served, the one too many is not
        # (the outputs' rows are several requests', in no order)
        one = ragged_case(lens=[n], H=2, seed=1)
        for name in ("q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias", "state", "out"):
            one[name] = case[name]
        for name in ("sources", "destinations"):
            one[name] = case[name][:1]
        alone = on_device(one)
        call_rule(ops()["prefill"], one, alone)
        np.testing.assert_array_equal(state[dst[0]], to_numpy(alone["state"])[dst[0]])
        np.testing.assert_array_equal(state[dst[-1]], case["state"][dst[-1]])


@pytest.mark.parametrize("op", ["prefill", "recurrent"])
def test_slots_far_apart(op):
    """Slots more than 2^31 elements apart: as in a pool without gaps."""
    import torch
    case = ragged_case(lens=[70, 30], H=2, seed=95, pool="bf16", slots=9, resume=(1,),
                       boundary={1: 20})
    case["sources"], case["destinations"] = np.array([0, 1], np.int32), np.array([2, 1], np.int32)
    case["boundaries"] = np.array([0, 3], np.int32)
    case["state"] = case["state"][:4]
    d = on_device(case)
    step = 2 ** 31 + 512
    far = torch.empty(3 * step + 2 * 128 * 128, dtype=torch.bfloat16, device="cuda")
    far = far.as_strided((4, 2, 128, 128), (step, 128 * 128, 128, 1))
    far.copy_(d["state"])
    near, d["state"] = d["state"], far
    call_rule(ops()[op], case, d)
    d["state"] = far.contiguous()
    del far
    verify(op, case, d)


def test_very_long_prompt():
    """Hundreds of chunks, many segments."""
    run_and_check("prefill", ragged_case(lens=[33000, 700], H=1, seed=98, boundary={0: 32897},
                                         resume=(1,), tail=1))
