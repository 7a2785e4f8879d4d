"""The tree operators where calls meet and sizes end: two streams at once,
captured graphs whose windows change between replays, batches of many empty,
inert and bad requests, hundreds of heads, rows and slots beyond 32 bits,
infinite gates, the same node twice in a path.  Against the oracles, with the
tolerances of the operators' own tests."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib

import test_gpu_draft_accept as ta
import test_gpu_tree as tg
import tree_testutil as tt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import _build
    assert torch.cuda.is_available()
    _build.build()
    _lib.load()


def trees_of(seed, sizes):
    rng = np.random.default_rng(seed)
    return [tt.random_tree(rng, n) if n else [] for n in sizes]


def fill(d, case):
    """The case's values into the tensors that are there."""
    fresh = tt.on_device(case)
    for n in fresh:
        if fresh[n] is not None:
            d[n].copy_(fresh[n])


def test_two_streams_at_once():
    """Every operator on two streams, other sizes on each, many times over:
    nothing is shared between them."""
    import torch
    rng = np.random.default_rng(1)
    sides = [torch.cuda.Stream() for _ in range(2)]
    sizes = [rng.integers(40, 65, 30), rng.integers(7, 33, 50)]
    verify = [tt.tree_case(trees_of(s, sizes[s]), 16, seed=60 + s, pending=0) for s in range(2)]
    select = [tg.select_case(trees_of(s, sizes[1 - s]), 9 + s, 62 + s, pending=0) for s in range(2)]
    accept = [ta.accept_case(trees_of(s, sizes[s]), 3001 + s, seed=64 + s) for s in range(2)]
    dv, dc, ds, da = ([tt.on_device(c) for c in cases] for cases in (verify, select, select, accept))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, side in enumerate(sides):
            with torch.cuda.stream(side):
                tg.run_verify(verify[s], dv[s], stream=side)
                tg.run_conv(select[s], dc[s], stream=side)
                ta.run_accept(accept[s], da[s], stream=side)
                tg.run_select(select[s], dc[s], windows=False, stream=side)
    for s, side in enumerate(sides):
        with torch.cuda.stream(side):
            tg.run_select(select[s], ds[s], stream=side)
    torch.cuda.synchronize()
    for s in range(2):
        tg.check_verify(verify[s], dv[s])
        tg.check_conv(select[s], dc[s])
        tg.check_select(select[s], dc[s], windows=False)
        tg.check_select(select[s], ds[s])
        ta.check_accept(accept[s], da[s])


@pytest.mark.parametrize("cap,pool", [(64, "f32"), (64, "bf16"), (32, "bf16"), (32, "f32"), (6, "f32")])
def test_a_graph_whose_windows_change(cap, pool):
    """One capture for up to `cap` nodes a request and a padded batch; replays
    with other trees, fewer tokens, requests gone empty or inert."""
    import torch
    H, B, rows = 3, 7, 7 * cap
    sizes = [[cap] * B, [1, 0, cap, cap // 2, 3, 0, 2], [0, 0, 0, 0, 0, 0, 5]]
    cases = []
    for s, lens in enumerate(sizes):
        kw = dict(tail=rows - sum(lens), inert=(2,) if s else (), pending=None)
        v = tt.tree_case(trees_of(s, lens), H, seed=70 + s, pool=pool, replay=pool == "f32", **kw)
        c = tg.select_case(trees_of(s, lens), H, 73 + s, **kw)
        a = ta.accept_case(trees_of(s, lens), 600, seed=76 + s, tail=rows - sum(lens))
        a["state_slots"] = v["state_slots"]
        for x in (v, c, a):
            x["Q"] = cap
        cases.append((v, c, a))
    d = [tt.on_device(c) for c in cases[0]]
    runs = (tg.run_verify, tg.run_conv, ta.run_accept)
    for run, case, on in zip(runs, cases[0], d):  # (their outputs are allocated)
        run(case, on)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tg.run_verify(cases[0][0], d[0])
        tg.run_conv(cases[0][1], d[1])
        ta.run_accept(cases[0][2], d[2])
        tg.run_select(cases[0][1], d[1])
    for (v, c, a) in cases[::-1] + cases:
        for on, case in zip(d, (v, c, a)):
            fill(on, case)
        graph.replay()
        torch.cuda.synchronize()
        tg.check_verify(v, d[0])
        tg.check_select(c, d[1])
        ta.check_accept(a, d[2])


@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("cap", [6, 20, 40])
def test_many_requests_of_every_kind(cap, H):
    """Empty windows with and without a replay, inert, rowless and bad
    requests among live ones, many to a CTA."""
    rng = np.random.default_rng(cap)
    B = 1100
    sizes = np.where(rng.random(B) < 0.6, 0, rng.integers(1, cap + 1, B))
    trees = trees_of(cap, sizes)
    inert, rowless = rng.permutation(B)[:300], rng.permutation(B)[:200]
    case = tg.select_case(trees, H, 80, inert=set(inert), rowless=set(rowless))
    case["node_corr"][:] = 123.0
    starts, live = case["query_start_loc"], case["state_slots"] > 0
    bad = [b for b in rng.permutation(B) if live[b] and sizes[b] > 1][:20]
    for b in bad:
        case["parents"][starts[b] + sizes[b] - 1] = sizes[b] - 1
    tg.check_verify(case, tg.run_verify(case), bad=len(bad))
    tg.check_conv(case, tg.run_conv(case), bad=len(bad))
    tg.check_select(case, tg.run_select(case))  # (goes by paths, not by parents)


@pytest.mark.parametrize("B,H,n", [(2, 700, 9), (1, 1024, 5), (2, 333, 34)])
def test_many_heads(B, H, n):
    case = tg.select_case(trees_of(n, [n, max(1, n - 3)][:B]), H, 81, rq=4)
    case["node_corr"][:] = 123.0
    tg.check_verify(case, tg.run_verify(case))
    tg.check_conv(case, tg.run_conv(case))
    tg.check_select(case, tg.run_select(case))


@pytest.mark.parametrize("n", [5, 12, 40])
def test_infinite_gates(n):
    """Gates and betas of both infinities: decays of 1 and e^lower_bound, a
    token that writes nothing or all."""
    case = tt.tree_case(trees_of(n, [n] * 40), 3, seed=82, pending=3)
    rng = np.random.default_rng(82)
    for name in ("raw_g", "raw_beta", "key_gate"):
        x = case[name] if name != "key_gate" else case[name][..., 128:]
        x[rng.random(x.shape) < 0.02] = 0x7F80
        x[rng.random(x.shape) < 0.02] = 0xFF80
    with np.errstate(over="ignore"):
        tg.check_verify(case, tg.run_verify(case))


@pytest.mark.parametrize("n", [6, 20, 64])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_state_row_that_is_not_finite(value, n):
    """It reaches its own output channel, and no other, of its head alone."""
    import torch
    case = tt.tree_case(trees_of(n, [n] * 4), 2, seed=83, pending=0)
    d = tg.run_verify(case)
    spoilt = tt.copy_case(case)
    spoilt["state"][case["state_slots"][1], 1, 77, 5] = value
    e = tg.run_verify(spoilt)
    for name in ("out", "node_corr"):
        got, want = e[name].float(), d[name].float()
        hit = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
        hit[n:2 * n, 1, 77] = True
        assert not torch.isfinite(got[hit]).any()
        assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("cap", [6, 20, 64])
@pytest.mark.parametrize("pool", ["f32", "bf16"])
def test_fewer_tokens_than_a_window_may_hold(pool, cap):
    """One token, and three in two requests, where windows may hold `cap`."""
    for sizes in ([1], [2, 0, 1]):
        case = tt.tree_case(trees_of(2, sizes), 2, seed=92, pool=pool, replay=pool == "f32")
        case["Q"] = cap
        tg.check_verify(case, tg.run_verify(case))
        tg.check_conv(case, tg.run_conv(case))


def test_rows_behind_the_last_hold_anything():
    """NaN in every row that belongs to no request, in slots and rows that
    none has, and between strides."""
    import torch
    case = tg.select_case(trees_of(9, [9, 30, 4]), 2, 84, tail=5)
    case["node_corr"][:] = 123.0
    for name in ("q", "k", "v", "raw_g", "raw_beta", "x"):
        case[name][-5:] = 0x7FC0
    for b in range(len(case["state"])):
        if b not in case["state_slots"]:
            case["state"][b], case["conv_state"][b] = np.nan, 0x7FC0
    for r in range(len(case["corr"])):
        if r not in case["record_rows"]:
            case["corr"][r], case["key_gate"][r] = np.nan, 0x7FC0
        else:  # behind the count
            n = max(0, int(case["pending"][r]))
            case["corr"][r, :, n:], case["key_gate"][r, :, n:] = np.nan, 0x7FC0
    d = tg.run_conv(case)
    tg.check_conv(case, d)
    live = np.isin(np.arange(len(case["state"])), case["state_slots"])
    d = tg.run_verify(case)
    got = tt.to_numpy(d["state"])
    assert np.isnan(got[~live]).all() and np.isfinite(got[live]).all()
    assert np.isfinite(tt.to_numpy(d["node_corr"])).all()
    clean = tt.copy_case(case)
    clean["state"][~live] = 0
    for name in ("corr", "key_gate"):
        clean[name][np.isnan(case["corr"]).any(-1)] = 0
    tg.check_verify(clean, tg.run_verify(clean))
    e = tg.run_verify(clean)
    for name in ("out", "node_corr"):
        assert torch.equal(d[name], e[name])


def test_accept_rows_beyond_32_bits():
    """Weights of more than 2^31 elements; windows that begin far from the
    first row."""
    import torch
    V, T = 1 << 20, 2100
    case = ta.accept_case(trees_of(3, [10, 40, 9]), 500, seed=85)
    n = len(case["tokens"])
    target = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    at = 700_000
    small = torch.from_numpy(case["target"]).cuda().to(torch.bfloat16)
    target[T - n:, at:at + 500] = small
    d = tt.on_device(case)
    pad = lambda x, v: torch.cat([torch.full((T - n,), v, dtype=x.dtype, device="cuda"), x])
    d["target"], d["tokens"] = target, pad(d["tokens"] + at, -9)
    d["parents"], d["accept_uniforms"] = pad(d["parents"], 99), pad(d["accept_uniforms"], 0.5)
    d["query_start_loc"] = d["query_start_loc"] + (T - n)
    ta.run_accept(case, d)
    case["target"] = tt.to_numpy(small)
    d["next"] -= at
    ta.check_accept(case, d)


def test_windows_beyond_32_bits():
    """Convolution windows further than 2^31 elements from the pool's start."""
    import torch
    case = tg.select_case(trees_of(4, [9, 12, 3]), 2, 86, extra_slots=0)
    d = tt.on_device(case)
    shape, stride = d["conv_state"].shape, 2 ** 30 + 8
    pool = torch.zeros(3 * stride + shape[1] * shape[2], dtype=torch.bfloat16, device="cuda")
    far = pool.as_strided(shape, (stride, shape[2], 1))
    far.copy_(d["conv_state"])
    d["conv_state"] = far
    tg.run_conv(case, d)
    tg.check_conv(case, d)
    tg.run_select(case, d)
    tg.check_select(case, d)


@pytest.mark.parametrize("rq,width", [(4, 10), (8, 5), (1, 10), (8, 3), (3, 4)])
def test_windows_of_another_length_than_the_records(rq, width):
    """Records of rq tokens beside windows of width - 2: each keeps its own
    layout, and a path fits both or is reported."""
    case = tg.select_case([tt.chain(8), tt.comb(20), tt.star(5), tt.chain(2)], 3, 91, rq=rq)
    rng = np.random.default_rng(91)
    case["conv_state"] = rng.integers(0x3F00, 0x4000, case["conv_state"].shape[:2] + (width,)).astype(np.uint16)
    too_long = int(((case["accepted"] > width - 2) & (case["state_slots"] > 0)).sum())
    tg.check_conv(case, tg.run_conv(case))
    tg.check_select(case, tg.run_select(case), bad=too_long)


def test_select_the_same_node_twice():
    """A path is what it says, a tree's or not."""
    case = tg.select_case([tt.star(9), tt.chain(4), tt.comb(64)], 2, 87)
    case["path"][:, :5] = [[3, 3, 0, 3, 8], [0, 0, 0, 0, 1], [63, 2, 2, 63, 7]]
    case["accepted"][:] = [5, 4, 5]
    tg.check_select(case, tg.run_select(case))


def test_every_slot_is_live_below_the_null_slot():
    """null_slot -1: slot 0 is a request's; 4: slots up to 4 are none's."""
    for null in (-1, 4):
        case = tg.select_case(trees_of(5, [7, 12, 3, 20, 9, 9]), 2, 88)
        case["node_corr"][:] = 123.0
        case["null_slot"] = null
        case["state_slots"][:] = [0, 5, 2, 6, 4, 1]
        tg.check_conv(case, tg.run_conv(case))
        tg.check_verify(case, tg.run_verify(case))
        tg.check_select(case, tg.run_select(case))


@pytest.mark.parametrize("probs", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["drafts", "trees"])
def test_accept_many_requests(kind, probs):
    """More than run at once, of a small vocabulary and of a larger one."""
    rng = np.random.default_rng(6)
    for B, V in ((3000, 5), (700, 777)):
        if kind == "drafts":
            trees = [tt.chain(int(n)) for n in rng.integers(0, 9, B)]
            case = ta.accept_case(trees, V, seed=89, probs=probs, draft=True, chains=True)
        else:
            trees = trees_of(7, rng.integers(0, 12, B))
            case = ta.accept_case(trees, V, seed=90, probs=probs)
        ta.check_accept(case, ta.run_accept(case))
