"""A step of trees in which one request cannot be served: what the calls in
their order leave of it, and of the requests beside it.

Every test runs two arms of the same steps, bit for bit the same inputs.  In
one the last request's tree, window, slot, row, tokens or path is spoilt for a
step; in the other the same request sits that step out (an inert slot: its
replay stays pending and its window where it is), or has no drafts in it (an
empty window: its replay is folded in, nothing is accepted).  Items are worked
out independently of one another, so all that the steps leave is equal bit for
bit."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib, synth

import tree_testutil as tt

pytestmark = pytest.mark.gpu

H, V = 2, 80
D = H * 128


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import _build
    assert torch.cuda.is_available()
    _build.build()
    _lib.load()


class Arm:
    """Four requests' slots, records and windows, and the loop over them."""

    def __init__(self, rq, width):
        from linear_attention_speculative_recoverssm_gb300 import DeferredRecoverSSM
        rng = np.random.default_rng(7)
        f32 = lambda *s, std=1.0: (rng.standard_normal(s) * std).astype(np.float32)
        bits = lambda *s, std=1.0: synth.to_bf16_bits(f32(*s, std=std))
        host = dict(state=f32(7, H, 128, 128, std=0.1), conv=bits(7, 3 * D, width),
                    w=bits(3, 4, D, std=0.5), A=rng.uniform(0, 1.5, H).astype(np.float32),
                    dt=f32(H, 128) - 2, slots=np.array([3, 1, 5, 2], np.int32),
                    rows=np.array([2, 0, 4, 1], np.int32), pending=np.zeros(5, np.int32),
                    corr=f32(5, H, rq, 128), kg=bits(5, H, rq, 256), status=np.zeros(1, np.int32))
        self.d = {n: tt.to_torch(a, "cuda") for n, a in host.items()}
        d = self.d
        self.loop = DeferredRecoverSSM(d["state"], d["slots"], d["rows"], d["pending"], d["corr"],
                                       d["kg"], d["A"], d["dt"], Q=rq, lower_bound=-5.0,
                                       q_scale=128 ** -0.5, status=d["status"])

    def step(self, seed, trees, *, spoil=None, eager=None, windows=True):
        """One step; `spoil` says what is wrong with the last request ("inert"
        and "empty" among it).  Everything that the step leaves."""
        import torch
        from linear_attention_speculative_recoverssm_gb300 import kda_draft_accept, kda_tree_conv
        d, B, T = self.d, len(trees), sum(map(len, trees))
        rng = np.random.default_rng(seed)
        bits = lambda *s: synth.to_bf16_bits(rng.standard_normal(s).astype(np.float32))
        x, g, beta = bits(T, 3 * D), bits(T, H, 128), bits(T, H)
        par, starts = tt.packed(trees), tt.starts_of(trees)
        # a token of its own for every node; the target likes its children: rows
        # that sum to one, nine parts in ten on them
        tokens = np.concatenate([np.arange(len(t)) for t in trees]).astype(np.int32)
        target = rng.dirichlet(np.full(V, 0.5), T)
        for b, tree in enumerate(trees):
            for a in range(len(tree)):
                kids = [t for t, up in enumerate(tree) if up == a]
                if kids:
                    target[starts[b] + a] *= 0.1
                    target[starts[b] + a, kids] += 0.9 / len(kids)
        u, un = rng.random(T).astype(np.float32) * 0.9, rng.random(B).astype(np.float32)
        Q, t0 = max(map(len, trees)), starts[-2]
        slots, rows = d["slots"].clone(), d["rows"].clone()
        if spoil == "inert":
            d["slots"][-1] = 0
        elif spoil == "empty":
            starts[-1] = t0
        elif spoil == "window":
            starts[-1] = T + 1
        elif spoil == "tree":
            par[t0 + 2] = 2
        elif spoil == "deep":
            par[t0:t0 + 9] = np.arange(-1, 8)
        elif spoil == "slot":
            d["slots"][-1] = d["state"].shape[0]
        elif spoil == "row":
            d["rows"][-1] = d["corr"].shape[0]
        elif spoil == "token":
            tokens[t0 + 1] = V
        dev = lambda a: tt.to_torch(a, "cuda")
        x, g, par = dev(x), dev(g), dev(par)
        q, k, v, out = (torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4))
        node_corr = torch.zeros((T, H, 128), device="cuda")
        accepted, nxt = torch.zeros((2, B), dtype=torch.int32, device="cuda")
        path = torch.zeros((B, 8), dtype=torch.int32, device="cuda")
        common = dict(Q=Q, query_start_loc=dev(starts))
        kda_tree_conv(x, d["w"], None, d["conv"], d["slots"], par, q, k, v, record_rows=d["rows"],
                      pending=d["pending"], status=d["status"], **common)
        self.loop.verify_tree(q, k, v, g, dev(beta), par, node_corr, out, **common)
        kda_draft_accept(dev(target.astype(np.float32)), dev(tokens), dev(u), dev(un), accepted, path,
                         nxt, parents=par, state_slots=d["slots"], status=d["status"], **common)
        if spoil == "path":
            path[-1, 1] = len(trees[-1])
        elif spoil == "negative":
            accepted[-1] = -3
        count = accepted.clone()
        wins = dict(x=x, conv_state=d["conv"]) if windows else {}
        self.accept(path, accepted, k, g, node_corr, par, eager=eager, **wins, **common)
        status = int(d["status"].item())
        assert status == (0 if spoil in (None, "inert", "empty") else _lib.KDA_ERR_ARG)
        d["status"].zero_()
        d["slots"].copy_(slots)
        d["rows"].copy_(rows)
        left = {n: d[n].clone() for n in ("state", "conv", "pending", "corr", "kg")}
        return dict(left, out=out[:t0], count=count, accepted=accepted, node_corr=node_corr[:t0])

    def accept(self, path, accepted, k, g, node_corr, par, *, eager, **kw):
        if eager is not None:
            eager = tt.to_torch(np.array(eager, np.uint8), "cuda")
        self.loop.accept_tree(path, accepted, k, g, node_corr, eager=eager, **kw)


def same(a, b, names):
    import torch
    for n in names:
        assert torch.equal(a[n], b[n]), n


LEFT = ("state", "conv", "pending", "corr", "kg", "out", "node_corr")


def two_arms(spoil, instead, trees, *, rq=8, width=10, flushed=False, eager=None, windows=True, arm=Arm):
    """A good step, the spoilt one (`instead` in the other arm), a good one and
    a flush; the state of the spoilt arm's middle step."""
    good = [tt.comb(7) if min(rq, width - 2) == 8 else tt.star(7), tt.chain(3), tt.star(6), tt.chain(4)]
    arms = [arm(rq, width), arm(rq, width)]
    first = [a.step(1, good, windows=windows) for a in arms]
    same(*first, LEFT)
    before = int(arms[0].d["pending"][1])  # the last request's row
    assert before > 0
    if flushed:
        for a in arms:
            a.loop.flush()
    middle = [a.step(2, trees, spoil=s, eager=eager, windows=windows)
              for a, s in zip(arms, (spoil, instead))]
    same(*middle, LEFT)
    assert int(middle[0]["pending"][1]) == (before if instead == "inert" else 0)
    last = [a.step(3, good, windows=windows) for a in arms]
    same(*last, LEFT + ("count",))
    for a in arms:
        a.loop.flush()
    same(arms[0].d, arms[1].d, ("state",))
    return middle[0]


LARGE = [tt.comb(11), tt.star(5), tt.chain(8), tt.comb(12)]
SMALL = [tt.comb(6), tt.star(5), tt.chain(4), tt.chain(5)]


@pytest.mark.parametrize("eager", [None, [0, 1, 0, 1]])
@pytest.mark.parametrize("trees,spoil", [(LARGE, "tree"), (SMALL, "tree"), (LARGE, "deep"),
                                         (LARGE, "window"), (SMALL, "window"), (LARGE, "slot"),
                                         (LARGE, "row")])
def test_what_verify_reports_stays_pending(trees, spoil, eager):
    """The tokens accepted before are not lost: the replay waits for the next
    step, and the window with it."""
    left = two_arms(spoil, "inert", trees, eager=eager)
    assert int(left["accepted"][-1]) == 0


@pytest.mark.parametrize("trees,spoil", [(LARGE, "tree"), (SMALL, "tree"), (LARGE, "deep"),
                                         (LARGE, "window"), (SMALL, "window")])
def test_behind_a_flush_nothing_is_pending(trees, spoil):
    """The replay was folded in by the flush: it must not be folded in twice."""
    two_arms(spoil, "empty", trees, flushed=True)


@pytest.mark.parametrize("flushed", [False, True])
def test_what_the_acceptance_alone_reports_is_as_empty(flushed):
    """A token outside the vocabulary: the rule was served, and the replay with
    it."""
    two_arms("token", "empty", LARGE, flushed=flushed)


DEEP = [tt.star(11), tt.star(5), tt.chain(3), tt.chain(8)]
FLAT = [tt.star(6), tt.star(5), tt.chain(3), tt.chain(5)]


@pytest.mark.parametrize("flushed,eager", [(False, None), (False, [0, 1, 0, 1]), (True, None)])
@pytest.mark.parametrize("trees,spoil,rq,width,windows", [
    (DEEP, "count", 4, 6, True),    # a path of eight tokens, records of four
    (FLAT, "count", 4, 6, True),
    (DEEP, "count", 8, 6, True),    # windows of four
    (DEEP, "count", 4, 10, True),
    (DEEP, "count", 4, 10, False),  # records alone
    (LARGE, "path", 8, 10, True),   # a node outside the window
    (LARGE, "negative", 8, 10, True),
])
def test_a_path_that_does_not_fit(trees, spoil, rq, width, windows, flushed, eager):
    """The replay before it was folded in, and nothing else is: no record of an
    earlier step is replayed in its place."""
    left = two_arms(spoil, "empty", trees, rq=rq, width=width, windows=windows, flushed=flushed,
                    eager=eager)
    assert int(left["accepted"][-1]) == 0
    if spoil == "count":
        assert int(left["count"][-1]) == len(trees[-1])


class Calls(Arm):
    """The same step by the library's calls."""

    def __init__(self, rq, width):
        super().__init__(rq, width)
        self.loop.verify_tree = self.verify

    def verify(self, q, k, v, g, beta, par, node_corr, out, **common):
        from linear_attention_speculative_recoverssm_gb300 import kda_tree_verify
        d = self.d
        kda_tree_verify(q, k, v, g, beta, d["A"], d["dt"], d["state"], d["slots"], par, node_corr, out,
                        lower_bound=-5.0, q_scale=128 ** -0.5, record_rows=d["rows"],
                        pending=d["pending"], corr=d["corr"], key_gate=d["kg"], status=d["status"],
                        **common)

    def accept(self, path, accepted, k, g, node_corr, par, *, eager, **common):
        import torch
        from linear_attention_speculative_recoverssm_gb300 import (kda_defer_commit, kda_tree_select,
                                                                   kda_tree_settle)
        d, status = self.d, dict(status=self.d["status"])
        rows, plan = torch.empty_like(d["rows"]), accepted.clone()
        window = {n: common[n] for n in ("Q", "query_start_loc")}
        most = min(d["corr"].shape[2], d["conv"].shape[2] - 2)
        kda_tree_settle(d["slots"], d["rows"], rows, path=path, accepted=accepted, most=most, parents=par,
                        n_tokens=len(par), n_slots=len(d["state"]), n_rows=len(d["corr"]), **window,
                        **status)
        kda_tree_select(path, accepted, k, g, node_corr, d["slots"], rows, d["corr"], d["kg"],
                        pending=d["pending"], **common, **status)
        plan.copy_(accepted)
        kda_defer_commit(d["slots"], plan, rows, d["pending"], **status)


@pytest.mark.parametrize("spoil,instead,trees,rq", [
    ("tree", "inert", LARGE, 8), ("window", "inert", LARGE, 8), ("slot", "inert", LARGE, 8),
    ("token", "empty", LARGE, 8), ("path", "empty", LARGE, 8), ("count", "empty", DEEP, 4)])
def test_by_the_calls(spoil, instead, trees, rq):
    left = two_arms(spoil, instead, trees, rq=rq, arm=Calls)
    assert int(left["accepted"][-1]) == 0


def test_select_moves_the_window_of_a_bad_one():
    """Nothing accepted and a bad window of tokens: reported, the convolution's
    window moved; a bad slot or row, or a count above zero: left alone."""
    import test_gpu_tree as tg
    case = tg.select_case([tt.chain(4)] * 6, 2, 60)
    case["accepted"][:] = [0, 2, 0, 0, 0, 1]
    case["query_start_loc"] = np.array([0, 70, 4, 8, 12, 16, 20], np.int32)  # 0 and 1 are bad
    case["state_slots"][2], case["record_rows"][3] = len(case["conv_state"]), len(case["corr"])
    case["state_slots"][4] = 0
    d = tg.run_select(case)
    assert tt.to_numpy(d["status"])[0] == _lib.KDA_ERR_ARG
    want, slot = case["conv_state"].copy(), case["state_slots"][0]
    n = max(0, int(case["pending"][case["record_rows"][0]]))
    off = n - 1 if n > 0 else 0
    want[slot, :, :3] = case["conv_state"][slot, :, off:off + 3]
    slot, row, t = case["state_slots"][5], case["record_rows"][5], 16 + case["path"][5, 0]
    n = max(0, int(case["pending"][row]))
    off = n - 1 if n > 0 else 0
    want[slot, :, :2] = case["conv_state"][slot, :, off + 1:off + 3]
    want[slot, :, 2] = case["x"][t]
    corr = case["corr"].copy()
    corr[row, :, 0] = case["node_corr"][t]
    np.testing.assert_array_equal(tt.to_numpy(d["conv_state"]), want)
    np.testing.assert_array_equal(tt.to_numpy(d["corr"]), corr)


def loop_over(d):
    from linear_attention_speculative_recoverssm_gb300 import DeferredRecoverSSM
    return DeferredRecoverSSM(d["state"], d["state_slots"], d["record_rows"], d["pending"], d["corr"],
                              d["key_gate"], d["A_log"], d["dt_bias"], Q=8, lower_bound=-5.0,
                              q_scale=128 ** -0.5, status=d["status"])


PER_STEP = ("q", "k", "v", "raw_g", "raw_beta", "parents", "path", "accepted", "x")


def one_step(loop, d, raw=False):
    kw = dict(Q=12)
    if raw:  # (the rule by the library's call)
        tt.call_verify(dict(lower_bound=-5.0, q_scale=128 ** -0.5, null_slot=0, Q=12), d)
    else:
        loop.verify_tree(d["q"], d["k"], d["v"], d["raw_g"], d["raw_beta"], d["parents"],
                         d["node_corr"], d["out"], **kw)
    loop.accept_tree(d["path"], d["accepted"], d["k"], d["raw_g"], d["node_corr"], x=d["x"],
                     conv_state=d["conv_state"], **kw)


def captured_cases():
    import test_gpu_tree as tg
    cases = []
    for seed in range(4):
        rng = np.random.default_rng(seed)
        case = tg.select_case([tt.random_tree(rng, 12) for _ in range(5)], 2, 90 + seed, inert=(1,))
        if seed % 2:  # (every other step; with a count that a caller made)
            case["parents"][2 * 12 + 5] = 5
            case["accepted"][3] = 9
        case["query_start_loc"] = None
        cases.append(case)
    return cases


@pytest.mark.parametrize("how", ["graph", "two graphs", "stream"])
def test_a_captured_step_settles_its_own_requests(how):
    """A step captured in one graph, or the rule and the acceptance in one each,
    replayed with good and bad trees in turn, leaves what eager steps leave."""
    import torch
    cases = captured_cases()
    arms = [tt.on_device(cases[0]) for _ in range(2)]
    eager, other = (loop_over(d) for d in arms)
    side = torch.cuda.Stream()
    if how != "stream":
        spare = tt.on_device(cases[0])
        one_step(loop_over(spare), spare)  # (all that a first call loads)
        torch.cuda.synchronize()
        d, graphs = arms[1], [torch.cuda.CUDAGraph() for _ in range(2 if how == "two graphs" else 1)]
        with torch.cuda.graph(graphs[0]):
            if how == "graph":
                one_step(other, d)
            else:
                other.verify_tree(d["q"], d["k"], d["v"], d["raw_g"], d["raw_beta"], d["parents"],
                                  d["node_corr"], d["out"], Q=12)
        if how == "two graphs":
            with torch.cuda.graph(graphs[1]):
                other.accept_tree(d["path"], d["accepted"], d["k"], d["raw_g"], d["node_corr"],
                                  x=d["x"], conv_state=d["conv_state"], Q=12)
    else:
        other.stream = side
    for n, case in enumerate(cases):
        fresh = tt.on_device(case)
        for d in arms:
            for name in PER_STEP:
                d[name].copy_(fresh[name])
        one_step(eager, arms[0])
        if how == "stream":
            side.wait_stream(torch.cuda.current_stream())
            one_step(other, arms[1])
            torch.cuda.current_stream().wait_stream(side)
        else:
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        same(*arms, ("state", "corr", "key_gate", "pending", "conv_state", "accepted", "status"))
        assert int(arms[0]["status"].item()) == (_lib.KDA_ERR_ARG if n % 2 else 0)
        for d in arms:
            d["status"].zero_()


def test_accept_tree_beside_the_librarys_verify():
    """Without verify_tree there is nothing that it reported: the paths that fit
    are taken."""
    import torch
    case = captured_cases()[0]
    arms = [tt.on_device(case) for _ in range(2)]
    for raw, d in zip((False, True), arms):
        one_step(loop_over(d), d, raw)
    torch.cuda.synchronize()
    same(*arms, ("state", "corr", "key_gate", "pending", "conv_state", "accepted", "status"))
    taken = case["accepted"].copy()
    taken[1] = 0
    got = tt.to_numpy(arms[1]["pending"])
    assert (got[case["record_rows"]] == np.where(case["state_slots"] > 0, taken,
                                                 case["pending"][case["record_rows"]])).all()


@pytest.mark.parametrize("by", ["flush", "prefill"])
def test_paths_longer_than_the_chains_windows(by):
    """Chains of three drafts beside records of eight: all that a tree's path left
    pending is folded in, as where chains have eight."""
    import torch
    arms = [Arm(8, 10), Arm(8, 10)]
    arms[1].loop.Q = 3
    deep = [tt.chain(8), tt.chain(8), tt.star(4), tt.chain(6)]
    left = [a.step(5, deep) for a in arms]
    same(*left, LEFT + ("count",))
    assert left[0]["count"].tolist() == [8, 8, 2, 6]
    for a in arms:
        if by == "flush":
            a.loop.flush()
        else:
            rng = np.random.default_rng(8)
            bits = lambda *s: tt.to_torch(synth.to_bf16_bits(rng.standard_normal(s).astype(np.float32)), "cuda")
            lens = np.array([5, 0, 9, 2])
            T, qsl = int(lens.sum()), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
            a.loop.prefill(bits(T, H, 128), bits(T, H, 128), bits(T, H, 128), bits(T, H, 128), bits(T, H),
                           tt.to_torch(qsl, "cuda"), bits(T, H, 128), Q=9, sources=a.d["slots"])
        assert int(a.d["status"].item()) == 0
    same(arms[0].d, arms[1].d, ("state", "pending"))
