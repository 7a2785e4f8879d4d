"""kda_draft_accept on the GPU against the oracle: paths and tokens are equal,
whatever the order of the sums.

Numbers are chosen by a generator and never on a border: a running sum of V
weights in FP64 is off by V 2^-53 < 2^-32 of the total at most, the kernel's by
some 2^-46; a uniform number hits a border of 2^20 that closely with a chance
of 2^20 2^-31 2 per draw at the very worst of spacings, some 1e-5 for the sizes
here."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib
from oracle import kda_oracle as ko
from oracle import tree_oracle as to

import tree_testutil as tt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import _build
    assert torch.cuda.is_available()
    _build.build()
    _lib.load()


def weights(rng, T, V, std, probs):
    z = np.exp(rng.standard_normal((T, V)) * std)
    p = (z / z.sum(1, keepdims=True)).astype(np.float32)
    return p if probs == "f32" else (p.view(np.uint32) >> 16).astype(np.uint16)


def as_f64(p):
    return ko.bf16_to_f64(p) if p.dtype == np.uint16 else p.astype(np.float64)


def accept_case(trees, V, *, seed, probs="f32", draft=False, chains=False, std=2.0, tail=0):
    rng = np.random.default_rng(seed)
    T = sum(map(len, trees)) + tail
    target = weights(rng, T, V, std, probs)
    case = dict(target=target, draft=None, tokens=rng.integers(0, V, T).astype(np.int32),
                parents=None if chains else np.concatenate([tt.packed(trees), np.full(tail, 5)]).astype(np.int32),
                query_start_loc=tt.starts_of(trees), accept_uniforms=rng.random(T).astype(np.float32),
                sample_uniforms=rng.random(len(trees)).astype(np.float32), state_slots=None,
                Q=max(max(map(len, trees)), 1), null_slot=0)
    start = case["query_start_loc"]
    if draft:
        q = as_f64(target)
        q = np.roll(q, 1, 0) * np.exp(rng.standard_normal((T, V)) * 0.4)
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
        case["draft"] = q if probs == "f32" else (q.view(np.uint32) >> 16).astype(np.uint16)
        q64 = as_f64(case["draft"])
        for t in range(T):
            case["tokens"][t] = np.searchsorted(np.cumsum(q64[t]), rng.random() * q64[t].sum())
        case["tokens"] = np.minimum(case["tokens"], V - 1).astype(np.int32)
    else:
        # the likeliest tokens of the parent's row, some of them twice
        for b, par in enumerate(trees):
            for t, a in enumerate(par):
                if a >= 0:
                    best = np.argsort(-as_f64(target[start[b] + a]))[:6]
                    case["tokens"][start[b] + t] = rng.choice(best)
    return case


def run_accept(case, d=None, **over):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_draft_accept
    d = tt.on_device(case) if d is None else d
    B = len(case["sample_uniforms"])
    if "accepted" not in d:
        d["accepted"], d["next"] = (torch.full((B,), 55, dtype=torch.int32, device="cuda") for _ in range(2))
        d["path"] = torch.full((B, 8), 55, dtype=torch.int32, device="cuda")
    kw = dict(Q=case["Q"], draft_probs=d["draft"], parents=d["parents"], state_slots=d["state_slots"],
              query_start_loc=d["query_start_loc"], null_slot=case["null_slot"], status=d["status"])
    kw.update(over)
    kda_draft_accept(d["target"], d["tokens"], d["accept_uniforms"], d["sample_uniforms"],
                     d["accepted"], d["path"], d["next"], **kw)
    return d


def check_accept(case, d, bad=0):
    with np.errstate(invalid="ignore"):
        *ref, n_bad = to.accept(
            target=as_f64(case["target"]), tokens=case["tokens"],
            accept_uniforms=case["accept_uniforms"], sample_uniforms=case["sample_uniforms"],
            Q=case["Q"], draft=None if case["draft"] is None else as_f64(case["draft"]),
            parents=case["parents"], state_slots=case["state_slots"],
            query_start_loc=case["query_start_loc"], null_slot=case["null_slot"])
    assert n_bad == bad and tt.to_numpy(d["status"])[0] == (_lib.KDA_ERR_ARG if bad else 0)
    for name, want in zip(("accepted", "path", "next"), ref):
        np.testing.assert_array_equal(tt.to_numpy(d[name]), want, err_msg=name)
    return ref


RNG = np.random.default_rng(1)
CHAINS = [tt.chain(n) for n in (8, 1, 2, 5, 8, 3, 7, 4, 6, 8)]
TREES = [tt.random_tree(RNG, n) for n in (1, 64, 17, 2, 33, 8, 32, 5)] + [tt.star(64), tt.comb(40)]


@pytest.mark.parametrize("V", [1, 2, 7, 511, 512, 513, 1000, 4096, 4099, 33000])
@pytest.mark.parametrize("probs", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["drafts", "chains", "trees"])
def test_accept(kind, probs, V):
    case = accept_case(TREES if kind == "trees" else CHAINS, V, seed=V, probs=probs,
                       draft=kind == "drafts", chains=kind != "trees", tail=2)
    check_accept(case, run_accept(case))


@pytest.mark.parametrize("V", [99999, 262144, 1 << 20])
def test_accept_large_vocabularies(V):
    """Flat weights: running sums a millionth apart."""
    case = accept_case([tt.chain(3), tt.chain(2)], V, seed=V, draft=True, chains=True, std=0.1)
    check_accept(case, run_accept(case))
    case = accept_case([tt.star(3), tt.chain(2)], V, seed=V + 1, std=0.1, probs="bf16")
    check_accept(case, run_accept(case))


def test_accept_rows_apart():
    """Rows of any stride and alignment."""
    import torch
    for probs, pads in (("f32", (1, 2, 4)), ("bf16", (1, 4, 8))):
        for pad in pads:
            case = accept_case(CHAINS, 1003, seed=pad, probs=probs, draft=True, chains=True)
            d = tt.on_device(case)
            for n, lead in (("target", 0), ("draft", pad)):
                x = d[n]
                wide = torch.full((x.shape[0], x.shape[1] + 2 * pad), float("nan"), dtype=x.dtype,
                                  device="cuda")
                wide[:, lead:lead + x.shape[1]] = x
                d[n] = wide[:, lead:lead + x.shape[1]]
            check_accept(case, run_accept(case, d))


@pytest.mark.parametrize("probs", ["f32", "bf16"])
def test_accept_nothing_left(probs):
    """Drafts from the target's own weights (nothing is left when one is
    refused: the target's row itself), one-hot rows, and children that hold
    all there is."""
    case = accept_case(CHAINS, 600, seed=3, probs=probs, draft=True, chains=True)
    case["draft"][1:] = case["target"][:-1]
    case["accept_uniforms"][:] = 1 - 2.0 ** -24
    case["draft"][:, ::2] = np.maximum(case["draft"][:, ::2], np.roll(case["target"], 1, 0)[:, ::2])
    check_accept(case, run_accept(case))
    one = 1.0 if probs == "f32" else 0x3F80
    case = accept_case(TREES, 600, seed=4, probs=probs)
    case["target"][:] = 0
    hot = RNG.integers(0, 600, len(case["target"]))
    case["target"][np.arange(len(hot)), hot] = one
    check_accept(case, run_accept(case))
    case = accept_case([tt.star(3)] * 4, 600, seed=5, probs=probs)
    case["target"][:] = 0
    for b in range(4):
        case["tokens"][3 * b + 1:3 * b + 3] = [7, 9]
        case["target"][3 * b, [7, 9]] = one if probs == "bf16" else 0.4
    case["accept_uniforms"][:] = [0.1, 0.9, 0.9] * 3 + [1 - 2.0 ** -24] * 3
    # (a child that is taken has a row of zeros: reported, with the path)
    check_accept(case, run_accept(case), bad=4 if probs == "bf16" else 3)


def test_accept_ends_of_the_uniforms():
    """0 takes the first weight above zero, the largest number below 1 one of
    the last; weights of zero at both ends are never taken."""
    case = accept_case([tt.chain(1)] * 6, 5000, seed=6, chains=True)
    case["target"][:, :700] = 0
    case["target"][:, -900:] = 0
    case["sample_uniforms"][:] = [0.0, 1 - 2.0 ** -24] * 3
    accepted, path, nxt = check_accept(case, run_accept(case))
    assert (nxt[::2] == 700).all() and (nxt[1::2] < 4100).all()


def test_accept_strange_weights():
    """NaN and negative weights count as zero; rows without a finite positive
    total are reported, with their paths."""
    for probs in ("f32", "bf16"):
        nan, neg, inf = ((np.nan, -1.0, np.inf) if probs == "f32" else (0x7FC0, 0xBF80, 0x7F80))
        case = accept_case(TREES, 900, seed=7, probs=probs)
        case["target"][:, 5:200:7] = nan
        case["target"][:, 6:300:5] = neg
        check_accept(case, run_accept(case))
        case = accept_case(CHAINS, 900, seed=8, probs=probs, draft=True, chains=True)
        case["draft"][:, 3:400:9] = nan
        case["target"][:, 4:400:11] = nan
        check_accept(case, run_accept(case))
        case = accept_case([tt.chain(1)] * 4, 900, seed=9, probs=probs, chains=True)
        case["target"][1] = 0
        case["target"][2, 17] = inf
        case["target"][3] = nan
        check_accept(case, run_accept(case), bad=3)


def test_accept_reports():
    case = accept_case([tt.comb(9) for _ in range(9)], 300, seed=10)
    start = case["query_start_loc"]
    case["tokens"][start[1] + 3], case["tokens"][start[2] + 8] = 300, -1
    case["parents"][start[3]] = 0
    case["parents"][start[4] + 2] = -1                       # a second root
    case["parents"][start[5] + 2] = 2
    case["parents"][start[6]:start[6] + 9] = tt.chain(9)     # nine deep
    case["tokens"][start[7]] = -5                            # (the root's is not looked at)
    check_accept(case, run_accept(case), bad=6)
    case = accept_case([tt.comb(9) for _ in range(3)], 300, seed=11)
    case["query_start_loc"][1] = 30
    check_accept(case, run_accept(case), bad=2)


def test_accept_inert_empty_and_uniform():
    case = accept_case([tt.chain(4), [], tt.comb(12), [], tt.chain(2)], 300, seed=12, tail=3)
    case["state_slots"] = np.array([3, 4, 0, -1, 2], np.int32)
    t = case["query_start_loc"][2]
    case["tokens"][t:t + 12], case["parents"][t:t + 12] = -9, 99
    check_accept(case, run_accept(case))
    case = accept_case([tt.comb(12)] * 5, 300, seed=13)
    case["query_start_loc"] = None
    check_accept(case, run_accept(case))


def test_accept_captured_and_on_another_stream():
    import torch
    cases = [accept_case(CHAINS, 5003, seed=20 + s, draft=True, chains=True) for s in range(3)]
    d = tt.on_device(cases[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run_accept(cases[0], d, stream=side)
    side.synchronize()
    check_accept(cases[0], d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_accept(cases[0], d)
    for case in cases:
        fresh = tt.on_device(case)
        for n in fresh:
            if fresh[n] is not None:
                d[n].copy_(fresh[n])
        graph.replay()
        torch.cuda.synchronize()
        check_accept(case, d)


def test_accept_is_lossless():
    """Many requests with the same weights: the first emitted token follows
    the target, by chains with a draft's probabilities and by trees, within
    five standard deviations of a count (some 1e-6 of chance a token)."""
    B, V = 1 << 16, 6
    rng = np.random.default_rng(30)
    p, q = rng.dirichlet(np.ones(V)).astype(np.float32), rng.dirichlet(np.ones(V)).astype(np.float32)
    for kind in ("draft", "tree"):
        n = 2 if kind == "draft" else 3
        tokens = np.zeros((B, n), np.int32)
        if kind == "draft":
            tokens[:, 1] = np.searchsorted(np.cumsum(q.astype(np.float64)), rng.random(B) * 0.999999)
        else:
            tokens[:, 1:] = [4, 1]
        case = dict(target=np.tile(p, (B * n, 1)), draft=np.tile(q, (B * n, 1)) if kind == "draft" else None,
                    tokens=tokens.ravel(), parents=None if kind == "draft" else np.tile(np.int32([-1, 0, 0]), B),
                    query_start_loc=None, accept_uniforms=rng.random(B * n).astype(np.float32),
                    sample_uniforms=rng.random(B).astype(np.float32), state_slots=None, Q=n, null_slot=0)
        d = run_accept(case)
        accepted, path, nxt = (tt.to_numpy(d[x]) for x in ("accepted", "path", "next"))
        first = np.where(accepted == 2, tokens[np.arange(B), np.maximum(path[:, 1], 0)], nxt)
        count = np.bincount(first, minlength=V)
        want = p.astype(np.float64) / p.astype(np.float64).sum()
        assert np.all(np.abs(count - B * want) <= 5 * np.sqrt(B * want * (1 - want)) + 1)
