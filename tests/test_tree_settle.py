"""kda_tree_settle: its refusals without a GPU; on the GPU, against the rules
that the header states, every kind of request among others."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _build, _lib
from oracle import tree_oracle as to

import tree_testutil as tt


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


A = 0x10000  # a 16-byte aligned stand-in address: never dereferenced below
OK, ARG = _lib.KDA_OK, _lib.KDA_ERR_ARG


def _settle(lib, **over):
    a = dict(path=A, accepted=A, most=8, slots=A, n_slots=4, rows=A, served=A, n_rows=3, parents=A, qsl=A, T=10,
             folded=0, to=A, B=2, Q=8, null=0, status=None, stream=None)
    return lib.kda_tree_settle(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), ARG), (dict(Q=0), ARG), (dict(Q=65), ARG), (dict(T=-1), ARG), (dict(null=-2), ARG),
    (dict(qsl=None), ARG), (dict(slots=None), ARG), (dict(to=None), ARG), (dict(n_slots=0), ARG),
    (dict(n_rows=0), ARG), (dict(rows=None, n_rows=1), ARG), (dict(B=0, slots=None), OK),
    (dict(accepted=None), ARG), (dict(most=-1), ARG), (dict(most=9), ARG),
])
def test_refusals(lib, over, code):
    assert _settle(lib, **over) == code


def test_binding_refusals(lib):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_tree_settle
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)

    def settle(**o):
        a = dict(state_slots=i32(2), record_rows=i32(2), rows=i32(2), Q=3, n_tokens=6, n_slots=4,
                 n_rows=3, accepted=i32(2), path=i32(2, 8), parents=i32(6), served=i32(2), query_start_loc=i32(3))
        return kda_tree_settle(**{**a, **o})

    for bad in (dict(rows=i32(2).long()), dict(accepted=torch.zeros(2)), dict(parents=i32(6).long())):
        with pytest.raises(TypeError):
            settle(**bad)
    for bad in (dict(rows=i32(3)), dict(served=i32(1)), dict(parents=i32(5)), dict(path=i32(2, 7)),
                dict(query_start_loc=i32(2)), dict(record_rows=i32(4)[::2]), dict()):
        with pytest.raises(ValueError):
            settle(**bad)


def rules(case, *, folded=False, trees=True, most=8):
    """(rows, accepted, whether one is reported) as the header has it."""
    T, n_slots, n_rows = len(case["q"]), len(case["state"]), len(case["corr"])
    to_rows, counts, bad = case["record_rows"].copy(), case["accepted"].copy(), 0
    wins = to.windows(case["query_start_loc"], len(to_rows), case["Q"], T)
    for b, (slot, row) in enumerate(zip(case["state_slots"], case["record_rows"])):
        if slot <= case["null_slot"] or row < 0:
            continue
        here = slot < n_slots and row < n_rows
        left = case["served"] is not None and case["served"][b] < 0
        good = here and not left and wins[b] is not None and \
            (not trees or to.tree(case["parents"], *wins[b]) is not None)
        if not good:
            bad, counts[b] = bad + 1, 0
            if left or not folded or not here:
                to_rows[b] = -1
        elif case["path"] is not None and \
                (not 0 <= counts[b] <= most or
                 any(not 0 <= t < wins[b][1] for t in case["path"][b, :counts[b]])):
            bad, counts[b] = bad + 1, 0
    return to_rows, counts, bad


def settle_case(B, seed, cap=12):
    """Requests of every kind: inert, rowless, empty, with bad trees, windows,
    slots, rows, and left by an earlier call."""
    rng = np.random.default_rng(seed)
    sizes = np.where(rng.random(B) < 0.2, 0, rng.integers(1, cap + 1, B))
    trees = [tt.random_tree(rng, int(n)) for n in sizes]
    case = tt.tree_case(trees, 1, seed=seed, inert=set(rng.permutation(B)[:B // 8]),
                        rowless=set(rng.permutation(B)[:B // 8]))
    case.update(accepted=rng.integers(-2, 9, B).astype(np.int32), served=case["record_rows"].copy(),
                path=rng.integers(0, np.maximum(sizes, 1)[:, None], (B, 8)).astype(np.int32), Q=cap)
    spoilt = rng.random((B, 8)) < 0.05
    case["path"][spoilt] = rng.choice([-1, cap, 1 << 30, -1 << 31], spoilt.sum())
    start = case["query_start_loc"]
    kinds = rng.integers(0, 12, B)
    for b in np.flatnonzero(sizes > 1):
        if kinds[b] == 0:
            case["parents"][start[b] + sizes[b] - 1] = rng.choice([sizes[b] - 1, 1 << 30, -2])
        elif kinds[b] == 1:
            case["state_slots"][b] = len(case["state"]) + int(rng.integers(0, 5))
        elif kinds[b] == 2:
            case["record_rows"][b] = len(case["corr"])
        elif kinds[b] == 3:
            case["served"][b] = -1
        elif kinds[b] == 4:  # its window and the one before it
            case["query_start_loc"][b] = start[b] + cap + 1 if rng.random() < 0.5 else -1
    return case


def run(case, **kw):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_tree_settle
    d = tt.on_device(case, ("state_slots", "path", "record_rows", "accepted", "parents", "served",
                            "query_start_loc"))
    rows = torch.full_like(d["state_slots"], 99)
    a = dict(rows=rows, Q=case["Q"], n_tokens=len(case["q"]), n_slots=len(case["state"]),
             n_rows=len(case["corr"]), accepted=d["accepted"], path=d["path"], parents=d["parents"],
             served=d["served"], query_start_loc=d["query_start_loc"], null_slot=case["null_slot"],
             status=d["status"])
    a.update({n: d[v] if isinstance(v, str) else v for n, v in kw.items()})
    kda_tree_settle(d["state_slots"], d["record_rows"], **a)
    return d, a["rows"]


def check(case, d, rows, **kw):
    want_rows, want_counts, bad = rules(case, **kw)
    np.testing.assert_array_equal(tt.to_numpy(rows), want_rows)
    np.testing.assert_array_equal(tt.to_numpy(d["accepted"]), want_counts)
    assert tt.to_numpy(d["status"])[0] == (ARG if bad else 0)
    for n in ("state_slots", "parents", "query_start_loc"):
        np.testing.assert_array_equal(tt.to_numpy(d[n]), case[n])


@pytest.mark.gpu
@pytest.mark.parametrize("folded", [False, True])
@pytest.mark.parametrize("served", [False, True])
@pytest.mark.parametrize("B,cap", [(1, 64), (9, 12), (1000, 12), (70, 64)])
def test_settle(lib, B, cap, served, folded):
    case = settle_case(B, B + cap, cap)
    if not served:
        case["served"] = None
    d, rows = run(case, folded=folded)
    check(case, d, rows, folded=folded)
    d, rows = run(case, folded=folded, parents=None, most=3)  # (no tree is looked at)
    check(case, d, rows, folded=folded, trees=False, most=3)
    d, rows = run(case, path=None)
    case["path"] = None
    check(case, d, rows)


@pytest.mark.gpu
def test_rows_over_the_rows(lib):
    """The result may stand where served or record_rows do; accepted may be
    missing."""
    case = settle_case(300, 5)
    for to_where in ("served", "record_rows"):
        d, rows = run(case, rows=to_where)
        check(case, d, rows)
    d, rows = run(case, accepted=None, path=None)
    np.testing.assert_array_equal(tt.to_numpy(rows), rules(case)[0])
    np.testing.assert_array_equal(tt.to_numpy(d["accepted"]), case["accepted"])
