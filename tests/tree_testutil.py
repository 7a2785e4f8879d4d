"""Cases of the tree operators' tests: trees, inputs as numpy arrays (BF16 as
bit patterns) and their device copies."""
from __future__ import annotations

import numpy as np

from kda_testutil import to_numpy, to_torch
from linear_attention_speculative_recoverssm_gb300 import synth

MARK = 0x4321  # what rows hold that nothing writes


def random_tree(rng, n, depth=8, roots=1):
    """Parents of a random tree of n nodes, `roots` of them on the checkpoint."""
    par, dep = [], []
    for t in range(n):
        while True:
            a = -1 if t < roots else int(rng.integers(0, t))
            if a < 0 or dep[a] < depth:
                break
        par.append(a)
        dep.append(1 if a < 0 else dep[a] + 1)
    return par


def chain(n):
    return list(range(-1, n - 1))


def star(n):
    return [-1] + [0] * (n - 1)


def comb(n):
    """A spine of eight nodes, leaves on its nodes in turn."""
    return chain(min(n, 8)) + [t % 7 for t in range(8, n)]


def packed(trees):
    return np.array([a for par in trees for a in par], dtype=np.int32)


def starts_of(trees):
    return np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)


def tree_case(trees, H, *, seed, pool="f32", replay=True, rq=8, tail=0, inert=(), rowless=(),
              lower_bound=-5.0, pending=None, memory=50.0, extra_slots=2):
    """Requests with the given trees, `tail` rows behind the last.  Gates,
    states and records as in the prompt operators' cases."""
    rng = np.random.default_rng(seed)
    B, T = len(trees), sum(map(len, trees)) + tail
    slots, rows = B + 1 + extra_slots, B + extra_slots
    n = lambda *s, std=1.0: (rng.standard_normal(s) * std).astype(np.float32)
    bits = synth.to_bf16_bits
    A_log = rng.uniform(0.0, 1.5, size=H).astype(np.float32)
    share = np.exp(rng.uniform(0, np.log(memory), size=(H, 128))) / (5.0 * memory)
    dt = (np.log(share / (1 - share)) / np.exp(A_log)[:, None]).astype(np.float32)
    state = n(slots, H, 128, 128, std=0.3)
    pend = rng.integers(0, rq + 1, size=rows).astype(np.int32)
    if pending is not None:
        pend[:] = pending
    D = H * 128
    return dict(
        q=bits(n(T, H, 128)), k=bits(n(T, H, 128)), v=bits(n(T, H, 128)),
        raw_g=bits(n(T, H, 128, std=0.7)), raw_beta=bits(n(T, H)), A_log=A_log, dt_bias=dt,
        state=state if pool == "f32" else bits(state),
        state_slots=np.where([b in inert for b in range(B)], 0,
                             rng.permutation(np.arange(1, slots))[:B]).astype(np.int32),
        record_rows=np.where([b in rowless for b in range(B)], -1,
                             rng.permutation(rows)[:B]).astype(np.int32),
        pending=pend if replay else None,
        corr=n(rows, H, rq, 128) if replay else None,
        key_gate=bits(n(rows, H, rq, 256)) if replay else None,
        parents=np.concatenate([packed(trees), np.full(tail, 77, dtype=np.int32)]).astype(np.int32),
        query_start_loc=starts_of(trees), Q=max(max(map(len, trees)), 1),
        node_corr=np.full((T, H, 128), 123.0, dtype=np.float32),
        out=np.full((T, H, 128), MARK, dtype=np.uint16),
        x=bits(n(T, 3 * D)), conv_weight=bits(n(3, 4, D, std=0.5)), conv_bias=bits(n(3 * D, std=0.1)),
        conv_state=bits(n(slots, 3 * D, rq + 2)),
        lower_bound=lower_bound, q_scale=128 ** -0.5, null_slot=0)


VERIFY = ("q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias", "state", "state_slots", "parents",
          "node_corr", "out", "record_rows", "pending", "corr", "key_gate", "query_start_loc")


def on_device(case, names=None):
    import torch
    d = {n: to_torch(a, "cuda") for n, a in case.items()
         if isinstance(a, np.ndarray) and (names is None or n in names)}
    for n, a in case.items():
        if a is None:
            d[n] = None
    d["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return d


def copy_case(case):
    return {k: a.copy() if isinstance(a, np.ndarray) else a for k, a in case.items()}


def call_verify(case, d, **over):
    from linear_attention_speculative_recoverssm_gb300 import kda_tree_verify
    kw = dict(Q=case["Q"], lower_bound=case["lower_bound"], q_scale=case["q_scale"],
              record_rows=d["record_rows"], pending=d["pending"], corr=d["corr"],
              key_gate=d["key_gate"], query_start_loc=d["query_start_loc"],
              null_slot=case["null_slot"], status=d["status"])
    kw.update(over)
    return kda_tree_verify(*(d[n] for n in ("q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias",
                                            "state", "state_slots", "parents", "node_corr", "out")),
                           **kw)


__all__ = ["MARK", "random_tree", "chain", "star", "comb", "packed", "starts_of", "tree_case",
           "VERIFY", "on_device", "copy_case", "call_verify", "to_numpy", "to_torch"]
