"""Cases of the prompt operators' tests: inputs as numpy arrays (BF16 as bit
patterns), their device copies, and the tolerances."""
from __future__ import annotations

import numpy as np

from kda_testutil import bf16_ulp, to_numpy, to_torch
from linear_attention_speculative_recoverssm_gb300 import synth
from oracle import kda_oracle as ko

# An output is rounded to BF16 once: off by half a step, 2^-8 of its value at
# most.  Before that the operators work in FP32: what is left of a decay's
# error.  A decay is good to 2^-22 (its two exponentials and reciprocal, each
# about 2^-23); a state entry that remembers M tokens has multiplied M of
# them, at most M 2^-22 off if all err one way, which for the tests' gates
# (mean decays below 0.98: M < 100 at 2^-3 of the value and less beyond) is
# below 2.5e-5 of the largest entry.  Sums of 128 products and of a chunk's
# tokens add less than 128 2^-24 = 8e-6 of their largest partial sums.
# Together under 1e-4 of the largest value, the tolerance of the verify
# kernels' states.
REL = 1e-4

# kda_prefill rounds the operands of the products that reach the outputs alone
# (and not the state) to 11 bits, 2^-11 of each at most: of Qd and S in Qd S^T,
# which leaves 2 2^-11 |Qd| |S row| (Cauchy-Schwarz, |Qd| <= 1); of q and k in
# A, |A| <= 1, and of A and U in A U, 4 2^-11 sum |u| over the chunk.  With the
# oracle's `sizes` (largest |S row| + 2 sum |u|), together 2^-10 sizes.  That
# bound has all roundings err one way; the framework's own tolerance of the
# outputs as a whole, 2e-3 in the 2-norm, is checked beside it.
QUERY = 2.0 ** -10
OUT_REL_L2 = 2e-3


def ragged_case(*, lens, H, seed, pool="f32", resume=None, boundary=None, inert=(), slots=None,
                lower_bound=-5.0, tail=0, memory=50.0):
    """Prompts of the given lengths packed one after the other, `tail` rows
    behind the last.  ``resume``: the requests with a source slot (default:
    every second one); ``boundary``: {request: m}; ``inert``: requests whose
    destination is the null slot."""
    rng = np.random.default_rng(seed)
    B, T = len(lens), sum(lens) + tail
    resume = set(range(1, B, 2)) if resume is None else set(resume)
    boundary = boundary or {}
    slots = 3 * B + 2 if slots is None else slots
    pick = rng.permutation(np.arange(1, slots))[:3 * B].astype(np.int32)
    src = np.where([b in resume for b in range(B)], pick[:B], 0).astype(np.int32)
    dst = np.where([b in inert for b in range(B)], 0, pick[B:2 * B]).astype(np.int32)
    bnd = np.array([pick[2 * B + b] if b in boundary else 0 for b in range(B)], dtype=np.int32)
    bl = np.array([boundary.get(b, 0) for b in range(B)], dtype=np.int32)
    n = lambda *s, std=1.0: (rng.standard_normal(s) * std).astype(np.float32)
    bits = synth.to_bf16_bits
    A_log = rng.uniform(0.0, 1.5, size=H).astype(np.float32)
    # channels that forget over 1 .. `memory` tokens
    share = np.exp(rng.uniform(0, np.log(memory), size=(H, 128))) / (5.0 * memory)
    dt = (np.log(share / (1 - share)) / np.exp(A_log)[:, None]).astype(np.float32)
    state = n(slots, H, 128, 128, std=0.3)
    return dict(
        q=bits(n(T, H, 128)), k=bits(n(T, H, 128)), v=bits(n(T, H, 128)),
        raw_g=bits(n(T, H, 128, std=0.7)), raw_beta=bits(n(T, H)), A_log=A_log, dt_bias=dt,
        state=state if pool == "f32" else bits(state), sources=src, destinations=dst,
        boundaries=bnd, boundary_lens=bl,
        query_start_loc=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32),
        out=np.full((T, H, 128), 0x4321, dtype=np.uint16),  # a mark: what is not written
        lower_bound=lower_bound, q_scale=128 ** -0.5, Q=max(max(lens), 1), null_slot=0)


RULE = ("q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias", "state", "sources",
        "destinations", "boundaries", "boundary_lens", "query_start_loc", "out")


def on_device(case, names=RULE):
    d = {n: None if case[n] is None else to_torch(case[n], "cuda") for n in names}
    d["status"] = to_torch(np.zeros(1, dtype=np.int32), "cuda")
    return d


def call_rule(fn, case, d, **over):
    kw = dict(Q=case["Q"], lower_bound=case["lower_bound"], q_scale=case["q_scale"],
              boundaries=d["boundaries"], boundary_lens=d["boundary_lens"],
              null_slot=case["null_slot"], status=d["status"])
    kw.update(over)
    args = [d[n] for n in ("q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias", "state",
                           "sources", "destinations")]
    if fn.__name__ == "kda_recurrent":
        return fn(*args, d["out"], query_start_loc=d["query_start_loc"], **kw)
    return fn(*args, d["query_start_loc"], d["out"], **kw)


def check_outputs(got_bits, ref_bits, ref_f64, live, slack=0.0):
    """Rows of `live` tokens within half a BF16 step plus REL of the head's
    largest plus `slack`, and within the framework's tolerance as a whole; the
    others bit for bit."""
    np.testing.assert_array_equal(got_bits[~live], ref_bits[~live])
    got, ref = ko.bf16_to_f64(got_bits[live]), ref_f64[live]
    if not ref.size:
        return
    scale = np.abs(ref).max(axis=(0, 2), keepdims=True)
    if not np.isscalar(slack):
        slack = slack[live]
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + REL * scale + slack), "outputs"
    assert np.linalg.norm(got - ref) <= OUT_REL_L2 * np.linalg.norm(ref), "outputs, rel-L2"


def check_states(got, ref, before):
    """Slots that the oracle changed, within REL of the slot's largest entry
    (BF16: and one step, two roundings of near values); the others bit for
    bit."""
    changed = (ref != before).reshape(len(ref), -1).any(axis=1)
    np.testing.assert_array_equal(got[~changed], before[~changed])
    for s in np.flatnonzero(changed):
        g, r = ko.state_to_f64(got[s]), ko.state_to_f64(ref[s])
        step = bf16_ulp(r) if got.dtype == np.uint16 else 0.0
        assert np.all(np.abs(g - r) <= step + REL * np.abs(r).max()), f"state of slot {s}"


__all__ = ["REL", "QUERY", "OUT_REL_L2", "ragged_case", "on_device", "call_rule", "check_outputs",
           "check_states", "to_numpy", "to_torch"]
