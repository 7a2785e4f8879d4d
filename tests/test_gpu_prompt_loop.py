"""Prompts in the middle of the decode loop: record rows with a replay pending
when a prompt comes, from the request before or from the request itself."""
import numpy as np
import pytest

from prompt_testutil import to_torch
from linear_attention_speculative_recoverssm_gb300 import synth

pytestmark = pytest.mark.gpu

H, B, Q, SLOTS = 2, 4, 3, 12
RULE = dict(lower_bound=-5.0, q_scale=128 ** -0.5)


def inputs(rng, T):
    bits = lambda *s, std=1.0: to_torch(
        synth.to_bf16_bits((rng.standard_normal(s) * std).astype(np.float32)), "cuda")
    return [bits(T, H, 128), bits(T, H, 128), bits(T, H, 128), bits(T, H, 128, std=0.7), bits(T, H)]


def i32(*a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def a_loop(rng, stream=None):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import DeferredRecoverSSM
    A_log = to_torch(rng.uniform(0, 1.5, H).astype(np.float32), "cuda")
    dt = to_torch((rng.standard_normal((H, 128)) - 2).astype(np.float32), "cuda")
    pool = to_torch(rng.standard_normal((SLOTS, H, 128, 128)).astype(np.float32), "cuda")
    loop = DeferredRecoverSSM(
        pool, i32(3, 5, 7, 9), i32(2, 0, 1, 3), torch.zeros(B, dtype=torch.int32, device="cuda"),
        torch.zeros((B, H, 8, 128), device="cuda"),
        torch.zeros((B, H, 8, 256), dtype=torch.bfloat16, device="cuda"), A_log, dt, Q=Q,
        status=torch.zeros(1, dtype=torch.int32, device="cuda"), stream=stream, **RULE)
    return loop


def empty(T):
    import torch
    return torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda")


def window(loop, x, accepted):
    out = empty(B * Q)
    loop.verify(*x, out)
    loop.accept(i32(*accepted))
    return out


@pytest.mark.parametrize("flushed", [False, True])
@pytest.mark.parametrize("side", [False, True])
def test_row_of_a_finished_request(flushed, side):
    """Requests 0 and 2 end with replays pending and their rows' next requests
    bring prompts: nothing of the old windows reaches them, and the replays of
    1 and 3 stay pending."""
    import torch
    rng = np.random.default_rng(1)
    loop = a_loop(rng, torch.cuda.Stream() if side else None)
    prompt, first, second = inputs(rng, 150), inputs(rng, B * Q), inputs(rng, B * Q)
    torch.cuda.synchronize()
    window(loop, first, (3, 2, 1, 3))
    if flushed:
        loop.flush()
    torch.cuda.synchronize()
    qsl = i32(0, 100, 100, 150, 150)
    clean = a_loop(np.random.default_rng(1), loop.stream)
    for name in ("state_pool", "corr", "key_gate", "pending"):
        getattr(clean, name).copy_(getattr(loop, name))
    clean.pending[loop.record_rows[[0, 2]].long()] = 0  # as if nothing had been before
    clean.flushed = loop.flushed
    torch.cuda.synchronize()
    outs = []
    for one in (loop, clean):
        out = empty(150)
        one.prefill(*prompt, qsl, out, Q=100)
        outs.append((out, window(one, second, (1, 2, 3, 0))))
        one.flush()
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(loop.state_pool, clean.state_pool)
    assert int(loop.status[0]) == 0
    # and what they are: the prompts alone, decoded
    from linear_attention_speculative_recoverssm_gb300 import kda_recurrent
    pool, ref = loop.state_pool.clone(), empty(150)
    kda_recurrent(*prompt, loop.A_log, loop.dt_bias, pool, i32(0, 0, 0, 0), loop.state_slots, ref,
                  Q=100, query_start_loc=qsl, **RULE)
    dec = empty(B * Q)
    kda_recurrent(*second, loop.A_log, loop.dt_bias, pool, loop.state_slots, i32(1, 0, 2, 0), dec,
                  Q=Q, **RULE)
    for t in (slice(0, Q), slice(2 * Q, 3 * Q)):
        a, b = outs[0][1][t].double(), dec[t].double()
        assert torch.linalg.norm(a - b) <= 2.0 ** -7 * torch.linalg.norm(b)


def test_prompt_after_decoded_tokens():
    """A request goes on from its own slot with accepted tokens still pending:
    they are part of what its next prompt goes on from, and are not replayed
    again; another's stay pending."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_recurrent
    rng = np.random.default_rng(2)
    loop = a_loop(rng)
    x, y, z = inputs(rng, B * Q), inputs(rng, 120), inputs(rng, B * Q)
    pool = loop.state_pool.clone()
    window(loop, x, (2, 3, 0, 1))
    before = loop.pending.clone()
    out, bnd = empty(120), i32(0, 11, 0, 10)
    loop.prefill(*y, i32(0, 0, 70, 70, 120), out, Q=70, sources=loop.state_slots, boundaries=bnd,
                 boundary_lens=i32(0, 20, 0, 33))
    assert loop.pending.tolist() == [0, int(before[1]), int(before[2]), 0]  # (rows 2, 0, 1, 3)
    # the same tokens one after the other
    n = (2, 3, 0, 1)
    at = [slice(b * Q, b * Q + n[b]) for b in range(B)]
    part = [torch.cat([t[s] for s in at]).contiguous() for t in x]
    own = loop.state_slots
    kda_recurrent(*part, loop.A_log, loop.dt_bias, pool, own, own, empty(6), Q=Q,
                  query_start_loc=i32(0, 2, 5, 5, 6), **RULE)
    ref = empty(120)
    kda_recurrent(*y, loop.A_log, loop.dt_bias, pool, own, own, ref, Q=70,
                  query_start_loc=i32(0, 0, 70, 70, 120), boundaries=bnd,
                  boundary_lens=i32(0, 20, 0, 33), **RULE)
    close = lambda a, b: torch.linalg.norm((a - b).double()) <= 2.0 ** -7 * torch.linalg.norm(b.double())
    # (records hold keys and gates in BF16: a step of each, 2^-8, of what three
    # tokens changed)
    assert close(out.float(), ref.float())
    for s in (5, 9, 10, 11):
        assert close(loop.state_pool[s], pool[s]), s
    loop.flush()  # now request 0's two tokens
    assert close(loop.state_pool[3], pool[3]) and close(loop.state_pool[7], pool[7])
    got, want = empty(B * Q), empty(B * Q)
    loop.verify(*z, got)
    kda_recurrent(*z, loop.A_log, loop.dt_bias, pool, own, i32(1, 2, 4, 6), want, Q=Q, **RULE)
    assert close(got.float(), want.float()) and int(loop.status[0]) == 0
