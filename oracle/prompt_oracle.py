"""FP64 CPU oracle of the prompt operators: the gated delta rule over ragged
prompts (``rule``), the layer's convolution over them (``conv``) and the slot
plan (``slot_plan``).  TEST INFRASTRUCTURE ONLY, like ``kda_oracle``, whose
exact conversions it uses; it shares no code with the library.

The rule is the stock sequential recurrence, token by token (page
"...cutedsl.kda.fused", module docstring, step 2):
S <- S diag(d_t); u_t = beta_t (v_t - S kn_t); S <- S + u_t kn_t^T;
o_t = S qn_t; whole heads at a time.
"""
from __future__ import annotations

import numpy as np

from .kda_oracle import bf16_to_f64, f64_to_bf16, f64_to_state, l2norm, sigmoid, state_to_f64


def _windows(qsl, B, Q, n_tokens):
    """(first token, length) of every request; None where the window is
    outside the activations or longer than Q."""
    out = []
    for b in range(B):
        t0, t1 = (b * Q, (b + 1) * Q) if qsl is None else (int(qsl[b]), int(qsl[b + 1]))
        out.append((t0, t1 - t0) if 0 <= t0 <= t1 <= n_tokens and t1 - t0 <= Q else None)
    return out


def _slots(b, n, sources, destinations, boundaries, boundary_lens, n_slots, null_slot):
    """(source, destination, boundary, m) with None for what is absent; None
    for a request that is left out."""
    dst = int(destinations[b])
    if dst <= null_slot:
        return (None, None, None, 0)
    src = int(sources[b])
    m = 0 if boundaries is None else int(boundary_lens[b])
    bnd = int(boundaries[b]) if m > 0 and boundaries[b] > null_slot else None
    if src >= n_slots or dst >= n_slots or (bnd is not None and bnd >= n_slots):
        return None
    return (src if src > null_slot else None, dst, bnd, min(m, n))


def rule(*, q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale, state, sources,
         destinations, out, Q, query_start_loc=None, boundaries=None, boundary_lens=None,
         null_slot=0, out_f64=None, sizes=None):
    """In place on ``state`` [slots, H, V, K] (FP32 or BF16 bits) and ``out``
    [T, H, V] (BF16 bits).  Returns the number of requests left out.
    ``out_f64`` [T, H, V], when given, takes the outputs before rounding.
    ``sizes`` [T, H, V], when given, takes the size of what the outputs are
    sums of: with q_scale and unit queries, the largest norm of the state row
    over the last 64 tokens plus twice the sum of |u| over them."""
    T, H, V = v.shape
    B = len(sources)
    a = np.exp(A_log.astype(np.float64))[:, None]
    dt = dt_bias.astype(np.float64)
    old = state.copy()  # sources are read before anything is written
    bad = 0
    for b, win in enumerate(_windows(query_start_loc, B, Q, T)):
        if win is None:
            bad += 1
            continue
        t0, n = win
        if n == 0:
            continue
        sl = _slots(b, n, sources, destinations, boundaries, boundary_lens, state.shape[0],
                    null_slot)
        if sl is None:
            bad += 1
            continue
        src, dst, bnd, m = sl
        if dst is None:
            out[t0:t0 + n] = 0
            if out_f64 is not None:
                out_f64[t0:t0 + n] = 0
            continue
        S = np.zeros(state.shape[1:]) if src is None else state_to_f64(old[src])
        norms, us = [np.sqrt((S * S).sum(-1))], []
        for t in range(t0, t0 + n):
            d = np.exp(lower_bound * sigmoid(a * (bf16_to_f64(raw_g[t]) + dt)))
            kn, qn = l2norm(bf16_to_f64(k[t])), l2norm(bf16_to_f64(q[t])) * q_scale
            beta = sigmoid(bf16_to_f64(raw_beta[t]))[:, None]
            S = S * d[:, None, :]
            u = beta * (bf16_to_f64(v[t]) - np.einsum("hvk,hk->hv", S, kn))
            S = S + u[:, :, None] * kn[:, None, :]
            o = np.einsum("hvk,hk->hv", S, qn)
            if sizes is not None:
                norms, us = norms[-64:] + [np.sqrt((S * S).sum(-1))], us[-63:] + [np.abs(u)]
                sizes[t] = abs(q_scale) * (np.max(norms, axis=0) + 2 * np.sum(us, axis=0))
            out[t] = f64_to_bf16(o)
            if out_f64 is not None:
                out_f64[t] = o
            if bnd is not None and t - t0 + 1 == m:
                state[bnd] = f64_to_state(S, state.dtype)
        state[dst] = f64_to_state(S, state.dtype)
    return bad


def conv(*, x, conv_weight, conv_bias, conv_state, sources, destinations, q, k, v, Q,
         query_start_loc=None, boundaries=None, boundary_lens=None, null_slot=0):
    """In place on ``conv_state`` [slots, 3 D, width] and q, k, v [T, H, 128]
    (all BF16 bits).  Returns the number of requests left out."""
    T, D3 = x.shape
    D = D3 // 3
    w = bf16_to_f64(conv_weight).transpose(1, 0, 2).reshape(4, D3)
    bias = np.zeros(D3) if conv_bias is None else bf16_to_f64(conv_bias)
    old = conv_state.copy()
    B, bad = len(sources), 0
    for b, win in enumerate(_windows(query_start_loc, B, Q, T)):
        if win is None:
            bad += 1
            continue
        t0, n = win
        if n == 0:
            continue
        sl = _slots(b, n, sources, destinations, boundaries, boundary_lens, conv_state.shape[0],
                    null_slot)
        if sl is None:
            bad += 1
            continue
        src, dst, bnd, m = sl
        if dst is None:
            continue
        head = np.zeros((3, D3), dtype=np.uint16) if src is None else old[src, :, :3].T
        line = np.concatenate([head, x[t0:t0 + n]])
        f = bf16_to_f64(line)
        z = bias + sum(w[i] * f[i:i + n] for i in range(4))
        y = f64_to_bf16(z * sigmoid(z)).reshape(n, 3, -1, 128)
        for i, o in enumerate((q, k, v)):
            o[t0:t0 + n] = y[:, i]
        if bnd is not None:
            conv_state[bnd, :, :3] = line[m:m + 3].T
        conv_state[dst, :, :3] = line[n:n + 3].T
    return bad


def slot_plan(*, computed_lens, new_lens, block_table, free_slots, free_head, block_size,
              null_slot=0):
    """Extends ``block_table`` in place; returns a dict of the outputs and the
    number of requests reported."""
    B, max_blocks = block_table.shape
    head = int(free_head)
    n_free = len(free_slots)
    bad = 0
    avail = n_free - head if 0 <= head <= n_free else 0
    taken, exhausted = 0, False
    qsl, rows = [0], []
    for b in range(B):
        c, n = int(computed_lens[b]), int(new_lens[b])
        qsl.append(qsl[-1] + max(n, 0))
        row = (null_slot, null_slot, null_slot, 0)
        rows.append(row)
        if c < 0 or n < 0 or c + n > max_blocks * block_size:
            bad += 1
            continue
        if n == 0:
            continue
        cur = (c - 1) // block_size if c > 0 else -1
        last = (c + n - 1) // block_size
        src = int(block_table[b, cur]) if c > 0 else null_slot
        if c > 0 and src <= null_slot:
            bad += 1
            continue
        m = last * block_size - c
        need = int(last != cur) + int(m > 0 and last - 1 != cur)
        if need and (exhausted or taken + need > avail):
            exhausted = True
            bad += 1
            continue
        bnd = null_slot
        if m > 0:
            for j in range(cur + 1, last - 1):
                block_table[b, j] = null_slot
            if last - 1 != cur:
                block_table[b, last - 1] = free_slots[head + taken]
                taken += 1
            bnd = int(block_table[b, last - 1])
        if last != cur:
            block_table[b, last] = free_slots[head + taken]
            taken += 1
        rows[-1] = (src, int(block_table[b, last]), bnd, max(m, 0))
    cols = np.array(rows, dtype=np.int32).reshape(B, 4)
    return dict(query_start_loc=np.array(qsl, dtype=np.int32), sources=cols[:, 0],
                destinations=cols[:, 1], boundaries=cols[:, 2], boundary_lens=cols[:, 3],
                free_next=np.array([head + taken], dtype=np.int32)), bad
