"""FP64 CPU oracle of the tree operators: the convolution over trees
(``conv``), the delta rule over trees (``verify``), drafts against the
target's probabilities (``accept``) and the accepted path to the front
(``select``).  TEST INFRASTRUCTURE ONLY, like ``kda_oracle``, whose exact
conversions it uses; it shares no code with the library.

The rule is the stock sequential recurrence (page "...cutedsl.kda.fused",
module docstring, step 2) taken down every path of a tree, one state a node.
"""
from __future__ import annotations

import numpy as np

from .kda_oracle import bf16_to_f64, f64_to_bf16, f64_to_state, l2norm, sigmoid, state_to_f64

MAX_NODES, MAX_DEPTH = 64, 8


def windows(qsl, B, Q, n_tokens):
    """(first token, length) of every request; None for a bad window."""
    out = []
    for b in range(B):
        t0, t1 = (b * Q, (b + 1) * Q) if qsl is None else (int(qsl[b]), int(qsl[b + 1]))
        out.append((t0, t1 - t0) if 0 <= t0 <= t1 <= n_tokens and t1 - t0 <= Q else None)
    return out


def tree(parents, t0, n):
    """The request's parents; None where they are no tree of the operators'."""
    par = list(range(-1, n - 1)) if parents is None else [int(a) for a in parents[t0:t0 + n]]
    depth = []
    for t, a in enumerate(par):
        if not -1 <= a < t:
            return None
        depth.append(1 if a < 0 else depth[a] + 1)
    return None if any(d > MAX_DEPTH for d in depth) else par


def _requests(*, state_slots, record_rows, pending, rq, n_slots, n_rows, parents, qsl, n_tokens,
              Q, null_slot, trees=True):
    """Per request: None (reported), or (slot or None, row or None, pending
    count, t0, parents or length)."""
    out = []
    for b, win in enumerate(windows(qsl, len(state_slots), Q, n_tokens)):
        if win is None:
            out.append(None)
            continue
        t0, n = win
        slot = int(state_slots[b])
        if slot <= null_slot:
            out.append((None, None, 0, t0, n))
            continue
        row = b if record_rows is None else int(record_rows[b])
        if slot >= n_slots or row >= n_rows:
            out.append(None)
            continue
        par = tree(parents, t0, n) if trees else n
        if par is None:
            out.append(None)
            continue
        m = 0
        if pending is not None and row >= 0:
            m = min(max(int(pending[row]), 0), rq)
        out.append((slot, row if row >= 0 else None, m, t0, par))
    return out


def conv(*, x, conv_weight, conv_bias, conv_state, state_slots, parents, q, k, v, Q,
         record_rows=None, pending=None, query_start_loc=None, null_slot=0, out_f64=None):
    """In place on q, k, v [T, H, 128] (BF16 bits; out_f64 [T, 3, H, 128]).
    Returns the number of requests reported."""
    T, D3 = x.shape
    D = D3 // 3
    w = bf16_to_f64(conv_weight).transpose(1, 0, 2).reshape(4, D3)
    bias = np.zeros(D3) if conv_bias is None else bf16_to_f64(conv_bias)
    reqs = _requests(state_slots=state_slots, record_rows=record_rows if pending is not None else None,
                     pending=pending, rq=conv_state.shape[2] - 2, n_slots=conv_state.shape[0],
                     n_rows=len(pending) if pending is not None else len(state_slots),
                     parents=parents, qsl=query_start_loc, n_tokens=T, Q=Q, null_slot=null_slot)
    for req in reqs:
        if req is None or req[0] is None:
            continue
        slot, _, m, t0, par = req
        off = m - 1 if m > 0 else 0
        above = bf16_to_f64(conv_state[slot, :, off:off + 3]).T  # oldest first
        node = bf16_to_f64(x[t0:t0 + len(par)])
        for t in range(len(par)):
            s, a = [node[t]], par[t]
            while len(s) < 4:
                if a >= 0:
                    s.append(node[a])
                    a = par[a]
                else:
                    s.append(above[3 + a])  # -1: the newest
                    a -= 1
            z = bias + sum(w[i] * s[3 - i] for i in range(4))
            y = (z * sigmoid(z)).reshape(3, -1, 128)
            for i, o in enumerate((q, k, v)):
                o[t0 + t] = f64_to_bf16(y[i])
            if out_f64 is not None:
                out_f64[t0 + t] = y
    return sum(req is None for req in reqs)


def verify(*, q, k, v, raw_g, raw_beta, A_log, dt_bias, lower_bound, q_scale, state, state_slots,
           parents, node_corr, out, Q, record_rows=None, pending=None, corr=None, key_gate=None,
           query_start_loc=None, null_slot=0, out_f64=None):
    """In place on ``state`` [slots, H, V, K] (FP32, or BF16 bits), node_corr
    [T, H, 128] and out (BF16 bits).  Returns the number reported."""
    T = len(q)
    replay = pending is not None
    reqs = _requests(state_slots=state_slots, record_rows=record_rows if replay else None,
                     pending=pending, rq=corr.shape[2] if replay else 0, n_slots=state.shape[0],
                     n_rows=len(corr) if replay else len(state_slots), parents=parents,
                     qsl=query_start_loc, n_tokens=T, Q=Q, null_slot=null_slot)
    a, dt = np.exp(A_log.astype(np.float64))[:, None], dt_bias.astype(np.float64)
    decay = lambda g: np.exp(lower_bound * sigmoid(a * (bf16_to_f64(g) + dt)))
    for req in reqs:
        if req is None:
            continue
        slot, row, m, t0, par = req
        if slot is None:
            out[t0:t0 + par] = 0
            if out_f64 is not None:
                out_f64[t0:t0 + par] = 0
            continue
        S0 = state_to_f64(state[slot])
        for t in range(m):
            kn = l2norm(bf16_to_f64(key_gate[row, :, t, :128]))
            S0 = S0 * decay(key_gate[row, :, t, 128:])[:, None]
            S0 = S0 + corr[row, :, t].astype(np.float64)[..., None] * kn[:, None]
        if m > 0:
            state[slot] = f64_to_state(S0, state.dtype)
        states = []
        for t, p in enumerate(par):
            S = (S0 if p < 0 else states[p]) * decay(raw_g[t0 + t])[:, None]
            kn, qn = l2norm(bf16_to_f64(k[t0 + t])), l2norm(bf16_to_f64(q[t0 + t])) * q_scale
            beta = sigmoid(bf16_to_f64(raw_beta[t0 + t]))[:, None]
            u = beta * (bf16_to_f64(v[t0 + t]) - np.einsum("hvk,hk->hv", S, kn))
            S = S + u[..., None] * kn[:, None]
            o = np.einsum("hvk,hk->hv", S, qn)
            states.append(S)
            node_corr[t0 + t] = u
            out[t0 + t] = f64_to_bf16(o)
            if out_f64 is not None:
                out_f64[t0 + t] = o
    return sum(req is None for req in reqs)


def accept(*, target, tokens, accept_uniforms, sample_uniforms, Q, draft=None, parents=None,
           state_slots=None, query_start_loc=None, null_slot=0):
    """(accepted [B], path [B, 8], next_tokens [B], number reported); target
    and draft [T, V] as float64."""
    B, V = len(sample_uniforms), target.shape[1]
    accepted, nexts = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    paths = np.full((B, MAX_DEPTH), -1, np.int32)
    bad = 0
    positive = lambda w: np.where(w > 0, w, 0.0)
    for b, win in enumerate(windows(query_start_loc, B, Q, len(tokens))):
        if win is None:
            bad += 1
            continue
        t0, n = win
        if n == 0 or (state_slots is not None and state_slots[b] <= null_slot):
            continue
        par = tree(parents, t0, n)
        x = [int(t) for t in tokens[t0:t0 + n]]
        if par is None or par[0] != -1 or min(par[1:], default=0) < 0 or \
                any(not 0 <= t < V for t in x[1:]):
            bad += 1
            continue
        path = [0]
        while True:
            cur = path[-1]
            p, u = target[t0 + cur], float(accept_uniforms[t0 + cur])
            children = [t for t in range(1, n) if par[t] == cur]
            taken, total, seen = None, 0.0, set()
            for t in children:
                if draft is not None:
                    hit = u * draft[t0 + t, x[t]] < positive(p[x[t]])
                elif x[t] in seen:
                    continue
                else:
                    seen.add(x[t])
                    total += float(positive(p[x[t]]))
                    hit = u < total
                if hit:
                    taken = t
                    break
            if taken is None:
                break
            path.append(taken)
        weight = positive(p)
        if children and draft is not None:
            q = draft[t0 + children[0]]
            weight = np.where(p > q, p - q, 0.0)
        elif children:
            weight = weight.copy()
            weight[[x[t] for t in children]] = 0.0
        if not weight.sum() > 0:
            weight = positive(p)
        accepted[b] = len(path)
        paths[b, :len(path)] = path
        sums = np.cumsum(weight.astype(np.longdouble))
        if not (sums[-1] > 0 and np.isfinite(sums[-1])):
            bad += 1
            continue
        past = np.flatnonzero((sums > np.longdouble(float(sample_uniforms[b])) * sums[-1]) & (weight > 0))
        nexts[b] = past[0] if len(past) else np.flatnonzero(weight > 0)[-1]
    return accepted, paths, nexts, bad


def select(*, path, accepted, k, raw_g, node_corr, state_slots, record_rows, corr, key_gate, Q,
           x=None, conv_state=None, pending=None, eager=None, query_start_loc=None, null_slot=0,
           n_slots=1 << 30):
    """In place on corr, key_gate and conv_state.  Returns the number
    reported."""
    width = conv_state.shape[2] if conv_state is not None else 0
    rq = corr.shape[2]
    reqs = _requests(state_slots=state_slots, record_rows=record_rows,
                     pending=pending if width else None, rq=width - 2,
                     n_slots=conv_state.shape[0] if width else n_slots, n_rows=len(corr),
                     parents=None, qsl=query_start_loc, n_tokens=len(k), Q=Q,
                     null_slot=null_slot, trees=False)
    bad = 0
    for b, req in enumerate(reqs):
        if req is None:
            bad += 1
            continue
        slot, row, m, t0, n = req
        if slot is None or row is None:
            continue
        count = int(accepted[b])
        if not 0 <= count <= (min(rq, width - 2) if width else rq) or \
                any(not 0 <= t < n for t in path[b, :count]):
            bad += 1
            continue
        at = [t0 + int(t) for t in path[b, :count]]
        corr[row, :, :count] = node_corr[at].transpose(1, 0, 2)
        key_gate[row, :, :count, :128] = k[at].transpose(1, 0, 2)
        key_gate[row, :, :count, 128:] = raw_g[at].transpose(1, 0, 2)
        if width:
            W = conv_state[slot].copy()
            off = m - 1 if m > 0 else 0
            if count == 0 or (eager is not None and eager[b]):
                conv_state[slot, :, :3] = np.concatenate([W[:, off:off + 3], x[at].T], 1)[:, -3:]
            else:
                conv_state[slot, :, :2] = W[:, off + 1:off + 3]
                conv_state[slot, :, 2:2 + count] = x[at].T
    return bad
