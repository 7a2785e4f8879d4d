"""The operators that take a prompt in and decode from it, as measured cases.

* ``prefill``: the gated delta rule of KDA over ragged prompts, from and to
  slots of a state pool (``kda_prefill``);
* ``recurrent``: the same rule token by token, one to a few tokens per
  request, the state advanced in place (``kda_recurrent``);
* ``conv``: the layer's short convolution and SiLU over ragged prompts, with
  the window that decoding goes on from (``kda_prefill_conv``);
* ``plan``: packed offsets, block table entries and slot maps from the
  requests' lengths (``kda_slot_plan``).

``run`` computes them in elementary torch operations where ``own`` is false,
and calls the library where it is true.
"""
import math
import random

import torch

own = False

DIM = 128          # key and value channels per head
CHUNK = 32         # tokens per step of the plain chunked form
LOWER_BOUND = -5.0
Q_SCALE = DIM ** -0.5
EPS = 1e-6         # inside the root of the L2 norms
NULL = 0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one short prompt on its own: the time to its first token
        dict(name="prefill-short", op="prefill", B=1, T=37, H=32, pool="f32", resume=False),
        # a scheduler's step of a few prompts that go on from a cached prefix,
        # each leaving a block boundary's state behind
        dict(name="prefill-resume", op="prefill", B=4, T=2047, H=32, pool="f32", resume=True),
        # one long document: nothing but its heads runs side by side
        dict(name="prefill-long", op="prefill", B=1, T=16384, H=32, pool="f32", resume=False),
        # a full batch of ragged prompts, BF16 checkpoints
        dict(name="prefill-batch", op="prefill", B=16, T=16384, H=32, pool="bf16", resume=False),
        # a wider model, prompts of a few thousand tokens, resumed
        dict(name="prefill-wide", op="prefill", B=6, T=8191, H=64, pool="f32", resume=True),
        # one user decoding
        dict(name="decode-one", op="recurrent", B=1, Q=1, H=32, pool="f32"),
        # a serving batch with BF16 checkpoints, three tokens per request
        dict(name="decode-bf16", op="recurrent", B=100, Q=3, H=32, pool="bf16"),
        # the largest serving batch
        dict(name="decode-batch", op="recurrent", B=512, Q=1, H=64, pool="f32"),
        # the convolution before a short prompt, and before a full batch
        dict(name="conv-short", op="conv", B=1, T=37, H=32, bias=False, resume=False),
        dict(name="conv-batch", op="conv", B=16, T=16384, H=32, bias=True, resume=True),
        # the slot maps of a small step and of a very large one
        dict(name="plan-step", op="plan", B=48, block=64, max_new=600, max_blocks=64),
        dict(name="plan-wide", op="plan", B=8192, block=16, max_new=4000, max_blocks=512),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "recurrent", "conv", "plan"])
    if op in ("prefill", "conv"):
        H = rng.choice([1, 2, 4, 7, 16, 32, 64])
        T = _log_int(rng, 1, 16384 * 32 // max(H, 32))
        B = _log_int(rng, 1, min(T, 64))
        c = dict(op=op, B=B, T=T, H=H, resume=rng.random() < 0.5)
        if op == "prefill":
            c["pool"] = rng.choice(["f32", "bf16"])
        else:
            c["bias"] = rng.random() < 0.5
        return c
    if op == "recurrent":
        H = rng.choice([1, 2, 4, 7, 16, 32, 64])
        return dict(op=op, B=_log_int(rng, 1, 16384 // H if H > 32 else 256), Q=rng.choice([1, 1, 2, 3, 5, 8]),
                    H=H, pool=rng.choice(["f32", "bf16"]))
    block = rng.choice([1, 8, 16, 64, 100, 256])
    max_blocks = _log_int(rng, 4, 512)
    return dict(op=op, B=_log_int(rng, 1, 8192), block=block,
                max_new=_log_int(rng, 1, max(1, block * max_blocks // 2)), max_blocks=max_blocks)


def _lens(case):
    """The prompts' lengths: a ragged split of T tokens over B requests, the
    same for every seed (they are part of the case)."""
    B, T = case["B"], case["T"]
    r = random.Random(B * 1000003 + T)
    cuts = sorted(r.sample(range(1, T), B - 1)) if B > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _boundary_lens(case):
    """Tokens of each prompt up to the last boundary of 64-token blocks inside
    it, counted from where its cached prefix ends; 0 where there is none."""
    lens = _lens(case)
    if not case["resume"]:
        return [0] * len(lens)
    prefix = [100 + 37 * b for b in range(len(lens))]
    return [max(0, (p + n - 1) // 64 * 64 - p) for p, n in zip(prefix, lens)]


# --------------------------------------------------------------------------
# what a program has in hand
# --------------------------------------------------------------------------

def _randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _gate_weights(gen, H):
    """Per-head A_log and per-channel dt_bias whose channels forget over one
    to a thousand tokens (log-uniform), as a trained layer's do."""
    A_log = torch.rand(H, generator=gen, device="cuda") * 1.5
    share = torch.exp(torch.rand(H, DIM, generator=gen, device="cuda") * math.log(1000.0)) / 5000.0
    dt_bias = torch.log(share / (1 - share)) / torch.exp(A_log)[:, None]
    return A_log, dt_bias


def _step_inputs(gen, s, T, H):
    bf = torch.bfloat16
    for name in ("q", "k", "v", "raw_g"):
        s[name] = _randn(gen, T, H, DIM).to(bf)
    s["raw_beta"] = _randn(gen, T, H).to(bf)
    s["A_log"], s["dt_bias"] = _gate_weights(gen, H)


def _slots(gen, n, first):
    return (torch.randperm(n, generator=gen, device="cuda") + first).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "plan":
        B, bs, mb = case["B"], case["block"], case["max_blocks"]
        room = bs * mb
        new = (torch.rand(B, generator=gen, device="cuda") ** 3 * case["max_new"]).long() + 1
        idle = torch.rand(B, generator=gen, device="cuda") < 0.05
        new = torch.where(idle, 0, new).clamp(max=room)
        at = (torch.rand(B, generator=gen, device="cuda") * (room - new + 1)).long()
        at = torch.where(torch.rand(B, generator=gen, device="cuda") < 0.3, 0, at)
        s["computed"], s["new"] = at.to(torch.int32), new.to(torch.int32)
        # each request has held a slot of its own for every block so far
        slots = torch.randperm(B * mb + 2 * B, generator=gen, device="cuda").to(torch.int32) + 1
        held = torch.arange(mb, device="cuda") < ((at + bs - 1) // bs)[:, None]
        s["table"] = torch.where(held, slots[:B * mb].view(B, mb), NULL).to(torch.int32)
        s["free"] = slots[B * mb:].contiguous()
        s["head"] = _int32([0])
        return s
    H, B = case["H"], case["B"]
    if op == "recurrent":
        T = B * case["Q"]
        _step_inputs(gen, s, T, H)
        pool = _randn(gen, B + 1, H, DIM, DIM, std=0.05)
        s["pool"] = pool if case["pool"] == "f32" else pool.to(torch.bfloat16)
        s["slots"] = _slots(gen, B, 1)
        return s
    lens = _lens(case)
    T = case["T"]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s["lens"], s["qsl"], s["max_len"] = lens, _int32(starts), max(lens)
    resume = case["resume"]
    # slots: the state a prompt goes on from, the one it leaves, and the one
    # of the last block boundary inside it
    slots = _slots(gen, 3 * B, 1)
    s["dst"] = slots[:B].contiguous()
    s["src"] = slots[B:2 * B].contiguous() if resume else _int32([NULL] * B)
    bnd = _boundary_lens(case)
    s["bnd_host"], s["bnd_lens"] = bnd, _int32(bnd)
    s["bnd"] = torch.where(s["bnd_lens"] > 0, slots[2 * B:], NULL).to(torch.int32)
    n_slots = 3 * B + 1
    if op == "prefill":
        _step_inputs(gen, s, T, H)
        pool = _randn(gen, n_slots, H, DIM, DIM, std=0.05)
        s["pool"] = pool if case["pool"] == "f32" else pool.to(torch.bfloat16)
    else:
        D = H * DIM
        s["x"] = _randn(gen, T, 3 * D).to(torch.bfloat16)
        s["w"] = _randn(gen, 3, 4, D, std=0.5).to(torch.bfloat16)
        s["bias"] = _randn(gen, 3 * D, std=0.1).to(torch.bfloat16) if case["bias"] else None
        s["conv_state"] = _randn(gen, n_slots, 3 * D, 6).to(torch.bfloat16)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    return {"prefill": _prefill, "recurrent": _recurrent, "conv": _conv, "plan": _plan}[s["op"]](s)


def _gate(s, raw_g):
    """log of the decay, [.., H, 128]."""
    a = torch.exp(s["A_log"])[:, None]
    return LOWER_BOUND * torch.sigmoid(a * (raw_g.float() + s["dt_bias"]))


def _unit(x):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _prefill(s):
    T, H = s["q"].shape[:2]
    out = torch.empty_like(s["v"])
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_prefill
        kda_prefill(s["q"], s["k"], s["v"], s["raw_g"], s["raw_beta"], s["A_log"], s["dt_bias"],
                    s["pool"], s["src"], s["dst"], s["qsl"], out, Q=s["max_len"],
                    lower_bound=LOWER_BOUND, q_scale=Q_SCALE, boundaries=s["bnd"],
                    boundary_lens=s["bnd_lens"])
        return {"out": out, "state": s["pool"]}
    # The tokens of every prompt in places of a padded table, its boundary at
    # a chunk's end, so that the state there is one that a chunk leaves.
    dev, C, B = out.device, CHUNK, len(s["lens"])
    lens, m = torch.tensor(s["lens"], device=dev), torch.tensor(s["bnd_host"], device=dev)
    m_up = (m + C - 1) // C * C
    steps = max((b + C - 1) // C + (n - b + C - 1) // C for n, b in zip(s["lens"], s["bnd_host"]))
    place = torch.arange(steps * C, device=dev)
    tok = torch.where(place < m_up[:, None], place, place - m_up[:, None] + m[:, None])
    live = torch.where(place < m_up[:, None], place < m[:, None], tok < lens[:, None])
    tok = torch.where(live, tok + s["qsl"][:-1].long()[:, None], T)
    grow = lambda x: torch.cat([x, torch.zeros_like(x[:1])])  # row T: no token
    q, k, v, raw_g, raw_beta = (grow(s[n]) for n in ("q", "k", "v", "raw_g", "raw_beta"))
    out_rows = torch.zeros(T + 1, H, DIM, dtype=out.dtype, device=dev)
    src, dst, bnd = s["src"].long(), s["dst"].long(), s["bnd"].long()
    S = s["pool"][src].float() * (src > NULL)[:, None, None, None]
    S_bnd = torch.zeros_like(S)
    tri = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    eye = torch.eye(C, device=dev)
    for c in range(steps):
        at, there = tok[:, c * C:(c + 1) * C], live[:, c * C:(c + 1) * C]
        heads = lambda x: x[at].transpose(1, 2)  # [B, H, C, ..]
        there = there[:, None, :, None]
        qn, kn = _unit(heads(q)) * Q_SCALE, _unit(heads(k)) * there
        g = _gate(s, raw_g[at]).transpose(1, 2) * there
        beta = torch.sigmoid(heads(raw_beta).float())[..., None] * there
        # the decays between two tokens of the chunk; their exponents are
        # differences of long sums, kept in 64 bits
        G = g.double().cumsum(2)
        between = (G[:, :, :, None] - G[:, :, None, :]).float().clamp_(max=0).exp_()
        between = between * tri[:, :, None]
        kk = (kn[:, :, :, None] * kn[:, :, None] * between).sum(-1)
        qk = (qn[:, :, :, None] * kn[:, :, None] * between).sum(-1)
        L = (beta * kk).tril(-1)
        # (I + L)^-1 = (I - L)(I + L^2)(I + L^4)...: L^C = 0
        inv, P = eye - L, L @ L
        inv = inv + inv @ P
        P = P @ P
        inv = inv + inv @ P
        P = P @ P
        inv = inv + inv @ P
        P = P @ P
        inv = inv + inv @ P
        down = G.exp().float()
        left = (G[:, :, -1:] - G).exp().float()
        R = heads(v).float() - (kn * down) @ S.transpose(-1, -2)
        U = inv @ (beta * R)
        o = (qn * down) @ S.transpose(-1, -2) + qk @ U
        S = S * down[:, :, -1:] + U.transpose(-1, -2) @ (kn * left)
        S_bnd = torch.where(((c + 1) * C == m_up)[:, None, None, None], S, S_bnd)
        out_rows[at] = o.transpose(1, 2).to(out.dtype)
    out.copy_(out_rows[:T])
    s["pool"][dst] = S.to(s["pool"].dtype)
    has = bnd > NULL
    s["pool"][torch.where(has, bnd, dst)] = torch.where(has[:, None, None, None], S_bnd, S).to(s["pool"].dtype)
    return {"out": out, "state": s["pool"]}


def _recurrent(s):
    out = torch.empty_like(s["v"])
    Q = s["case"]["Q"]
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_recurrent
        kda_recurrent(s["q"], s["k"], s["v"], s["raw_g"], s["raw_beta"], s["A_log"], s["dt_bias"],
                      s["pool"], s["slots"], s["slots"], out, Q=Q, lower_bound=LOWER_BOUND,
                      q_scale=Q_SCALE)
        return {"out": out, "state": s["pool"]}
    slots = s["slots"].long()
    S = s["pool"][slots].float()
    for t in range(Q):
        q, k = _unit(s["q"][t::Q]) * Q_SCALE, _unit(s["k"][t::Q])
        S = S * torch.exp(_gate(s, s["raw_g"][t::Q]))[:, :, None]
        beta = torch.sigmoid(s["raw_beta"][t::Q].float())[..., None]
        u = beta * (s["v"][t::Q].float() - (S * k[:, :, None]).sum(-1))
        S = S + u[..., None] * k[:, :, None]
        out[t::Q] = (S * q[:, :, None]).sum(-1).to(out.dtype)
    s["pool"][slots] = S.to(s["pool"].dtype)
    return {"out": out, "state": s["pool"]}


def _conv(s):
    T, D = s["x"].shape[0], s["x"].shape[1] // 3
    H = D // DIM
    q, k, v = (torch.empty(T, H, DIM, dtype=torch.bfloat16, device=s["x"].device) for _ in range(3))
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_prefill_conv
        kda_prefill_conv(s["x"], s["w"], s["bias"], s["conv_state"], s["src"], s["dst"], s["qsl"],
                         q, k, v, Q=s["max_len"], boundaries=s["bnd"], boundary_lens=s["bnd_lens"])
        return {"q": q, "k": k, "v": v, "window": s["conv_state"]}
    x, dev = s["x"], s["x"].device
    src, dst, bnd = s["src"].long(), s["dst"].long(), s["bnd"].long()
    old = s["conv_state"][src][:, :, :3].transpose(1, 2) * (src > NULL)[:, None, None]  # [B, 3, 3 D]
    starts = s["qsl"][:-1].long()
    request = torch.bucketize(torch.arange(T, device=dev), s["qsl"][1:].long(), right=True)

    def entry(b, at):
        """Entry `at` of request b's inputs; -3 .. -1 are the window's."""
        from_x = x[(starts[b] + at).clamp(0, T - 1)]
        return torch.where((at < 0)[:, None], old[b, (at + 3).clamp(0, 2)], from_x)

    t = torch.arange(T, device=dev) - starts[request]
    w = s["w"].float().permute(1, 0, 2).reshape(4, 3 * D)
    y = sum(w[i] * entry(request, t + i - 3).float() for i in range(4))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = (y * torch.sigmoid(y)).to(torch.bfloat16)
    for i, o in enumerate((q, k, v)):
        o.copy_(y[:, i * D:(i + 1) * D].reshape(T, H, DIM))
    b = torch.arange(len(s["lens"]), device=dev)
    n = s["qsl"].long().diff()
    to = torch.where(bnd > NULL, bnd, dst)
    m = torch.where(bnd > NULL, s["bnd_lens"].long(), n)
    end = [torch.stack([entry(b, at - 3 + i) for i in range(3)], dim=2) for at in (n, m)]
    s["conv_state"][dst, :, :3] = end[0]
    s["conv_state"][to, :, :3] = end[1]
    return {"q": q, "k": k, "v": v, "window": s["conv_state"]}


def _plan(s):
    B, bs = s["case"]["B"], s["case"]["block"]
    dev = s["computed"].device
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_slot_plan
        qsl = torch.empty(B + 1, dtype=torch.int32, device=dev)
        src, dst, bnd, bnd_lens = torch.empty(4, B, dtype=torch.int32, device=dev)
        nxt = torch.empty(1, dtype=torch.int32, device=dev)
        kda_slot_plan(s["computed"], s["new"], s["table"], s["free"], s["head"], nxt, qsl, src,
                      dst, bnd, bnd_lens, block_size=bs)
        return dict(qsl=qsl, sources=src, destinations=dst, boundaries=bnd, boundary_lens=bnd_lens,
                    free_next=nxt, table=s["table"])
    c, n, table = s["computed"].long(), s["new"].long(), s["table"]
    live = n > 0
    last = (c + n - 1) // bs                 # the block the state ends in
    cur = torch.where(c > 0, (c - 1) // bs, -1)  # the block it is in now
    crosses = live & (last * bs > c)
    new_last = live & (last != cur)
    new_bnd = crosses & (last - 1 != cur)
    need = new_last.long() + new_bnd.long()
    first = s["head"].long() + need.cumsum(0) - need
    free = s["free"]
    take = lambda at: free[at.clamp(0, free.shape[0] - 1)]
    rows = torch.arange(B, device=dev)
    slot_last = torch.where(new_last, take(first + new_bnd.long()), table[rows, last.clamp(min=0)])
    slot_bnd = torch.where(new_bnd, take(first), table[rows, (last - 1).clamp(min=0)])
    src = torch.where(live & (c > 0), table[rows, cur.clamp(min=0)], NULL)
    j = torch.arange(table.shape[1], device=dev)
    skipped = live[:, None] & (j > cur[:, None]) & (j < (last - 1)[:, None])
    filled = torch.where(skipped, NULL, table)
    filled = torch.where(new_bnd[:, None] & (j == (last - 1)[:, None]), slot_bnd[:, None], filled)
    table.copy_(torch.where(new_last[:, None] & (j == last[:, None]), slot_last[:, None], filled))
    qsl = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    qsl[1:] = n.cumsum(0)
    i32 = lambda x: x.to(torch.int32)
    return dict(qsl=qsl, sources=i32(src), destinations=i32(torch.where(live, slot_last, NULL)),
                boundaries=i32(torch.where(crosses, slot_bnd, NULL)),
                boundary_lens=i32(torch.where(crosses, last * bs - c, 0)),
                free_next=i32(s["head"] + need.sum()), table=table)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op, B = case["op"], case["B"]
    if op == "plan":
        # lengths in; offsets, four maps out; a table entry read and at most
        # two free slots read and two entries written per request
        return {"bytes": 4.0 * B * (2 + 1 + 4 + 1 + 4), "flops": 0.0}
    H = case["H"]
    if op == "conv":
        D, T = H * DIM, case["T"]
        held = 3 * 3 * D * 2.0 * B
        return {"bytes": 12.0 * D * T + 24.0 * D + held * (3 if case["resume"] else 1),
                "flops": 3.0 * D * T * 12}
    T = B * case["Q"] if op == "recurrent" else case["T"]
    page = H * DIM * DIM * (4.0 if case["pool"] == "f32" else 2.0)
    if op == "recurrent":
        pages = 2 * B
    else:
        # the boundary's state where the prompt crosses one
        pages = B + (B if case["resume"] else 0) + sum(m > 0 for m in _boundary_lens(case))
    return {"bytes": T * H * (5 * 2.0 * DIM + 2) + pages * page, "flops": 7.0 * DIM * DIM * T * H}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_rule, "recurrent": _exact_rule, "conv": _exact_conv, "plan": _exact_plan}[s["op"]](s)


def _exact_rule(s):
    """The recurrence token by token: S <- S diag(d); u = beta (v - S k);
    S <- S + u k^T; o = S q."""
    case = s["case"]
    f = lambda x: x.to(torch.float64)
    pool = f(s["pool"])
    if s["op"] == "recurrent":
        B, Q = case["B"], case["Q"]
        lens, m = [Q] * B, [0] * B
        src = dst = s["slots"].long()
        bnd = torch.zeros_like(src)
        starts = torch.arange(B, device=src.device) * Q
    else:
        lens, m = s["lens"], s["bnd_host"]
        src, dst, bnd = s["src"].long(), s["dst"].long(), s["bnd"].long()
        starts = s["qsl"][:-1].long()
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=src.device)
    # requests longest first, so that those still running are a leading part
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    o_idx = torch.tensor(order, device=src.device)
    starts_o = starts[o_idx]
    S = pool[src[o_idx]] * (src[o_idx] > NULL)[:, None, None, None]
    a, dt = torch.exp(f(s["A_log"]))[:, None], f(s["dt_bias"])
    running = len(order)
    for t in range(max(lens)):
        while lens[order[running - 1]] <= t:
            running -= 1
        at = starts_o[:running] + t
        k, q = f(s["k"][at]), f(s["q"][at])
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS) * Q_SCALE
        d = torch.exp(LOWER_BOUND / (1 + torch.exp(-a * (f(s["raw_g"][at]) + dt))))
        beta = 1 / (1 + torch.exp(-f(s["raw_beta"][at])))
        part = S[:running]
        part.mul_(d[:, :, None])
        u = beta[..., None] * (f(s["v"][at]) - torch.einsum("bhvk,bhk->bhv", part, k))
        part.addcmul_(u[..., None], k[:, :, None])
        out[at] = torch.einsum("bhvk,bhk->bhv", part, q)
        for i in range(running):
            if m[order[i]] == t + 1:
                pool[bnd[order[i]]] = S[i]
    pool[dst[o_idx]] = S
    return {"out": out, "state": pool}


def _exact_conv(s):
    f = lambda x: x.to(torch.float64)
    D = s["x"].shape[1] // 3
    H = D // DIM
    w = f(s["w"]).transpose(0, 1).reshape(4, 3 * D)
    window, ys, at = f(s["conv_state"]), [], 0
    for b, n in enumerate(s["lens"]):
        src, dst, bnd = int(s["src"][b]), int(s["dst"][b]), int(s["bnd"][b])
        head = f(s["conv_state"][src, :, :3]).t() if src > NULL else torch.zeros(3, 3 * D, dtype=torch.float64, device=w.device)
        line = torch.cat([head, f(s["x"][at:at + n])])
        y = w[0] * line[:n] + w[1] * line[1:n + 1] + w[2] * line[2:n + 2] + w[3] * line[3:n + 3]
        if s["bias"] is not None:
            y = y + f(s["bias"])
        ys.append(y / (1 + torch.exp(-y)))
        window[dst, :, :3] = line[n:n + 3].t()
        if bnd > NULL:
            m = s["bnd_host"][b]
            window[bnd, :, :3] = line[m:m + 3].t()
        at += n
    y = torch.cat(ys)
    q, k, v = (y[:, i * D:(i + 1) * D].reshape(-1, H, DIM) for i in range(3))
    return {"q": q, "k": k, "v": v, "window": window}


def _exact_plan(s):
    bs = s["case"]["block"]
    computed, new, free = s["computed"].tolist(), s["new"].tolist(), s["free"].tolist()
    table = s["table"].cpu().numpy().copy()
    head = int(s["head"])
    qsl, maps = [0], []
    for b, (c, n) in enumerate(zip(computed, new)):
        qsl.append(qsl[-1] + n)
        if n == 0:
            maps.append((NULL, NULL, NULL, 0))
            continue
        cur, last = (c - 1) // bs if c else -1, (c + n - 1) // bs
        source = int(table[b, cur]) if c else NULL
        table[b, cur + 1:max(cur + 1, last - 1)] = NULL
        boundary, length = NULL, 0
        if last * bs > c:
            length = last * bs - c
            if last - 1 != cur:
                table[b, last - 1] = free[head]
                head += 1
            boundary = int(table[b, last - 1])
        if last != cur:
            table[b, last] = free[head]
            head += 1
        maps.append((source, int(table[b, last]), boundary, length))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    src, dst, bnd, bnd_lens = (i32([r[i] for r in maps]) for i in range(4))
    return dict(qsl=i32(qsl), sources=src, destinations=dst, boundaries=bnd, boundary_lens=bnd_lens,
                free_next=i32([head]), table=torch.from_numpy(table))
