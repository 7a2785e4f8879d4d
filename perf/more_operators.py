"""The operators of speculation with trees of drafted tokens, as measured cases.

* ``conv``: the layer's short convolution and SiLU over the nodes of a tree,
  each behind its own ancestors (``kda_tree_conv``);
* ``verify``: the gated delta rule of KDA over a tree of drafted tokens, from
  the request's checkpoint, the pending replay folded in (``kda_tree_verify``);
* ``accept``: the drafted tokens against the target's probabilities, from
  given random numbers, and the token that follows (``kda_draft_accept``);
* ``select``: the accepted path's records and inputs moved to where the next
  step's replay and convolution read them (``kda_tree_select``).

``run`` computes them in elementary torch operations where ``own`` is false,
and calls the library where it is true.
"""
import math
import random

import torch

own = False

DIM = 128          # key and value channels per head
DEPTH = 8          # tokens of the longest path of a tree
LOWER_BOUND = -5.0
Q_SCALE = DIM ** -0.5
EPS = 1e-6         # inside the root of the L2 norms


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one user: a small tree through one layer
        dict(name="conv-one", op="conv", B=1, N=15, H=32, ragged=False, bias=False),
        # a full batch's trees
        dict(name="conv-batch", op="conv", B=128, N=33, H=64, ragged=True, bias=True),
        # one user: a small tree, a replay pending
        dict(name="verify-one", op="verify", B=1, N=15, H=32, ragged=False, pool="f32", replay=True),
        # a serving batch, trees of different sizes
        dict(name="verify-ragged", op="verify", B=48, N=32, H=32, ragged=True, pool="f32", replay=True),
        # BF16 checkpoints, which are only read
        dict(name="verify-bf16", op="verify", B=100, N=24, H=32, ragged=False, pool="bf16", replay=False),
        # the largest: wide trees of a full batch, a wider model
        dict(name="verify-wide", op="verify", B=128, N=64, H=64, ragged=False, pool="f32", replay=True),
        # one user: a chain of three drafts with their probabilities
        dict(name="accept-one", op="accept", B=1, N=4, V=32000, tree=False, draft=True, probs="f32", ragged=False),
        # a full batch of chains
        dict(name="accept-batch", op="accept", B=256, N=8, V=131072, tree=False, draft=True, probs="f32",
             ragged=False),
        # trees of the likeliest tokens, an odd vocabulary, BF16 probabilities
        dict(name="accept-tree", op="accept", B=64, N=24, V=100003, tree=True, draft=False, probs="bf16",
             ragged=True),
        # one user's path, and those of the largest batch
        dict(name="select-one", op="select", B=1, N=15, H=32, ragged=False),
        dict(name="select-batch", op="select", B=256, N=32, H=64, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "verify", "verify", "accept", "accept", "select"])
    ragged = rng.random() < 0.5
    if op == "accept":
        V = _log_int(rng, 1000, 131072)
        tree = rng.random() < 0.5
        N = _log_int(rng, 1, 64 if tree else 8)
        B = _log_int(rng, 1, max(1, min(256, 256 * 131072 * 8 // (V * max(N, 8)))))
        return dict(op=op, B=B, N=N, V=V, tree=tree, draft=not tree and rng.random() < 0.7,
                    probs=rng.choice(["f32", "bf16"]), ragged=ragged)
    H = rng.choice([1, 2, 4, 7, 16, 32, 64])
    N = _log_int(rng, 1, 64)
    B = _log_int(rng, 1, 128)
    c = dict(op=op, B=B, N=N, H=H, ragged=ragged)
    if op == "verify":
        c["pool"] = rng.choice(["f32", "f32", "bf16"])
        c["replay"] = c["pool"] == "f32" and rng.random() < 0.7
    if op == "conv":
        c["bias"] = rng.random() < 0.5
    return c


def _lens(case):
    """Nodes of each request's window, the same for every seed (they are part
    of the case)."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return [N] * B
    r = random.Random(B * 1000003 + N)
    return [max(1, r.randint((N + 1) // 2, N)) for _ in range(B)]


# --------------------------------------------------------------------------
# what a program has in hand
# --------------------------------------------------------------------------

def _randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _trees(seed, lens):
    """Each node's parent, within its request: node 0 is the last accepted
    token, and a draft hangs on any node before it, more often on a late one,
    DEPTH tokens deep at most."""
    r = random.Random(seed)
    parents, depths = [], []
    for n in lens:
        par, dep = [-1], [1]
        for t in range(1, n):
            while True:
                a = int(t * r.random() ** 0.6)
                if dep[a] < DEPTH:
                    break
            par.append(a)
            dep.append(dep[a] + 1)
        parents.append(par)
        depths.append(dep)
    return parents, depths


def _gate_weights(gen, H):
    """Per-head A_log and per-channel dt_bias whose channels forget over one
    to a thousand tokens (log-uniform), as a trained layer's do."""
    A_log = torch.rand(H, generator=gen, device="cuda") * 1.5
    share = torch.exp(torch.rand(H, DIM, generator=gen, device="cuda") * math.log(1000.0)) / 5000.0
    dt_bias = torch.log(share / (1 - share)) / torch.exp(A_log)[:, None]
    return A_log, dt_bias


def _slots(gen, n, first):
    return (torch.randperm(n, generator=gen, device="cuda") + first).to(torch.int32)


def _accepted_paths(seed, parents, depths):
    """A path down from each tree's root, as sampling leaves it."""
    r = random.Random(seed + 1)
    paths = []
    for par in parents:
        path = [0]
        while len(path) < DEPTH:
            children = [t for t, a in enumerate(par) if a == path[-1]]
            if not children or r.random() < 0.25:
                break
            path.append(r.choice(children))
        paths.append(path)
    return paths


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, B = case["op"], case["B"]
    lens = _lens(case)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    T = starts[-1]
    parents, depths = _trees(int(seed), lens)
    s = dict(op=op, case=case, lens=lens, starts=starts, max_len=max(lens), T=T,
             qsl=_int32(starts) if case["ragged"] else None)
    bf = torch.bfloat16
    if op == "accept":
        return _prepare_accept(case, gen, s, parents)
    H = case["H"]
    D = H * DIM
    s["parents_host"] = parents
    s["parents"] = _int32([a for par in parents for a in par])
    s["slots"], s["rows"] = _slots(gen, B, 1), _slots(gen, B, 0)
    s["pending"] = torch.randint(1, DEPTH + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    if op in ("conv", "select"):
        s["x"] = _randn(gen, T, 3 * D).to(bf)
        s["conv_state"] = _randn(gen, B + 1, 3 * D, DEPTH + 2).to(bf)
    if op == "conv":
        s["w"] = _randn(gen, 3, 4, D, std=0.5).to(bf)
        s["bias"] = _randn(gen, 3 * D, std=0.1).to(bf) if case["bias"] else None
        return s
    s["corr"] = _randn(gen, B, H, DEPTH, DIM)
    s["key_gate"] = _randn(gen, B, H, DEPTH, 2 * DIM).to(bf)
    for name in ("k", "raw_g") if op == "select" else ("q", "k", "v", "raw_g"):
        s[name] = _randn(gen, T, H, DIM).to(bf)
    if op == "select":
        s["node_corr"] = _randn(gen, T, H, DIM)
        paths = _accepted_paths(int(seed), parents, depths)
        s["paths_host"] = paths
        s["accepted"] = _int32([len(p) for p in paths])
        s["path"] = _int32([p + [-1] * (DEPTH - len(p)) for p in paths])
        return s
    s["raw_beta"] = _randn(gen, T, H).to(bf)
    s["A_log"], s["dt_bias"] = _gate_weights(gen, H)
    pool = _randn(gen, B + 1, H, DIM, DIM, std=0.05)
    s["pool"] = pool if case["pool"] == "f32" else pool.to(bf)
    return s


def _prepare_accept(case, gen, s, parents):
    """A target's next-token probabilities after every node; drafts drawn from
    a draft model's probabilities (chains), or its likeliest tokens, a row's
    children one after the other (trees)."""
    B, V, T = case["B"], case["V"], s["T"]
    dtype = torch.float32 if case["probs"] == "f32" else torch.bfloat16
    logits = _randn(gen, T, V, std=3.0)
    if case["tree"]:
        near = logits + _randn(gen, T, V, std=0.5)
        best = near.topk(8, dim=-1).indices.to(torch.int32).cpu()
        del near
        tokens, base = [], 0
        for par in parents:
            given = {}
            for a in par:
                if a < 0:
                    tokens.append(0)
                    continue
                i = given.get(a, 0)
                given[a] = i + 1
                tokens.append(int(best[base + a, i % 8]))  # (a ninth child repeats the first)
            base += len(par)
        s["tokens"] = _int32(tokens)
        s["parents_host"] = parents
        s["parents"] = _int32([a for par in parents for a in par])
        s["draft"] = None
    else:
        # row t: what token t was drawn from, behind token t - 1
        behind = torch.roll(logits, 1, 0) + _randn(gen, T, V, std=0.7)
        q = torch.softmax(behind, dim=-1).to(dtype)
        del behind
        s["tokens"] = torch.cat([torch.multinomial(part.float(), 1, generator=gen)[:, 0]
                                 for part in q.split(256)]).to(torch.int32)
        s["parents_host"] = s["parents"] = None
        s["draft"] = q if case["draft"] else None
    s["target"] = torch.softmax(logits, dim=-1).to(dtype)
    s["u"] = torch.rand(T, generator=gen, device="cuda")
    s["u_next"] = torch.rand(B, generator=gen, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    return {"conv": _conv, "verify": _verify, "accept": _accept, "select": _select}[s["op"]](s)


def _table(s):
    """(index of every node in the packed rows [B, N], whether there is one)."""
    dev = "cuda"
    place = torch.arange(s["max_len"], device=dev)
    lens = torch.tensor(s["lens"], device=dev)
    starts = torch.tensor(s["starts"][:-1], device=dev)
    live = place < lens[:, None]
    return torch.where(live, starts[:, None] + place, 0), live


def _conv(s):
    T, D = s["T"], s["x"].shape[1] // 3
    H = D // DIM
    q, k, v = (torch.empty(T, H, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_tree_conv
        kda_tree_conv(s["x"], s["w"], s["bias"], s["conv_state"], s["slots"], s["parents"], q, k, v,
                      Q=s["max_len"], record_rows=s["rows"], pending=s["pending"],
                      query_start_loc=s["qsl"])
        return {"q": q, "k": k, "v": v}
    x = s["x"]
    tok, live = _table(s)
    request = torch.repeat_interleave(torch.arange(len(s["lens"]), device="cuda"),
                                      torch.tensor(s["lens"], device="cuda"))
    first = torch.tensor(s["starts"], device="cuda")[request]
    off = (s["pending"].long()[s["rows"].long()] - 1)[request]  # the window's first live entry
    window = s["conv_state"][s["slots"].long()]
    parent = s["parents"].long()

    # `at`: a node (packed), or -1, -2, -3 .. for the window's entries from the end
    def up(at):
        a = torch.where(at >= 0, parent[at.clamp(min=0)], 0)
        return torch.where(at >= 0, torch.where(a >= 0, first + a, -1), at - 1)

    def entry(at):
        back = (off + 3 + at.clamp(max=-1)).clamp(min=0)  # -1: the newest of the three
        old = window[request, :, back]
        return torch.where((at >= 0)[:, None], x[at.clamp(min=0)], old).float()

    w = s["w"].float().permute(1, 0, 2).reshape(4, 3 * D)
    at = torch.arange(T, device="cuda")
    y = w[3] * entry(at)
    for i in (2, 1, 0):
        at = up(at)
        y = y + w[i] * entry(at)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = (y * torch.sigmoid(y)).to(torch.bfloat16)
    for i, o in enumerate((q, k, v)):
        o.copy_(y[:, i * D:(i + 1) * D].reshape(T, H, DIM))
    return {"q": q, "k": k, "v": v}


def _unit(x):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _log_decay(s, raw_g):
    a = torch.exp(s["A_log"])[:, None]
    return LOWER_BOUND * torch.sigmoid(a * (raw_g.float() + s["dt_bias"]))


def _verify(s):
    T, H = s["q"].shape[:2]
    replay = s["case"]["replay"]
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_tree_verify
        out = torch.empty_like(s["v"])
        node_corr = torch.empty(T, H, DIM, device="cuda")
        records = dict(record_rows=s["rows"], pending=s["pending"], corr=s["corr"],
                       key_gate=s["key_gate"]) if replay else {}
        kda_tree_verify(s["q"], s["k"], s["v"], s["raw_g"], s["raw_beta"], s["A_log"], s["dt_bias"],
                        s["pool"], s["slots"], s["parents"], node_corr, out, Q=s["max_len"],
                        lower_bound=LOWER_BOUND, q_scale=Q_SCALE, query_start_loc=s["qsl"], **records)
        return {"out": out, "node_corr": node_corr, "state": s["pool"]}
    slots = s["slots"].long()
    S = s["pool"][slots].float()  # [B, H, V, K]
    if replay:
        rows = s["rows"].long()
        n = s["pending"].long()[rows]
        kg = s["key_gate"][rows]
        corr = s["corr"][rows]
        live = (torch.arange(DEPTH, device="cuda") < n[:, None])[:, None, :, None]
        g = torch.where(live, _log_decay(s, kg[..., DIM:].transpose(1, 2)).transpose(1, 2), 0)
        left = g.flip(2).cumsum(2).flip(2)  # from token t's decay to the end
        kp = torch.where(live, _unit(kg[..., :DIM]), 0) * torch.exp(left - g)
        S = S * torch.exp(left[:, :, :1]) + corr.transpose(-1, -2) @ kp
        s["pool"][slots] = S
    tok, there = _table(s)
    heads = lambda x: x[tok].transpose(1, 2)  # [B, H, N, ..]
    N = tok.shape[1]
    par = torch.where(there, s["parents"].long()[tok], -1)
    # which nodes are on the way to which, themselves included
    anc = torch.eye(N, dtype=torch.bool, device="cuda").expand(tok.shape[0], N, N).clone()
    for t in range(1, N):
        above = anc.gather(1, par[:, t].clamp(min=0)[:, None, None].expand(-1, 1, N))[:, 0]
        anc[:, t] |= above & (par[:, t] >= 0)[:, None]
    g = _log_decay(s, s["raw_g"][tok]).transpose(1, 2)
    # (its exponents are differences of sums: in 64 bits)
    G = torch.einsum("bts,bhsk->bhtk", anc.double(), g.double())
    qn, kn = _unit(heads(s["q"])) * Q_SCALE, _unit(heads(s["k"]))
    beta = torch.sigmoid(heads(s["raw_beta"]).float())[..., None]
    down, back = torch.exp(G), kn.double() * torch.exp(-G)
    kd, qd = kn.double() * down, qn.double() * down
    kk = torch.where(anc[:, None], kd @ back.transpose(-1, -2), 0).float().tril(-1)
    qk = torch.where(anc[:, None], qd @ back.transpose(-1, -2), 0).float()
    w, y = kd.float() @ S.transpose(-1, -2), qd.float() @ S.transpose(-1, -2)
    u = beta * (heads(s["v"]).float() - w)
    for t in range(1, N):
        u[:, :, t] -= beta[:, :, t] * (kk[:, :, t, None, :t] @ u[:, :, :t])[:, :, 0]
    o = y + qk @ u
    packed = lambda x: x.transpose(1, 2)[there].contiguous()
    return {"out": packed(o).to(torch.bfloat16), "node_corr": packed(u), "state": s["pool"]}


def _accept(s):
    B = len(s["lens"])
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_draft_accept
        accepted, next_tokens = torch.empty(2, B, dtype=torch.int32, device="cuda")
        path = torch.empty(B, DEPTH, dtype=torch.int32, device="cuda")
        kda_draft_accept(s["target"], s["tokens"], s["u"], s["u_next"], accepted, path, next_tokens,
                         Q=s["max_len"], draft_probs=s["draft"], parents=s["parents"],
                         query_start_loc=s["qsl"])
        return {"accepted": accepted, "path": path, "next_tokens": next_tokens}
    # probabilities next to a border: in 64 bits
    target, draft = s["target"], s["draft"]
    node, there = _table(s)
    N = node.shape[1]
    tokens = s["tokens"].long()[node]
    if s["parents"] is None:
        par = torch.arange(-1, N - 1, device="cuda").expand(B, N)
    else:
        par = s["parents"].long()[node]
    row = node.gather(1, par.clamp(min=0))
    p = target[row, tokens].double()
    u = s["u"].double()[node]
    # a child whose token an earlier child of the same node has is never taken
    same = (tokens[:, :, None] == tokens[:, None]) & (par[:, :, None] == par[:, None])
    first = ~(same & there[:, None]).tril(-1).any(-1)
    place = torch.arange(N, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    going = torch.ones(B, dtype=torch.bool, device="cuda")
    path = [cur]
    for _ in range(DEPTH - 1):
        child = there & (par == cur[:, None]) & first & (place > 0)
        at_u = u.gather(1, cur[:, None])
        if draft is not None:
            taken = child & (at_u * draft[node, tokens].double() < p)
        else:
            taken = child & (at_u < torch.where(child, p, 0).cumsum(1))
        going = going & taken.any(1)
        cur = torch.where(going, taken.int().argmax(1), cur)
        path.append(torch.where(going, cur, -1))
    path = torch.stack(path, 1)
    accepted = (path >= 0).sum(1)
    # the token behind the path: from what the refused drafts leave
    last = node.gather(1, cur[:, None])[:, 0]
    weight = target[last].double()
    whole = weight
    child = there & (par == cur[:, None]) & (place > 0)
    if draft is not None:
        # (an arm that ends has no child to refuse)
        refused = child.any(1)
        behind = node.gather(1, child.int().argmax(1)[:, None])[:, 0]
        left = (weight - draft[behind].double()).clamp(min=0)
        weight = torch.where(refused[:, None], left, weight)
    else:
        # (a column for what is no child)
        weight = torch.cat([weight, torch.zeros(B, 1, dtype=torch.float64, device="cuda")], 1)
        weight.scatter_(1, torch.where(child, tokens, weight.shape[1] - 1), 0.0)
        weight = weight[:, :-1]
    weight = torch.where((weight.sum(1) > 0)[:, None], weight, whole)
    run_sum = weight.cumsum(1)
    goal = s["u_next"].double()[:, None] * run_sum[:, -1:]
    next_tokens = (run_sum > goal).int().argmax(1)
    i32 = lambda x: x.to(torch.int32)
    return {"accepted": i32(accepted), "path": i32(path), "next_tokens": i32(next_tokens)}


def _select(s):
    corr, key_gate, window = s["corr"], s["key_gate"], s["conv_state"]
    if own:
        from linear_attention_speculative_recoverssm_gb300 import kda_tree_select
        kda_tree_select(s["path"], s["accepted"], s["k"], s["raw_g"], s["node_corr"], s["slots"],
                        s["rows"], corr, key_gate, Q=s["max_len"], x=s["x"], conv_state=window,
                        pending=s["pending"], query_start_loc=s["qsl"])
        return {"corr": corr, "key_gate": key_gate, "window": window}
    rows, slots = s["rows"].long(), s["slots"].long()
    n = s["accepted"].long()[:, None]
    starts = torch.tensor(s["starts"][:-1], device="cuda")[:, None]
    place = torch.arange(DEPTH, device="cuda")
    on = place < n
    tok = torch.where(on, starts + s["path"].long(), 0)
    pick = lambda new, old: torch.where(on[:, None, :, None], new[tok].transpose(1, 2), old[rows])
    corr[rows] = pick(s["node_corr"], corr)
    key_gate[rows] = pick(torch.cat([s["k"], s["raw_g"]], -1), key_gate)
    # two entries from before the path, then its inputs
    old = window[slots]
    off = (s["pending"].long()[rows] - 1)[:, None] + 1
    entries = old.transpose(1, 2)  # [B, DEPTH + 2, 3 D]
    head = entries.gather(1, (off + torch.arange(2, device="cuda"))[:, :, None].expand(-1, -1, entries.shape[2]))
    tail = torch.where(on[:, :, None], s["x"][tok], entries[:, 2:])
    window[slots] = torch.cat([head, tail], 1).transpose(1, 2)
    return {"corr": corr, "key_gate": key_gate, "window": window}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op, B, lens = case["op"], case["B"], _lens(case)
    T = float(sum(lens))
    if op == "accept":
        # one target row a request, and its drafts' row where one was refused
        rows = B * (2 if case["draft"] else 1)
        return {"bytes": rows * case["V"] * (4.0 if case["probs"] == "f32" else 2.0), "flops": 2.0 * rows * case["V"]}
    H = case["H"]
    D = H * DIM
    if op == "conv":
        return {"bytes": 12.0 * D * T + 24.0 * D + 18.0 * D * B, "flops": 3.0 * D * T * 12}
    if op == "select":
        # some four tokens a path
        n = 4.0 * B
        return {"bytes": n * H * DIM * 2 * 8.0 + n * 12.0 * D + 24.0 * D * B, "flops": 0.0}
    page = H * DIM * DIM * (4.0 if case["pool"] == "f32" else 2.0)
    replayed = 4.5 * B if case["replay"] else 0.0
    return {"bytes": T * H * (5 * 2.0 * DIM + 2 + 4.0 * DIM) + B * page * (2 if case["replay"] else 1)
            + replayed * H * DIM * 8.0,
            "flops": T * H * 4.0 * DIM * DIM + replayed * H * 2.0 * DIM * DIM}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "verify": _exact_verify, "accept": _exact_accept,
            "select": _exact_select}[s["op"]](s)


def _f64(x):
    return x.to(torch.float64)


def _exact_conv(s):
    D = s["x"].shape[1] // 3
    H = D // DIM
    w = _f64(s["w"]).transpose(0, 1).reshape(4, 3 * D)
    rows, slots = s["rows"].tolist(), s["slots"].tolist()
    pending = s["pending"].tolist()
    ys = []
    for b, par in enumerate(s["parents_host"]):
        n, t0 = len(par), s["starts"][b]
        off = pending[rows[b]] - 1
        # the window's three entries, oldest first, then the nodes
        line = torch.cat([_f64(s["conv_state"][slots[b], :, off:off + 3]).t(), _f64(s["x"][t0:t0 + n])])
        taps = []
        for t in range(n):
            way = [t]
            while len(way) < 4:
                way.append(par[way[-1]] if way[-1] >= 0 else way[-1] - 1)
            taps.append([3 + a for a in reversed(way)])
        y = sum(w[i] * line[[tap[i] for tap in taps]] for i in range(4))
        if s["bias"] is not None:
            y = y + _f64(s["bias"])
        ys.append(y / (1 + torch.exp(-y)))
    y = torch.cat(ys)
    return {name: y[:, i * D:(i + 1) * D].reshape(-1, H, DIM) for i, name in enumerate("qkv")}


def _exact_verify(s):
    """The recurrence down every path: S <- S diag(d); u = beta (v - S k);
    S <- S + u k^T; o = S q."""
    H = s["q"].shape[1]
    pool = _f64(s["pool"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    us = torch.zeros_like(out)
    a, dt = torch.exp(_f64(s["A_log"]))[:, None], _f64(s["dt_bias"])
    unit = lambda x: _f64(x) / torch.sqrt((_f64(x) ** 2).sum(-1, keepdim=True) + EPS)
    decay = lambda g: torch.exp(LOWER_BOUND / (1 + torch.exp(-a * (_f64(g) + dt))))
    rows, slots, pending = s["rows"].tolist(), s["slots"].tolist(), s["pending"].tolist()
    for b, par in enumerate(s["parents_host"]):
        S = pool[slots[b]]
        if s["case"]["replay"]:
            r = rows[b]
            for t in range(pending[r]):
                key = unit(s["key_gate"][r, :, t, :DIM])
                S = S * decay(s["key_gate"][r, :, t, DIM:])[:, None] + _f64(s["corr"][r, :, t])[..., None] * key[:, None]
            pool[slots[b]] = S
        span = slice(s["starts"][b], s["starts"][b + 1])
        q, k, v = unit(s["q"][span]) * Q_SCALE, unit(s["k"][span]), _f64(s["v"][span])
        d, beta = decay(s["raw_g"][span]), 1 / (1 + torch.exp(-_f64(s["raw_beta"][span])))
        states = []
        for t, p in enumerate(par):
            St = (S if p < 0 else states[p]) * d[t][:, None]
            u = beta[t][:, None] * (v[t] - (St * k[t][:, None]).sum(-1))
            St = St + u[..., None] * k[t][:, None]
            out[span.start + t], us[span.start + t] = (St * q[t][:, None]).sum(-1), u
            states.append(St)
    return {"out": out, "node_corr": us, "state": pool}


def _exact_accept(s):
    import numpy as np
    host = lambda x: x.double().cpu().numpy()
    tokens, u, u_next = s["tokens"].tolist(), host(s["u"]), host(s["u_next"])
    target, draft = s["target"], s["draft"]
    accepted, paths, nexts = [], [], []
    for b, n in enumerate(s["lens"]):
        t0 = s["starts"][b]
        par = list(range(-1, n - 1)) if s["parents_host"] is None else s["parents_host"][b]
        path = [0]
        while True:
            cur = path[-1]
            row = host(target[t0 + cur])
            children, seen = [], set()
            for t in range(1, n):
                if par[t] == cur and tokens[t0 + t] not in seen:
                    seen.add(tokens[t0 + t])
                    children.append(t)
            taken, cum, q = None, 0.0, None
            for t in children:
                x = tokens[t0 + t]
                if draft is not None:
                    q = host(draft[t0 + t])
                    hit = u[t0 + cur] * q[x] < row[x]
                else:
                    cum += row[x]
                    hit = u[t0 + cur] < cum
                if hit:
                    taken = t
                    break
            if taken is None:
                break
            path.append(taken)
        weight = row.copy()
        if q is not None:
            weight = np.maximum(row - q, 0.0)
        elif draft is None:
            weight[[tokens[t0 + t] for t in children]] = 0.0
        if not weight.sum() > 0:
            weight = row
        sums = np.cumsum(weight)
        nexts.append(int(np.argmax(sums > u_next[b] * sums[-1])))
        accepted.append(len(path))
        paths.append(path + [-1] * (DEPTH - len(path)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return {"accepted": i32(accepted), "path": i32(paths), "next_tokens": i32(nexts)}


def _exact_select(s):
    corr, kg, window = _f64(s["corr"]), _f64(s["key_gate"]), _f64(s["conv_state"])
    rows, slots, pending = s["rows"].tolist(), s["slots"].tolist(), s["pending"].tolist()
    for b, path in enumerate(s["paths_host"]):
        r, t0 = rows[b], s["starts"][b]
        W = window[slots[b]].clone()
        off = pending[r] - 1
        window[slots[b], :, 0], window[slots[b], :, 1] = W[:, off + 1], W[:, off + 2]
        for i, t in enumerate(path):
            corr[r, :, i] = _f64(s["node_corr"][t0 + t])
            kg[r, :, i, :DIM], kg[r, :, i, DIM:] = _f64(s["k"][t0 + t]), _f64(s["raw_g"][t0 + t])
            window[slots[b], :, 2 + i] = _f64(s["x"][t0 + t])
    return {"corr": corr, "key_gate": kg, "window": window}
