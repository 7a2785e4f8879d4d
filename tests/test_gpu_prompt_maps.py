"""kda_slot_plan and kda_prefill_conv against the oracle, and the prompt
operators one after the other as a server uses them."""
import numpy as np
import pytest

from oracle import kda_oracle as ko
from oracle import prompt_oracle as po
from prompt_testutil import to_numpy, to_torch
from linear_attention_speculative_recoverssm_gb300 import synth

pytestmark = pytest.mark.gpu

I32 = np.int32


def plan_case(B, block_size, max_blocks, seed, n_free=None, max_new=None):
    rng = np.random.default_rng(seed)
    room = block_size * max_blocks
    new = rng.integers(0, (max_new or room) + 1, size=B).clip(0, room)
    computed = (rng.random(B) * (room - new + 1)).astype(np.int64)
    computed[rng.random(B) < 0.3] = 0
    table = np.zeros((B, max_blocks), dtype=I32)
    slots = rng.permutation(B * max_blocks + 2 * B) + 1
    for b in range(B):
        held = -(-int(computed[b]) // block_size)
        table[b, :held] = slots[b * max_blocks:b * max_blocks + held]
    free = slots[B * max_blocks:].astype(I32)
    if n_free is not None:
        free = free[:n_free]
    return dict(computed_lens=computed.astype(I32), new_lens=new.astype(I32), block_table=table,
                free_slots=free, free_head=np.array([0], dtype=I32), block_size=block_size)


def run_plan(case, same_head=False, null_slot=0):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_slot_plan
    B = len(case["new_lens"])
    d = {n: to_torch(case[n], "cuda") for n in ("computed_lens", "new_lens", "free_slots",
                                                "free_head")}
    # rows further apart than their size, marks between them
    wide = torch.full((B, case["block_table"].shape[1] + 3), -77, dtype=torch.int32, device="cuda")
    wide[:, :-3] = to_torch(case["block_table"], "cuda")
    table = wide[:, :-3]
    i32 = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")
    out = dict(query_start_loc=i32(B + 1), sources=i32(B), destinations=i32(B),
               boundaries=i32(B), boundary_lens=i32(B))
    nxt = d["free_head"] if same_head else i32(1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda_slot_plan(d["computed_lens"], d["new_lens"], table, d["free_slots"], d["free_head"], nxt,
                  *out.values(), block_size=case["block_size"], null_slot=null_slot,
                  status=status)
    got = {n: to_numpy(t) for n, t in out.items()}
    got["free_next"] = to_numpy(nxt)
    assert bool((wide[:, -3:] == -77).all())
    return got, to_numpy(table.contiguous()), int(status[0])


def check_plan(case, **kw):
    got, table, status = run_plan(case, **kw)
    ref_table = case["block_table"].copy()
    ref, bad = po.slot_plan(**{**case, "block_table": ref_table,
                               "free_head": case["free_head"][0]},
                            null_slot=kw.get("null_slot", 0))
    for n, r in ref.items():
        np.testing.assert_array_equal(got[n], r, err_msg=n)
    np.testing.assert_array_equal(table, ref_table)
    assert (status != 0) == (bad > 0)
    return status, bad


@pytest.mark.parametrize("B", [1, 31, 33, 1000, 1024, 1025, 8192, 8193, 20000])
@pytest.mark.parametrize("block_size,max_blocks", [(1, 5), (16, 20), (100, 3)])
def test_plan(B, block_size, max_blocks):
    assert check_plan(plan_case(B, block_size, max_blocks, seed=B + block_size),
                      same_head=B % 2 == 0)[1] == 0


def test_plan_long_prompts():
    check_plan(plan_case(40, 16, 5000, seed=3))


@pytest.mark.parametrize("B,n_free", [(40, 0), (40, 1), (40, 2), (40, 31), (3000, 2000),
                                      (9000, 9001)])
def test_plan_runs_out_of_slots(B, n_free):
    status, bad = check_plan(plan_case(B, 16, 20, seed=n_free, n_free=n_free))
    assert bad > 0 and status == -7


def test_plan_reports_bad_requests():
    case = plan_case(200, 16, 20, seed=4, max_new=50)
    case["new_lens"][3] = -5
    case["computed_lens"][4] = -1
    case["new_lens"][5] = 16 * 20 + 1
    case["computed_lens"][6], case["new_lens"][6] = 2 ** 31 - 1, 2 ** 31 - 1
    case["new_lens"][6] = 16 * 20 + 3  # keep the packed total in range
    case["computed_lens"][7], case["new_lens"][7] = 20, 5
    case["block_table"][7, 1] = 0  # its state is not held
    status, bad = check_plan(case)
    assert status == -1 and bad == 5


@pytest.mark.parametrize("head", [-1, 1000])
def test_plan_bad_head(head):
    case = plan_case(20, 16, 20, seed=6, n_free=30)
    case["free_head"][0] = head
    got, table, status = run_plan(case)
    assert status != 0 and got["free_next"][0] == head
    np.testing.assert_array_equal(table, np.where(table == case["block_table"], table, 0))
    fresh = (case["computed_lens"] == 0) & (case["new_lens"] > 0)
    assert np.all(got["destinations"][fresh] == 0)


@pytest.mark.parametrize("B", [3, 5000])
def test_plan_captured(B):
    """Captured on another stream and replayed on other lengths: the plan
    that an eager call makes."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_slot_plan
    cases = [plan_case(B, 16, 8, seed=s) for s in (31, 32)]
    dev = "cuda"
    names = ("computed_lens", "new_lens", "block_table", "free_slots", "free_head")
    d = {n: to_torch(cases[0][n], dev) for n in names}
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)
    out = [i32(B + 1)] + [i32(B) for _ in range(4)]
    nxt, side = i32(1), torch.cuda.Stream()
    call = lambda: kda_slot_plan(*d.values(), nxt, *out, block_size=16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for case in cases:
        for n in names:
            d[n].copy_(to_torch(case[n], dev))
        graph.replay()
        torch.cuda.synchronize()
        ref_table = case["block_table"].copy()
        ref, bad = po.slot_plan(computed_lens=case["computed_lens"], new_lens=case["new_lens"],
                                block_table=ref_table, free_slots=case["free_slots"],
                                free_head=0, block_size=16)
        assert bad == 0
        np.testing.assert_array_equal(to_numpy(d["block_table"]), ref_table)
        for n, t in zip(("query_start_loc", "sources", "destinations", "boundaries",
                         "boundary_lens"), out):
            np.testing.assert_array_equal(to_numpy(t), ref[n])
        assert int(nxt[0]) == int(np.asarray(ref["free_next"]).reshape(-1)[0])


@pytest.mark.parametrize("resume", [(), (0, 1, 2)])
def test_conv_captured(resume):
    """The same for the convolution, whose windows are advanced in place."""
    import torch
    cases = [conv_case([30, 1, 70], 2, seed=s, resume=resume) for s in (33, 34)]
    for c in cases[1:]:
        for n in ("sources", "destinations"):
            c[n] = cases[0][n]
    d = {n: None if a is None else to_torch(a, "cuda") for n, a in cases[0].items() if n != "Q"}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run_conv(cases[0], d)
    for c in cases:
        for n, a in c.items():
            if n != "Q":
                d[n].copy_(to_torch(a, "cuda"))
        graph.replay()
        torch.cuda.synchronize()
        check_conv(c, d)


def test_plan_no_requests():
    case = plan_case(0, 16, 20, seed=7, n_free=0)
    case["free_slots"] = np.arange(1, 4, dtype=I32)
    case["free_head"][0] = 2
    got, _, status = run_plan(case)
    assert status == 0 and got["free_next"][0] == 2 and list(got["query_start_loc"]) == [0]


def test_plan_other_null_slot():
    case = plan_case(100, 16, 20, seed=8)
    case["block_table"][case["block_table"] == 0] = -1
    check_plan(case, null_slot=-1)


# --------------------------------------------------------------------------
# convolution
# --------------------------------------------------------------------------

def conv_case(lens, H, seed, width=6, bias=True, resume=None, boundary=None, inert=(), tail=0):
    rng = np.random.default_rng(seed)
    B, T, D3 = len(lens), sum(lens) + tail, 3 * H * 128
    resume = set(range(1, B, 2)) if resume is None else set(resume)
    boundary = boundary or {}
    bits = lambda *s, std=1.0: synth.to_bf16_bits((rng.standard_normal(s) * std).astype(np.float32))
    pick = (rng.permutation(3 * B) + 1).astype(I32)
    return dict(
        x=bits(T, D3), conv_weight=bits(3, 4, H * 128, std=0.5),
        conv_bias=bits(D3, std=0.2) if bias else None, conv_state=bits(3 * B + 1, D3, width),
        sources=np.where([b in resume for b in range(B)], pick[:B], 0).astype(I32),
        destinations=np.where([b in inert for b in range(B)], 0, pick[B:2 * B]).astype(I32),
        boundaries=np.array([pick[2 * B + b] if b in boundary else 0 for b in range(B)], dtype=I32),
        boundary_lens=np.array([boundary.get(b, 0) for b in range(B)], dtype=I32),
        query_start_loc=np.concatenate([[0], np.cumsum(lens)]).astype(I32),
        q=np.full((T, H, 128), 0x4321, dtype=np.uint16),
        k=np.full((T, H, 128), 0x4321, dtype=np.uint16),
        v=np.full((T, H, 128), 0x4321, dtype=np.uint16), Q=max(max(lens), 1))


def run_conv(case, d=None, **kw):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill_conv
    if d is None:
        d = {n: None if a is None else to_torch(a, "cuda") for n, a in case.items() if n != "Q"}
    d["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda_prefill_conv(d["x"], d["conv_weight"], d["conv_bias"], d["conv_state"], d["sources"],
                     d["destinations"], d["query_start_loc"], d["q"], d["k"], d["v"], Q=case["Q"],
                     boundaries=d["boundaries"], boundary_lens=d["boundary_lens"],
                     status=d["status"], **kw)
    return d


def check_conv(case, d, bad=0):
    ref = {n: None if a is None else (a.copy() if isinstance(a, np.ndarray) else a)
           for n, a in case.items()}
    assert po.conv(**ref) == bad
    np.testing.assert_array_equal(to_numpy(d["conv_state"]), ref["conv_state"])
    assert (int(d["status"][0]) != 0) == (bad > 0)
    for n in ("q", "k", "v"):
        got, want = to_numpy(d[n]), ref[n]
        kept = want == case[n]
        np.testing.assert_array_equal(got[kept], want[kept])
        g, w = ko.bf16_to_f64(got), ko.bf16_to_f64(want)
        # half a step each side of the oracle's rounded value, and the FP32
        # sum of five terms and the sigmoid: 8 2^-23 of the terms' size (< 16)
        assert np.all(np.abs(g - w) <= 2.0 ** -7 * np.abs(w) + 1.6e-5), n


@pytest.mark.parametrize("lens", [[1], [2], [3], [4], [1, 1, 1, 1, 1], [16, 15, 17], [0, 14, 2, 0, 33],
                                  [13, 3, 1, 2, 40, 0, 100]])
@pytest.mark.parametrize("H,width", [(1, 3), (2, 6), (5, 10)])
def test_conv_ragged(lens, H, width):
    boundary = {b: max(1, n // 2) for b, n in enumerate(lens) if n and b % 3 != 1}
    case = conv_case(lens, H, seed=len(lens) + sum(lens), width=width, bias=H != 2,
                     boundary=boundary, tail=4, inert=(4,))
    check_conv(case, run_conv(case))


@pytest.mark.parametrize("H,tokens", [(16, 900), (16, 1700), (17, 3500)])
def test_conv_longer_runs(H, tokens):
    """Enough tokens that a thread takes runs of 16, 32 and 64 of them:
    requests that end and begin everywhere in a run."""
    rng = np.random.default_rng(tokens)
    lens = [int(n) for n in rng.integers(0, 90, size=tokens // 90)] + [64, 1, 2, 63, 65, 128]
    lens.append(max(tokens - sum(lens), 1))
    boundary = {b: max(1, n // 3) for b, n in enumerate(lens) if n and b % 3 != 1}
    case = conv_case(lens, H, seed=tokens, width=4, boundary=boundary, tail=5, inert=(2, 7))
    check_conv(case, run_conv(case))


@pytest.mark.parametrize("width", [3, 4, 5, 6, 7, 8, 9, 10])
def test_conv_every_width(width):
    """Windows of every width, one-token prompts among them, some advanced in
    place and some left as a boundary in their own source."""
    lens = [1, 1, 2, 1, 3, 1, 4, 1, 7, 1]
    case = conv_case(lens, 3, seed=width, width=width, resume=range(9), boundary={2: 1, 6: 3, 8: 4})
    case["destinations"][:4] = case["sources"][:4]
    case["boundaries"][6] = case["sources"][6]
    check_conv(case, run_conv(case))


def test_conv_slots_far_apart():
    """Windows more than 2^31 elements apart: as in a pool without gaps."""
    import torch
    case = conv_case([5, 40], 2, seed=96, resume=(1,), boundary={1: 7})
    case["sources"], case["destinations"] = np.array([0, 1], I32), np.array([2, 1], I32)
    case["boundaries"], case["conv_state"] = np.array([0, 3], I32), case["conv_state"][:4]
    d = {n: None if a is None else to_torch(a, "cuda") for n, a in case.items() if n != "Q"}
    step, (_, D3, width) = 2 ** 31 + 512, case["conv_state"].shape
    far = torch.empty(3 * step + D3 * width, dtype=torch.bfloat16, device="cuda")
    far = far.as_strided((4, D3, width), (step, width, 1))
    far.copy_(d["conv_state"])
    d["conv_state"] = far
    run_conv(case, d)
    d["conv_state"] = far.contiguous()
    del far
    check_conv(case, d)


@pytest.mark.parametrize("null_slot", [-1, 4])
def test_conv_other_null_slots(null_slot):
    """Slot 0 is a slot where the null slot is -1; slots up to it are none."""
    case = conv_case([3, 20, 5, 1], 2, seed=60, boundary={1: 9})
    case["sources"][case["sources"] == 0] = null_slot  # (fresh, none reads slot 0 but its writer)
    case["destinations"][3] = case["sources"][3] = 0
    case["null_slot"] = null_slot
    d = {n: None if a is None else to_torch(a, "cuda") for n, a in case.items()
         if n not in ("Q", "null_slot")}
    check_conv(case, run_conv(case, d, null_slot=null_slot))


def test_conv_in_place_and_shared():
    """Windows left in their own source (as destination or as boundary), for
    prompts of one to many runs, and one source for several requests."""
    lens = [1, 2, 3, 40, 17, 64]
    case = conv_case(lens, 2, seed=5, resume=range(6), boundary={1: 1, 3: 2, 5: 63})
    s = case["sources"]
    s[0], s[2], s[4] = case["destinations"][0], case["destinations"][2], case["destinations"][4]
    s[1], s[5] = case["boundaries"][1], case["boundaries"][5]
    check_conv(case, run_conv(case))
    case = conv_case(lens, 2, seed=6, resume=range(6))
    case["sources"][:] = case["sources"][0]
    check_conv(case, run_conv(case))


def test_conv_reports_and_uniform():
    case = conv_case([20, 5, 9], 2, seed=7)
    case["Q"] = 19
    case["destinations"][1] = case["conv_state"].shape[0]
    check_conv(case, run_conv(case), bad=2)
    case = conv_case([7] * 5, 2, seed=8)
    d = {n: None if a is None else to_torch(a, "cuda") for n, a in case.items() if n != "Q"}
    d["query_start_loc"] = None
    check_conv(case, run_conv(case, d))


def test_conv_equals_the_layer_prologue():
    """On windows of 8 tokens with nothing pending it is the layer's own
    convolution, bit for bit, and so are the windows' entries 0 .. 2."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_layer_prologue
    c = synth.layer_case(B=6, H=2, Q=8, slots=16, seed=3)
    B, Q = 6, 8
    slots = c["state_slots"]
    d = {n: to_torch(c[n], "cuda") for n in ("x", "conv_weight", "conv_bias", "conv_state", "f_a",
                                             "f_b", "state_slots")}
    outs = [torch.zeros((B * Q, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    window = d["conv_state"].clone()
    kda_layer_prologue(d["x"], d["conv_weight"], d["conv_bias"], d["conv_state"], d["f_a"],
                       d["f_b"], d["state_slots"], None, None, *outs, Q=Q)
    case = dict(x=c["x"], conv_weight=c["conv_weight"], conv_bias=c["conv_bias"],
                conv_state=to_numpy(window), sources=slots, destinations=slots,
                boundaries=None, boundary_lens=None, query_start_loc=None, Q=Q,
                q=np.zeros((B * Q, 2, 128), dtype=np.uint16),
                k=np.zeros((B * Q, 2, 128), dtype=np.uint16),
                v=np.zeros((B * Q, 2, 128), dtype=np.uint16))
    e = run_conv(case)
    for got, want in zip((e["q"], e["k"], e["v"]), outs):
        np.testing.assert_array_equal(to_numpy(got), to_numpy(want))
    live = slots[slots > 0]
    got = to_numpy(e["conv_state"])[live][:, :, :3]
    # the layer leaves W_1, W_2, x_0 .. x_7; the last three are its entries 7 ..
    np.testing.assert_array_equal(got, to_numpy(d["conv_state"])[live][:, :, Q - 1:Q + 2])


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------

def test_serving_a_batch():
    """Plan, convolution, prefill and decode steps as a server runs them,
    prompts arriving in two parts, against the oracle over each request's
    whole sequence; the cached blocks hold the states at their boundaries."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import (kda_prefill, kda_prefill_conv,
                                                               kda_recurrent, kda_slot_plan)
    H, B, bs, max_blocks = 2, 5, 32, 12
    rng = np.random.default_rng(11)
    steps = [[70, 33, 0, 128, 5], [10, 64, 97, 1, 0], [1, 1, 1, 1, 1], [1, 1, 1, 1, 1]]
    total = np.sum(steps, axis=0)
    bits = lambda *s, std=1.0: synth.to_bf16_bits((rng.standard_normal(s) * std).astype(np.float32))
    D = H * 128
    seq = [dict(x=bits(n, 3 * D), raw_g=bits(n, H, 128), raw_beta=bits(n, H)) for n in total]
    w, bias = bits(3, 4, D, std=0.5), bits(3 * D, std=0.1)
    A_log = rng.uniform(0, 1.5, H).astype(np.float32)
    dt = (rng.standard_normal((H, 128)) - 2).astype(np.float32)
    n_slots = 64
    dev = "cuda"
    pool = torch.randn((n_slots, H, 128, 128), device=dev)
    conv_pool = torch.randn((n_slots, 3 * D, 6), device=dev).to(torch.bfloat16)
    table = torch.zeros((B, max_blocks), dtype=torch.int32, device=dev)
    free = torch.arange(1, n_slots, dtype=torch.int32, device=dev)
    head = torch.zeros(1, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    done = np.zeros(B, dtype=I32)
    outs = [[] for _ in range(B)]
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)
    for new in steps:
        new = np.array(new, dtype=I32)
        qsl, src, dst, bnd, bl = i32(B + 1), i32(B), i32(B), i32(B), i32(B)
        kda_slot_plan(to_torch(done, dev), to_torch(new, dev), table, free, head, head, qsl, src,
                      dst, bnd, bl, block_size=bs, status=status)
        pack = lambda name: to_torch(np.concatenate(
            [seq[b][name][done[b]:done[b] + new[b]] for b in range(B)]), dev)
        T, Q = int(new.sum()), int(new.max())
        q, k, v, out = (torch.zeros((T, H, 128), dtype=torch.bfloat16, device=dev)
                        for _ in range(4))
        kda_prefill_conv(pack("x"), to_torch(w, dev), to_torch(bias, dev), conv_pool, src, dst,
                         qsl, q, k, v, Q=Q, boundaries=bnd, boundary_lens=bl, status=status)
        common = dict(Q=Q, lower_bound=-5.0, q_scale=128 ** -0.5, boundaries=bnd,
                      boundary_lens=bl, status=status)
        args = (q, k, v, pack("raw_g"), pack("raw_beta"), to_torch(A_log, dev), to_torch(dt, dev),
                pool, src, dst)
        if Q == 1:
            kda_recurrent(*args, out, query_start_loc=qsl, **common)
        else:
            kda_prefill(*args, qsl, out, **common)
        got, at = to_numpy(out), 0
        for b in range(B):
            outs[b].append(got[at:at + new[b]])
            at += new[b]
        done += new
    assert int(status[0]) == 0
    rows = to_numpy(table)
    for b in range(B):
        n = int(total[b])
        qkv = [np.zeros((n, H, 128), dtype=np.uint16) for _ in range(3)]
        one = np.array([1], dtype=I32)
        po.conv(x=seq[b]["x"], conv_weight=w, conv_bias=bias,
                conv_state=np.zeros((2, 3 * D, 6), dtype=np.uint16), sources=one * 0,
                destinations=one, q=qkv[0], k=qkv[1], v=qkv[2], Q=n)
        # the state at every block boundary that a call's end or boundary left
        ends = np.cumsum([s[b] for s in steps])
        starts = ends - [s[b] for s in steps]
        for p in sorted({int(e) for e in ends if e} |
                        {int((e - 1) // bs * bs) for e, s in zip(ends, starts)
                         if (e - 1) // bs * bs > s}):
            state = np.zeros((2, H, 128, 128), dtype=np.float32)
            f64 = np.zeros((n, H, 128))
            ref_out = np.zeros((n, H, 128), dtype=np.uint16)
            po.rule(q=qkv[0][:p], k=qkv[1][:p], v=qkv[2][:p], raw_g=seq[b]["raw_g"][:p],
                    raw_beta=seq[b]["raw_beta"][:p], A_log=A_log, dt_bias=dt, lower_bound=-5.0,
                    q_scale=128 ** -0.5, state=state, sources=one * 0, destinations=one,
                    out=ref_out[:p], Q=p, out_f64=f64[:p])
            if p % bs == 0 or p == n:
                slot = rows[b, (p - 1) // bs]
                err = np.abs(to_numpy(pool)[slot] - state[1]).max()
                # q, k, v of kernel and oracle may differ by one BF16 step in
                # places (2^-8 of a key, in a state that averages over keys)
                assert slot > 0 and err <= 2.0 ** -8 * np.abs(state[1]).max(), (b, p)
        got = ko.bf16_to_f64(np.concatenate(outs[b]))
        scale = np.abs(f64).max(axis=(0, 2), keepdims=True)
        assert np.all(np.abs(got - f64) <= 2.0 ** -7 * np.abs(f64) + 2.0 ** -8 * scale), b


def test_plan_feeds_the_commit():
    """The plan of accepted counts is kda_commit's sources, destinations and
    boundaries: the committed states equal the oracle's."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import (KDA_STATE_F32, kda_commit,
                                                               kda_slot_plan, layer_tables)
    B, H, Q, bs, max_blocks = 6, 2, 8, 16, 8
    c = synth.replay_verify_case(B=B, H=H, Q=Q, slots=40, seed=21)
    rng = np.random.default_rng(22)
    computed = np.array([5, 16, 30, 0, 31, 12], dtype=I32)
    accepted = np.array([8, 3, 7, 4, 1, 0], dtype=I32)
    table = np.zeros((B, max_blocks), dtype=I32)
    slots = rng.permutation(np.arange(1, 40)).astype(I32)
    for b in range(B):
        held = -(-int(computed[b]) // bs)
        table[b, :held] = slots[b * 3:b * 3 + held]
    free = slots[18:]
    computed[3], table[3, 0] = 2, slots[17]  # a commit goes on from a state
    ref_table = table.copy()
    ref, bad = po.slot_plan(computed_lens=computed, new_lens=accepted, block_table=ref_table,
                            free_slots=free, free_head=0, block_size=bs)
    assert bad == 0
    dev = "cuda"
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)
    src, dst, bnd, bl = i32(B), i32(B), i32(B), i32(B)
    acc = to_torch(accepted, dev)
    kda_slot_plan(to_torch(computed, dev), acc, to_torch(table, dev), to_torch(free, dev),
                  torch.zeros(1, dtype=torch.int32, device=dev), i32(1), i32(B + 1), src, dst,
                  bnd, bl, block_size=bs)
    state0 = rng.standard_normal((40, H, 128, 128)).astype(np.float32)
    state, corr, kg = to_torch(state0, dev), to_torch(c["corr"], dev), to_torch(c["key_gate"], dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kda_commit(*layer_tables([state], [corr], [kg], dev), to_torch(c["A_log"][None], dev),
               to_torch(c["dt_bias"][None], dev), src, acc, dst, state_dtype=KDA_STATE_F32,
               lower_bound=c["lower_bound"], L=1, H=H, B=B, Q=Q, n_slots=40, n_rows=B,
               boundaries=bnd, boundary_lens=bl, status=status)
    want = [dict(state=state0.copy(), corr=c["corr"], key_gate=c["key_gate"])]
    ko.commit(layers=want, A_log=c["A_log"][None], dt_bias=c["dt_bias"][None],
              sources=ref["sources"], commit_lens=accepted, destinations=ref["destinations"],
              lower_bound=c["lower_bound"], Q=Q, B=B, H=H, boundaries=ref["boundaries"],
              boundary_lens=ref["boundary_lens"])
    assert int(status[0]) == 0
    assert np.abs(to_numpy(state) - want[0]["state"]).max() <= 1e-4 * np.abs(want[0]["state"]).max()


def test_prompts_before_speculation():
    """DeferredRecoverSSM takes prompts in, whole and in two parts beside an
    empty window and an inert request, then verifies and commits windows: the
    outputs and states of kda_recurrent over the same tokens."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import DeferredRecoverSSM, kda_recurrent
    H, B, Q, slots = 2, 4, 3, 9
    lens, window = [100, 70, 0, 50], [Q] * B
    rng = np.random.default_rng(91)
    bits = lambda *s, std=1.0: to_torch(
        synth.to_bf16_bits((rng.standard_normal(s) * std).astype(np.float32)), "cuda")
    T = sum(lens)
    dev = "cuda"
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    x = [bits(T, H, 128), bits(T, H, 128), bits(T, H, 128), bits(T, H, 128, std=0.7), bits(T, H)]
    y = [bits(B * Q, H, 128) for _ in range(3)] + [bits(B * Q, H, 128, std=0.7), bits(B * Q, H)]
    A_log = to_torch(rng.uniform(0, 1.5, H).astype(np.float32), dev)
    dt = to_torch((rng.standard_normal((H, 128)) - 2).astype(np.float32), dev)
    first = torch.randn((slots, H, 128, 128), device=dev)
    pool, own = first.clone(), i32(3, 5, 7, 0)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    loop = DeferredRecoverSSM(pool, own, i32(0, 1, 2, 3),
                              torch.zeros(B, dtype=torch.int32, device=dev),
                              torch.zeros((B, H, 8, 128), device=dev),
                              torch.zeros((B, H, 8, 256), dtype=torch.bfloat16, device=dev),
                              A_log, dt, Q=Q, lower_bound=-5.0, q_scale=128 ** -0.5,
                              status=status)
    out = torch.zeros((T, H, 128), dtype=torch.bfloat16, device=dev)
    cut = i32(0, 64, 134, 134, 184)  # request 0 in two parts
    part = [torch.cat([t[:64], t[100:]]) for t in x]
    o = torch.zeros_like(part[2])
    loop.prefill(*part, cut, o, Q=70)
    rest = [t[64:100].contiguous() for t in x]
    o2 = torch.zeros_like(rest[2])
    loop.prefill(*rest, i32(0, 36, 36, 36, 36), o2, Q=36, sources=own)
    out[:64], out[100:], out[64:100] = o[:64], o[64:], o2
    ref_pool, ref = first.clone(), torch.zeros_like(out)
    common = dict(lower_bound=-5.0, q_scale=128 ** -0.5)
    kda_recurrent(*x, A_log, dt, ref_pool, i32(0, 0, 0, 0), own, ref, Q=100,
                  query_start_loc=i32(0, 100, 170, 170, 220), **common)
    # two evaluations of one rule, each output rounded once and the chunked
    # form's query products before that (11 bits): half a step each and the
    # operators' tolerance
    def close(a, b):
        a, b = a.double(), b.double()
        assert torch.linalg.norm(a - b) <= 2.0 ** -8 * 2 * torch.linalg.norm(b)
    close(out, ref)
    assert torch.equal(pool[[0, 1, 2, 4, 6, 7, 8]], first[[0, 1, 2, 4, 6, 7, 8]])
    err = (pool - ref_pool).abs().max()
    assert err <= 1e-4 * ref_pool[[3, 5]].abs().max()
    # a window verified and accepted whole is that window decoded
    got, want = (torch.zeros((B * Q, H, 128), dtype=torch.bfloat16, device=dev) for _ in range(2))
    loop.verify(*y, got)
    loop.accept(i32(Q, Q, Q, 0))
    loop.flush()
    kda_recurrent(*y, A_log, dt, ref_pool, own, own, want, Q=Q, **common)
    close(got[:3 * Q], want[:3 * Q])
    # (the records hold keys and gates in BF16: a step of each, 2^-8, in a state
    # that three tokens changed)
    assert (pool - ref_pool)[[3, 5, 7]].abs().max() <= 3 * 2.0 ** -7 * ref_pool[[3, 5, 7]].abs().max()
    assert int(status[0]) == 0
