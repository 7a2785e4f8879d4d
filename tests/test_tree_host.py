"""The tree operators without a GPU: what the C entry points and the binding
refuse before anything is launched, and the oracle's own pins."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _build, _lib
from oracle import kda_oracle as ko
from oracle import prompt_oracle as po
from oracle import tree_oracle as to

import tree_testutil as tt


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


A = 0x10000  # a 16-byte aligned stand-in address: never dereferenced below
OK, ARG, ALIGN, UNSUPPORTED = (_lib.KDA_OK, _lib.KDA_ERR_ARG, _lib.KDA_ERR_ALIGN,
                               _lib.KDA_ERR_UNSUPPORTED)
TAIL = dict(B=2, H=2, Q=8, null=0, status=None, stream=None)
SIZES = [
    (dict(B=-1), ARG), (dict(H=0), ARG), (dict(H=1025), ARG), (dict(Q=0), ARG), (dict(Q=65), ARG),
    (dict(T=-1), ARG), (dict(null=-2), ARG), (dict(n_slots=0), ARG),
    (dict(qsl=None), ARG),                           # windows of Q nodes: T = B Q
    (dict(B=2 ** 30), ARG), (dict(slots=None), ARG),
]


def _conv(lib, **over):
    a = dict(x=A, w=A, bias=A, cs=A, stride=3 * 256 * 10, width=10, n_slots=4, slots=A, rows=A,
             pending=A, n_rows=3, parents=A, qsl=A, T=10, q=A, k=A, v=A, **TAIL)
    return lib.kda_tree_conv(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", SIZES + [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(cs=None), ARG), (dict(q=None), ARG),
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(width=2), ARG), (dict(width=11), ARG),
    (dict(stride=100), ARG), (dict(n_rows=0), ARG), (dict(rows=None, n_rows=1), ARG),
    (dict(parents=None, Q=9), ARG),
    (dict(x=A + 2), ALIGN), (dict(w=A + 8), ALIGN), (dict(bias=A + 2), ALIGN),
    (dict(cs=A + 4), ALIGN), (dict(q=A + 8), ALIGN), (dict(stride=3 * 256 * 10 + 4), ALIGN),
    (dict(B=0, x=None), OK), (dict(T=0, x=None), OK),
])
def test_conv_refusals(lib, over, code):
    assert _conv(lib, **over) == code


def _verify(lib, **over):
    a = dict(q=A, k=A, v=A, g=A, beta=A, A_log=A, dt=A, lb=-5.0, qs=0.1, pool=A, dtype=0,
             stride=2 * 128 * 128, n_slots=4, slots=A, parents=A, qsl=A, T=10, rows=A, pending=A,
             corr=A, kg=A, cs=2 * 8 * 128, ks=2 * 8 * 256, n_rows=3, rq=8, node_corr=A, out=A,
             **TAIL)
    return lib.kda_tree_verify(*{**a, **over}.values())


NO_REPLAY = dict(pending=None, corr=None, kg=None)


@pytest.mark.parametrize("over,code", SIZES + [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(g=None), ARG),
    (dict(beta=None), ARG), (dict(A_log=None), ARG), (dict(dt=None), ARG), (dict(pool=None), ARG),
    (dict(node_corr=None), ARG), (dict(out=None), ARG), (dict(pending=None), ARG),
    (dict(corr=None), ARG), (dict(kg=None), ARG), (dict(rq=0), ARG), (dict(rq=9), ARG),
    (dict(n_rows=0), ARG), (dict(rows=None, n_rows=1), ARG), (dict(stride=100), ARG),
    (dict(cs=100), ARG), (dict(ks=100), ARG), (dict(parents=None, Q=9), ARG),
    (dict(qs=float("nan")), ARG), (dict(qs=float("inf")), ARG),
    (dict(q=A + 2), ALIGN), (dict(k=A + 8), ALIGN), (dict(v=A + 4), ALIGN), (dict(g=A + 8), ALIGN),
    (dict(pool=A + 8), ALIGN), (dict(dt=A + 4), ALIGN), (dict(node_corr=A + 4), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(corr=A + 4), ALIGN), (dict(kg=A + 2), ALIGN),
    (dict(stride=2 * 128 * 128 + 1), ALIGN), (dict(cs=2 * 8 * 128 + 2), ALIGN),
    (dict(ks=2 * 8 * 256 + 4), ALIGN), (dict(NO_REPLAY, dtype=1, stride=2 * 128 * 128 + 4), ALIGN),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=1), UNSUPPORTED), (dict(lb=11.0), UNSUPPORTED),
    (dict(lb=-11.0), UNSUPPORTED), (dict(lb=float("nan")), UNSUPPORTED),
    (dict(B=0, q=None, slots=None), OK), (dict(NO_REPLAY, T=0, q=None), OK),
])
def test_verify_refusals(lib, over, code):
    assert _verify(lib, **over) == code


def _accept(lib, **over):
    a = dict(target=A, draft=None, dtype=0, ts=100, ds=100, vocab=100, tokens=A, parents=A, u=A,
             un=A, slots=None, qsl=A, T=10, accepted=A, path=A, next=A, B=2, Q=8, null=0,
             status=None, stream=None)
    return lib.kda_draft_accept(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), ARG), (dict(Q=0), ARG), (dict(Q=65), ARG), (dict(T=-1), ARG), (dict(qsl=None, T=17), ARG),
    (dict(qsl=None), ARG), (dict(null=-2), ARG), (dict(B=2 ** 29), ARG),
    (dict(target=None), ARG), (dict(tokens=None), ARG), (dict(u=None), ARG), (dict(un=None), ARG),
    (dict(accepted=None), ARG), (dict(path=None), ARG), (dict(next=None), ARG),
    (dict(vocab=0), ARG), (dict(vocab=(1 << 20) + 1), ARG), (dict(ts=99), ARG),
    (dict(parents=None, draft=A, ds=99), ARG),
    (dict(draft=A), ARG),                            # draft probabilities go with chains
    (dict(parents=None, Q=9), ARG),
    (dict(target=A + 2), ALIGN), (dict(dtype=1, target=A + 1), ALIGN),
    (dict(parents=None, draft=A + 1), ALIGN), (dict(dtype=2), UNSUPPORTED),
    (dict(B=0, target=None), OK),
])
def test_accept_refusals(lib, over, code):
    assert _accept(lib, **over) == code


def _select(lib, **over):
    a = dict(path=A, accepted=A, eager=None, k=A, g=A, node_corr=A, slots=A, rows=A, pending=A, corr=A, kg=A,
             cs=2 * 8 * 128, ks=2 * 8 * 256, n_rows=3, rq=8, x=A, conv=A, stride=3 * 256 * 10,
             width=10, n_slots=4, qsl=A, T=10, **TAIL)
    return lib.kda_tree_select(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", SIZES + [
    (dict(path=None), ARG), (dict(accepted=None), ARG), (dict(k=None), ARG), (dict(g=None), ARG),
    (dict(node_corr=None), ARG), (dict(corr=None), ARG), (dict(kg=None), ARG), (dict(x=None), ARG),
    (dict(conv=None), ARG), (dict(rq=0), ARG), (dict(rq=9), ARG), (dict(width=2), ARG),
    (dict(width=11), ARG), (dict(n_rows=0), ARG), (dict(rows=None, n_rows=1), ARG),
    (dict(cs=100), ARG), (dict(ks=100), ARG), (dict(stride=100), ARG),
    (dict(path=A + 4), ALIGN), (dict(k=A + 8), ALIGN), (dict(g=A + 8), ALIGN),
    (dict(node_corr=A + 8), ALIGN), (dict(corr=A + 8), ALIGN), (dict(kg=A + 8), ALIGN),
    (dict(x=A + 8), ALIGN), (dict(conv=A + 8), ALIGN), (dict(cs=2 * 8 * 128 + 2), ALIGN),
    (dict(stride=3 * 256 * 10 + 4), ALIGN), (dict(B=0, path=None), OK),
])
def test_select_refusals(lib, over, code):
    assert _select(lib, **over) == code


def test_binding_refusals(lib):
    """Types, shapes, layouts and devices, before the library is reached (CPU
    tensors: a call that passed them all would be refused for its device)."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import (kda_draft_accept, kda_tree_conv,
                                                               kda_tree_select, kda_tree_verify)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i32 = lambda *s: z(*s, dt=torch.int32)
    f32 = lambda *s: z(*s, dt=torch.float32)
    T, H, B = 6, 2, 2
    heads = lambda: z(T, H, 128)

    def verify(**o):
        a = dict(q=heads(), k=heads(), v=heads(), raw_g=heads(), raw_beta=z(T, H), A_log=f32(H),
                 dt_bias=f32(H, 128), state_pool=f32(3, H, 128, 128), state_slots=i32(B),
                 parents=i32(T), node_corr=f32(T, H, 128), out=heads(), Q=3, lower_bound=-5.0,
                 q_scale=0.1)
        a.update(o)
        return kda_tree_verify(**a)

    for bad in (dict(q=f32(T, H, 128)), dict(node_corr=heads()), dict(parents=z(T)),
                dict(state_pool=z(3, H, 128, 128, dt=torch.float16)), dict(A_log=z(H))):
        with pytest.raises(TypeError):
            verify(**bad)
    for bad in (dict(k=z(T, H, 64)), dict(parents=i32(T + 1)), dict(out=z(T, H, 256)[..., ::2]),
                dict(pending=i32(4)), dict(corr=f32(4, H, 8, 128)), dict(),
                dict(state_pool=f32(3, 128, 128, H).permute(0, 3, 1, 2))):
        with pytest.raises(ValueError):
            verify(**bad)

    def accept(**o):
        a = dict(target_probs=f32(T, 50), tokens=i32(T), accept_uniforms=f32(T),
                 sample_uniforms=f32(B), accepted=i32(B), path=i32(B, 8), next_tokens=i32(B), Q=3)
        a.update(o)
        return kda_draft_accept(**a)

    for bad in (dict(target_probs=z(T, 50, dt=torch.float16)),
                dict(tokens=z(T, dt=torch.int64)), dict(accept_uniforms=f32(T).double())):
        with pytest.raises(TypeError):
            accept(**bad)
    for bad in (dict(target_probs=f32(T)), dict(draft_probs=f32(T, 49)), dict(path=i32(B, 7)),
                dict(draft_probs=f32(T, 50), parents=i32(T)), dict(draft_probs=f32(T - 1, 50)),
                dict(target_probs=f32(50, T).t()), dict()):
        with pytest.raises(ValueError):
            accept(**bad)

    def conv(**o):
        a = dict(x=z(T, 768), conv_weight=z(3, 4, 256), conv_bias=None, conv_state=z(3, 768, 10),
                 state_slots=i32(B), parents=i32(T), q=heads(), k=heads(), v=heads(), Q=3)
        a.update(o)
        return kda_tree_conv(**a)

    with pytest.raises(TypeError):
        conv(conv_bias=f32(768))
    for bad in (dict(x=z(T, 767)), dict(conv_state=z(3, 767, 10)), dict(parents=i32(T - 1)), dict()):
        with pytest.raises(ValueError):
            conv(**bad)

    def select(**o):
        a = dict(path=i32(B, 8), accepted=i32(B), k=heads(), raw_g=heads(),
                 node_corr=f32(T, H, 128), state_slots=i32(B), record_rows=i32(B),
                 corr=f32(3, H, 8, 128), key_gate=z(3, H, 8, 256), Q=3)
        a.update(o)
        return kda_tree_select(**a)

    with pytest.raises(TypeError):
        select(node_corr=heads())
    for bad in (dict(x=z(T, 768)), dict(key_gate=z(3, H, 7, 256)), dict(key_gate=z(4, H, 8, 256)),
                dict(pending=i32(2)), dict(path=i32(B, 4)), dict()):
        with pytest.raises(ValueError):
            select(**bad)


# --------------------------------------------------------------------------
# the oracle
# --------------------------------------------------------------------------

def test_oracle_chain_is_the_stock_rule():
    """On chains the tree rule is the prompt operators' sequential one, and
    the replay the step oracle's."""
    trees = [tt.chain(5), tt.chain(8), tt.chain(1)]
    case = tt.tree_case(trees, 2, seed=1)
    mine = tt.copy_case(case)
    to.verify(**{n: mine[n] for n in tt.VERIFY}, Q=8, lower_bound=-5.0, q_scale=case["q_scale"])
    state = case["state"].copy()
    for b in range(3):
        slot, row = case["state_slots"][b], case["record_rows"][b]
        for h in range(2):
            n = int(case["pending"][row])
            state[slot, h] = ko.replay_item(
                state[slot, h].astype(np.float64), case["corr"][row, h].astype(np.float64),
                ko.bf16_to_f64(case["key_gate"][row, h, :, :128]),
                ko.bf16_to_f64(case["key_gate"][row, h, :, 128:]), n, case["A_log"][h],
                case["dt_bias"][h], -5.0)[0]
    np.testing.assert_allclose(mine["state"], state.astype(np.float32), rtol=0, atol=1e-6)
    out = np.zeros_like(case["out"])
    f64 = np.zeros(out.shape)
    po.rule(q=case["q"], k=case["k"], v=case["v"], raw_g=case["raw_g"], raw_beta=case["raw_beta"],
            A_log=case["A_log"], dt_bias=case["dt_bias"], lower_bound=-5.0,
            q_scale=case["q_scale"], state=mine["state"].copy(), sources=case["state_slots"],
            destinations=case["state_slots"], out=out, Q=8,
            query_start_loc=case["query_start_loc"], out_f64=f64)
    # (the second starts from the state rounded to FP32)
    np.testing.assert_allclose(ko.bf16_to_f64(mine["out"]), f64, rtol=2.0 ** -8, atol=1e-5)


@pytest.mark.parametrize("seed", [0, 1])
def test_oracle_accept_is_lossless(seed):
    """Chain of two drafts, vocabulary of four: over all draws of the drafts
    (by their probabilities) and a fine grid of uniforms, the first emitted
    token follows the target."""
    rng = np.random.default_rng(seed)
    V, G = 4, 64
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    target = np.stack([p, rng.dirichlet(np.ones(V))])
    grid = (np.arange(G) + 0.5) / G
    got = np.zeros(V)
    for x in range(V):
        u, s = (g.ravel() for g in np.meshgrid(grid, grid))
        B = len(u)
        acc, path, nxt, bad = to.accept(
            target=np.tile(target, (B, 1)), draft=np.tile(np.stack([q, q]), (B, 1)),
            tokens=np.tile([0, x], B), accept_uniforms=np.stack([u, u], 1).ravel(),
            sample_uniforms=s, Q=2)
        assert bad == 0
        first = np.where(acc == 2, x, nxt)
        got += q[x] * np.bincount(first, minlength=V) / B
    # a grid of G points has each border off by at most half a cell: two
    # borders of u and V of s
    assert np.abs(got - p).max() <= (1 + V) / G
    # a tree of two likely tokens, taken for sure
    u, s = (g.ravel() for g in np.meshgrid(grid, grid))
    B = len(u)
    acc, path, nxt, bad = to.accept(
        target=np.tile(np.stack([p, p, p]), (B, 1)), tokens=np.tile([0, 2, 1], B),
        parents=np.tile([-1, 0, 0], B), accept_uniforms=np.repeat(u, 3), sample_uniforms=s, Q=3)
    first = np.where(acc == 2, np.where(path[:, 1] == 1, 2, 1), nxt)
    assert bad == 0 and np.abs(np.bincount(first, minlength=V) / B - p).max() <= (2 + V) / G


def test_oracle_trees():
    assert to.tree(np.array([-1, 0, 1, 2, 3, 4, 5, 6, 0]), 0, 9) is not None
    assert to.tree(np.array([-1, 0, 1, 2, 3, 4, 5, 6, 7]), 0, 9) is None  # nine deep
    assert to.tree(np.array([0]), 0, 1) is None
    assert to.tree(np.array([-1, -2]), 0, 2) is None
    assert to.tree(np.array([-1, 2, 0]), 0, 3) is None
    assert to.tree(None, 0, 8) == tt.chain(8)
