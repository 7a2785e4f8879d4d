"""The prompt operators without a GPU: what the C entry points and the
binding refuse before anything is launched, and the oracle's own pins."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _build, _lib
from oracle import kda_oracle as ko
from oracle import prompt_oracle as po


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


A = 0x10000  # a 16-byte aligned stand-in address: never dereferenced below
OK, ARG, ALIGN, UNSUPPORTED = (_lib.KDA_OK, _lib.KDA_ERR_ARG, _lib.KDA_ERR_ALIGN,
                               _lib.KDA_ERR_UNSUPPORTED)

RULE = dict(q=A, k=A, v=A, g=A, beta=A, A_log=A, dt=A, lb=-5.0, qs=0.1, pool=A, dtype=0,
            stride=2 * 128 * 128, n_slots=4, src=A, dst=A, bnd=None, bl=None, qsl=A, T=10, out=A)
TAIL = dict(B=2, H=2, Q=8, null=0, status=None, stream=None)


def _recurrent(lib, **over):
    return lib.kda_recurrent(*{**RULE, **TAIL, **over}.values())


def _prefill(lib, **over):
    need = lib.kda_prefill_workspace_bytes(10, 2, 2)
    return lib.kda_prefill(*{**RULE, "ws": A, "bytes": need, **TAIL, **over}.values())


@pytest.mark.parametrize("call", [_recurrent, _prefill])
@pytest.mark.parametrize("over,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(g=None), ARG),
    (dict(beta=None), ARG), (dict(A_log=None), ARG), (dict(dt=None), ARG), (dict(pool=None), ARG),
    (dict(out=None), ARG), (dict(src=None), ARG), (dict(dst=None), ARG), (dict(bnd=A), ARG),
    (dict(bl=A), ARG), (dict(B=-1), ARG), (dict(H=0), ARG), (dict(H=1025), ARG), (dict(Q=0), ARG),
    (dict(T=-1), ARG), (dict(n_slots=0), ARG), (dict(null=-2), ARG), (dict(stride=100), ARG),
    (dict(qsl=None), ARG),                                  # windows of Q tokens: T = B Q
    (dict(T=2 ** 30), ARG), (dict(B=2 ** 30), ARG),         # rows beyond 31 bits
    (dict(qs=float("nan")), ARG), (dict(qs=float("inf")), ARG),
    (dict(q=A + 2), ALIGN), (dict(k=A + 8), ALIGN), (dict(v=A + 4), ALIGN), (dict(g=A + 8), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(pool=A + 8), ALIGN), (dict(dt=A + 4), ALIGN),
    (dict(stride=2 * 128 * 128 + 1), ALIGN),
    (dict(dtype=1, stride=2 * 128 * 128 + 4), ALIGN),
    (dict(dtype=2), UNSUPPORTED), (dict(lb=0.5), UNSUPPORTED), (dict(lb=-11.0), UNSUPPORTED),
    (dict(lb=float("nan")), UNSUPPORTED),
    (dict(B=0, q=None, src=None), OK), (dict(T=0, q=None, src=None), OK),
])
def test_rule_refusals(lib, call, over, code):
    assert call(lib, **over) == code


def test_prefill_workspace(lib):
    assert lib.kda_prefill_workspace_bytes(-1, 1, 1) == -1
    assert lib.kda_prefill_workspace_bytes(1, -1, 1) == -1
    assert lib.kda_prefill_workspace_bytes(1, 1, 0) == -1
    sizes = [lib.kda_prefill_workspace_bytes(t, 3, 4) for t in (0, 1, 100, 1000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] >= 0
    need = lib.kda_prefill_workspace_bytes(10, 2, 2)
    if need:
        assert _prefill(lib, bytes=need - 1) == ARG
        assert _prefill(lib, ws=None) == ARG
        assert _prefill(lib, ws=A + 8) == ALIGN


@pytest.mark.parametrize("over,code", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(cs=None), ARG), (dict(q=None), ARG),
    (dict(width=2), ARG), (dict(width=11), ARG), (dict(stride=100), ARG), (dict(H=0), ARG),
    (dict(src=None), ARG), (dict(bnd=A), ARG), (dict(T=-1), ARG), (dict(qsl=None), ARG),
    (dict(x=A + 2), ALIGN), (dict(bias=A + 2), ALIGN), (dict(v=A + 8), ALIGN),
    (dict(stride=3 * 256 * 6 + 4), ALIGN), (dict(B=0), OK), (dict(T=0), OK),
])
def test_conv_refusals(lib, over, code):
    base = dict(x=A, w=A, bias=None, cs=A, stride=3 * 256 * 6, width=6, n_slots=4, src=A, dst=A,
                bnd=None, bl=None, qsl=A, T=10, q=A, k=A, v=A, **TAIL)
    assert lib.kda_prefill_conv(*{**base, **over}.values()) == code


@pytest.mark.parametrize("over", [
    dict(B=-1), dict(B=2 ** 24 + 1), dict(max_blocks=0), dict(stride=3), dict(n_free=-1), dict(bs=0), dict(null=-2),
    dict(head=None), dict(nxt=None), dict(qsl=None), dict(c=None), dict(n=None), dict(table=None),
    dict(free=None), dict(src=None), dict(dst=None), dict(bnd=None), dict(bl=None),
])
def test_plan_refusals(lib, over):
    base = dict(c=A, n=A, table=A, stride=4, max_blocks=4, free=A, n_free=3, head=A, nxt=A, qsl=A,
                src=A, dst=A, bnd=A, bl=A, B=2, bs=16, null=0, status=None, stream=None)
    assert lib.kda_slot_plan(*{**base, **over}.values()) == ARG


def test_slots_error_string(lib):
    assert lib.kda_error_string(_lib.KDA_ERR_SLOTS) == b"no free state slot left"


def _cpu_rule(**over):
    import torch
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = torch.zeros
    t = dict(q=z((4, 2, 128), dtype=bf), k=z((4, 2, 128), dtype=bf), v=z((4, 2, 128), dtype=bf),
             raw_g=z((4, 2, 128), dtype=bf), raw_beta=z((4, 2), dtype=bf), A_log=z(2),
             dt_bias=z((2, 128)), state_pool=z((3, 2, 128, 128)), sources=z(1, dtype=i32),
             destinations=z(1, dtype=i32), query_start_loc=z(2, dtype=i32),
             out=z((4, 2, 128), dtype=bf))
    t.update(over)
    return t


@pytest.mark.parametrize("name,make,error", [
    ("q", lambda z, d: z((4, 2, 128)), TypeError),
    ("raw_g", lambda z, d: z((4, 2, 128), dtype=d.float16), TypeError),
    ("state_pool", lambda z, d: z((3, 2, 128, 128), dtype=d.float16), TypeError),
    ("sources", lambda z, d: z(1, dtype=d.int64), TypeError),
    ("k", lambda z, d: z((4, 3, 128), dtype=d.bfloat16), ValueError),
    ("v", lambda z, d: z((5, 2, 128), dtype=d.bfloat16), ValueError),
    ("raw_beta", lambda z, d: z((2, 4), dtype=d.bfloat16), ValueError),
    ("dt_bias", lambda z, d: z((2, 64)), ValueError),
    ("state_pool", lambda z, d: z((3, 2, 128, 64)), ValueError),
    ("state_pool", lambda z, d: z((3, 2, 128, 128)).transpose(2, 3), ValueError),
    ("k", lambda z, d: z((4, 2, 256), dtype=d.bfloat16)[:, :, ::2], ValueError),
    ("query_start_loc", lambda z, d: z(3, dtype=d.int32), ValueError),
    ("destinations", lambda z, d: z(2, dtype=d.int32), ValueError),
    ("out", lambda z, d: z((4, 2, 128), dtype=d.bfloat16), ValueError),  # not on a GPU
])
def test_binding_refuses_tensors(lib, name, make, error):
    """Types, shapes, layouts and devices are checked before the call."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill, kda_recurrent
    t = _cpu_rule(**{name: make(torch.zeros, torch)})
    with pytest.raises(error):
        kda_prefill(*t.values(), Q=4, lower_bound=-5.0, q_scale=1.0)
    t["query_start_loc"], out = t["out"], t["query_start_loc"]
    with pytest.raises(error):
        kda_recurrent(*list(t.values())[:-1], Q=4, lower_bound=-5.0, q_scale=1.0,
                      query_start_loc=out)


def test_binding_refuses_maps_and_layers(lib):
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill_conv, kda_slot_plan
    z, i32, bf = torch.zeros, torch.int32, torch.bfloat16
    one = z(1, dtype=i32)
    plan = [one, one, z((1, 4), dtype=i32), one, one, one, z(2, dtype=i32), one, one, one, one]
    for i, bad in ((0, z(1)), (2, z((2, 4), dtype=i32)), (4, z(2, dtype=i32)),
                   (6, z(3, dtype=i32)), (2, z((4, 1), dtype=i32).t())):
        with pytest.raises((TypeError, ValueError)):
            kda_slot_plan(*[bad if j == i else a for j, a in enumerate(plan)], block_size=4)
    with pytest.raises(ValueError, match="CUDA"):
        kda_slot_plan(*plan, block_size=4)
    q = z((4, 2, 128), dtype=bf)
    conv = [z((4, 768), dtype=bf), z((3, 4, 256), dtype=bf), None, z((2, 768, 6), dtype=bf), one,
            one, z(2, dtype=i32), q, q, q]
    for i, bad in ((0, z((4, 512), dtype=bf)), (1, z((3, 3, 256), dtype=bf)), (3, z((2, 768, 6))),
                   (2, z(256, dtype=bf)), (8, z((4, 2, 64), dtype=bf))):
        with pytest.raises((TypeError, ValueError)):
            kda_prefill_conv(*[bad if j == i else a for j, a in enumerate(conv)], Q=4)


# --------------------------------------------------------------------------
# the oracle against hand work and the stock oracle
# --------------------------------------------------------------------------

def test_oracle_rule_equals_the_stock_oracle():
    """A prompt of 20 tokens in two parts equals the stock recurrence's state
    and outputs (kda_oracle, head by head)."""
    from prompt_testutil import ragged_case
    case = ragged_case(lens=[20], H=2, seed=1, resume=(0,), boundary={0: 7})
    src, dst, bnd = (int(case[n][0]) for n in ("sources", "destinations", "boundaries"))
    S0 = case["state"][src].astype(np.float64)
    f64 = np.zeros(case["v"].shape)
    po.rule(out_f64=f64, **case)
    f = ko.bf16_to_f64
    for h in range(2):
        ops = [f(case[n][:, h]) for n in ("q", "k", "v", "raw_g", "raw_beta")]
        a, dt = float(case["A_log"][h]), case["dt_bias"][h].astype(np.float64)
        _, o = ko.verify_item(S0[h], *ops, a, dt, -5.0, 128 ** -0.5)
        np.testing.assert_allclose(f64[:, h], o, rtol=1e-10, atol=1e-12)
        for slot, n in ((bnd, 7), (dst, 20)):
            S = ko.advance_item(S0[h], *[x[:n] for x in ops[1:]], n, a, dt, -5.0)
            np.testing.assert_array_equal(case["state"][slot, h], S.astype(np.float32))


def test_oracle_conv_by_hand():
    one = ko.f64_to_bf16(np.array([1.0]))[0]
    x = np.zeros((2, 384), dtype=np.uint16)
    x[:, 5] = ko.f64_to_bf16(np.array([2.0, 4.0]))
    w = np.zeros((3, 4, 128), dtype=np.uint16)
    w[0, 3, 5], w[0, 0, 5] = one, one
    window = np.zeros((3, 384, 4), dtype=np.uint16)
    window[1, 5, 0] = ko.f64_to_bf16(np.array([8.0]))[0]
    q, k, v = (np.zeros((2, 1, 128), dtype=np.uint16) for _ in range(3))
    i32 = lambda x: np.array([x], dtype=np.int32)
    po.conv(x=x, conv_weight=w, conv_bias=None, conv_state=window, sources=i32(1),
            destinations=i32(2), q=q, k=k, v=v, Q=2)
    silu = lambda z: ko.f64_to_bf16(np.array([z / (1 + np.exp(-z))]))[0]
    assert q[0, 0, 5] == silu(8.0 + 2.0) and q[1, 0, 5] == silu(4.0)
    assert list(ko.bf16_to_f64(window[2, 5, :3])) == [0.0, 2.0, 4.0]


def test_oracle_plan_by_hand():
    table = np.array([[7, 0, 0, 0], [0, 0, 0, 0], [9, 0, 0, 0], [5, 0, 0, 0]], dtype=np.int32)
    got, bad = po.slot_plan(computed_lens=[10, 0, 16, 3], new_lens=[10, 60, 4, 0],
                            block_table=table, free_slots=[20, 21, 22, 23, 24], free_head=1,
                            block_size=16)
    assert bad == 0
    # 0: 10 -> 20 tokens, block 0 (slot 7) ends at 16: its boundary; ends in a
    # new block.  1: 60 fresh tokens, blocks 0 and 1 passed over, 2 kept at
    # 48, ends in 3.  2: goes on at a block's end.  3: idle.
    assert list(got["sources"]) == [7, 0, 9, 0]
    assert list(got["destinations"]) == [21, 23, 24, 0]
    assert list(got["boundaries"]) == [7, 22, 0, 0]
    assert list(got["boundary_lens"]) == [6, 48, 0, 0]
    assert list(got["query_start_loc"]) == [0, 10, 70, 74, 74] and got["free_next"][0] == 5
    assert table.tolist() == [[7, 21, 0, 0], [0, 0, 22, 23], [9, 24, 0, 0], [5, 0, 0, 0]]
