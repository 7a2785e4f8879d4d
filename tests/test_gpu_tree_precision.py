"""kda_tree_verify holds 24 bits of what its products are made of.

The corrections of ordinary cases are compared at 1e-4 of a head's largest
value, which a product of two BF16 parts (16 bits) would pass by far.  Here all
128 channels of a vector hold one value, so that what an operand loses adds up
in place of cancelling, gates and betas are infinite (decays of 1, beta of 1),
and every correction has a closed form:
  "state": nodes on the checkpoint, v = 0, rows of the page s_r:
      u_t = -128 s_r c_t rsqrt(128 c_t^2 + 1e-6);
  "pairs": an empty page, a node (v = 1) and its child (v = 0) in turn:
      u_child = -128 c_t c_p rsqrt(..) rsqrt(..).

Tolerance, relative, in 2^-24: a norm's root (2 units in the last place) 4 and
two products behind it 2, for a pair twice: 12; decays, betas and their divisions
4; operands' parts and the products left out 2 for each of two products: 4; the
sum of 128, in eight steps of the tensor core, each off by 2^-22 of what is there
so far, 18 (by FMA 16 + 3 + 1 roundings at most), of smaller products' sums 2; the
last product's step 4; one rounding each of v - w and of the split sums 4: 48,
2.9e-6.  The third part of an operand is worth up to 2^-17 = 128 2^-24; the
values below are those that need it, which the tests without a GPU show by
planting its loss in an emulation."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib, synth
from oracle import kda_oracle as ko

import tree_testutil as tt

TOL = 48 * 2.0 ** -24
EPS = float(np.float32(1e-6))


def bf16(x):
    return ko.bf16_to_f64(ko.f64_to_bf16(np.asarray(x, dtype=np.float64)))


def parts(x):
    """Three BF16 parts, each the nearest to what the ones before leave."""
    out = []
    for _ in range(3):
        out.append(bf16(x))
        x = x - out[-1]
    return out


def unit(c):
    """A channel of the normalised vector of 128 times c."""
    return c / np.sqrt(128 * c * c + EPS)


def missing(x):
    """What two parts leave of x, relative."""
    hi, mid, _ = parts(x)
    return np.abs(x - hi - mid) / np.abs(x)


# BF16 values whose unit vectors need the third part most, and FP32 rows that do
CS = bf16(np.unique(bf16(np.exp(np.linspace(np.log(8e-5), np.log(3e-4), 4000)))))
CS = CS[np.argsort(-missing(unit(CS)))]
ROWS = np.float32(2.0) ** np.arange(-6, 2).repeat(16) * np.concatenate(
    [np.linspace(1, 1.9, 64), 1 + 2.0 ** -9 + 2.0 ** -17 - 2.0 ** -23 * np.arange(1, 65)])
ROWS = ROWS.astype(np.float32)


def pair_keys(n):
    """Keys of n / 2 nodes and their children, the products of the first half of
    which need the third part."""
    a, b = np.meshgrid(CS, CS, indexing="ij")
    order = np.argsort(-missing(128 * unit(a) * unit(b)), axis=None)
    take = np.concatenate([order[:n // 4], np.argsort(-missing(unit(a)), axis=None)[:n - n // 4]])
    return np.stack([a.ravel()[take], b.ravel()[take]], 1).ravel()[:n]


def product(a, b, lost=""):
    """The six products of parts that are kept, as a sum in FP64."""
    pa, pb = parts(a), parts(b)
    if "a" in lost:
        pa[2] = pa[2] * 0
    if "b" in lost:
        pb[2] = pb[2] * 0
    return sum(pa[i] * pb[j] for i, j in ((2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)))


def emulated(kind, c, rows, lost=None):
    """Corrections [nodes, 128] with products in parts, the third part of one
    operand left out: S, X or R of "state", X, Y or T of "pairs"."""
    k = unit(c)
    if kind == "state":
        w = 128 * product(rows[None], k[:, None], {"S": "a", "X": "b"}.get(lost, ""))
        return product(-w, np.ones_like(w), "a" if lost == "R" else "")
    up, down = k[0::2], k[1::2]
    p = 128 * product(down, up, {"X": "a", "Y": "b"}.get(lost, ""))
    t = product(np.ones_like(p), -p, "b" if lost == "T" else "")
    u = np.stack([np.ones_like(t), t], 1).ravel()
    return np.repeat(u[:, None], 128, 1)


def exact(kind, c, rows):
    k = unit(c)
    if kind == "state":
        return -128 * rows.astype(np.float64)[None] * k[:, None]
    u = np.ones(len(c))
    u[1::2] = -128 * k[0::2] * k[1::2]
    return np.repeat(u[:, None], 128, 1)


def keys(kind, n):
    return CS[:n] if kind == "state" else pair_keys(n)


@pytest.mark.parametrize("n", [4, 20, 64])
@pytest.mark.parametrize("kind,operands", [("state", "SXR"), ("pairs", "XYT")])
def test_two_parts_would_be_seen(kind, operands, n):
    c = keys(kind, n)
    want = exact(kind, c, ROWS)
    off = lambda lost: (np.abs(emulated(kind, c, ROWS, lost) - want) / np.abs(want)).max()
    assert off(None) < 4 * 2.0 ** -24
    for lost in operands:
        assert off(lost) > 1.5 * TOL, lost


@pytest.fixture(scope="module")
def lib():
    from linear_attention_speculative_recoverssm_gb300 import _build
    _build.build()
    return _lib.load()


@pytest.mark.gpu
# windows of few nodes by FMA, and on the tensor cores, up to 32 nodes and more
@pytest.mark.parametrize("B,H,n", [(2, 2, 4), (200, 8, 4), (2, 2, 6), (160, 5, 6), (2, 2, 20),
                                   (30, 8, 32), (2, 2, 40), (12, 16, 64)])
@pytest.mark.parametrize("kind", ["state", "pairs"])
@pytest.mark.parametrize("pool", ["f32", "bf16"])
def test_corrections_hold_24_bits(lib, kind, pool, B, H, n):
    if kind == "state":
        trees = [[-1] * n] * B
    else:
        trees = [[t - 1 if t % 2 else -1 for t in range(n)]] * B
    case = tt.tree_case(trees, H, seed=1, pool=pool, replay=False)
    c = keys(kind, n)
    rows = ROWS if pool == "f32" else bf16(ROWS).astype(np.float32)
    inf = 0x7F80
    case["k"][:] = np.tile(synth.to_bf16_bits(c.astype(np.float32)), B)[:, None, None]
    case["raw_g"][:], case["raw_beta"][:] = inf | 0x8000, inf
    case["v"][:] = 0
    state = np.zeros((1, 1, 128, 128), np.float32)
    if kind == "state":
        state[:] = rows[:, None]
    else:
        case["v"].reshape(B, n, H, 128)[:, 0::2] = 0x3F80  # 1
    case["state"][:] = state if pool == "f32" else synth.to_bf16_bits(state)
    d = tt.on_device(case)
    tt.call_verify(case, d)
    assert int(d["status"].item()) == 0
    got = tt.to_numpy(d["node_corr"]).reshape(B, n, H, 128).astype(np.float64)
    want = exact(kind, c, rows)[None, :, None]
    off = np.abs(got - want) / np.abs(want)
    assert off.max() <= TOL, off.max() * 2.0 ** 24
