"""kda_tree_verify's kernels where the tests of single shapes do not take them:
windows of five and six nodes in batches large enough for the tensor cores, of
every page type, and pages beyond 32 bits for every kernel."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib

import test_gpu_tree as tg
import tree_testutil as tt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import _build
    assert torch.cuda.is_available()
    _build.build()
    _lib.load()


def trees_of(seed, sizes):
    rng = np.random.default_rng(seed)
    return [tt.random_tree(rng, int(n)) for n in sizes]


@pytest.mark.parametrize("pool,replay", [("f32", True), ("f32", False), ("bf16", False)])
@pytest.mark.parametrize("cap", [4, 5, 6])
def test_small_windows_in_large_batches(cap, pool, replay):
    sizes = np.random.default_rng(cap).integers(1, cap + 1, 170)
    sizes[0] = cap
    case = tt.tree_case(trees_of(cap, sizes), 4, seed=cap, pool=pool, replay=replay, inert=(3, 9),
                        rowless=(4,) if replay else ())
    assert case["Q"] == cap
    tg.check_verify(case, tg.run_verify(case))


@pytest.mark.parametrize("pool", ["f32", "bf16"])
@pytest.mark.parametrize("n,B", [(4, 3), (4, 100), (9, 3), (40, 3)])
def test_pages_beyond_32_bits(n, B, pool):
    """The last page further than 2^31 elements from the first."""
    import torch
    case = tt.tree_case(trees_of(n, [n] * B), 2, seed=14, pool=pool, replay=pool == "f32", extra_slots=0)
    d = tt.on_device(case)
    slots, pages = case["state"].shape[0], 2 * 128 * 128
    stride = max(pages, 2 ** 31 // (slots - 1) + 64 - 2 ** 31 // (slots - 1) % 8)
    pool_mem = torch.zeros((slots - 1) * stride + pages, dtype=d["state"].dtype, device="cuda")
    far = pool_mem.as_strided(d["state"].shape, (stride, 128 * 128, 128, 1))
    assert (slots - 1) * stride > 2 ** 31 and slots - 1 in case["state_slots"]
    far.copy_(d["state"])
    d["state"] = far
    tg.run_verify(case, d)
    tg.check_verify(case, d)
