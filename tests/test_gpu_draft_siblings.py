"""kda_draft_accept where a warp's lanes need what the others have read: many
siblings with few different tokens, nodes that leave the reading early (roots,
empty lanes), one request by several CTAs.  Paths and tokens equal the
oracle's, call after call."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _lib

import test_gpu_draft_accept as ta
import tree_testutil as tt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import _build
    assert torch.cuda.is_available()
    _build.build()
    _lib.load()


@pytest.mark.parametrize("probs", ["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(3, 9000), (40, 700), (900, 64)])
def test_siblings_share_tokens(B, V, probs):
    """Children hold one of four tokens: most are never taken, and the sums run
    over the first of each alone.  3 requests go to 8 CTAs each, 40 to 4, 900 to
    one."""
    rng = np.random.default_rng(B)
    sizes = rng.choice([64, 63, 33, 32, 31, 2, 1], B)
    trees = [tt.star(int(n)) if rng.random() < 0.5 else
             [-1] + [int(a) for a in rng.integers(0, min(3, int(n) - 1) + 1, int(n) - 1).clip(max=np.arange(int(n) - 1))]
             for n in sizes]
    case = ta.accept_case(trees, V, seed=B + V, probs=probs, std=1.0)
    start = case["query_start_loc"]
    for b, par in enumerate(trees):
        few = rng.integers(0, V, 4)
        case["tokens"][start[b]:start[b] + len(par)] = rng.choice(few, len(par))
        # half of the weight on the four, so that paths go down and end
        for t in range(len(par)):
            p = ta.as_f64(case["target"][start[b] + t])
            p = p / p.sum() * 0.5
            np.add.at(p, few, 0.125)
            p = p.astype(np.float32)
            case["target"][start[b] + t] = p if probs == "f32" else (p.view(np.uint32) >> 16).astype(np.uint16)
    d = ta.run_accept(case)
    ref = ta.check_accept(case, d)
    assert len(set(ref[0])) > 1
    for _ in range(10):
        for name in ("accepted", "path", "next"):
            d[name].fill_(55)
        ta.run_accept(case, d)
        for name, want in zip(("accepted", "path", "next"), ref):
            np.testing.assert_array_equal(tt.to_numpy(d[name]), want, err_msg=name)
