"""What kda_prefill asks for as workspace, and that it stays inside it."""
import numpy as np
import pytest

from linear_attention_speculative_recoverssm_gb300 import _build, _lib


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def test_size_follows_the_windows(lib):
    size = lib.kda_prefill_workspace_bytes_for
    for args in ((-1, 1, 1, 1, 0), (1, -1, 1, 1, 0), (1, 1, 0, 1, 0), (1, 1, 1025, 1, 0),
                 (1, 1, 1, 0, 0)):
        assert size(*args) == -1
    # no window longer than 40 tokens: none at all, however many there are
    assert size(512 * 37, 512, 64, 37, 1) == size(4096 * 40, 4096, 32, 40, 1) == 0
    assert size(40, 3, 32, 10000, 1) == lib.kda_prefill_workspace_bytes(40, 3, 32) == 0
    assert size(0, 0, 1, 1, 0) == size(100, 0, 1, 100, 0) == 0
    for T, B, H in ((41, 1, 1), (1000, 7, 5), (16384, 16, 32), (4096 * 41, 4096, 2)):
        sizes = [size(T, B, H, Q, 1) for Q in (1, 40, 41, 64, 100, 1000, T, 2 * T)]
        assert sizes == sorted(sizes) and sizes[2] > 0
        assert sizes[-1] == sizes[-2] == lib.kda_prefill_workspace_bytes(T, B, H)
        assert size(T, B, H, T, 0) <= size(T, B, H, T, 1)
    # an image of a chunk, 128.6 KB, and no more than 2 % beside it, for windows
    # of whole chunks without boundaries (a chunk more where the windows may differ)
    image, need = 1029 * 128, size(64 * 256, 1, 32, 64 * 256, 0)
    assert 32 * 256 * image <= need <= 1.02 * 32 * 257 * image + 64 * 1024 * 32


@pytest.mark.gpu
@pytest.mark.parametrize("lens,bounds", [([40] * 20, True), ([41], False), ([41, 1], True),
                                         ([64, 128, 192], False), ([70, 24, 25, 26, 300], True),
                                         ([4100], False), ([4100, 64], True), ([65] * 60, False)])
def test_stays_inside(lens, bounds):
    """A workspace of exactly the size asked for, marks before and behind it;
    none where none is asked for."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import (kda_prefill,
                                                               kda_prefill_workspace_bytes)
    from prompt_testutil import call_rule, on_device, ragged_case
    from test_gpu_prompt_rule import verify
    case = ragged_case(lens=lens, H=3, seed=len(lens) + lens[0],
                       boundary={b: n // 2 for b, n in enumerate(lens)} if bounds else None)
    if not bounds:
        case["boundaries"] = case["boundary_lens"] = None
    need = kda_prefill_workspace_bytes(sum(lens), len(lens), 3, case["Q"], bounds)
    assert (need == 0) == (max(lens) <= 40)
    room = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    d = on_device(case)
    call_rule(kda_prefill, case, d, workspace=room[256:256 + need])
    verify("prefill", case, d)
    assert bool((room[:256] == 0x5a).all()) and bool((room[256 + need:] == 0x5a).all())


@pytest.mark.gpu
def test_too_small_is_refused():
    import torch
    from linear_attention_speculative_recoverssm_gb300 import (KdaError, kda_prefill,
                                                               kda_prefill_workspace_bytes)
    from prompt_testutil import call_rule, on_device, ragged_case
    case = ragged_case(lens=[41, 64], H=2, seed=1)
    need = kda_prefill_workspace_bytes(105, 2, 2, 64, True)
    d = on_device(case)
    before = d["state"].clone()
    with pytest.raises(KdaError):
        call_rule(kda_prefill, case, d,
                  workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(before, d["state"])


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["default", "zero", "side", "address", "none"])
def test_workspace_belongs_to_the_call_s_stream(which, monkeypatch):
    """What the binding allocates is of the stream that the kernels run on:
    another stream's next allocation does not take it while they run."""
    import torch
    from linear_attention_speculative_recoverssm_gb300 import kda_prefill
    from prompt_testutil import call_rule, on_device, ragged_case
    from test_gpu_prompt_rule import verify
    case = ragged_case(lens=[70, 100], H=2, seed=3)
    d = on_device(case)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    stream, want = {"default": (torch.cuda.default_stream(), 0), "zero": (0, 0),
                    "side": (side, side.cuda_stream), "none": (None, other.cuda_stream),
                    "address": (side.cuda_stream, side.cuda_stream)}[which]
    seen, empty = [], torch.empty
    def noted(*args, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)
    with torch.cuda.stream(other):
        monkeypatch.setattr(torch, "empty", noted)
        call_rule(kda_prefill, case, d, stream=stream)
        monkeypatch.undo()
    torch.cuda.synchronize()
    assert seen == [want]
    verify("prefill", case, d)
