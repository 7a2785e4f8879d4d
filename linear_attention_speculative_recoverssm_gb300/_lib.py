"""ctypes binding of libkda_recoverssm.so (argument marshalling only).

Every function here takes torch tensors on the GPU, reads their data
pointers, sizes and strides, and calls the C entry point of the same name on
the current CUDA stream (or the given one).  All compute runs in the
library's kernels; there is no fallback: if the library is missing, import
fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda_recoverssm.so")

# status codes (include/kda_recoverssm.h)
KDA_OK = 0
KDA_ERR_ARG = -1
KDA_ERR_ALIGN = -2
KDA_ERR_UNSUPPORTED = -3
KDA_ERR_CUDA = -4
KDA_ERR_TIMEOUT = -5
KDA_ERR_SCRATCH = -6
KDA_ERR_SLOTS = -7
KDA_LAYER_STEP_NOALLOC_MAX_BYTES = 16 * 1024 * 1024
KDA_STATE_F32 = 0
KDA_STATE_BF16 = 1
KDA_PROBS_F32 = 0
KDA_PROBS_BF16 = 1
KDA_TREE_MAX_NODES = 64
KDA_TREE_MAX_DEPTH = 8
KDA_MAX_VOCAB = 1 << 20

EXPORTS = ("kda_abi_version", "kda_error_string", "kda_check_status", "kda_verify",
           "kda_replay_verify", "kda_replay_verify_layers",
           "kda_commit", "kda_defer_commit", "kda_flush_plan", "kda_selftest_wait_timeout",
           "kda_layer_prologue", "kda_layer_epilogue", "kda_layer_step_workspace_bytes",
           "kda_layer_step", "kda_layer_step_noalloc", "kda_slot_plan", "kda_prefill_conv",
           "kda_prefill_workspace_bytes", "kda_prefill_workspace_bytes_for", "kda_prefill",
           "kda_recurrent", "kda_tree_conv", "kda_tree_verify", "kda_draft_accept",
           "kda_tree_settle", "kda_tree_select")

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float

_SIGS = {
    "kda_abi_version": ([], _I),
    "kda_error_string": ([_I], ctypes.c_char_p),
    "kda_check_status": ([_P, _P], _I),
    "kda_verify": ([_P] * 7 + [_F, _F, _P, _I, _I64, _I, _P, _P, _I, _P, _P, _P, _I64, _I64,
                               _I, _I, _P, _I, _I, _I, _I, _P, _P], _I),
    "kda_replay_verify": ([_P] * 7 + [_F, _F, _P, _I64, _I, _P, _P, _I, _P, _P, _P, _P, _I64,
                                      _I64, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P],
                          _I),
    "kda_replay_verify_layers": ([_P] * 7 + [_F, _F, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I,
                                             _I, _P, _I, _I, _I, _I, _I, _P, _P], _I),
    "kda_commit": ([_P] * 14 + [_I, _F, _I, _I, _I, _I, _I, _I, _I, _P, _P], _I),
    "kda_defer_commit": ([_P] * 5 + [_I, _I, _I, _P, _P], _I),
    "kda_flush_plan": ([_P] * 7 + [_I, _I, _I, _I, _P, _P], _I),
    "kda_selftest_wait_timeout": ([_P, _P], _I),
    "kda_layer_prologue": ([_P] * 4 + [_I64] + [_P] * 5 + [_I, _I, _I] + [_P] * 4
                           + [_I, _I, _I, _I, _P, _P], _I),
    "kda_layer_epilogue": ([_P, _P, _P, _F, _P, _I, _I, _P], _I),
    "kda_layer_step_workspace_bytes": ([_I, _I, _I], _I64),
    "kda_layer_step_noalloc": ([_P] * 4 + [_I64] + [_P] * 5 + [_F, _F, _P, _I64, _I, _P, _P, _P,
                                                           _P, _P, _I64, _I64, _I, _I, _P, _P, _F,
                                                           _P, _I, _I, _I, _I, _P, _P], _I),
    "kda_layer_step": ([_P] * 4 + [_I64] + [_P] * 5 + [_F, _F, _P, _I64, _I, _P, _P, _P, _P, _P,
                                                   _I64, _I64, _I, _I, _P, _P, _F, _P, _P, _I64,
                                                   _I, _I, _I, _I, _P, _P], _I),
    "kda_slot_plan": ([_P] * 3 + [_I64, _I, _P, _I] + [_P] * 7 + [_I, _I, _I, _P, _P], _I),
    "kda_prefill_conv": ([_P] * 4 + [_I64, _I, _I] + [_P] * 5 + [_I] + [_P] * 3
                         + [_I, _I, _I, _I, _P, _P], _I),
    "kda_prefill_workspace_bytes": ([_I, _I, _I], _I64),
    "kda_prefill_workspace_bytes_for": ([_I, _I, _I, _I, _I], _I64),
    "kda_prefill": ([_P] * 7 + [_F, _F, _P, _I, _I64, _I] + [_P] * 5 + [_I, _P, _P, _I64]
                    + [_I, _I, _I, _I, _P, _P], _I),
    "kda_recurrent": ([_P] * 7 + [_F, _F, _P, _I, _I64, _I] + [_P] * 5 + [_I, _P]
                      + [_I, _I, _I, _I, _P, _P], _I),
    "kda_tree_conv": ([_P] * 4 + [_I64, _I, _I, _P, _P, _P, _I, _P, _P, _I, _P, _P, _P]
                      + [_I, _I, _I, _I, _P, _P], _I),
    "kda_tree_verify": ([_P] * 7 + [_F, _F, _P, _I, _I64, _I, _P, _P, _P, _I, _P, _P, _P, _P,
                                    _I64, _I64, _I, _I, _P, _P] + [_I, _I, _I, _I, _P, _P], _I),
    "kda_draft_accept": ([_P, _P, _I, _I64, _I64, _I] + [_P] * 6 + [_I, _P, _P, _P]
                         + [_I, _I, _I, _P, _P], _I),
    "kda_tree_settle": ([_P, _P, _I, _P, _I, _P, _P, _I, _P, _P, _I, _I, _P] + [_I, _I, _I, _P, _P], _I),
    "kda_tree_select": ([_P] * 11 + [_I64, _I64, _I, _I, _P, _P, _I64, _I, _I, _P, _I]
                        + [_I, _I, _I, _I, _P, _P], _I),
}

_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library once; raise ImportError if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(
            f"{p} is missing: build it with `python -m "
            "linear_attention_speculative_recoverssm_gb300._build` "
            "(or __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


class KdaError(RuntimeError):
    def __init__(self, fn, code):
        msg = load().kda_error_string(code).decode()
        super().__init__(f"{fn} returned {code} ({msg})")
        self.code = code


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, code, raise_on_error):
    if code != KDA_OK and raise_on_error:
        raise KdaError(fn, code)
    return code


def _expect(t, dtype, name):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _check_step_dtypes(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_slots, record_rows,
                       corr, key_gate, out):
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("raw_g", raw_g), ("raw_beta", raw_beta),
                    ("key_gate", key_gate), ("out", out)):
        _expect(t, torch.bfloat16, name)
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias), ("corr", corr)):
        _expect(t, torch.float32, name)
    for name, t in (("state_slots", state_slots), ("record_rows", record_rows)):
        _expect(t, torch.int32, name)


def kda_check_status(status, *, stream=None):
    """The code held by the device status word ``status`` (int32 tensor),
    read back after the work already enqueued on the stream (this call waits
    for that stream)."""
    import torch
    _expect(status, torch.int32, "status")
    return load().kda_check_status(_ptr(status), _stream(stream))


def kda_verify(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, state_slots, corr,
               key_gate, out, *, Q, lower_bound, q_scale, record_rows=None,
               query_start_loc=None, null_slot=0, status=None, stream=None,
               raise_on_error=True):
    """Stock verify of one window (state read only).  Shapes as in
    include/kda_recoverssm.h; state_pool is float32 or bfloat16; the
    activations' first dimension is the token count (B*Q without
    query_start_loc)."""
    import torch
    _check_step_dtypes(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_slots, record_rows,
                       corr, key_gate, out)
    _expect(query_start_loc, torch.int32, "query_start_loc")
    dtype = KDA_STATE_F32 if state_pool.dtype == torch.float32 else KDA_STATE_BF16
    if state_pool.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("state_pool must be float32 or bfloat16")
    B = state_slots.shape[0]
    H = q.shape[1]
    rc = load().kda_verify(
        _ptr(q), _ptr(k), _ptr(v), _ptr(raw_g), _ptr(raw_beta), _ptr(A_log), _ptr(dt_bias),
        lower_bound, q_scale, _ptr(state_pool), dtype, state_pool.stride(0),
        state_pool.shape[0], _ptr(state_slots), _ptr(query_start_loc), q.shape[0],
        _ptr(record_rows), _ptr(corr), _ptr(key_gate), corr.stride(0), key_gate.stride(0),
        corr.shape[0], corr.shape[2], _ptr(out), B, H, Q, null_slot, _ptr(status),
        _stream(stream))
    return _check("kda_verify", rc, raise_on_error)


def kda_replay_verify(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, state_slots,
                      record_rows, pending, corr, key_gate, out, *, Q, lower_bound, q_scale,
                      boundary_slots=None, boundary_lens=None, query_start_loc=None,
                      null_slot=0, split=0, status=None, stream=None, raise_on_error=True):
    """Fused replay + verify (FP32 state pool, written in place)."""
    import torch
    _check_step_dtypes(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_slots, record_rows,
                       corr, key_gate, out)
    _expect(query_start_loc, torch.int32, "query_start_loc")
    _expect(state_pool, torch.float32, "state_pool")
    _expect(pending, torch.int32, "pending")
    B = state_slots.shape[0]
    H = q.shape[1]
    rc = load().kda_replay_verify(
        _ptr(q), _ptr(k), _ptr(v), _ptr(raw_g), _ptr(raw_beta), _ptr(A_log), _ptr(dt_bias),
        lower_bound, q_scale, _ptr(state_pool), state_pool.stride(0), state_pool.shape[0],
        _ptr(state_slots), _ptr(query_start_loc), q.shape[0], _ptr(record_rows), _ptr(pending),
        _ptr(corr), _ptr(key_gate), corr.stride(0), key_gate.stride(0), corr.shape[0],
        corr.shape[2], _ptr(boundary_slots), _ptr(boundary_lens), _ptr(out), B, H, Q,
        null_slot, split, _ptr(status), _stream(stream))
    return _check("kda_replay_verify", rc, raise_on_error)


def kda_replay_verify_layers(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pools, state_slots,
                             record_rows, pending, corrs, key_gates, out, *, Q, lower_bound,
                             q_scale, null_slot=0, status=None, stream=None,
                             raise_on_error=True):
    """Fused replay + verify over L layers in one launch: q, k, v, raw_g, out
    [L, B*Q, H, 128] and raw_beta [L, B*Q, H] layer-stacked; A_log [L, H],
    dt_bias [L, H, 128]; state_pools, corrs, key_gates lists of the L
    layers' FP32 pools, FP32 corrections and BF16 key/gate records (their
    addresses and strides are passed as host arrays); the index arrays are
    shared by the layers."""
    import torch
    L = len(state_pools)
    if not (len(corrs) == len(key_gates) == L):
        raise ValueError("state_pools, corrs and key_gates must list the same layers")
    for t in state_pools:
        _expect(t, torch.float32, "state_pools[l]")
    for t in corrs:
        _expect(t, torch.float32, "corrs[l]")
    if any(t.shape[2] != corrs[0].shape[2] for t in list(corrs) + list(key_gates)):
        raise ValueError("every layer's records must hold the same number of tokens")
    for t in key_gates:
        _expect(t, torch.bfloat16, "key_gates[l]")
    _check_step_dtypes(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_slots, record_rows,
                       corrs[0], key_gates[0], out)
    _expect(pending, torch.int32, "pending")
    ptrs = lambda ts: (ctypes.c_void_p * L)(*[t.data_ptr() for t in ts])
    strides = lambda ts: (ctypes.c_int64 * L)(*[t.stride(0) for t in ts])
    B = state_slots.shape[0]
    H = q.shape[2]
    rc = load().kda_replay_verify_layers(
        _ptr(q), _ptr(k), _ptr(v), _ptr(raw_g), _ptr(raw_beta), _ptr(A_log), _ptr(dt_bias),
        lower_bound, q_scale, ptrs(state_pools), strides(state_pools),
        min(t.shape[0] for t in state_pools), _ptr(state_slots), _ptr(record_rows),
        _ptr(pending), ptrs(corrs), ptrs(key_gates), strides(corrs), strides(key_gates),
        min(min(t.shape[0] for t in corrs), min(t.shape[0] for t in key_gates)),
        corrs[0].shape[2], _ptr(out), L,
        B, H, Q, null_slot, _ptr(status), _stream(stream))
    return _check("kda_replay_verify_layers", rc, raise_on_error)


def kda_commit(state_ptrs, corr_ptrs, kg_ptrs, state_strides, corr_strides, kg_strides, A_log,
               dt_bias, sources, commit_lens, destinations, *, state_dtype, lower_bound, L, H,
               B, Q, n_slots, n_rows, boundaries=None, boundary_lens=None, record_rows=None,
               null_slot=0, status=None, stream=None, raise_on_error=True):
    """Standalone commit over L layers; the six tables are device int64
    tensors of [L] addresses / strides (see layer_tables)."""
    rc = load().kda_commit(
        _ptr(state_ptrs), _ptr(corr_ptrs), _ptr(kg_ptrs), _ptr(state_strides),
        _ptr(corr_strides), _ptr(kg_strides), _ptr(A_log), _ptr(dt_bias), _ptr(sources),
        _ptr(commit_lens), _ptr(destinations), _ptr(boundaries), _ptr(boundary_lens),
        _ptr(record_rows), state_dtype, lower_bound, null_slot, L, H, B, Q, n_slots, n_rows,
        _ptr(status), _stream(stream))
    return _check("kda_commit", rc, raise_on_error)


def layer_tables(states, corrs, key_gates, device):
    """The per-layer address and stride tables kda_commit reads, as device
    int64 tensors: (state_ptrs, corr_ptrs, kg_ptrs, state_strides,
    corr_strides, kg_strides)."""
    import torch
    mk = lambda xs: torch.tensor(xs, dtype=torch.int64, device=device)
    return (mk([s.data_ptr() for s in states]), mk([c.data_ptr() for c in corrs]),
            mk([g.data_ptr() for g in key_gates]), mk([s.stride(0) for s in states]),
            mk([c.stride(0) for c in corrs]), mk([g.stride(0) for g in key_gates]))


def kda_defer_commit(state_slots, commit_lens, record_rows, pending, *, eager=None, null_slot=0,
                     status=None, stream=None, raise_on_error=True):
    rc = load().kda_defer_commit(
        _ptr(state_slots), _ptr(commit_lens), _ptr(record_rows), _ptr(pending), _ptr(eager),
        state_slots.shape[0], null_slot, pending.shape[0], _ptr(status), _stream(stream))
    return _check("kda_defer_commit", rc, raise_on_error)


def kda_flush_plan(state_slots, record_rows, pending, commit_lens, final_slots, boundary_slots,
                   boundary_lens, *, Q, null_slot=0, status=None, stream=None,
                   raise_on_error=True):
    rc = load().kda_flush_plan(
        _ptr(state_slots), _ptr(record_rows), _ptr(pending), _ptr(commit_lens),
        _ptr(final_slots), _ptr(boundary_slots), _ptr(boundary_lens), state_slots.shape[0], Q,
        null_slot, pending.shape[0], _ptr(status), _stream(stream))
    return _check("kda_flush_plan", rc, raise_on_error)


def kda_selftest_wait_timeout(status, *, stream=None, raise_on_error=True):
    """Failure-detection self-test: a device wait that runs out writes
    KDA_ERR_TIMEOUT to ``status`` (device int32)."""
    rc = load().kda_selftest_wait_timeout(_ptr(status), _stream(stream))
    return _check("kda_selftest_wait_timeout", rc, raise_on_error)


def kda_layer_prologue(x, conv_weight, conv_bias, conv_state, f_a, f_b, state_slots,
                       record_rows, pending, q, k, v, raw_g, *, Q, rq=None, null_slot=0,
                       status=None, stream=None, raise_on_error=True):
    """The layer's convolution + SiLU, gate projection and window rewrite
    (shapes as in include/kda_recoverssm.h; conv_state [slots, 3*H*128,
    rq + 2])."""
    import torch
    for name, t in (("x", x), ("conv_weight", conv_weight), ("conv_bias", conv_bias),
                    ("conv_state", conv_state), ("f_a", f_a), ("f_b", f_b), ("q", q), ("k", k),
                    ("v", v), ("raw_g", raw_g)):
        _expect(t, torch.bfloat16, name)
    for name, t in (("state_slots", state_slots), ("record_rows", record_rows),
                    ("pending", pending)):
        _expect(t, torch.int32, name)
    rq = conv_state.shape[2] - 2 if rq is None else rq
    rc = load().kda_layer_prologue(
        _ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state), conv_state.stride(0),
        _ptr(f_a), _ptr(f_b), _ptr(state_slots), _ptr(record_rows), _ptr(pending),
        conv_state.shape[0], 0 if pending is None else pending.shape[0], rq, _ptr(q), _ptr(k),
        _ptr(v), _ptr(raw_g), state_slots.shape[0], q.shape[1], Q, null_slot, _ptr(status),
        _stream(stream))
    return _check("kda_layer_prologue", rc, raise_on_error)


def kda_layer_epilogue(o, gate, norm_weight, out, *, eps, stream=None, raise_on_error=True):
    """The gated RMSNorm of the step's outputs o [T, H, 128] into out
    [T, H*128]."""
    import torch
    _expect(o, torch.bfloat16, "o")
    _expect(gate, torch.bfloat16, "gate")
    _expect(out, torch.bfloat16, "out")
    _expect(norm_weight, torch.float32, "norm_weight")
    rc = load().kda_layer_epilogue(_ptr(o), _ptr(gate), _ptr(norm_weight), eps, _ptr(out),
                                   o.shape[0], o.shape[1], _stream(stream))
    return _check("kda_layer_epilogue", rc, raise_on_error)


def kda_layer_step_workspace_bytes(B, H, Q):
    """Bytes of workspace kda_layer_step needs (the step's q, k, v, raw_g)."""
    return load().kda_layer_step_workspace_bytes(B, H, Q)


def kda_layer_step(x, conv_weight, conv_bias, conv_state, f_a, f_b, raw_beta, A_log, dt_bias,
                   state_pool, state_slots, record_rows, pending, corr, key_gate, gate,
                   norm_weight, out, workspace, *, Q, lower_bound, q_scale, eps, rq=None,
                   null_slot=0, status=None, stream=None, raise_on_error=True):
    """One model-layer step (convolution + SiLU, gate projection, fused
    replay + verify with the gated RMSNorm folded in): out [B*Q, H*128]
    BF16.  ``workspace`` is a device tensor of at least
    kda_layer_step_workspace_bytes(B, H, Q) bytes; afterwards it holds the
    step's q, k, v, raw_g ([B*Q, H, 128] BF16 each, in that order)."""
    import torch
    for name, t in (("x", x), ("conv_weight", conv_weight), ("conv_bias", conv_bias),
                    ("conv_state", conv_state), ("f_a", f_a), ("f_b", f_b),
                    ("raw_beta", raw_beta), ("key_gate", key_gate), ("gate", gate),
                    ("out", out)):
        _expect(t, torch.bfloat16, name)
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias), ("state_pool", state_pool),
                    ("corr", corr), ("norm_weight", norm_weight)):
        _expect(t, torch.float32, name)
    for name, t in (("state_slots", state_slots), ("record_rows", record_rows),
                    ("pending", pending)):
        _expect(t, torch.int32, name)
    rq = corr.shape[2] if rq is None else rq
    B = state_slots.shape[0]
    H = A_log.shape[0]
    nbytes = workspace.numel() * workspace.element_size()
    rc = load().kda_layer_step(
        _ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state), conv_state.stride(0),
        _ptr(f_a), _ptr(f_b), _ptr(raw_beta), _ptr(A_log), _ptr(dt_bias), lower_bound, q_scale,
        _ptr(state_pool), state_pool.stride(0), state_pool.shape[0], _ptr(state_slots),
        _ptr(record_rows), _ptr(pending), _ptr(corr), _ptr(key_gate), corr.stride(0),
        key_gate.stride(0), corr.shape[0], rq, _ptr(gate), _ptr(norm_weight), eps, _ptr(out),
        _ptr(workspace), nbytes, B, H, Q, null_slot, _ptr(status), _stream(stream))
    return _check("kda_layer_step", rc, raise_on_error)


def kda_layer_step_noalloc(x, conv_weight, conv_bias, conv_state, f_a, f_b, raw_beta, A_log,
                           dt_bias, state_pool, state_slots, record_rows, pending, corr,
                           key_gate, gate, norm_weight, out, *, Q, lower_bound, q_scale, eps,
                           rq=None, null_slot=0, status=None, stream=None,
                           raise_on_error=True):
    """kda_layer_step without a workspace, for callers that cannot allocate
    device memory on the decode path: the step's operands go to the
    library's own fixed array (KDA_LAYER_STEP_NOALLOC_MAX_BYTES per GPU), so
    nothing is allocated.  Calls larger than that raise KDA_ERR_SCRATCH;
    calls that overlap on the GPU share the array and must be ordered."""
    import torch
    for name, t in (("x", x), ("conv_weight", conv_weight), ("conv_bias", conv_bias),
                    ("conv_state", conv_state), ("f_a", f_a), ("f_b", f_b),
                    ("raw_beta", raw_beta), ("key_gate", key_gate), ("gate", gate),
                    ("out", out)):
        _expect(t, torch.bfloat16, name)
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias), ("state_pool", state_pool),
                    ("corr", corr), ("norm_weight", norm_weight)):
        _expect(t, torch.float32, name)
    for name, t in (("state_slots", state_slots), ("record_rows", record_rows),
                    ("pending", pending)):
        _expect(t, torch.int32, name)
    rq = corr.shape[2] if rq is None else rq
    B = state_slots.shape[0]
    H = A_log.shape[0]
    rc = load().kda_layer_step_noalloc(
        _ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state), conv_state.stride(0),
        _ptr(f_a), _ptr(f_b), _ptr(raw_beta), _ptr(A_log), _ptr(dt_bias), lower_bound, q_scale,
        _ptr(state_pool), state_pool.stride(0), state_pool.shape[0], _ptr(state_slots),
        _ptr(record_rows), _ptr(pending), _ptr(corr), _ptr(key_gate), corr.stride(0),
        key_gate.stride(0), corr.shape[0], rq, _ptr(gate), _ptr(norm_weight), eps, _ptr(out),
        B, H, Q, null_slot, _ptr(status), _stream(stream))
    return _check("kda_layer_step_noalloc", rc, raise_on_error)


# ---------------------------------------------------------------------------
# prompts and plain decoding
# ---------------------------------------------------------------------------

def _expect_tensors(device, *specs):
    """The prompt operators' tensors, (name, tensor or None, type, shape) each:
    their types, shapes and layouts (contiguous), and that all are on
    `device`, a GPU."""
    index = device.index
    for name, t, dtype, shape in specs:
        if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                         and t.get_device() == index):
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if device.type == "cuda":
            raise ValueError(f"{name} must be on {device}, got {t.device}")
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, got {device}")


def _expect_rows(device, name, t, dtype, inner):
    """A pool or table: rows of shape `inner` (None: any size), each
    contiguous, any stride from one to the next."""
    if t.dtype is dtype and t.is_contiguous() and t.get_device() == device.index:
        # (the usual pool: what follows takes 3 us)
        n = t.shape[1:]
        if n == inner or (inner[-1] is None and len(n) == len(inner) and n[:-1] == inner[:-1]):
            return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(inner) + 1 or any(w is not None and w != n
                                        for w, n in zip(inner, t.shape[1:])):
        raise ValueError(f"{name} must have shape {('any', *inner)}, got {tuple(t.shape)}")
    want = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != want:
            raise ValueError(f"{name} must be contiguous but for the stride of its rows")
        want *= n
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _call_on(device, stream, call):
    """call(stream's address) with the device of the call's tensors the
    current one; the device's current stream where none is given."""
    import torch
    if stream is None:
        # (torch.cuda.current_stream builds a Stream object: 3 us of a call
        # that takes 13)
        address = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        address = stream if isinstance(stream, int) else stream.cuda_stream
    if device.index == torch._C._cuda_getDevice():
        return call(address)
    with torch.cuda.device(device):
        return call(address)


def _address(t):
    return None if t is None else t.data_ptr()


def _row_stride(t, minimum):
    """Elements from one slot to the next (the pool of a single slot may have
    any stride there: nothing uses it)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), minimum)


def kda_slot_plan(computed_lens, new_lens, block_table, free_slots, free_head, free_next,
                  query_start_loc, sources, destinations, boundaries, boundary_lens, *,
                  block_size, null_slot=0, status=None, stream=None, raise_on_error=True):
    """Packed offsets, block table entries and slot maps from the requests'
    lengths (the rules are in include/kda_recoverssm.h).  In: computed_lens,
    new_lens [B], block_table [B, max_blocks] (rows of any stride; extended in
    place), free_slots [n], free_head [1].  Out: free_next [1] (may be
    free_head), query_start_loc [B + 1], sources, destinations, boundaries,
    boundary_lens [B].  All int32."""
    import torch
    i32, dev = torch.int32, computed_lens.device
    B = computed_lens.shape[0]
    one, per = (1,), (B,)
    _expect_tensors(dev, ("computed_lens", computed_lens, i32, per), ("new_lens", new_lens, i32, per),
                    ("free_slots", free_slots, i32, (free_slots.numel(),)),
                    ("free_head", free_head, i32, one), ("free_next", free_next, i32, one),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("sources", sources, i32, per), ("destinations", destinations, i32, per),
                    ("boundaries", boundaries, i32, per),
                    ("boundary_lens", boundary_lens, i32, per), ("status", status, i32, one))
    _expect_rows(dev, "block_table", block_table, i32, (None,))
    if block_table.shape[0] != B:
        raise ValueError(f"block_table must have {B} rows, got {block_table.shape[0]}")
    rc = _call_on(dev, stream, lambda st: load().kda_slot_plan(
            computed_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
            _row_stride(block_table, block_table.shape[1]), block_table.shape[1],
            free_slots.data_ptr(), free_slots.shape[0], free_head.data_ptr(),
            free_next.data_ptr(), query_start_loc.data_ptr(), sources.data_ptr(),
            destinations.data_ptr(), boundaries.data_ptr(), boundary_lens.data_ptr(), B,
            block_size, null_slot, _address(status), st))
    return _check("kda_slot_plan", rc, raise_on_error)


def kda_prefill_conv(x, conv_weight, conv_bias, conv_state, sources, destinations,
                     query_start_loc, q, k, v, *, Q, boundaries=None, boundary_lens=None,
                     null_slot=0, status=None, stream=None, raise_on_error=True):
    """The layer's convolution + SiLU over ragged prompts: x [T, 3*H*128] to
    q, k, v [T, H, 128], the windows of conv_state [slots, 3*H*128, width]
    read at ``sources`` and left at ``destinations`` (and after boundary_lens
    tokens at ``boundaries``).  Q: at least the longest window;
    query_start_loc None: windows of Q tokens."""
    import torch
    bf, i32, dev = torch.bfloat16, torch.int32, x.device
    T, H, _ = q.shape
    D, B = H * 128, sources.shape[0]
    per, heads = (B,), (T, H, 128)
    _expect_tensors(dev, ("x", x, bf, (T, 3 * D)), ("conv_weight", conv_weight, bf, (3, 4, D)),
                    ("conv_bias", conv_bias, bf, (3 * D,)), ("q", q, bf, heads),
                    ("k", k, bf, heads), ("v", v, bf, heads), ("sources", sources, i32, per),
                    ("destinations", destinations, i32, per),
                    ("boundaries", boundaries, i32, per),
                    ("boundary_lens", boundary_lens, i32, per),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    _expect_rows(dev, "conv_state", conv_state, bf, (3 * D, None))
    rc = _call_on(dev, stream, lambda st: load().kda_prefill_conv(
            x.data_ptr(), conv_weight.data_ptr(), _address(conv_bias), conv_state.data_ptr(),
            _row_stride(conv_state, 3 * D * conv_state.shape[2]), conv_state.shape[2],
            conv_state.shape[0], sources.data_ptr(), destinations.data_ptr(),
            _address(boundaries), _address(boundary_lens), _address(query_start_loc), T,
            q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, Q, null_slot, _address(status), st))
    return _check("kda_prefill_conv", rc, raise_on_error)


def _rule_args(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, sources, destinations,
               query_start_loc, out, boundaries, boundary_lens, status):
    """Checks of kda_prefill's and kda_recurrent's tensors; the pool's type
    and stride."""
    import torch
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, q.device
    T, H, _ = q.shape
    B = sources.shape[0]
    per, heads = (B,), (T, H, 128)
    if state_pool.dtype != f32 and state_pool.dtype != bf:
        raise TypeError("state_pool must be float32 or bfloat16")
    _expect_tensors(dev, ("q", q, bf, heads), ("k", k, bf, heads), ("v", v, bf, heads),
                    ("raw_g", raw_g, bf, heads), ("out", out, bf, heads),
                    ("raw_beta", raw_beta, bf, (T, H)), ("A_log", A_log, f32, (H,)),
                    ("dt_bias", dt_bias, f32, (H, 128)), ("sources", sources, i32, per),
                    ("destinations", destinations, i32, per),
                    ("boundaries", boundaries, i32, per),
                    ("boundary_lens", boundary_lens, i32, per),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    _expect_rows(dev, "state_pool", state_pool, state_pool.dtype, (H, 128, 128))
    return (KDA_STATE_F32 if state_pool.dtype == f32 else KDA_STATE_BF16,
            _row_stride(state_pool, H * 128 * 128))


def kda_prefill_workspace_bytes(n_tokens, B, H, Q=None, boundaries=True):
    """Bytes of workspace kda_prefill needs for n_tokens packed tokens of B
    requests; with ``Q`` (and ``boundaries`` False where there are none) for
    windows of up to Q tokens, which may be far less (0 for Q <= 40)."""
    if Q is None:
        return load().kda_prefill_workspace_bytes(n_tokens, B, H)
    return load().kda_prefill_workspace_bytes_for(n_tokens, B, H, Q, int(boundaries))


def kda_prefill(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, sources, destinations,
                query_start_loc, out, *, Q, lower_bound, q_scale, boundaries=None,
                boundary_lens=None, workspace=None, null_slot=0, status=None, stream=None,
                raise_on_error=True):
    """The gated delta rule over ragged prompts, in chunks: q, k, v, raw_g,
    out [T, H, 128], raw_beta [T, H] BF16; the states of state_pool
    [slots, H, 128, 128] (float32 or bfloat16) read at ``sources`` (a fresh
    start at null_slot) and left at ``destinations`` (and after boundary_lens
    tokens at ``boundaries``).  Q: at least the longest window;
    query_start_loc None: windows of Q tokens.  ``workspace``: a device
    tensor of kda_prefill_workspace_bytes(T, B, H, Q, boundaries is not None)
    bytes that nothing else uses meanwhile; None takes it from torch's
    allocator for this call."""
    import torch
    dtype, slot_stride = _rule_args(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, sources,
                                    destinations, query_start_loc, out, boundaries,
                                    boundary_lens, status)
    T, H, _ = q.shape
    B = sources.shape[0]
    if workspace is not None and (not workspace.is_contiguous() or workspace.device != q.device):
        raise ValueError("workspace must be a contiguous tensor on the operands' device")
    lib = load()

    def call(st):
        ws = workspace
        if ws is None:
            need = max(0, lib.kda_prefill_workspace_bytes_for(T, B, H, Q, boundaries is not None))
            if stream is None:
                ws = torch.empty(need, dtype=torch.uint8, device=q.device)
            else:
                # of the call's own stream: the allocator hands it on there (the
                # default one has no address: ExternalStream(0) is another)
                own = (torch.cuda.ExternalStream(st) if st
                       else torch.cuda.default_stream(q.device))
                with torch.cuda.stream(own):
                    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        nbytes = ws.numel() * ws.element_size()
        return lib.kda_prefill(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_g.data_ptr(), raw_beta.data_ptr(),
            A_log.data_ptr(), dt_bias.data_ptr(), lower_bound, q_scale, state_pool.data_ptr(),
            dtype, slot_stride, state_pool.shape[0], sources.data_ptr(), destinations.data_ptr(),
            _address(boundaries), _address(boundary_lens), _address(query_start_loc), T,
            out.data_ptr(), ws.data_ptr() if nbytes else None, nbytes, B, H, Q, null_slot,
            _address(status), st)

    rc = _call_on(q.device, stream, call)
    return _check("kda_prefill", rc, raise_on_error)


def kda_recurrent(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, sources, destinations,
                  out, *, Q, lower_bound, q_scale, query_start_loc=None, boundaries=None,
                  boundary_lens=None, null_slot=0, status=None, stream=None,
                  raise_on_error=True):
    """The gated delta rule token by token, for decoding: arguments as
    kda_prefill's; query_start_loc None: windows of Q tokens."""
    dtype, slot_stride = _rule_args(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, sources,
                                    destinations, query_start_loc, out, boundaries,
                                    boundary_lens, status)
    T, H, _ = q.shape
    rc = _call_on(q.device, stream, lambda st: load().kda_recurrent(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_g.data_ptr(), raw_beta.data_ptr(),
            A_log.data_ptr(), dt_bias.data_ptr(), lower_bound, q_scale, state_pool.data_ptr(),
            dtype, slot_stride, state_pool.shape[0], sources.data_ptr(), destinations.data_ptr(),
            _address(boundaries), _address(boundary_lens), _address(query_start_loc), T,
            out.data_ptr(), sources.shape[0], H, Q, null_slot, _address(status), st))
    return _check("kda_recurrent", rc, raise_on_error)


# ---------------------------------------------------------------------------
# trees of drafted tokens
# ---------------------------------------------------------------------------

def kda_tree_conv(x, conv_weight, conv_bias, conv_state, state_slots, parents, q, k, v, *, Q,
                  record_rows=None, pending=None, query_start_loc=None, null_slot=0, status=None,
                  stream=None, raise_on_error=True):
    """The layer's convolution + SiLU over trees of drafted tokens: x
    [T, 3*H*128] to q, k, v [T, H, 128], each node behind its own ancestors
    (``parents`` [T], within the request, -1 above a root; None: chains) and
    the windows of conv_state [slots, 3*H*128, width] (read only), whose live
    entries the pending counts tell.  Q: at least the largest tree;
    query_start_loc None: trees of Q nodes."""
    import torch
    bf, i32, dev = torch.bfloat16, torch.int32, x.device
    T, H, _ = q.shape
    D, B = H * 128, state_slots.shape[0]
    per, heads = (B,), (T, H, 128)
    _expect_tensors(dev, ("x", x, bf, (T, 3 * D)), ("conv_weight", conv_weight, bf, (3, 4, D)),
                    ("conv_bias", conv_bias, bf, (3 * D,)), ("q", q, bf, heads),
                    ("k", k, bf, heads), ("v", v, bf, heads),
                    ("state_slots", state_slots, i32, per), ("parents", parents, i32, (T,)),
                    ("record_rows", record_rows, i32, per),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    n_rows = 0
    if pending is not None:
        n_rows = pending.shape[0]
        _expect_tensors(dev, ("pending", pending, i32, (n_rows,)))
    _expect_rows(dev, "conv_state", conv_state, bf, (3 * D, None))
    rc = _call_on(dev, stream, lambda st: load().kda_tree_conv(
            x.data_ptr(), conv_weight.data_ptr(), _address(conv_bias), conv_state.data_ptr(),
            _row_stride(conv_state, 3 * D * conv_state.shape[2]), conv_state.shape[2],
            conv_state.shape[0], state_slots.data_ptr(), _address(record_rows),
            _address(pending), n_rows, _address(parents), _address(query_start_loc), T,
            q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, Q, null_slot, _address(status), st))
    return _check("kda_tree_conv", rc, raise_on_error)


def _expect_records(dev, corr, key_gate, H):
    """Record rows: corr [rows, H, rq, 128], key_gate [rows, H, rq, 256]; the
    rows' strides."""
    import torch
    rq = corr.shape[2] if corr.dim() == 4 else 0
    _expect_rows(dev, "corr", corr, torch.float32, (H, rq, 128))
    _expect_rows(dev, "key_gate", key_gate, torch.bfloat16, (H, rq, 256))
    if key_gate.shape[0] != corr.shape[0]:
        raise ValueError(f"key_gate must have {corr.shape[0]} rows, got {key_gate.shape[0]}")
    return _row_stride(corr, H * rq * 128), _row_stride(key_gate, H * rq * 256)


def kda_tree_verify(q, k, v, raw_g, raw_beta, A_log, dt_bias, state_pool, state_slots, parents,
                    node_corr, out, *, Q, lower_bound, q_scale, record_rows=None, pending=None,
                    corr=None, key_gate=None, query_start_loc=None, null_slot=0, status=None,
                    stream=None, raise_on_error=True):
    """The delta rule over trees of drafted tokens: q, k, v, raw_g, out
    [T, H, 128], raw_beta [T, H] BF16, every node from the state behind its
    ancestors (``parents`` as in kda_tree_conv), starting from the request's
    page of state_pool [slots, H, 128, 128]; node_corr [T, H, 128] FP32 takes
    the nodes' corrections.  With ``pending`` [rows], corr and key_gate (a
    float32 pool) the pending replay of a request's record row is folded into
    its page first; without, the pool (float32 or bfloat16) is only read."""
    import torch
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, q.device
    T, H, _ = q.shape
    B = state_slots.shape[0]
    per, heads = (B,), (T, H, 128)
    dtype = state_pool.dtype
    if dtype != f32 and dtype != bf:
        raise TypeError("state_pool must be float32 or bfloat16")
    _expect_tensors(dev, ("q", q, bf, heads), ("k", k, bf, heads), ("v", v, bf, heads),
                    ("raw_g", raw_g, bf, heads), ("out", out, bf, heads),
                    ("node_corr", node_corr, f32, heads), ("raw_beta", raw_beta, bf, (T, H)),
                    ("A_log", A_log, f32, (H,)), ("dt_bias", dt_bias, f32, (H, 128)),
                    ("state_slots", state_slots, i32, per), ("parents", parents, i32, (T,)),
                    ("record_rows", record_rows, i32, per),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    _expect_rows(dev, "state_pool", state_pool, dtype, (H, 128, 128))
    if (pending is None) != (corr is None) or (corr is None) != (key_gate is None):
        raise ValueError("pending, corr and key_gate come together")
    n_rows = rq = corr_stride = kg_stride = 0
    if pending is not None:
        corr_stride, kg_stride = _expect_records(dev, corr, key_gate, H)
        n_rows, rq = corr.shape[0], corr.shape[2]
        _expect_tensors(dev, ("pending", pending, i32, (n_rows,)))
    rc = _call_on(dev, stream, lambda st: load().kda_tree_verify(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_g.data_ptr(), raw_beta.data_ptr(),
            A_log.data_ptr(), dt_bias.data_ptr(), lower_bound, q_scale, state_pool.data_ptr(),
            KDA_STATE_F32 if dtype == f32 else KDA_STATE_BF16,
            _row_stride(state_pool, H * 128 * 128), state_pool.shape[0], state_slots.data_ptr(),
            _address(parents), _address(query_start_loc), T, _address(record_rows),
            _address(pending), _address(corr), _address(key_gate), corr_stride, kg_stride, n_rows,
            rq, node_corr.data_ptr(), out.data_ptr(), B, H, Q, null_slot, _address(status), st))
    return _check("kda_tree_verify", rc, raise_on_error)


def kda_draft_accept(target_probs, tokens, accept_uniforms, sample_uniforms, accepted, path,
                     next_tokens, *, Q, draft_probs=None, parents=None, state_slots=None,
                     query_start_loc=None, null_slot=0, status=None, stream=None,
                     raise_on_error=True):
    """Drafted ``tokens`` [T] against the target's next-token probabilities
    target_probs [T, vocab] (float32 or bfloat16, rows of any stride, each
    summing to one), from uniform numbers accept_uniforms [T] (one a node, for
    its children) and sample_uniforms [B] in [0, 1).  Chains with draft_probs
    [T, vocab] (what each token was drawn from; rows as target_probs'), or
    trees (``parents``) and chains of drafts that were taken for sure.  Out, int32: accepted [B] (tokens of the path,
    the root among them), path [B, 8] (its nodes, -1 behind), next_tokens [B]
    (drawn from the target after the path).  The rules are in
    include/kda_recoverssm.h."""
    import torch
    f32, i32, dev = torch.float32, torch.int32, target_probs.device
    if target_probs.dim() != 2:
        raise ValueError("target_probs must have shape (tokens, vocab)")
    T, V = target_probs.shape
    B = sample_uniforms.shape[0]
    dtype, per = target_probs.dtype, (B,)
    if dtype != f32 and dtype != torch.bfloat16:
        raise TypeError("target_probs must be float32 or bfloat16")
    if draft_probs is not None and parents is not None:
        raise ValueError("draft_probs go with chains: parents must be None")
    _expect_tensors(dev, ("tokens", tokens, i32, (T,)),
                    ("accept_uniforms", accept_uniforms, f32, (T,)),
                    ("sample_uniforms", sample_uniforms, f32, per),
                    ("accepted", accepted, i32, per), ("path", path, i32, (B, KDA_TREE_MAX_DEPTH)),
                    ("next_tokens", next_tokens, i32, per), ("parents", parents, i32, (T,)),
                    ("state_slots", state_slots, i32, per),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    _expect_rows(dev, "target_probs", target_probs, dtype, (V,))
    draft_stride = 0
    if draft_probs is not None:
        _expect_rows(dev, "draft_probs", draft_probs, dtype, (V,))
        if draft_probs.shape[0] != T:
            raise ValueError(f"draft_probs must have {T} rows, got {draft_probs.shape[0]}")
        draft_stride = _row_stride(draft_probs, V)
    rc = _call_on(dev, stream, lambda st: load().kda_draft_accept(
            target_probs.data_ptr(), _address(draft_probs),
            KDA_PROBS_F32 if dtype == f32 else KDA_PROBS_BF16, _row_stride(target_probs, V),
            draft_stride, V, tokens.data_ptr(), _address(parents), accept_uniforms.data_ptr(),
            sample_uniforms.data_ptr(), _address(state_slots), _address(query_start_loc), T,
            accepted.data_ptr(), path.data_ptr(), next_tokens.data_ptr(), B, Q, null_slot,
            _address(status), st))
    return _check("kda_draft_accept", rc, raise_on_error)


def kda_tree_settle(state_slots, record_rows, rows, *, Q, n_tokens, n_slots, n_rows, path=None,
                    accepted=None, most=KDA_TREE_MAX_DEPTH, parents=None, served=None,
                    query_start_loc=None, folded=False, null_slot=0, status=None, stream=None,
                    raise_on_error=True):
    """Between kda_draft_accept and kda_tree_select: record_rows [B] to ``rows``
    [B] (int32; they may be one), -1 for the requests that kda_tree_verify
    reported, whose replays are still pending (bad windows, slots, rows and,
    with ``parents`` [n_tokens], trees), and 0 to their ``accepted``.  Select and
    kda_defer_commit, called with ``rows``, leave those as they were.  With
    ``path`` [B, 8], 0 too to the counts above ``most`` (what records, rq, and
    windows, width - 2, hold) and to those of paths outside their windows.
    ``served``: the rows of an earlier call of the same step, beside the verify
    (``parents`` are not needed then).  ``folded``: the replays were folded in
    otherwise, and such a request keeps its row.  n_slots, n_rows: of the state
    pool and of the records."""
    import torch
    i32, dev, B = torch.int32, state_slots.device, state_slots.shape[0]
    per = (B,)
    _expect_tensors(dev, ("state_slots", state_slots, i32, per),
                    ("record_rows", record_rows, i32, per), ("rows", rows, i32, per),
                    ("served", served, i32, per), ("accepted", accepted, i32, per),
                    ("path", path, i32, (B, KDA_TREE_MAX_DEPTH)),
                    ("parents", parents, i32, (n_tokens,)),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    rc = _call_on(dev, stream, lambda st: load().kda_tree_settle(
            _address(path), _address(accepted), most, state_slots.data_ptr(), n_slots,
            _address(record_rows), _address(served), n_rows, _address(parents),
            _address(query_start_loc), n_tokens, int(folded), rows.data_ptr(), B, Q, null_slot,
            _address(status), st))
    return _check("kda_tree_settle", rc, raise_on_error)


def kda_tree_select(path, accepted, k, raw_g, node_corr, state_slots, record_rows, corr, key_gate,
                    *, Q, x=None, conv_state=None, pending=None, eager=None, query_start_loc=None,
                    null_slot=0, status=None, stream=None, raise_on_error=True):
    """The accepted paths (``path`` [B, 8] and ``accepted`` [B], as
    kda_draft_accept leaves them) to the front of the requests' records: the
    nodes' corrections, keys and raw gates to corr [rows, H, rq, 128] and
    key_gate [rows, H, rq, 256]; with x [T, 3*H*128] and conv_state
    [slots, 3*H*128, width] (and ``pending`` as kda_tree_conv had it), the
    path's inputs to the convolution windows as well.  kda_defer_commit then
    makes the path the pending replay; rows that it will leave without one,
    being committed at once, are marked in ``eager`` (uint8 [B])."""
    import torch
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, k.device
    T, H, _ = k.shape
    D, B = H * 128, state_slots.shape[0]
    per, heads = (B,), (T, H, 128)
    if (x is None) != (conv_state is None):
        raise ValueError("x and conv_state come together")
    _expect_tensors(dev, ("path", path, i32, (B, KDA_TREE_MAX_DEPTH)),
                    ("accepted", accepted, i32, per), ("eager", eager, torch.uint8, per),
                    ("k", k, bf, heads),
                    ("raw_g", raw_g, bf, heads), ("node_corr", node_corr, f32, heads),
                    ("state_slots", state_slots, i32, per),
                    ("record_rows", record_rows, i32, per), ("x", x, bf, (T, 3 * D)),
                    ("query_start_loc", query_start_loc, i32, (B + 1,)),
                    ("status", status, i32, (1,)))
    corr_stride, kg_stride = _expect_records(dev, corr, key_gate, H)
    n_rows = corr.shape[0]
    _expect_tensors(dev, ("pending", pending, i32, (n_rows,)))
    n_slots, slot_stride, width = 0x7fffffff, 0, 0
    if conv_state is not None:
        _expect_rows(dev, "conv_state", conv_state, bf, (3 * D, None))
        n_slots, width = conv_state.shape[0], conv_state.shape[2]
        slot_stride = _row_stride(conv_state, 3 * D * width)
    rc = _call_on(dev, stream, lambda st: load().kda_tree_select(
            path.data_ptr(), accepted.data_ptr(), _address(eager), k.data_ptr(),
            raw_g.data_ptr(), node_corr.data_ptr(), state_slots.data_ptr(),
            _address(record_rows), _address(pending), corr.data_ptr(), key_gate.data_ptr(), corr_stride, kg_stride,
            n_rows, corr.shape[2], _address(x), _address(conv_state), slot_stride, width, n_slots,
            _address(query_start_loc), T, B, H, Q, null_slot, _address(status), st))
    return _check("kda_tree_select", rc, raise_on_error)
