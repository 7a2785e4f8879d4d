"""The deferred RecoverSSM of one layer across speculative decode steps.

A runner verifies a window per step, samples, and then must fold the
accepted tokens into each request's checkpoint.  The deferred form (page
"...cutedsl.kda.fused", module docstring; page "...recoverssm.kernels",
``_defer_commit_kernel`` and ``_prepare_flush_plan_kernel``) does not commit
after sampling: the accepted count becomes the request's pending replay, and
the next verify replays it in the same pass over the state.  This class only
sequences the library's entry points in that order; every step runs in the
library's kernels (and what a prompt does to the pending counts in a few of
torch's), on the given stream, with no host synchronisation, so a sequence of
steps can be captured in a CUDA graph.

* ``prefill``: prompts are taken into their requests' checkpoints before the
  first step (in one call or in parts);
* ``verify``: the fused replay + verify, or the stock verify (no replay) when
  the pending replays were just folded in by ``flush``;
* ``accept``: the accepted counts become the pending replays (defer); rows
  marked eager are committed at once from the records this step wrote;
* ``verify_tree`` and ``accept_tree``: the same two for a tree of drafted
  tokens in place of a chain (any step may be either); kda_draft_accept makes
  the accepted path from the target's probabilities between them;
* ``flush``: every pending replay is folded into its checkpoint in place
  (flush plan + commit); the next ``verify`` is then the stock one, because
  the plan leaves the pending counts as they are.
"""
from __future__ import annotations

from ._lib import (KDA_STATE_F32, kda_commit, kda_defer_commit, kda_flush_plan,
                   kda_prefill, kda_replay_verify, kda_tree_select, kda_tree_settle,
                   kda_tree_verify, kda_verify, layer_tables)


class DeferredRecoverSSM:
    """One layer's checkpoints, records and pending counts (device tensors,
    owned by the caller): state_pool FP32 [slots, H, 128, 128]; state_slots
    and record_rows int32 [B] (every live request needs a record row to be
    deferred); pending int32 [rows]; corr FP32 [rows, H, RQ, 128]; key_gate
    BF16 [rows, H, RQ, 256]; A_log FP32 [H]; dt_bias FP32 [H, 128]."""

    def __init__(self, state_pool, state_slots, record_rows, pending, corr, key_gate, A_log,
                 dt_bias, *, Q, lower_bound, q_scale, null_slot=0, split=0, status=None,
                 stream=None):
        import torch
        self.state_pool, self.state_slots, self.record_rows = state_pool, state_slots, record_rows
        self.pending, self.corr, self.key_gate = pending, corr, key_gate
        self.A_log, self.dt_bias = A_log, dt_bias
        self.Q, self.lower_bound, self.q_scale = Q, lower_bound, q_scale
        self.null_slot, self.split, self.status, self.stream = null_slot, split, status, stream
        self.B, self.H = state_slots.shape[0], A_log.shape[0]
        dev = state_pool.device
        # the commit's one-layer address tables and the flush plan's outputs,
        # made once so that no step allocates or copies from the host
        self._tables = layer_tables([state_pool], [corr], [key_gate], dev)
        self._plan = {name: torch.zeros(self.B, dtype=torch.int32, device=dev)
                      for name in ("commit_lens", "final_slots", "boundary_slots",
                                   "boundary_lens")}
        self._fresh = torch.full((self.B,), self.null_slot, dtype=torch.int32, device=dev)
        self._none = torch.zeros(self.B, dtype=torch.int32, device=dev)
        self._no_row = torch.tensor(-1, dtype=torch.int32, device=dev)
        # the record rows of the requests that verify_tree served, for accept_tree
        self._rows = torch.full((self.B,), -1, dtype=torch.int32, device=dev)
        self._settled = False  # they are this step's
        self.flushed = False

    def _commit(self, commit_lens, destinations, boundaries=None, boundary_lens=None):
        kda_commit(*self._tables, self.A_log, self.dt_bias, self.state_slots, commit_lens,
                   destinations, state_dtype=KDA_STATE_F32, lower_bound=self.lower_bound,
                   L=1, H=self.H, B=self.B, Q=self.corr.shape[2],
                   n_slots=self.state_pool.shape[0], n_rows=self.corr.shape[0],
                   boundaries=boundaries, boundary_lens=boundary_lens,
                   record_rows=self.record_rows, null_slot=self.null_slot, status=self.status,
                   stream=self.stream)

    def _on_stream(self):
        """torch's operations on the loop's stream."""
        import contextlib
        import torch
        if self.stream is None:
            return contextlib.nullcontext()
        stream = self.stream
        if isinstance(stream, int):
            dev = self.state_pool.device
            stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                      else torch.cuda.default_stream(dev))
        return torch.cuda.stream(stream)

    def prefill(self, q, k, v, raw_g, raw_beta, query_start_loc, out, *, Q, sources=None,
                boundaries=None, boundary_lens=None, workspace=None):
        """Prompts (q, k, v, raw_g BF16 [T, H, 128], raw_beta BF16 [T, H],
        packed by query_start_loc [B + 1], windows of up to Q tokens) through
        the rule, outputs to out: each request's state is left in its own
        slot, from which ``verify`` goes on, and after boundary_lens tokens
        in ``boundaries`` (int32 [B] each).  A request with an empty window is
        left alone, its pending replay too.  ``sources`` (int32 [B]): the slots
        to go on from, the null slot for a fresh start (None: all fresh;
        ``state_slots`` for a prompt's later parts, or for what follows decoded
        tokens).  A request that goes on from its own slot has its pending
        replay folded in first; whatever was pending in the record row of a
        request that gets a prompt is gone afterwards."""
        import torch
        common = dict(null_slot=self.null_slot, status=self.status, stream=self.stream)
        with self._on_stream():
            prompted = query_start_loc[1:] > query_start_loc[:-1]
            rows = torch.where(prompted, self.record_rows, self._no_row)
            resumed = None
            if sources is not None and not self.flushed:
                resumed = torch.where(sources == self.state_slots, rows, self._no_row)
        if sources is None:
            sources = self._fresh
        if resumed is not None:
            p = self._plan
            kda_flush_plan(self.state_slots, resumed, self.pending, p["commit_lens"],
                           p["final_slots"], p["boundary_slots"], p["boundary_lens"],
                           Q=self.corr.shape[2], **common)
            self._commit(p["commit_lens"], p["final_slots"])
        kda_prefill(q, k, v, raw_g, raw_beta, self.A_log, self.dt_bias, self.state_pool, sources,
                    self.state_slots, query_start_loc, out, Q=Q, lower_bound=self.lower_bound,
                    q_scale=self.q_scale, boundaries=boundaries, boundary_lens=boundary_lens,
                    workspace=workspace, **common)
        # (no accepted token is pending in those rows: the counts stay zero)
        kda_defer_commit(self.state_slots, self._none, rows, self.pending, **common)

    def verify(self, q, k, v, raw_g, raw_beta, out, query_start_loc=None):
        """Verify this step's window (q, k, v, raw_g BF16 [T, H, 128],
        raw_beta BF16 [T, H]; T = B*Q, or packed windows of q_b <= Q tokens
        given by query_start_loc [B + 1]) into out BF16 [T, H, 128], writing
        the window's records.  With windows of different lengths the counts
        passed to ``accept`` must not exceed each request's q_b."""
        common = dict(Q=self.Q, lower_bound=self.lower_bound, q_scale=self.q_scale,
                      null_slot=self.null_slot, status=self.status, stream=self.stream,
                      query_start_loc=query_start_loc)
        if self.flushed:
            kda_verify(q, k, v, raw_g, raw_beta, self.A_log, self.dt_bias, self.state_pool,
                       self.state_slots, self.corr, self.key_gate, out,
                       record_rows=self.record_rows, **common)
        else:
            kda_replay_verify(q, k, v, raw_g, raw_beta, self.A_log, self.dt_bias,
                              self.state_pool, self.state_slots, self.record_rows,
                              self.pending, self.corr, self.key_gate, out, split=self.split,
                              **common)

    def accept(self, accepted, eager=None):
        """After sampling: ``accepted`` (int32 [B], overwritten: it ends as
        the commit plan, non-zero only on eager rows) becomes each request's
        pending replay; ``eager`` (uint8 [B] or None) marks rows committed
        now instead."""
        self._accept(accepted, self.record_rows, eager)

    def _accept(self, accepted, rows, eager):
        kda_defer_commit(self.state_slots, accepted, rows, self.pending, eager=eager,
                         null_slot=self.null_slot, status=self.status, stream=self.stream)
        if eager is not None:
            self._commit(accepted, self.state_slots)
        self.flushed = self._settled = False

    def verify_tree(self, q, k, v, raw_g, raw_beta, parents, node_corr, out, *, Q,
                    query_start_loc=None):
        """Verify this step's trees of up to Q drafted tokens (q, k, v, raw_g,
        out BF16 [T, H, 128], raw_beta BF16 [T, H], parents int32 [T]; T =
        B*Q, or packed by query_start_loc [B + 1]), every node from the state
        behind its ancestors.  node_corr FP32 [T, H, 128] takes the nodes'
        corrections, for ``accept_tree``; the records are not written.  No path
        is longer than what the records and convolution windows hold.  A
        request that is reported (a bad tree or window) keeps its pending
        replay, ``accept_tree`` included."""
        replay = {} if self.flushed else dict(pending=self.pending, corr=self.corr,
                                              key_gate=self.key_gate)
        kda_tree_verify(q, k, v, raw_g, raw_beta, self.A_log, self.dt_bias, self.state_pool,
                        self.state_slots, parents, node_corr, out, Q=Q,
                        lower_bound=self.lower_bound, q_scale=self.q_scale,
                        record_rows=self.record_rows, query_start_loc=query_start_loc,
                        null_slot=self.null_slot, status=self.status, stream=self.stream, **replay)
        if not self.flushed:
            self._settle(q.shape[0], parents=parents, Q=Q, query_start_loc=query_start_loc)
            self._settled = True

    def _settle(self, n_tokens, **kw):
        """The record rows of the requests that go on, to self._rows."""
        kda_tree_settle(self.state_slots, self.record_rows, self._rows, n_tokens=n_tokens,
                        n_slots=self.state_pool.shape[0], n_rows=self.corr.shape[0],
                        null_slot=self.null_slot, status=self.status, stream=self.stream, **kw)

    def accept_tree(self, path, accepted, k, raw_g, node_corr, *, Q, query_start_loc=None, x=None,
                    conv_state=None, eager=None):
        """After sampling from the trees of ``verify_tree``: the accepted paths
        (path int32 [B, 8], accepted int32 [B], overwritten as in ``accept``)
        move to the front of the records, and with x and conv_state their
        inputs to the layer's convolution windows; then as ``accept``.  A
        request that ``verify_tree`` reported comes out as it went in; a path
        that the records or windows cannot hold is reported and not taken."""
        most = self.corr.shape[2]
        if conv_state is not None:
            most = max(0, min(most, conv_state.shape[2] - 2))
        # (behind a flush every replay is in its checkpoint, whatever the trees were)
        self._settle(k.shape[0], path=path, accepted=accepted, most=most, folded=self.flushed,
                     served=self._rows if self._settled else None, Q=Q,
                     query_start_loc=query_start_loc)
        kda_tree_select(path, accepted, k, raw_g, node_corr, self.state_slots, self._rows,
                        self.corr, self.key_gate, Q=Q, x=x, conv_state=conv_state,
                        pending=self.pending, eager=eager, query_start_loc=query_start_loc,
                        null_slot=self.null_slot, status=self.status, stream=self.stream)
        self._accept(accepted, self._rows, eager)

    def flush(self):
        """Fold every pending replay into its checkpoint, in place."""
        # (a tree's path may fill a record row, beyond a chain's window)
        p = self._plan
        kda_flush_plan(self.state_slots, self.record_rows, self.pending, p["commit_lens"],
                       p["final_slots"], p["boundary_slots"], p["boundary_lens"],
                       Q=self.corr.shape[2], null_slot=self.null_slot, status=self.status,
                       stream=self.stream)
        self._commit(p["commit_lens"], p["final_slots"], p["boundary_slots"],
                     p["boundary_lens"])
        self.flushed = True
