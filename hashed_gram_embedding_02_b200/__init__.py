"""Engram conditional-memory forward path for NVIDIA B200 (sm_100a).

The compute lives in ``libengram.so`` (CUDA kernels behind the C ABI declared
in ``include/engram.h``); :mod:`.binding` is its ctypes binding with the same
function names, and :class:`Engram` is a small convenience owner of a context
plus its workspace.  PyTorch is used only for device memory and streams.
"""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional

from .binding import (  # noqa: F401  (re-exported C ABI names)
    ENGRAM_BF16, ENGRAM_F32, ENGRAM_FP8, ENGRAM_ERR_CANON, ENGRAM_ERR_INDEX, ENGRAM_ERR_TIMEOUT, ENGRAM_ERR_TOKEN,
    ENGRAM_E_CUDA, ENGRAM_E_DEVICE, ENGRAM_E_HOST, ENGRAM_E_INVAL, ENGRAM_E_NOMEM, ENGRAM_E_TIMEOUT,
    ENGRAM_E_UNSUPPORTED,
    ENGRAM_INVALID_INDEX, ENGRAM_OK, EXPORTS, LIB_PATH, EngramError, engram_config, engram_conv, engram_create,
    ENGRAM_NOALLOC_SCRATCH_BYTES, engram_destroy, engram_device_status, engram_forward, engram_forward_noalloc,
    engram_forward_host, engram_gate_conv, engram_gather, engram_gather_staged, engram_hash, engram_host_dedupe,
    engram_host_fetch, engram_host_tier_create, engram_host_tier_destroy, engram_host_tier_stats,
    engram_host_workspace_bytes, engram_pack_rows, engram_debug_stall_next, engram_debug_ffn_cut, engram_host_tier_debug,
    ENGRAM_INJECT_LIST_WAIT, ENGRAM_INJECT_PACK_ABANDON, engram_host_cache_enable, engram_host_cache_reset,
    engram_host_cache_stats, engram_shard_range, engram_forward_sharded, engram_ipc_export, engram_ipc_open,
    engram_ipc_close, ENGRAM_IPC_HANDLE_BYTES, ENGRAM_MAX_SHARDS, engram_multibranch_workspace_bytes,
    engram_forward_multibranch, ENGRAM_MAX_BRANCHES, engram_table_grad_workspace_bytes, engram_table_grad,
    engram_table_sgd, engram_host_tier_map, engram_grad_route_workspace_bytes, engram_grad_route,
    engram_grad_combine_workspace_bytes, engram_grad_combine, engram_shard_sgd,
    engram_embed, engram_embed_grad_workspace_bytes, engram_embed_grad, engram_add_norm,
    engram_add_norm_grad_workspace_bytes, engram_add_norm_grad, engram_ffn_workspace_bytes, engram_ffn,
    engram_ffn_saved_bytes, engram_ffn_grad_workspace_bytes, engram_ffn_grad, ENGRAM_ACT_SILU, ENGRAM_ACT_GELU,
    engram_last_error, engram_profile_enable, engram_profile_read, engram_project, engram_remap, engram_strerror,
    engram_workspace_bytes, make_config)


class _Here:
    """No change of stream."""

    def __enter__(self):
        pass

    def __exit__(self, *_):
        pass


_HERE = _Here()


def _on_stream(stream):
    """Context in which tensors are allocated for work on `stream` (a torch
    stream, a raw handle, or None: the current stream), so that the caching
    allocator hands their memory on only in that stream's order."""
    if stream is None:
        return _HERE
    import torch
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


_ACTS = {"silu": ENGRAM_ACT_SILU, "gelu": ENGRAM_ACT_GELU}


class NormOut(NamedTuple):
    """Outputs of :meth:`Engram.add_norm`; those not asked for are None."""

    sum: Optional[object]
    y: Optional[object]
    q: Optional[object]
    q_scale: Optional[object]
    rstd: Optional[object]


class Engram:
    """Owns one engram_ctx (bound to the current device) and a workspace,
    grown on demand (or reserved up front for B sequences of L rows)."""

    def __init__(self, cfg: engram_config, B: int = 0, L: int = 0):
        import torch
        self.cfg = cfg
        self.ctx = engram_create(cfg)
        self.device = torch.device("cuda", torch.cuda.current_device())
        self.workspace = None
        self.workspace_bytes = 0
        if B and L:
            self.reserve(B, L)

    def reserve(self, B: int, L: int):
        import torch
        need = engram_workspace_bytes(self.ctx, B, L)
        if need > self.workspace_bytes:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            self.workspace_bytes = need

    def close(self):
        if self.ctx:
            engram_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def G(self) -> int:
        return (self.cfg.hidden + 127) // 128

    def forward(self, tok, P, tables, h, Wk, Wv, conv_w, y, *, t_begin: int = 0, gq=None, gk=None,
                conv_state=None, alpha_out=None, add_residual: bool = False, stream=None):
        B, T = tok.shape[0], tok.shape[1]
        self.reserve(B, T - t_begin)
        engram_forward(self.ctx, tok, B, T, tok.stride(0), t_begin, P, tables, h, Wk, Wv, gq, gk, conv_w,
                       conv_state, y, alpha_out, add_residual, self.workspace, self.workspace_bytes, stream)
        return y

    def forward_multibranch(self, tok, P, tables, h, Wk, Wv, conv_w, y, *, t_begin: int = 0, gq=None, gk=None,
                            k_scale=None, v_scale=None, conv_state=None, alpha_out=None, add_residual: bool = False,
                            stream=None):
        """M-branch forward: h [M][n][d], Wk [M][d][d_mem], gq/gk [M][d],
        conv_state [M][B][w-1][d], y [M][n][d], alpha_out [M][n]."""
        import torch
        M = h.shape[0]
        B, T = tok.shape[0], tok.shape[1]
        need = engram_multibranch_workspace_bytes(self.ctx, M, B, T - t_begin)
        if need > getattr(self, "mb_workspace_bytes", 0):
            self.mb_workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            self.mb_workspace_bytes = need
        engram_forward_multibranch(self.ctx, M, tok, B, T, tok.stride(0), t_begin, P, tables, h, Wk, Wv, gq, gk,
                                   k_scale, v_scale, conv_w, conv_state, y, alpha_out, add_residual, self.mb_workspace,
                                   self.mb_workspace_bytes, stream)
        return y

    def forward_sharded(self, tok, P, shard_ptrs, h, Wk, Wv, conv_w, y, *, t_begin: int = 0, gq=None, gk=None,
                        conv_state=None, alpha_out=None, add_residual: bool = False, stream=None):
        """The forward with the tables split into shards (device pointers
        valid on this GPU, in shard order: ShardedTables.ptrs)."""
        B, T = tok.shape[0], tok.shape[1]
        self.reserve(B, T - t_begin)
        engram_forward_sharded(self.ctx, tok, B, T, tok.stride(0), t_begin, P, shard_ptrs, h, Wk, Wv, gq, gk, conv_w,
                               conv_state, y, alpha_out, add_residual, self.workspace, self.workspace_bytes, stream)
        return y

    def forward_host(self, tok_host, P, tables, h_host, Wk, Wv, conv_w, y_host, *, t_begin: int = 0, gq=None,
                     gk=None, conv_state=None, add_residual: bool = False, chunk_rows: int = 0, stream=None):
        """The forward with tok, h and y in host memory (pinned CPU tensors
        overlap their copies with the compute); returns y_host, complete once
        the stream is synchronised."""
        import torch
        B, T = tok_host.shape[0], tok_host.shape[1]
        need = engram_host_workspace_bytes(self.ctx, B, T, t_begin, chunk_rows)
        if need > getattr(self, "host_workspace_bytes", 0):
            self.host_workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            self.host_workspace_bytes = need
        engram_forward_host(self.ctx, tok_host, B, T, tok_host.stride(0), t_begin, P, tables, h_host, Wk, Wv, gq, gk,
                            conv_w, conv_state, y_host, add_residual, chunk_rows, self.host_workspace,
                            self.host_workspace_bytes, stream)
        return y_host

    def table_grad(self, idx, d_e, stream=None):
        """Sparse gradient of the tables from dL/de: (rows [U] int64 global
        rows, grad [U][D] fp32), U read back from the device (a sync)."""
        import torch
        n_tok = idx.shape[0]
        n = max(1, n_tok * idx.shape[1])
        need = engram_table_grad_workspace_bytes(self.ctx, n_tok)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        rows = torch.empty(n, dtype=torch.int64, device=self.device)
        grad = torch.empty(n, self.cfg.row_dim, dtype=torch.float32, device=self.device)
        cnt = torch.zeros(1, dtype=torch.int64, device=self.device)
        engram_table_grad(self.ctx, idx, n_tok, d_e, rows, grad, cnt, ws, need, stream)
        U = int(cnt.item())
        return rows[:U], grad[:U], cnt

    def grad_route(self, rows, grad, n_pairs, n_shards: int, stream=None):
        """This rank's (row, gradient) pairs split by the shard that owns the
        row: (send_rows, send_grad, send_counts), the counts an int64 [n_shards]
        tensor on the device, the segments in shard order."""
        import torch
        max_rows = rows.shape[0]
        send_rows = torch.empty(max(1, max_rows), dtype=torch.int64, device=self.device)
        send_grad = torch.empty(max(1, max_rows), self.cfg.row_dim, dtype=torch.float32, device=self.device)
        send_counts = torch.empty(n_shards, dtype=torch.int64, device=self.device)
        need = engram_grad_route_workspace_bytes(self.ctx)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        engram_grad_route(self.ctx, n_shards, rows, grad, n_pairs, max_rows, send_rows, send_grad, send_counts, ws,
                          need, stream)
        return send_rows, send_grad, send_counts

    def grad_combine(self, pair_rows, pair_grad, n_shards: int, shard: int, stream=None):
        """The pairs received by shard `shard`, summed per row: (rows [U]
        int64 global rows, grad [U][D] fp32, count), U read back (a sync)."""
        import torch
        n = pair_rows.shape[0]
        need = engram_grad_combine_workspace_bytes(self.ctx, n)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        rows = torch.empty(max(1, n), dtype=torch.int64, device=self.device)
        grad = torch.empty(max(1, n), self.cfg.row_dim, dtype=torch.float32, device=self.device)
        cnt = torch.zeros(1, dtype=torch.int64, device=self.device)
        engram_grad_combine(self.ctx, n_shards, shard, pair_rows, pair_grad, n, rows, grad, cnt, ws, need, stream)
        U = int(cnt.item())
        return rows[:U], grad[:U], cnt

    def shard_sgd(self, n_shards: int, shard: int, rows, grad, n_unique, shard_table, lr: float, stream=None):
        """shard_table[row - first] -= lr * grad for the listed global rows."""
        engram_shard_sgd(self.ctx, n_shards, shard, rows, grad, n_unique, rows.shape[0], shard_table, lr, stream)

    # ---- the residual stream around the module.  With a stream given, the work
    # and the tensors made here belong to it: a caller that uses them on
    # another stream orders the two (wait_stream, record_stream).

    @functools.cached_property
    def dtype(self):
        """torch dtype of the hidden states (h, Y)"""
        import torch
        return torch.float32 if self.cfg.dtype == ENGRAM_F32 else torch.bfloat16

    def _want(self, name: str, t, shape, dtype):
        """Refuse a tensor of another device, dtype or shape, or with gaps."""
        if t.shape == shape and t.dtype is dtype and t.device == self.device and t.is_contiguous():
            return
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the context on {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} is {t.dtype}, needs {dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
        raise ValueError(f"{name} must be contiguous")

    def _want_tokens(self, tok, t_begin: int):
        """(B, T, row stride) of a token tensor whose rows may be wider than T."""
        import torch
        if tok.ndim != 2:
            raise ValueError(f"tok has {tok.ndim} dimensions, needs 2")
        if tok.dtype is not torch.int32 or tok.device != self.device:
            raise ValueError(f"tok is {tok.dtype} on {tok.device}, needs torch.int32 on {self.device}")
        B, T = tok.shape
        if T > 1 and tok.stride(1) != 1:
            raise ValueError("the ids of a sequence must be adjacent in memory")
        if not 0 <= t_begin <= T:
            raise ValueError(f"t_begin = {t_begin} is outside [0, {T}]")
        stride = tok.stride(0) if B > 1 else T
        if stride < T:
            raise ValueError(f"the sequences overlap: row stride {stride} below T = {T}")
        return B, T, stride

    def embed(self, tok, E, *, t_begin: int = 0, scale: float = 1.0, out=None, stream=None):
        """Hidden states scale * E[tok] of positions t_begin .. T-1: [B*L][d]."""
        import torch
        B, T, stride = self._want_tokens(tok, t_begin)
        n, d = B * (T - t_begin), self.cfg.hidden
        self._want("E", E, (self.cfg.vocab, d), self.dtype)
        if out is None:
            with _on_stream(stream):
                out = torch.empty(n, d, dtype=E.dtype, device=self.device)
        else:
            self._want("out", out, (n, d), E.dtype)
        engram_embed(self.ctx, tok, B, T, stride, t_begin, E, scale, out, stream)
        return out

    def embed_grad(self, tok, d_h, *, t_begin: int = 0, scale: float = 1.0, out=None, accumulate: bool = False,
                   stream=None):
        """Gradient of E from that of the hidden states: fp32 [V][d], written
        to `out` (or a new tensor), or added to `out` with accumulate."""
        import torch
        B, T, stride = self._want_tokens(tok, t_begin)
        n, d = B * (T - t_begin), self.cfg.hidden
        self._want("d_h", d_h, (n, d), self.dtype)
        if accumulate and out is None:
            raise ValueError("accumulate needs the gradient to add to (out)")
        if n > 1 << 24:
            raise ValueError(f"{n} rows, at most 2^24 in one call")
        V = self.cfg.vocab
        if out is not None:
            self._want("out", out, (V, d), torch.float32)
        with _on_stream(stream):
            if out is None:
                out = torch.empty(V, d, dtype=torch.float32, device=self.device)
            need = engram_embed_grad_workspace_bytes(self.ctx, n)
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        engram_embed_grad(self.ctx, tok, B, T, stride, t_begin, d_h, scale, out, accumulate, ws, need, stream)
        return out

    def add_norm(self, x, res=None, *, gain=None, sum: bool = True, y: bool = True, q: bool = False,
                 rstd: bool = False, stream=None) -> NormOut:
        """s = x + res and its RMSNorm: the sum, the normed rows (y), their E4M3
        form with a scale per row (q), and 1/rms per row (rstd, for the
        backward), as asked for."""
        import torch
        d = self.cfg.hidden
        n = x.shape[0]
        self._want("x", x, (n, d), self.dtype)
        if res is not None:
            self._want("res", res, (n, d), self.dtype)
        if gain is not None:
            self._want("gain", gain, (d,), torch.float32)
        with _on_stream(stream):
            o = NormOut(torch.empty_like(x) if sum else None, torch.empty_like(x) if y else None,
                        torch.empty_like(x, dtype=torch.float8_e4m3fn) if q else None,
                        torch.empty(n, dtype=torch.float32, device=self.device) if q else None,
                        torch.empty(n, dtype=torch.float32, device=self.device) if rstd else None)
        engram_add_norm(self.ctx, x, res, n, gain, *o, stream)
        return o

    def add_norm_grad(self, d_y, sum, rstd, *, gain=None, d_sum=None, need_gain: bool = True, stream=None):
        """(d_x, d_gain): d_x is the gradient of x and of res; d_gain is None
        without need_gain."""
        import torch
        d = self.cfg.hidden
        n = d_y.shape[0]
        self._want("d_y", d_y, (n, d), self.dtype)
        self._want("sum", sum, (n, d), self.dtype)
        self._want("rstd", rstd, (n,), torch.float32)
        if d_sum is not None:
            self._want("d_sum", d_sum, (n, d), self.dtype)
        if gain is not None:
            self._want("gain", gain, (d,), torch.float32)
        with _on_stream(stream):
            d_x = torch.empty_like(d_y)
            d_gain = torch.empty(d, dtype=torch.float32, device=self.device) if need_gain else None
            need = engram_add_norm_grad_workspace_bytes(self.ctx, n) if need_gain else 0
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need_gain else None
        engram_add_norm_grad(self.ctx, d_y, d_sum, sum, rstd, n, gain, d_x, d_gain, ws, need, stream)
        return d_x, d_gain

    def _ffn_args(self, x, Wgu, Wd, act: str, x_dtype, w_dtype):
        """(n, f, activation code) of a feed-forward call's common tensors."""
        import torch
        d = self.cfg.hidden
        if act not in _ACTS:
            raise ValueError(f"act is {act!r}, needs one of {sorted(_ACTS)}")
        if Wd.dim() != 2:
            raise ValueError(f"Wd has {Wd.dim()} dimensions, needs 2")
        n, f = x.shape[0], Wd.shape[1]
        self._want("x", x, (n, d), x_dtype)
        self._want("Wgu", Wgu, (2 * f, d), w_dtype)
        self._want("Wd", Wd, (d, f), torch.bfloat16)
        return n, f, _ACTS[act]

    def ffn(self, x, Wgu, Wd, *, act: str = "silu", x_scale=None, gu_scale=None, res=None, save: bool = False,
            stream=None):
        """Gated feed-forward block (act(x Wg^T) * x Wu^T) Wd^T (+ res), Wgu the
        rows of Wg then Wu; in an FP8 context x and Wgu are E4M3 with a scale
        per row (x_scale, gu_scale).  Returns y, or (y, saved) with save: the
        bytes that :meth:`ffn_grad` reads (bf16 contexts)."""
        import torch
        f8 = self.cfg.dtype == ENGRAM_FP8
        dt = torch.float8_e4m3fn if f8 else torch.bfloat16
        n, f, a = self._ffn_args(x, Wgu, Wd, act, dt, dt)
        if (x_scale is None or gu_scale is None) if f8 else (x_scale is not None or gu_scale is not None):
            raise ValueError("x_scale and gu_scale go with an FP8 context, and are required there")
        if save and f8:
            raise ValueError("save is for the backward, which takes bf16 contexts")
        if f8:
            self._want("x_scale", x_scale, (n,), torch.float32)
            self._want("gu_scale", gu_scale, (2 * f,), torch.float32)
        if res is not None:
            self._want("res", res, (n, self.cfg.hidden), torch.bfloat16)
        need = engram_ffn_workspace_bytes(self.ctx, n, f)
        with _on_stream(stream):
            y = torch.empty(n, self.cfg.hidden, dtype=torch.bfloat16, device=self.device)
            saved = torch.empty(engram_ffn_saved_bytes(self.ctx, n, f), dtype=torch.uint8, device=self.device) if save else None
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        engram_ffn(self.ctx, x, x_scale, n, f, a, Wgu, gu_scale, Wd, res, y, saved, ws, need, stream)
        return (y, saved) if save else y

    def ffn_grad(self, d_y, x, saved, Wgu, Wd, *, act: str = "silu", stream=None):
        """(d_x, d_Wgu, d_Wd) from the gradient of y and the forward's x and saved."""
        import torch
        bf = torch.bfloat16
        n, f, a = self._ffn_args(x, Wgu, Wd, act, bf, bf)
        self._want("d_y", d_y, (n, self.cfg.hidden), bf)
        self._want("saved", saved, (engram_ffn_saved_bytes(self.ctx, n, f),), torch.uint8)
        need = engram_ffn_grad_workspace_bytes(self.ctx, n, f)
        with _on_stream(stream):
            d_x, d_Wgu, d_Wd = torch.empty_like(x), torch.empty_like(Wgu), torch.empty_like(Wd)
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        engram_ffn_grad(self.ctx, d_y, x, saved, n, f, a, Wgu, Wd, d_x, d_Wgu, d_Wd, ws, need, stream)
        return d_x, d_Wgu, d_Wd

    def status(self, stream=None):
        return engram_device_status(self.ctx, stream)


class HostTier:
    """Owns one engram_host_tier: tables in host memory, rows fetched per
    batch (engram_host_dedupe -> engram_host_fetch -> engram_gather_staged)."""

    def __init__(self, engram: "Engram", host_tables, max_lookups: int, n_threads: int = 8):
        self.engram = engram
        self.host_tables = host_tables          # keeps the host memory alive
        self.tier = engram_host_tier_create(engram.ctx, host_tables, max_lookups, n_threads)

    def close(self):
        if self.tier:
            engram_host_tier_destroy(self.tier)
            self.tier = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def dedupe(self, idx, n_tok: int, stream=None):
        engram_host_dedupe(self.tier, idx, n_tok, stream)

    def fetch(self, side_stream) -> int:
        return engram_host_fetch(self.tier, side_stream)

    def gather(self, n_tok: int, e_cat, stream=None):
        engram_gather_staged(self.tier, n_tok, e_cat, stream)
        return e_cat

    def stats(self):
        return engram_host_tier_stats(self.tier)

    def map_tables(self):
        """Fetch rows with a GPU kernel reading the mapped host tables."""
        engram_host_tier_map(self.tier)

    def enable_cache(self, capacity_rows: int, min_count: int = 2):
        engram_host_cache_enable(self.tier, capacity_rows, min_count)

    def reset_cache(self, stream=None):
        engram_host_cache_reset(self.tier, stream)

    def cache_stats(self):
        return engram_host_cache_stats(self.tier)

    def debug(self, inject: int, wait_limit_s: float):
        engram_host_tier_debug(self.tier, inject, wait_limit_s)


def exchange_shards(local_ptr: int, rank: int, world: int, all_gather, export=None, open_=None):
    """Shard pointers valid on this rank's GPU for every rank's shard.

    One process per GPU; rank r holds shard r at the device pointer
    ``local_ptr``.  Each rank exports its shard (an IPC handle and offset),
    ``all_gather(obj) -> [obj of rank 0, ..., obj of rank world-1]`` collects
    every rank's export (``torch.distributed.all_gather_object`` in a job),
    and each rank maps the others' shards into its own address space.
    Returns (pointers in shard order, mapping bases to close later).  The
    export/open functions default to the library's IPC calls; the host logic
    is the same with any pair."""
    export = engram_ipc_export if export is None else export
    open_ = engram_ipc_open if open_ is None else open_
    mine = export(local_ptr) if world > 1 else None
    every = all_gather(mine) if world > 1 else [mine]
    if len(every) != world:
        raise RuntimeError(f"expected {world} shard exports, got {len(every)}")
    ptrs, bases = [], []
    for g in range(world):
        if g == rank:
            ptrs.append(int(local_ptr))
            continue
        handle, offset = every[g]
        ptr, base = open_(handle, offset)
        ptrs.append(ptr)
        bases.append(base)
    return ptrs, bases


class ShardedTables:
    """This rank's shard of the tables (rank r of ``world`` holds shard r, the
    global rows ``engram_shard_range`` gives it) and the pointers of every
    shard on this rank's GPU.  ``fill(first_row, n_rows, out)`` writes the
    shard's rows into ``out`` ([n_rows][D] on the device).  Mappings of
    other ranks' shards are closed by :meth:`close`; all ranks must keep
    their shard alive until every rank is done with it (a barrier)."""

    def __init__(self, engram: "Engram", world: int, rank: int, row_dim: int, dtype, device, fill, all_gather=None,
                 export=None, open_=None, close=None):
        import torch
        self.first, self.rows = engram_shard_range(engram.ctx, world, rank)
        self.local = torch.empty(max(1, self.rows), row_dim, dtype=dtype, device=device)
        if self.rows:
            fill(self.first, self.rows, self.local[: self.rows])
        torch.cuda.synchronize(device)
        self._close = engram_ipc_close if close is None else close
        self.ptrs, self._bases = exchange_shards(self.local.data_ptr(), rank, world, all_gather, export, open_)

    def close(self):
        for b in self._bases:
            self._close(b)
        self._bases = []


def all_to_all_pairs(send_rows, send_grad, send_counts, all_to_all_single=None):
    """The backward's exchange of (row, gradient) pairs between the ranks.

    ``send_counts[g]`` pairs of this rank are for rank g (one shard per rank),
    in segments of ``send_rows`` / ``send_grad`` in rank order (what
    :meth:`Engram.grad_route` writes).  First the counts go round (one int64
    from every rank to every rank), then the segments, with the split sizes
    those counts give.  Returns (recv_rows, recv_grad, recv_counts as a host
    list): the pairs sent to this rank by rank 0, then rank 1, and so on.
    ``all_to_all_single`` defaults to ``torch.distributed``'s (NCCL between
    GPUs, gloo on CPU); reading the counts on the host is a sync."""
    import torch
    if all_to_all_single is None:
        import torch.distributed as dist
        all_to_all_single = dist.all_to_all_single
    recv_counts = torch.empty_like(send_counts)
    all_to_all_single(recv_counts, send_counts)
    in_split = [int(x) for x in send_counts.tolist()]
    out_split = [int(x) for x in recv_counts.tolist()]
    if min(in_split + out_split, default=0) < 0:
        raise RuntimeError(f"negative pair count in {in_split} / {out_split}")
    n_send, n_recv = sum(in_split), sum(out_split)
    if n_send > send_rows.shape[0]:
        raise RuntimeError(f"{n_send} pairs to send, the send buffers hold {send_rows.shape[0]}")
    D = send_grad.shape[1]
    recv_rows = torch.empty(n_recv, dtype=send_rows.dtype, device=send_rows.device)
    recv_grad = torch.empty(n_recv, D, dtype=send_grad.dtype, device=send_grad.device)
    all_to_all_single(recv_rows, send_rows[:n_send], out_split, in_split)
    all_to_all_single(recv_grad, send_grad[:n_send], out_split, in_split)
    return recv_rows, recv_grad, out_split


def sharded_table_step(engram: Engram, tables: ShardedTables, idx, d_e, lr: float, rank: int, world: int,
                       all_to_all_single=None):
    """One update of sharded tables from this rank's batch: the sparse
    gradient of the rows the batch looked up (engram_table_grad), routed to
    the ranks that own them (engram_grad_route), exchanged
    (:func:`all_to_all_pairs`), summed per row in rank order
    (engram_grad_combine) and applied to this rank's shard
    (engram_shard_sgd).  Every rank calls it with its own batch; returns the
    (rows, gradient) applied to this rank's shard."""
    rows, grad, cnt = engram.table_grad(idx, d_e)
    send_rows, send_grad, send_counts = engram.grad_route(rows, grad, cnt, world)
    recv_rows, recv_grad, _ = all_to_all_pairs(send_rows, send_grad, send_counts, all_to_all_single)
    r, g, u = engram.grad_combine(recv_rows, recv_grad, world, rank)
    engram.shard_sgd(world, rank, r, g, u, tables.local, lr)
    return r, g
