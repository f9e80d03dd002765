"""hwkv: per-head budgeted KV residency on one GB300.

The grouped-cache runtime of "HeadWiseKV: Budgeted Per-Head Cache Residency for Hybrid
Long-Context Language Models" (blog summary; abstract and section "Grouped-Cache
Runtime"): every KV head of a global-attention layer keeps a static window of its most
recent tokens in ceil(w / block_size) paged blocks, and decode attention reads only that
resident window.

``binding`` exposes the C ABI of ``include/hwkv.h`` under the same names; ``Pool`` below
is a convenience wrapper that owns the device buffers (allocated with torch).
"""
from __future__ import annotations

from contextlib import nullcontext
from typing import Optional

import torch

from . import binding
from .binding import (HWKV_BF16, HWKV_E4M3, HWKV_F32, HWKV_KERNEL_AUTO, HWKV_KERNEL_SIMT, HWKV_KERNEL_TENSOR, DecodeLaunch, HwkvError, RopeTable, Score,
                      hwkv_abi_version, hwkv_advance_positions, hwkv_append, hwkv_append_decode_attn, hwkv_block_table,
                      hwkv_check_device_errors, hwkv_kernel_launches,
                      hwkv_decode_attn, hwkv_decode_attn_score, hwkv_decode_attn_shared,
                      hwkv_decode_shared_workspace_bytes, hwkv_decode_workspace_bytes, hwkv_materialize, hwkv_pool_bytes,
                      hwkv_pool_create, hwkv_pool_destroy, hwkv_pool_geometry, hwkv_prefill_attn,
                      hwkv_prefill_attn_score, hwkv_prefill_plan, hwkv_prefill_workspace_bytes, hwkv_rope, hwkv_rope_append, hwkv_rope_table, hwkv_set_block_table, hwkv_set_decode_config,
                      hwkv_set_prefill_config, hwkv_wait_selftest)

__all__ = [
    "Pool", "DecodeLaunch", "HwkvError", "RopeTable", "Score", "binding", "rope_table", "HWKV_F32", "HWKV_BF16", "HWKV_E4M3", "HWKV_KERNEL_AUTO", "HWKV_KERNEL_TENSOR",
    "HWKV_KERNEL_SIMT", "hwkv_abi_version", "hwkv_advance_positions", "hwkv_append", "hwkv_append_decode_attn", "hwkv_block_table",
    "hwkv_check_device_errors", "hwkv_kernel_launches",
    "hwkv_decode_attn", "hwkv_decode_attn_score", "hwkv_decode_attn_shared", "hwkv_decode_shared_workspace_bytes",
    "hwkv_decode_workspace_bytes", "hwkv_materialize", "hwkv_pool_bytes", "hwkv_pool_create",
    "hwkv_pool_destroy", "hwkv_pool_geometry", "hwkv_prefill_attn", "hwkv_prefill_attn_score", "hwkv_prefill_plan", "hwkv_prefill_workspace_bytes", "hwkv_rope", "hwkv_rope_append", "hwkv_rope_table",
    "hwkv_set_block_table", "hwkv_set_decode_config", "hwkv_set_prefill_config", "hwkv_wait_selftest",
]


_ROPE_LAYOUTS = {"half": binding.HWKV_ROPE_HALF, "interleaved": binding.HWKV_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"none": binding.HWKV_ROPE_SCALE_NONE, "linear": binding.HWKV_ROPE_SCALE_LINEAR,
                  "ntk": binding.HWKV_ROPE_SCALE_NTK, "by_parts": binding.HWKV_ROPE_SCALE_BY_PARTS}


def rope_table(head_dim: int, rot_dim: Optional[int] = None, base: float = 10000.0, layout: str = "half",
               scaling: str = "none", factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0,
               beta_slow: float = 1.0) -> RopeTable:
    """The table ``Pool.rope`` turns heads of ``head_dim`` with: pairs of the first ``rot_dim`` dims
    (all by default), ``layout`` "half" (i, i + rot_dim / 2) or "interleaved" (2i, 2i + 1),
    frequencies base^(-2i / rot_dim) scaled for longer contexts by ``scaling`` "none", "linear",
    "ntk" or "by_parts".  by_parts ramps over a pair's turns in original_len positions and scales by
    0.1 ln(factor) + 1; a configuration that ramps over the pair's index, or keeps magnitude 1, sets the
    table's ``freq[i]`` and ``magnitude`` itself (see hwkv_rope_table in the header)."""
    rot_dim = head_dim if rot_dim is None else rot_dim
    if rot_dim > head_dim:
        raise ValueError(f"rot_dim {rot_dim} exceeds head_dim {head_dim}")
    if layout not in _ROPE_LAYOUTS or scaling not in _ROPE_SCALINGS:
        raise ValueError(f"unknown rope layout {layout!r} or scaling {scaling!r}")
    return hwkv_rope_table(rot_dim, _ROPE_LAYOUTS[layout], base, _ROPE_SCALINGS[scaling], factor, original_len, beta_fast,
                           beta_slow)


def _on(stream):
    """Where tensors that a call on ``stream`` makes are allocated and filled."""
    if stream is None:
        return nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class Pool:
    """A per-head paged KV pool on the current CUDA device.

    The pool buffer is one torch uint8 allocation of exactly ``hwkv_pool_bytes`` bytes
    (the pre-serving prediction), bound with ``hwkv_pool_create``.  With dtype
    ``torch.float8_e4m3fn`` it holds 8-bit codes and a scale per 16 slots (``scales``); queries,
    new rows and outputs are then bf16 (``io_dtype``).
    """

    def __init__(self, layers: int, kv_heads: int, head_dim: int, block_size: int, windows, num_seqs: int,
                 dtype: torch.dtype, q_heads: Optional[int] = None, device=None, stream=None):
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        self.block_size, self.num_seqs, self.dtype = block_size, num_seqs, dtype
        elem = (torch.float32, torch.bfloat16, torch.float8_e4m3fn)[binding._dtype_code(dtype)]
        self.io_dtype = torch.bfloat16 if elem == torch.float8_e4m3fn else elem
        self.q_heads = q_heads or kv_heads
        self.nbytes = hwkv_pool_bytes(layers, kv_heads, head_dim, block_size, windows, num_seqs, dtype)
        device = torch.device(device or "cuda")
        self.buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self._device_index = self.buffer.get_device()
        self.handle = hwkv_pool_create(layers, kv_heads, head_dim, block_size, windows, num_seqs, dtype,
                                       self.buffer, stream)
        _, total, block_bytes = hwkv_pool_geometry(self.handle)
        self._blocks = self.buffer[:total * block_bytes].view(elem).view(total, 2, block_size, head_dim)
        self._scales = None
        if elem == torch.float8_e4m3fn:
            groups = block_size // 16
            area = self.buffer[total * block_bytes:total * block_bytes + total * groups * 8]
            self._scales = area.view(torch.float32).view(total, groups, 2)
        self.workspace = None
        self.prefill_workspace = None
        self._prefill_captured = False
        self.shared_workspace = None
        self._outgrown = []  # workspaces that captured graphs (or other streams) may still use
        self._size_workspace()

    def _size_workspace(self):
        need = hwkv_decode_workspace_bytes(self.handle, self.q_heads)
        if self.workspace is None or self.workspace.numel() < need:
            if self.workspace is not None:  # seldom: the group or the configuration grew
                self._outgrown.append(self.workspace)
            self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=self.buffer.device)

    def set_decode_config(self, split_tokens: int = 0, kernel: int = HWKV_KERNEL_AUTO, workers: int = 0):
        hwkv_set_decode_config(self.handle, split_tokens, workers, kernel)
        self._size_workspace()

    def geometry(self):
        return hwkv_pool_geometry(self.handle)

    def blocks(self) -> torch.Tensor:
        """View of the pool as [total_blocks][2][block_size][head_dim] elements (the codes of an
        8-bit pool)."""
        return self._blocks

    def scales(self) -> torch.Tensor:
        """View of an 8-bit pool's scales, fp32 [total_blocks][block_size / 16][2 (K, V)]: a value
        of ``blocks()`` stands for its code times the scale of its 16 slots."""
        if self._scales is None:
            raise ValueError("only an 8-bit pool has scales")
        return self._scales

    def _check_io(self, *tensors):
        # an 8-bit pool does not share its element type with the tensors passed to it
        if self._scales is not None:
            for t in tensors:
                if t is not None and t.dtype != torch.bfloat16:
                    raise ValueError(f"an 8-bit pool takes bf16 tensors (got {t.dtype})")

    def block_table(self, seq: int, layer: int, kv_head: int):
        return hwkv_block_table(self.handle, seq, layer, kv_head)

    def set_block_table(self, table, stream=None):
        hwkv_set_block_table(self.handle, table, stream)

    def materialize(self, layer: int, k_full, v_full, lens, stream=None):
        self._check_io(k_full, v_full)
        hwkv_materialize(self.handle, layer, k_full, v_full, lens, stream)

    def append(self, layer: int, k_new, v_new, pos, stream=None):
        self._check_io(k_new, v_new)
        hwkv_append(self.handle, layer, k_new, v_new, pos, stream)

    def decode(self, layer: int, q, scale: float, lens, out=None, stream=None, early_reads: bool = False,
               softcap: float = 0.0, slopes=None):
        """Attention of q [B][Hq][D] at lengths ``lens`` (after the append).  softcap > 0 caps the scores
        at softcap * tanh(score / softcap); slopes (float32 [Hq]) lowers them by slope * distance."""
        if out is None:
            out = torch.empty_like(q)
        self._check_io(q, out)
        if q.shape[1] != self.q_heads:
            self.q_heads = q.shape[1]
            self._size_workspace()
        if softcap == 0 and slopes is None:
            hwkv_decode_attn(self.handle, layer, q, scale, lens, out, self.workspace, stream, early_reads)
        else:
            hwkv_decode_attn_score(self.handle, layer, q, binding.score(scale, softcap, slopes, q), lens, out,
                                   self.workspace, None, None, stream, early_reads)
        return out

    def append_decode(self, layer: int, q, scale: float, k_new, v_new, pos, out=None, stream=None,
                      early_reads: bool = False, softcap: float = 0.0, slopes=None):
        """Append the new token (positions ``pos``) and decode at ``pos + 1`` in one call.
        softcap, slopes: as ``decode``.
        early_reads: the caller's guarantee of HWKV_DECODE_EARLY_READS (lengths, block table
        and this layer's pool not written by the kernel just before in the stream)."""
        if out is None:
            out = torch.empty_like(q)
        self._check_io(q, k_new, v_new, out)
        if q.shape[1] != self.q_heads:
            self.q_heads = q.shape[1]
            self._size_workspace()
        if softcap == 0 and slopes is None:
            hwkv_append_decode_attn(self.handle, layer, q, scale, k_new, v_new, pos, out, self.workspace, stream,
                                    early_reads)
        else:
            hwkv_decode_attn_score(self.handle, layer, q, binding.score(scale, softcap, slopes, q), pos, out,
                                   self.workspace, k_new, v_new, stream, early_reads)
        return out

    def shared_decode(self, layer: int, prefix: "Pool", q, scale: float, lens, prefix_of, prefix_lens, k_new=None, v_new=None,
                      out=None, stream=None, softcap: float = 0.0, slopes=None):
        """Attention of q [B][Hq][D] whose sequences continue prefixes kept once in the pool ``prefix``: sequence s has
        lens[s] tokens of its own in this pool (after the append; with k_new and v_new [B][Hkv][D] the length before it) behind
        the prefix_lens[f] tokens of prefix f = prefix_of[s] (negative: behind none).  int32 [B], [B] and
        [prefix.num_seqs].  softcap, slopes: as ``decode``.  Keeps a workspace, grown on demand; one that
        is outgrown stays, for a captured graph or another stream may still use it.  The calls of a pool share it: no two at
        once, on two streams or in two graphs.  What is allocated belongs to ``stream``."""
        if out is None:
            with _on(stream):
                out = torch.empty_like(q)
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new go together")
        shape = q.shape
        if out is not q and out.shape != shape:
            raise ValueError("out must match q")
        self._check_row(q, "q", shape[-2])
        self._check_row(out, "out", shape[-2])
        if k_new is not None:
            self._check_row(k_new, "k_new", self.kv_heads)
            self._check_row(v_new, "v_new", self.kv_heads)
        if not (self._is_counts(lens) and self._is_counts(prefix_of) and prefix._is_counts(prefix_lens)):
            raise ValueError(f"lens and prefix_of must hold {self.num_seqs} values, prefix_lens {prefix.num_seqs}, in a row on "
                             f"{self.buffer.device}")
        args = (layer, q, binding.score(scale, softcap, slopes, q), lens, prefix_of, prefix_lens, out)
        if self.shared_workspace is not None:
            try:
                hwkv_decode_attn_shared(self.handle, prefix.handle, *args, self.shared_workspace, k_new, v_new, stream)
                return out
            except HwkvError as e:
                if e.status != binding.HWKV_ERR_WORKSPACE_TOO_SMALL:
                    raise
                self._outgrown.append(self.shared_workspace)
        need = hwkv_decode_shared_workspace_bytes(self.handle, prefix.handle, q.shape[1])
        with _on(stream):
            self.shared_workspace = torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
        hwkv_decode_attn_shared(self.handle, prefix.handle, *args, self.shared_workspace, k_new, v_new, stream)
        return out

    def decode_launch(self, layer: int, q, scale: float, lens, out, k_new=None, v_new=None, stream=None,
                      early_reads: bool = False, softcap: float = 0.0, slopes=None) -> DecodeLaunch:
        """A prepared launch of decode (k_new None, ``lens`` = lengths after the append) or of the
        fused append + decode (``lens`` = positions) on fixed buffers: calling it launches."""
        self._check_io(q, out, k_new, v_new)
        if q.shape[1] != self.q_heads:
            self.q_heads = q.shape[1]
            self._size_workspace()
        return DecodeLaunch(self.handle, layer, q, scale, lens, out, self.workspace, k_new, v_new, stream, early_reads,
                            softcap, slopes)

    def prefill(self, layer: int, q, scale: float, k_new, v_new, pos, n, out=None, stream=None, softcap: float = 0.0,
                slopes=None):
        """Chunked prefill: q [B][n_max][Hq][D], k_new/v_new [B][n_max][Hkv][D]; pos, n int32 [B];
        softcap, slopes: as ``decode``.
        Keeps a workspace for the split of long key streams, grown on demand; one that a capture has
        used stays when it is outgrown."""
        if out is None:
            out = torch.zeros_like(q)
        need = hwkv_prefill_workspace_bytes(self.handle, layer, q.shape[2], q.shape[1])
        if need and (self.prefill_workspace is None or self.prefill_workspace.numel() < need):
            if self._prefill_captured:
                self._outgrown.append(self.prefill_workspace)
                self._prefill_captured = False
            self.prefill_workspace = torch.empty(need, dtype=torch.uint8, device=self.buffer.device)
        workspace = self.prefill_workspace if need else None
        if need and torch.cuda.is_current_stream_capturing():
            self._prefill_captured = True
        if softcap == 0 and slopes is None:
            hwkv_prefill_attn(self.handle, layer, q, scale, k_new, v_new, pos, n, out, workspace, stream)
        else:
            hwkv_prefill_attn_score(self.handle, layer, q, binding.score(scale, softcap, slopes, q), k_new, v_new,
                                    pos, n, out, workspace, stream)
        return out

    def set_prefill_config(self, max_stages: int = 0):
        hwkv_set_prefill_config(self.handle, max_stages)

    def advance_positions(self, pos, out=None, delta: int = 1, stream=None):
        """out = pos + delta on the device with a library kernel (in place when out is None)."""
        out = pos if out is None else out
        hwkv_advance_positions(self.handle, pos, out, delta, stream)
        return out

    def rope(self, table: RopeTable, q, k, pos, n=None, q_out=None, k_out=None, stream=None):
        """Rotary positions: turns q [B][n_max][Hq][D] and k [B][n_max][Hkv][D] (or single rows
        [B][heads][D]; either may be None) at positions pos[s] + row, rows below n[s] (all when n is
        None).  Inputs may be slices of a fused projection.  Outputs default to new tensors (zeros past
        n); pass q_out=q, k_out=k to work in place.  Returns (q_out, k_out)."""
        new = torch.empty if n is None else torch.zeros
        if q is not None:
            self._check_rows(q, "q")
            if q_out is None:
                q_out = new(q.shape, dtype=q.dtype, device=q.device)
        if k is not None:
            if self._check_rows(k, "k") != self.kv_heads:
                raise ValueError(f"k must hold {self.kv_heads} heads")
            if k_out is None:
                k_out = new(k.shape, dtype=k.dtype, device=k.device)
        at = self._device_index
        if (q_out is not None and q_out.get_device() != at) or (k_out is not None and k_out.get_device() != at):
            raise ValueError(f"outputs must lie on {self.buffer.device}")
        if not self._is_counts(pos) or not (n is None or self._is_counts(n)):
            raise ValueError(f"positions and row counts must hold {self.num_seqs} values in a row on {self.buffer.device}")
        hwkv_rope(self.handle, table, q, k, pos, n, q_out, k_out, stream)
        return q_out, k_out

    def rope_append(self, layer: int, table: Optional[RopeTable], q, k, v, pos, n=None, q_out=None, k_out=None, turn_pos=None,
                    stream=None):
        """Rotary positions on the way into the pool, in one launch: q [B][n_max][Hq][D] and k [B][n_max][Hkv][D]
        (or single rows [B][heads][D]) turn at positions turn_pos[s] + row (pos[s] + row by default), and the
        turned k and v are stored at positions pos[s] + row, rows below n[s] (all when n is None).  q may be None;
        table None turns nothing.  q_out defaults to a new tensor of ``stream`` (zeros past n); pass q_out=q to work in place.
        k_out, when given, receives the turned keys too.  Returns (q_out, k_out)."""
        at = self._device_index
        if q is not None:
            if self._check_rows(q, "q") % self.kv_heads:
                raise ValueError(f"q must hold a multiple of {self.kv_heads} heads")
            if q_out is None:
                with _on(stream):
                    q_out = (torch.empty if n is None else torch.zeros)(q.shape, dtype=q.dtype, device=q.device)
            elif q_out.get_device() != at:
                raise ValueError(f"outputs must lie on {self.buffer.device}")
        elif q_out is not None:
            raise ValueError("q_out goes with q")
        if self._check_rows(k, "k") != self.kv_heads or self._check_rows(v, "v") != self.kv_heads:
            raise ValueError(f"k and v must hold {self.kv_heads} heads")
        if k_out is not None and k_out.get_device() != at:
            raise ValueError(f"outputs must lie on {self.buffer.device}")
        if not self._is_counts(pos) or not (n is None or self._is_counts(n)) or not (turn_pos is None or self._is_counts(turn_pos)):
            raise ValueError(f"positions and row counts must hold {self.num_seqs} values in a row on {self.buffer.device}")
        hwkv_rope_append(self.handle, layer, table, q, k, v, pos, n, turn_pos, q_out, k_out, stream)
        return q_out, k_out

    def _check_rows(self, t, name) -> int:
        shape = t.shape
        if (t.dtype != self.io_dtype or len(shape) < 3 or shape[0] != self.num_seqs or shape[-1] != self.head_dim
                or t.get_device() != self._device_index):
            raise ValueError(f"{name} must hold {self.io_dtype} rows of head_dim {self.head_dim} for "
                             f"{self.num_seqs} sequences on {self.buffer.device}")
        return shape[-2]

    def _check_row(self, t, name, heads):
        if (t.dtype != self.io_dtype or t.shape != (self.num_seqs, heads, self.head_dim) or not t.is_contiguous()
                or t.get_device() != self._device_index):
            raise ValueError(f"{name} must be contiguous {self.io_dtype} [{self.num_seqs}][{heads}][{self.head_dim}] on "
                             f"{self.buffer.device}")

    def _is_counts(self, t) -> bool:
        return t.get_device() == self._device_index and t.numel() >= self.num_seqs and t.is_contiguous()

    def check_device_errors(self, stream=None) -> int:
        return hwkv_check_device_errors(self.handle, stream)

    def close(self):
        if getattr(self, "handle", None):
            hwkv_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
