"""A whole decode step captured in a CUDA graph.

The C ABI is capture-safe: lengths and positions are device tensors, launch shapes depend
only on the pool's static geometry, nothing is allocated inside a call, and the tensor-core
kernel launches as a programmatic dependent so consecutive layers keep their overlap inside
the graph.  ``DecodeStepGraph`` records, for every layer, the append of the new token and the
windowed attention (``hwkv_append_decode_attn``, or ``hwkv_append`` + ``hwkv_decode_attn``),
followed by the advance of the positions (``hwkv_advance_positions``), and replays that whole
step with one launch from the host: every kernel of a replayed step is the library's.  With a
rotary table each layer's queries and new keys are first turned at the step's positions
(``hwkv_rope``).  Inputs are read from, and outputs written to, the static buffers it owns.
"""
from __future__ import annotations

import torch


class DecodeStepGraph:
    """Captured decode step of every layer of ``pool``.

    Static buffers (fill them before ``replay``):
      q     [layers][B][q_heads][D]   queries of the step
      k_new [layers][B][kv_heads][D]  new keys, v_new likewise
      pos   [B] int32                 lengths before the append; the step adds 1 to them
    Output: out [layers][B][q_heads][D].
    rope: a ``rope_table`` when q and k_new come without their rotary positions.
    softcap, slopes: capped or distance-biased scores, as in ``Pool.decode``.
    """

    def __init__(self, pool, scale: float, q_heads: int, pos0, fused: bool = True, rope=None, softcap: float = 0.0,
                 slopes=None):
        dev = pool.buffer.device
        L, B, H, D = pool.layers, pool.num_seqs, pool.kv_heads, pool.head_dim
        dt = pool.io_dtype
        self.pool = pool
        self.q = torch.zeros((L, B, q_heads, D), dtype=dt, device=dev)
        self.k_new = torch.zeros((L, B, H, D), dtype=dt, device=dev)
        self.v_new = torch.zeros_like(self.k_new)
        self.out = torch.zeros_like(self.q)
        self.pos = torch.as_tensor(pos0, dtype=torch.int32, device=dev).clone()
        self.lens = torch.empty_like(self.pos)
        if q_heads != pool.q_heads:
            pool.q_heads = q_heads
            pool._size_workspace()
        self.rope = rope
        self._score = {"softcap": softcap, "slopes": slopes}
        self._q, self._k = self.q, self.k_new  # what the attention reads
        if rope is not None:
            self._q, self._k = torch.empty_like(self.q), torch.empty_like(self.k_new)
        self.scale = float(scale)
        self.fused = fused
        self.graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            with torch.cuda.graph(self.graph, stream=side):
                self._record()
        torch.cuda.current_stream(dev).wait_stream(side)

    def _record(self):
        p = self.pool
        if not self.fused:
            p.advance_positions(self.pos, out=self.lens)  # lengths after the append
        for l in range(p.layers):
            if self.rope is not None:
                p.rope(self.rope, self.q[l], self.k_new[l], self.pos, q_out=self._q[l], k_out=self._k[l])
            if self.fused:
                # the kernel just before is the rotary one, or after layer 0 the previous layer's
                # attention: neither writes the positions or this layer's pool
                p.append_decode(l, self._q[l], self.scale, self._k[l], self.v_new[l], self.pos, out=self.out[l],
                                early_reads=l > 0 or self.rope is not None, **self._score)
            else:
                p.append(l, self._k[l], self.v_new[l], self.pos)
                p.decode(l, self._q[l], self.scale, self.lens, out=self.out[l], **self._score)
        p.advance_positions(self.pos)  # the next step's positions

    def replay(self):
        self.graph.replay()
