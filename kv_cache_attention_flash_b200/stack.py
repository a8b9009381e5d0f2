"""A stack of Flash-Cache layer steps chained through the residual stream.

The pages describe one layer's hot path ("Flash-dLLM: I/O-Aware KV Caching
and Parallel Decoding for Fast, Memory-Efficient Diffusion LLMs", ai4snews
summary, paragraph 1). A model runs it once per layer, and a layer's output
reaches the next layer through the attention block's output projection and
the residual stream. Per layer l this module runs

    out_l   = fused layer step on x_l          (fdllm_layer_step, bf16 out)
    x_{l+1} = x_l + out_l W_o,l                (fdllm_oproj with the residual,
                                                in place over x)

With feed-forward weights the block's second half follows,

    x_{l+1} += (silu(x_{l+1} W_gate) * (x_{l+1} W_up)) W_down    (two fdllm_linear)

and `decode` runs the same layers for one new token a sequence: fdllm_linear
for the projections, fdllm_decode_attention for the attention over the same
pools. The norms of a full transformer block are not part of the path and are
left out. Host orchestration only: every arithmetic step runs in the library's
kernels, in stream order.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import (FlashCache, _on, fdllm_last_launch_count, fdllm_layer_step, fdllm_linear,
               fdllm_oproj)


class LayerStack:
    """Chained layers over one FlashCache (one pool slice per layer).

    wqkv[l]: bf16 [H, 3H]; w_o[l]: bf16 [H, H]. mlp[l], when given:
    (W_gate, W_up, W_down), bf16 [H, F], [H, F] and [F, H]. run() updates x in
    place (x_0 in, x_L out) and returns the last layer's attention mass."""

    def __init__(self, cache: FlashCache, wqkv: Sequence[torch.Tensor],
                 w_o: Sequence[torch.Tensor], mlp: Optional[Sequence] = None):
        if len(wqkv) != len(w_o):
            raise ValueError("one W_o per layer")
        if mlp is not None and len(mlp) != len(wqkv):
            raise ValueError("feed-forward weights for every layer, or for none")
        self.cache = cache
        self.wqkv = list(wqkv)
        self.w_o = list(w_o)
        self.mlp = None if mlp is None else list(mlp)
        self.n_layers = len(self.wqkv)
        self._out = None
        self.launches = 0

    def run(self, cu_rows, seq_lens, x: torch.Tensor, positions: torch.Tensor,
            block_table: torch.Tensor, view_mask: Optional[torch.Tensor] = None,
            slots: Optional[torch.Tensor] = None, attn_mass: Optional[torch.Tensor] = None,
            stream=None, x_out: Optional[torch.Tensor] = None, outs=None):
        """One pass through the stack. With x_out, x stays as it is: the
        first projection writes the residual stream into x_out and the later
        layers update x_out in place; without it, x is updated in place.
        `outs`, a dict, receives a copy of each layer's bf16 out when given
        (for tests). Returns (the final residual stream, attn_mass)."""
        R, H = x.shape
        if self._out is None or self._out.shape != (R, H):
            self._out = torch.empty(R, H, dtype=torch.bfloat16, device=x.device)
        mb = int(block_table.shape[1])
        n = 0
        cur = x
        dst = x if x_out is None else x_out
        for l in range(self.n_layers):
            fdllm_layer_step(self.cache.handle, l, cu_rows, seq_lens, mb, cur, self.wqkv[l],
                             positions, block_table, view_mask, self._out, attn_mass, slots,
                             False, stream)
            n += fdllm_last_launch_count()
            if outs is not None:
                outs[l] = self._out.clone()
            fdllm_oproj(self._out, self.w_o[l], y=dst, residual=cur, stream=stream,
                        status=self.cache.status)
            n += fdllm_last_launch_count()
            n += self._feed_forward(l, dst, stream, self.cache.status)
            cur = dst
        self.launches = n
        return dst, attn_mass

    def _feed_forward(self, l: int, x: torch.Tensor, stream, status, outs=None) -> int:
        """x += (silu(x W_gate) * (x W_up)) W_down in place; launches made."""
        if self.mlp is None:
            return 0
        gate, up, down = self.mlp[l]
        h = fdllm_linear(x, up, act="silu", w_gate=gate, status=status, stream=stream)
        n = fdllm_last_launch_count()
        if outs is not None:
            outs["ff_in"], outs["ff_hidden"] = x.clone(), h
        fdllm_linear(h, down, residual=x, y=x, status=status, stream=stream)
        return n + fdllm_last_launch_count()

    def decode(self, x: torch.Tensor, positions: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, slots: Optional[torch.Tensor] = None,
               x_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream=None, outs=None) -> torch.Tensor:
        """One new token a sequence through the stack: x bf16 [B, H], the
        token's position, the slot its k and v go to (default: the position)
        and the slots it sees, itself included (device int32 [B] each:
        "seq_positions", "seq_slots" and "seq_lens" of fdllm_plan_blocks, not
        its row outputs, whose entries move up where a request has no row; a
        request without a row writes nothing and its x means nothing). The residual
        stream ends in x_out (default: x). A call may be captured after a
        first one outside a capture has built the cache's RoPE tables. Device-
        side errors are raised by the cache's next check(), or written to
        `status` alone when that is given. `outs`, a dict, receives each
        layer's intermediate results (for tests)."""
        if stream is not None:
            with _on(stream, x):
                return self.decode(x, positions, block_table, seq_lens, slots, x_out, status, None,
                                   outs)
        status = self.cache.status if status is None else status
        H = x.shape[1]
        n = 0
        cur = x
        dst = x if x_out is None else x_out
        for l in range(self.n_layers):
            qkv = fdllm_linear(cur, self.wqkv[l], out_dtype=torch.float32, status=status)
            n += fdllm_last_launch_count()
            out, _ = self.cache.decode(l, qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:], positions,
                                       block_table, seq_lens, slots, out_dtype=torch.bfloat16,
                                       status=status)
            n += fdllm_last_launch_count()
            o = None
            if outs is not None:
                o = outs[l] = {"x": cur.clone(), "qkv": qkv, "out": out}
            fdllm_linear(out, self.w_o[l], residual=cur, y=dst, status=status)
            n += fdllm_last_launch_count()
            if o is not None:
                o["y"] = dst.clone()
            n += self._feed_forward(l, dst, None, status, o)
            cur = dst
        self.launches = n
        return dst
