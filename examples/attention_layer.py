"""Attention of one decoder layer with everything 4-bit: Q4_K projections, Q4_0 paged KV cache.

Two prompts of different lengths enter the cache in chunks, then both sequences are decoded a token
at a time.  The weights and the rows that stand for tokens are synthetic; what is shown is how the
calls go together:

  prompt chunk   qk_gemv (q, k, v) -> qk_kv_append -> qk_kv_read (the prefix and the chunk) -> qk_attn_prompt -> qk_gemv
  decode step    qk_gemv (q, k, v) -> qk_kv_append -> qk_attn_paged -> qk_gemv

Run it on the GPU:  python examples/attention_layer.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemv_quantize_amd as qk
from quantized_gemv_quantize_amd import synth


class AttentionLayer:
    """Projections and cache of one layer.  Pages are handed out in order; a server has an allocator here."""

    def __init__(self, hidden, heads, kv_heads, dim, sequences, positions, page=64, seed=0):
        rng = np.random.default_rng(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.page = hidden, heads, kv_heads, dim, page
        self.w_qkv = torch.from_numpy(synth.q4_K_blocks(rng, (heads + 2 * kv_heads) * dim, hidden)).cuda()
        self.w_out = torch.from_numpy(synth.q4_K_blocks(rng, hidden, heads * dim)).cuda()
        per_seq = -(-positions // page)
        n_pages = sequences * per_seq
        bytes_ = qk.qk_kv_page_bytes(qk.QK_TYPE_Q4_0, page, dim)
        self.pages = torch.zeros((n_pages, kv_heads, bytes_), dtype=torch.uint8, device="cuda")
        order = rng.permutation(n_pages).astype(np.int32).reshape(sequences, per_seq)
        self.table = torch.from_numpy(order).cuda()
        angle = np.arange(positions)[:, None] * 10000.0 ** (-2.0 * np.arange(dim // 2) / dim)
        self.rope = torch.from_numpy(np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)).cuda()

    def _project(self, w, n_out, x):
        return qk.qk_gemv(qk.QK_TYPE_Q4_K, w, n_out, x.shape[1], qk.qk_quantize_act(qk.QK_TYPE_Q8_K, x), x.shape[0])

    def _append(self, x, cu, start):
        """q, k, v of the rows of x; k and v go to the cache, the rotated q comes back."""
        h, hk, d = self.heads, self.kv_heads, self.dim
        y = self._project(self.w_qkv, (h + 2 * hk) * d, x).view(x.shape[0], h + 2 * hk, d)
        return qk.qk_kv_append(self.pages, self.page, self.table, cu, start, y[:, h:h + hk], y[:, h + hk:], q=y[:, :h],
                               rope=self.rope)

    def cached(self, lengths):
        """k and v of the first lengths[i] positions of each sequence, packed, and where each begins."""
        cu = _int32(np.concatenate([[0], np.cumsum(lengths)]))
        return *qk.qk_kv_read(self.pages, self.page, self.table, cu, torch.zeros_like(cu[1:]), int(sum(lengths)), self.dim), cu

    def chunk(self, x, new, past):
        """Rows x of sequences that have past[i] positions already and get new[i] more."""
        cu = _int32(np.concatenate([[0], np.cumsum(new)]))
        q = self._append(x, cu, _int32(past))
        k, v, cu_k = self.cached([a + b for a, b in zip(new, past)])
        return self._out(qk.qk_attn_prompt(q, k, v, cu, cu_k))

    def step(self, x, cu, start):
        """One row of every sequence; cu and start stay on the device, so a captured graph follows them."""
        q = self._append(x, cu, start)
        return self._out(qk.qk_attn_paged(self.pages, self.page, self.table, cu, start, q)), q

    def _out(self, attended):
        return self._project(self.w_out, self.hidden, attended.flatten(1))


def _int32(values):
    return torch.from_numpy(np.asarray(values, np.int32)).cuda()


def main(hidden=4096, heads=32, kv_heads=8, dim=128, lengths=(700, 93), chunk=256, steps=16):
    torch.manual_seed(0)
    layer = AttentionLayer(hidden, heads, kv_heads, dim, len(lengths), max(lengths) + steps)
    past = [0] * len(lengths)
    while past != list(lengths):
        new = [min(chunk, n - p) for n, p in zip(lengths, past)]
        layer.chunk(torch.randn(sum(new), hidden, device="cuda"), new, past)
        past = [p + m for p, m in zip(past, new)]
    cu, start = _int32(range(len(lengths) + 1)), _int32(lengths)
    for _ in range(steps):
        y, q = layer.step(torch.randn(len(lengths), hidden, device="cuda"), cu, start)
        start += 1
    # the last step once more with the cache read back and attended as a prompt: the same values
    k, v, cu_k = layer.cached([n + steps for n in lengths])
    again = layer._out(qk.qk_attn_prompt(q, k, v, cu, cu_k))
    off = float((y - again).abs().max() / again.abs().max())
    print(f"prompts of {lengths} in chunks of {chunk}, {steps} decode steps; paged against read back: {off:.2g} of the largest output",
          flush=True)
    return off


if __name__ == "__main__":
    main()
