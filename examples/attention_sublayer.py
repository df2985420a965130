"""The attention sub-layer behind an engram layer, as a decoder runs it.

engram_forward updates the FP32 highway; one of its streams then goes through
  engram_residual_norm   (bf16, for the projection)
  engram_project         (query, key and value side by side)
  engram_kv_append       (keys and values to the paged 8-bit cache, rotated; queries rotated in place)
  engram_attention       (over the cache)
  engram_project         (output)
  engram_residual_norm   (adds the output to the stream in place and leaves its norm as e4m3 codes
                          with e8m0 scales, for the sub-layer behind)
for a prompt and then for single tokens.  Synthetic weights; run it with
    python examples/attention_sublayer.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from deepseek_v4_engram_hash_gb300 import _lib as E  # noqa: E402
from deepseek_v4_engram_hash_gb300 import configs  # noqa: E402


class AttentionSublayer:
    """Weights, cache and workspaces of one sub-layer over `batch` sequences of up to `max_seq` tokens."""

    def __init__(self, dim, n_heads, n_kv_heads, head_dim, batch, max_seq, page_tokens=64, rope_dim=None, theta=10000.0,
                 scale_block=32, eps=1e-6, seed=0, device="cuda"):
        self.dim, self.H, self.KH, self.D = dim, n_heads, n_kv_heads, head_dim
        self.batch, self.eps, self.block = batch, eps, scale_block
        g = torch.Generator(device=device).manual_seed(seed)
        width = (n_heads + 2 * n_kv_heads) * head_dim

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).bfloat16()

        self.wqkv, self.wo = weight(width, dim), weight(dim, n_heads * head_dim)
        self.norm_in, self.norm_out = (1 + 0.1 * torch.randn(dim, generator=g, device=device) for _ in range(2))
        rot = head_dim if rope_dim is None else rope_dim
        at = torch.arange(max_seq, device=device, dtype=torch.float64)[:, None]
        f = theta ** (-torch.arange(rot // 2, device=device, dtype=torch.float64) / (rot // 2))
        self.angles = torch.stack([(at * f).cos(), (at * f).sin()], -1).float().contiguous()
        self.rope = E.Rope(self.angles, max_seq, rot)
        # every sequence has its pages; their order in the cache does not matter
        pages = -(-max_seq // page_tokens)
        order = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(seed))
        self.page_table = order.to(torch.int32).view(batch, pages).to(device)
        shape = (batch * pages, n_kv_heads, page_tokens, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in "kv")
        self.k_scales, self.v_scales = (torch.zeros(shape[:2], dtype=torch.uint8, device=device) for _ in "kv")
        self.cache = E.KvCache(self.k, self.v, self.k_scales, self.v_scales, shape[0], n_kv_heads, page_tokens, head_dim)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.attn = E.Attention()
        self._buffers = {}

    def _call(self, T):
        """The batch descriptor and buffers of calls with T tokens a sequence."""
        if T not in self._buffers:
            rows, dev = self.batch * T, self.k.device
            b = {"plan": E.KvBatch(self.page_table, self.kv_len, None, self.batch, self.page_table.shape[1], rows, T),
                 "x": torch.empty(rows, self.dim, dtype=torch.bfloat16, device=dev),
                 "qkv": torch.empty(rows, self.wqkv.shape[0], dtype=torch.bfloat16, device=dev),
                 "o": torch.empty(rows, self.H * self.D, dtype=torch.bfloat16, device=dev),
                 "y": torch.empty(rows, self.dim, dtype=torch.bfloat16, device=dev),
                 "codes": torch.empty(rows, self.dim, dtype=torch.uint8, device=dev),
                 "scales": torch.empty(rows, self.dim // self.block, dtype=torch.uint8, device=dev)}
            self._buffers[T] = b
        return self._buffers[T]

    def forward(self, d_h, stream_no, T):
        """d_h [batch * T, hc, dim] f32: one stream's attention, in place; its norm as (codes, e8m0 scales).  Only enqueues work."""
        b, rows, H, KH, D, BF16 = self._call(T), self.batch * T, self.H, self.KH, self.D, E.ENGRAM_T_BF16
        h, wide = d_h[:, stream_no], d_h.stride(0)
        E.engram_residual_norm(None, BF16, h, E.ENGRAM_T_F32, None, self.norm_in, rows, self.dim, self.eps,
                               E.ENGRAM_FMT_BF16, 0, b["x"], None, res_stride=wide)
        E.engram_project(b["x"], self.wqkv, rows, self.dim, self.wqkv.shape[0], b["qkv"])
        q, k, v = b["qkv"][:, : H * D], b["qkv"][:, H * D: (H + KH) * D], b["qkv"][:, (H + KH) * D:]
        st = b["qkv"].stride(0)
        self.kv_len += T
        E.engram_kv_append(self.cache, b["plan"], BF16, k, st, v, st, q, st, q, st, H, self.rope)
        E.engram_attention(self.attn, self.cache, b["plan"], BF16, q, st, H, D ** -0.5, 0, b["o"], 0)
        E.engram_project(b["o"], self.wo, rows, H * D, self.dim, b["y"])
        E.engram_residual_norm(b["y"], BF16, h, E.ENGRAM_T_F32, h, self.norm_out, rows, self.dim, self.eps,
                               E.ENGRAM_FMT_FP8_E8M0, self.block, b["codes"], b["scales"], res_stride=wide)
        return b["codes"], b["scales"]


def main():
    from deepseek_v4_engram_hash_gb300 import runner, synth
    import numpy as np
    import __graft_entry__
    __graft_entry__.build()
    cfg = configs.V41_DECODE
    prompt, steps = 512, 8
    eng = runner.EngramSetup(cfg, batch=1, max_tokens=prompt)
    sub = AttentionSublayer(cfg.dim, 32, 8, 128, batch=1, max_seq=prompt + steps)
    pos = 0
    for T in [prompt] + [1] * steps:
        ids = eng.ids_for(f"attention{pos}", T)
        d_h = torch.from_numpy(synth.highway(cfg, np.arange(pos, pos + T))).cuda()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        eng.forward(ids, pos, d_h)
        begin.record()
        codes, scales = sub.forward(d_h, 0, T)
        end.record()
        rc = E.engram_check()
        assert rc == 0, E.strerror(rc)
        print(f"{T} token(s) at {pos}: sub-layer {begin.elapsed_time(end) * 1e3:.0f} us, |h| {d_h[:, 0].norm().item():.3f}, "
              f"codes {tuple(codes.shape)}, scales {tuple(scales.shape)}")
        pos += T


if __name__ == "__main__":
    main()
