"""The experts' sub-layer behind an engram layer and its attention, as a decoder runs it.

The attention sub-layer leaves the norm of its stream as e4m3 codes with a power-of-two scale for
each 128 of a row; these go through
  engram_project_fp8     (router: logits in f32)
  engram_route           (experts and weights of every token, and the lists of pairs by expert)
  engram_glu_fp8         (the experts' gated products, rows gathered by the lists, output in 8 bits)
  engram_project_fp8     (their second products, by pair)
  engram_glu_fp8, engram_project_fp8   (the shared expert: the same without lists)
  engram_combine         (the weighted sum, onto the shared expert's output)
  engram_residual_norm   (adds it to the stream in place and leaves the next block's norm)
Synthetic weights; run it with
    python examples/experts_sublayer.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from deepseek_v4_engram_hash_gb300 import _lib as E  # noqa: E402
from deepseek_v4_engram_hash_gb300 import configs  # noqa: E402

BLOCK = 128


def fp8_weight(w, gated=False):
    """w [n_experts, parts, n, k] f32 -> (descriptor, codes, e8m0 scales): one power of two for each 128 x 128."""
    n_experts, parts, n, k = w.shape
    p = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK)).view(n_experts, parts, -(-n // BLOCK), BLOCK, -(-k // BLOCK), BLOCK)
    m, e = torch.frexp(p.abs().amax((3, 5)))
    e = torch.where(m <= 0.875, e - 9, e - 8)                  # the smallest e with amax <= 448 * 2^e
    codes = torch.ldexp(p, -e[:, :, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = codes.view(n_experts, parts, -(-n // BLOCK) * BLOCK, -1)[:, :, :n, :k].contiguous()
    scales = (e + 127).to(torch.uint8)
    return E.Fp8Weight(codes, scales, E.ENGRAM_FMT_FP8_E8M0, n_experts, n, k, gated), codes, scales


class ExpertsSublayer:
    """Weights and buffers for calls of up to `max_tokens` tokens."""

    def __init__(self, dim, inter, n_experts, top_k, shared_inter, max_tokens, n_groups=8, top_groups=4, scale=2.5, limit=0.0,
                 eps=1e-6, seed=0, device="cuda"):
        self.dim, self.inter, self.shared_inter, self.n_experts, self.top_k = dim, inter, shared_inter, n_experts, top_k
        self.limit, self.eps = limit, eps
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n_mats, parts, n, k):
            w = torch.randn(n_mats, parts, n, k, generator=g, device=device) * k ** -0.5
            return fp8_weight(w, parts == 2)

        self.gate = weight(1, 1, n_experts, dim)
        self.up, self.down = weight(n_experts, 2, inter, dim), weight(n_experts, 1, dim, inter)
        self.shared_up, self.shared_down = weight(1, 2, shared_inter, dim), weight(1, 1, dim, shared_inter)
        self.bias = 0.01 * torch.randn(n_experts, generator=g, device=device)
        self.norm = 1 + 0.1 * torch.randn(dim, generator=g, device=device)
        self.router = E.Router(n_experts, top_k, E.ENGRAM_SCORE_SIGMOID, n_groups, top_groups, 2, True, scale)
        pairs = max_tokens * top_k

        def empty(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=device)

        self.logits = empty(max_tokens, n_experts, dtype=torch.float32)
        self.ids, self.weights = empty(max_tokens, top_k, dtype=torch.int32), empty(max_tokens, top_k, dtype=torch.float32)
        self.offsets, self.pairs = empty(n_experts + 1, dtype=torch.int32), empty(pairs, dtype=torch.int32)
        self.ws_bytes = max(E.engram_route_workspace_bytes(n_experts, t) for t in (max_tokens, min(max_tokens, 8192)))
        self.ws = empty(max(1, self.ws_bytes), dtype=torch.uint8)
        self.a, self.a_scales = empty(pairs, inter, dtype=torch.uint8), empty(pairs, -(-inter // BLOCK), dtype=torch.uint8)
        self.b, self.b_scales = empty(max_tokens, shared_inter, dtype=torch.uint8), empty(max_tokens, -(-shared_inter // BLOCK), dtype=torch.uint8)
        self.y, self.out = empty(pairs, dim, dtype=torch.bfloat16), empty(max_tokens, dim, dtype=torch.bfloat16)
        self.next = empty(max_tokens, dim, dtype=torch.bfloat16)

    def forward(self, codes, scales, T, h=None):
        """codes [T, dim] and e8m0 scales [T, dim / 128] of T tokens -> their outputs [T, dim] bf16; added to h [T, dim] f32 (rows
        h.stride(0) apart) in place where it is given.  Only enqueues work."""
        fmt, k, dim = E.ENGRAM_FMT_FP8_E8M0, self.top_k, self.dim
        lists = E.ExpertLists(self.offsets, self.pairs, self.n_experts, k, T)
        E.engram_project_fp8(codes, 0, scales, fmt, T, self.gate[0], None, E.ENGRAM_T_F32, self.logits, 0)
        E.engram_route(self.router, E.ENGRAM_T_F32, self.logits, 0, self.bias, T, self.ids, self.weights, lists, self.ws, self.ws_bytes)
        E.engram_glu_fp8(codes, 0, scales, fmt, T, self.up[0], lists, self.limit, fmt, self.a, self.a_scales)
        E.engram_project_fp8(self.a, 0, self.a_scales, fmt, T * k, self.down[0], lists, E.ENGRAM_T_BF16, self.y, 0)
        E.engram_glu_fp8(codes, 0, scales, fmt, T, self.shared_up[0], None, self.limit, fmt, self.b, self.b_scales)
        E.engram_project_fp8(self.b, 0, self.b_scales, fmt, T, self.shared_down[0], None, E.ENGRAM_T_BF16, self.out, 0)
        E.engram_combine(self.y, E.ENGRAM_T_BF16, 0, self.weights, T, k, dim, self.out, E.ENGRAM_T_BF16, 0, E.ENGRAM_T_BF16, self.out, 0)
        if h is not None:
            E.engram_residual_norm(self.out, E.ENGRAM_T_BF16, h, E.ENGRAM_T_F32, h, self.norm, T, dim, self.eps, E.ENGRAM_FMT_BF16, 0,
                                   self.next, None, res_stride=h.stride(0))
        return self.out[:T]


def main():
    import numpy as np
    import __graft_entry__
    __graft_entry__.build()
    from deepseek_v4_engram_hash_gb300 import runner, synth
    from examples.attention_sublayer import AttentionSublayer
    cfg = configs.V41_DECODE
    prompt, steps = 512, 8
    eng = runner.EngramSetup(cfg, batch=1, max_tokens=prompt)
    attention = AttentionSublayer(cfg.dim, 32, 8, 128, batch=1, max_seq=prompt + steps, scale_block=BLOCK)
    experts = ExpertsSublayer(cfg.dim, 1024, 64, 8, 2048, max_tokens=prompt)
    pos = 0
    for T in [prompt] + [1] * steps:
        ids = eng.ids_for(f"experts{pos}", T)
        d_h = torch.from_numpy(synth.highway(cfg, np.arange(pos, pos + T))).cuda()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        eng.forward(ids, pos, d_h)
        codes, scales = attention.forward(d_h, 0, T)
        begin.record()
        experts.forward(codes, scales, T, d_h[:, 0])
        end.record()
        rc = E.engram_check()
        assert rc == 0, E.strerror(rc)
        print(f"{T} token(s) at {pos}: experts {begin.elapsed_time(end) * 1e3:.0f} us, |h| {d_h[:, 0].norm().item():.3f}, "
              f"{int((experts.offsets.diff() > 0).sum())} of {experts.n_experts} experts used")
        pos += T


if __name__ == "__main__":
    main()
