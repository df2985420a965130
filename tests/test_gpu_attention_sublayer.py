"""The attention sub-layer's operators together, as examples/attention_sublayer.py
runs them behind an engram: the highway after a prompt and after single tokens
against the same steps in 64 bits.

The cache's own codes are taken for the keys and values (their bits are tested
by themselves); of the rest every step rounds to bf16 once (2^-8): x, q k v, the
rotated queries, the attention's output and the output projection, whose
errors add up under the final sum's 4 x 2^-8 of the largest y, with the
attention's own bound below one more.
"""
import os
import sys

import numpy as np
import pytest
import torch

import sublayer_ref as R
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    import __graft_entry__
    __graft_entry__.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    assert torch.cuda.is_available()
    return _lib


def _example():
    path = os.path.join(ROOT, "examples")
    if path not in sys.path:
        sys.path.insert(0, path)
    import attention_sublayer
    return attention_sublayer


@pytest.mark.parametrize("batch,dim,H,KH,D,pt,steps", [
    (1, 128, 4, 2, 64, 16, (16, 1, 1)),
    (3, 256, 8, 2, 64, 32, (5, 1, 40, 2, 1)),           # a second chunk behind cached tokens
    (2, 512, 4, 4, 128, 64, (70, 1)),
])
def test_sublayer_matches_64_bits(E, batch, dim, H, KH, D, pt, steps):
    ex = _example()
    hc, stream_no = 2, 1
    sub = ex.AttentionSublayer(dim, H, KH, D, batch, sum(steps), page_tokens=pt, seed=batch)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = 0
    for T in steps:
        h0 = torch.randn(batch * T, hc, dim, generator=g, device="cuda")
        d_h = h0.clone()
        codes, scales = sub.forward(d_h, stream_no, T)
        assert E.engram_check() == 0
        assert torch.equal(d_h[:, 0], h0[:, 0])
        h = h0[:, stream_no].double()
        x = h / torch.sqrt(h.square().mean(1, keepdim=True) + sub.eps) * sub.norm_in.double()
        q = (x @ sub.wqkv.double().T)[:, : H * D].view(batch, T, H, D)
        k, v = (R.dequant(c, s)[sub.page_table.long()].permute(0, 1, 3, 2, 4).reshape(batch, -1, KH, D)
                for c, s in ((sub.k, sub.k_scales), (sub.v, sub.v_scales)))
        at = torch.arange(pos, pos + T, device="cuda")
        o = torch.stack([R.attention(R.rotate(q[b], sub.angles, at, D, False), k[b, : pos + T], v[b, : pos + T], at, D ** -0.5, 0)[0]
                         for b in range(batch)]).view(batch * T, H * D)
        y = o @ sub.wo.double().T
        want = h + y
        assert ((d_h[:, stream_no].double() - want).abs() <= 5 * 2.0 ** -8 * y.abs().amax()).all()
        r = d_h[:, stream_no].double()
        n = r / torch.sqrt(r.square().mean(1, keepdim=True) + sub.eps) * sub.norm_out.double()
        n = n.view(batch * T, -1, sub.block)
        s = R.pow2(scales.int() - 127)[..., None]
        assert (n.abs().amax(2) <= 448 * s[..., 0]).all()
        got = R.e4m3_values().cuda()[codes.long()].view_as(n) * s
        assert ((got - n).abs() <= 0.5 * R.e4m3_step(n / s) * s * (1 + 1e-9) + 2.5e-6 * n.abs()).all()
        pos += T


def test_prompt_equals_its_chunks(E):
    """A prompt at once and in chunks: the same positions see the same tokens; only block scales that grew in between round differently."""
    ex = _example()
    outs = []
    g = torch.Generator(device="cuda").manual_seed(5)
    h0 = torch.randn(96, 1, 256, generator=g, device="cuda")
    for parts in ((96,), (64, 31, 1)):
        sub = ex.AttentionSublayer(256, 4, 2, 64, 1, 96, page_tokens=32, seed=9)
        rows, at = [], 0
        for T in parts:
            d_h = h0[at: at + T].clone()
            sub.forward(d_h, 0, T)
            rows.append(d_h)
            at += T
        outs.append(torch.cat(rows))
    assert E.engram_check() == 0
    y = (outs[0] - h0).abs().amax()
    assert (outs[0] - outs[1]).abs().max() <= y / 8          # a code's own rounding is 2^-4 of it
    assert torch.equal(outs[0][:64], outs[1][:64]) or (outs[0][:64] - outs[1][:64]).abs().max() <= y / 8
    assert np.isfinite(outs[1].cpu().numpy()).all()
