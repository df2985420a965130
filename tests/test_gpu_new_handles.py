"""A handle is ready on every stream when its create returns, whatever the default stream is still doing."""
import pytest
import torch

import sublayer_glue as U
import test_gpu_attention as A
from deepseek_v4_engram_hash_gb300 import configs, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    import __graft_entry__
    __graft_entry__.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    assert torch.cuda.is_available()
    return _lib


def _leave_old_bytes():
    """Device memory of small and large allocations goes back to the driver full of ones."""
    old = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in [1 << 8] * 64 + [1 << 22] * 16]
    torch.cuda.synchronize()
    del old
    torch.cuda.empty_cache()


def _busy_default_stream(ms=200):
    """Work of some `ms` on the default stream, which the host does not wait for."""
    torch.cuda._sleep(int(ms * 1e6))                       # about 1.9e6 clocks a ms at most, so no less than half of it


@pytest.mark.parametrize("new", [1, 40])
def test_attention_on_a_new_workspace(E, new):
    """Split rows on a non-blocking stream, at once after the create: all counters are zero, as on a used workspace."""
    KH, H, D, pt, n = 2, 8, 128, 64, 20000
    table = U.pages_for([n], pt, 320)
    cache = U.Cache(E, 320, KH, pt, D)
    U.fill_random(cache, table, [n], 3)
    q = A._queries(new, H, D, 0, 5)
    plan = U.batch(E, table, [new], [n])
    out, lse = torch.zeros_like(q), torch.zeros(new, H, device="cuda")
    want = A._run(E, E.Attention(), cache, plan, q, H, 0.1, 0, 0)
    side = torch.cuda.Stream()
    _leave_old_bytes()
    E.Attention().close()                                   # modules are loaded; its memory is free again
    _busy_default_stream()
    attn = E.Attention()
    E.engram_attention(attn, cache.desc, plan, 0, q, 0, H, 0.1, 0, out, 0, lse, stream=side)
    assert E.engram_check(side) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_hash_on_a_new_hasher(E):
    """Positions behind tokens that were never hashed look back on zeros, on a non-blocking stream at once after the create."""
    cfg = configs.TINY
    t = synth.hash_tables(cfg)
    g = E.make_geom(cfg.n_layers, cfg.max_ngram, cfg.n_heads, cfg.head_dim, cfg.dim, cfg.hc, cfg.scale_block, cfg.vocab)
    tabs = E.Tables(g, t["token_map"], t["pad_token_id"], t["multipliers"], t["primes"], t["offsets"])
    d_ids = torch.from_numpy(synth.token_ids(cfg, "new-hasher", 5)[None]).cuda()
    want, got = (torch.zeros((1, 5, cfg.n_layers, cfg.cols), dtype=torch.int64, device="cuda") for _ in range(2))
    settled = E.Hasher(tabs, 1, 4096)
    torch.cuda.synchronize()
    E.engram_hash(settled, d_ids, 5, 7, want)
    side = torch.cuda.Stream()
    _leave_old_bytes()
    _busy_default_stream()
    hs = E.Hasher(tabs, 1, 4096)
    E.engram_hash(hs, d_ids, 5, 7, got, stream=side)
    assert E.engram_check(side) == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want)
