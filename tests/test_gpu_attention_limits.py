"""engram_attention at the ends of its ranges, against its definition in 64 bits.

test_gpu_attention.py has the bounds of ordinary inputs; here the inputs are such
that a tighter one can be derived, which each test does.
"""
import math

import pytest
import torch

import sublayer_glue as U
import sublayer_ref as R
import test_gpu_attention as A

pytestmark = pytest.mark.gpu
LN2 = float(torch.tensor(math.log(2.0), dtype=torch.float32))    # times log2(e): 1 to within 2^-24


@pytest.fixture(scope="module")
def E():
    import __graft_entry__
    __graft_entry__.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    assert torch.cuda.is_available()
    return _lib


@pytest.fixture(scope="module")
def attn(E):
    return E.Attention()


@pytest.mark.parametrize("new", [1, 20])
def test_weights_far_under_the_largest_count(E, attn, new):
    """One token of weight 1 and value 0, all others of weight 2^-28 and value 1: out = m 2^-28 / (1 + m 2^-28) for m others.

    The scores in log2 units are whole to within 2^-24 of 28; with a bound at least 4 under the row's largest the weights
    are multiples of f16's least number, 2^-24, so out keeps 2^-10 of itself before it is rounded to bf16.  With the
    bound at the largest they would be 0 in the product and not in the sum."""
    KH, D, pt, n = 304, 64, 128, 2048                     # as many heads as it takes for whole sequences on one SM
    table = U.pages_for([n], pt, 16)
    cache = U.Cache(E, 16, KH, pt, D, fill=0, scale=127)
    cache.k[:, :, :, 0] = 0xDE                            # -28
    cache.v.fill_(0x38)                                   # 1
    first = int(table[0, 0])
    cache.k[first, :, 0, 0], cache.v[first, :, 0] = 0, 0
    q = torch.zeros(new, KH, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    out, lse = A._run(E, attn, cache, U.batch(E, table, [new], [n]), q.view(new, -1), KH, LN2, 0, 0)
    others = torch.arange(n - new, n, device="cuda", dtype=torch.float64)[:, None]
    want = others * 2.0 ** -28 / (1 + others * 2.0 ** -28)
    got = out.double()
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want).all(), (got.min(), got.max())
    assert ((lse.double() - torch.log1p(others * 2.0 ** -28)).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("pt", [16, 32, 64, 128])
@pytest.mark.parametrize("H,new,D,ty", [(4, 1, 128, 0), (6, 5, 64, 1), (16, 40, 128, 0), (2, 300, 64, 0)])
def test_nothing_behind_the_window_is_read(E, attn, H, new, D, ty, pt):
    """Pages that no row sees may be given back: their entries hold anything, their bytes and those before the first
    visible token of a page are NaN.  No error, and the same bits."""
    KH, window = 2, 100
    kv = [1337, 333, 1025]
    news = [new, min(new, 333), max(1, new // 2)]
    table = U.pages_for(kv, pt, sum(-(-t // pt) for t in kv) + 1, seed=pt)
    cache = U.Cache(E, sum(-(-t // pt) for t in kv) + 1, KH, pt, D)
    free = (set(range(cache.n_pages)) - set(table.flatten().tolist())).pop()
    U.fill_random(cache, table, kv, 3)
    q = A._queries(sum(news), H, D, ty, 5)
    want = A._run(E, attn, cache, U.batch(E, table, news, kv), q, H, 0.1, window, ty)
    A._check(cache, table, news, kv, q, H, 0.1, window, ty, *want)
    for b, (n, t) in enumerate(zip(news, kv)):
        first = max(0, t - n - window + 1)
        for i in range(first // pt):
            page = int(table[b, i])
            for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
                codes[page], scales[page] = 127, 255
            table[b, i] = (-7, cache.n_pages, 1 << 30, free, page)[i % 5]
        if first % pt:
            page = int(table[b, first // pt])
            cache.k[page, :, : first % pt], cache.v[page, :, : first % pt] = 127, 255
    got = A._run(E, attn, cache, U.batch(E, table, news, kv), q, H, 0.1, window, ty)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,new", [(4, 1), (16, 40)])
@pytest.mark.parametrize("vbyte", [61, 127, 247, 253, 254])
def test_every_value_scale_up_to_the_largest(E, attn, H, new, vbyte):
    """Value blocks of one scale, up to 2^127: outputs are those of scale 1 times it, and the log-sum-exp is the same."""
    KH, D, pt, n = 2, 64, 16, 200
    table = U.pages_for([n], pt, 14)
    cache = U.Cache(E, 14, KH, pt, D)
    U.fill_random(cache, table, [n], 3, spread=0)
    cache.v.copy_(torch.where(cache.v & 127 == 127, cache.v, cache.v & 0xB7))    # under 2: no output past bf16's range
    q = A._queries(new, H, D, 0, 5)
    plan = U.batch(E, table, [new], [n])
    cache.vs.fill_(vbyte)
    out, lse = A._run(E, attn, cache, plan, q, H, 0.1, 0, 0)
    A._check(cache, table, [new], [n], q, H, 0.1, 0, 0, out, lse)
