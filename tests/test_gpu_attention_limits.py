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


@pytest.mark.parametrize("H,KH,D,pt,new,kv", [(8, 2, 128, 16, [1, 1, 1], [900, 33, 130]), (4, 1, 64, 64, [3], [700]),
                                              (8, 2, 128, 64, [70, 5], [300, 290]), (16, 1, 64, 16, [257], [600])])
@pytest.mark.parametrize("down", [0, 6])
def test_large_scores_with_exact_products(E, attn, H, KH, D, pt, new, kv, down):
    """Whole-number queries and keys: every sum of products is a whole number under 2^24, so it is exact in any order.

    With scale = ln 2 2^-down the scores in log2 units are whole multiples of 2^-down (up to thousands) to within the
    roundings of the scale, of the sum with the value's exponent, of the bound and of the differences with it: under
    6 x 2^-24 T, T the largest |t|.  So a weight is right to 2^-22 T, and its quotient by the sum to 2^-21 T, to 2^-20
    (the exponentials) and to 2^-11 (f16), or to 2^-32 of the largest where f16 has no more bits; sums are f32."""
    scale = LN2 * 2.0 ** -down
    table = U.pages_for(kv, pt, sum(-(-t // pt) for t in kv) + 2)
    cache = U.Cache(E, sum(-(-t // pt) for t in kv) + 2, KH, pt, D)
    U.fill_random(cache, table, kv, 3)
    g = torch.Generator(device="cuda").manual_seed(7)
    whole = torch.randint(-8, 9, cache.k.shape, generator=g, device="cuda").float().to(torch.float8_e4m3fn).view(torch.uint8)
    cache.k.copy_(torch.where(cache.k & 127 == 127, cache.k, whole))             # what no token holds stays NaN
    cache.ks.copy_(torch.where(cache.ks == 255, cache.ks, torch.full_like(cache.ks, 127)))
    q = (torch.randint(-8, 9, (sum(new), H * D), generator=g, device="cuda") * 8).bfloat16()
    out, lse = A._run(E, attn, cache, U.batch(E, table, new, kv), q, H, scale, 0, 0)
    row = 0
    for b, (n, t) in enumerate(zip(new, kv)):
        k, v = U.sequence_tokens(R, cache, table, b, t)
        pos = torch.arange(t - n, t, device="cuda")
        qs = q[row: row + n].double().view(n, H, D)
        want, wl, mass, _, big = R.attention(qs, k, v, pos, scale, 0)
        T = 16 + max(float((qs[:, h] @ k[:, h // (H // KH)].T).abs().max()) for h in range(H)) * 2.0 ** -down
        got, gl = out[row: row + n].double().view(n, H, D), lse[row: row + n].double()
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -20 * T) * mass + (t * 2.0 ** -31 + 2.0 ** -22) * big[..., None]
        assert ((got - want).abs() <= tol).all(), (b, T, ((got - want).abs() / tol.clamp(min=1e-30)).max())
        assert ((gl - wl).abs() <= 2.0 ** -21 * T + 2.0 ** -20 * (1 + wl.abs())).all()
        row += n


@pytest.mark.parametrize("ty", [0, 1])
def test_prompt_and_chunks_leave_the_same_pages_and_outputs(E, attn, ty):
    """96 tokens at once and as 64 + 31 + 1 from the same inputs: the two pages that the first chunk fills are equal bit
    for bit, and each output is within its bound of the 64-bit one over its own cache."""
    KH, H, D, pt, n = 2, 8, 128, 32, 96
    table = U.pages_for([n], pt, 4)
    w = A._queries(n, H + 2 * KH, D, ty, 4)
    st = w.stride(0)
    caches = []
    for parts in ((96,), (64, 31, 1)):
        cache = U.Cache(E, 4, KH, pt, D)
        at = 0
        for T in parts:
            x = w[at: at + T]
            q, k, v = x[:, : H * D], x[:, H * D: (H + KH) * D], x[:, (H + KH) * D:]
            plan = U.batch(E, table, [T], [at + T])
            E.engram_kv_append(cache.desc, plan, ty, k, st, v, st, None, 0, None, 0, 0)
            out, lse = torch.empty(T, H * D, dtype=w.dtype, device="cuda"), torch.empty(T, H, device="cuda")
            E.engram_attention(attn, cache.desc, plan, ty, q, st, H, D ** -0.5, 0, out, 0, lse)
            assert E.engram_check() == 0
            A._check(cache, table, [T], [at + T], q, H, D ** -0.5, 0, ty, out, lse)
            at += T
            if at == 64:
                first = [c[table[0, :2].long()].clone() for c in cache.tensors()]
        caches.append(cache)
    for one, chunked in zip(caches[0].tensors(), first):
        assert torch.equal(one[table[0, :2].long()], chunked)


@pytest.mark.parametrize("H,new", [(4, 1), (16, 40)])
@pytest.mark.parametrize("apart", [60, 100])
def test_value_scales_far_apart(E, attn, H, new, apart):
    """Value blocks of one sequence up to 2^100 apart, the smallest at 2^-66: the small ones keep their whole weight."""
    KH, D, pt, n = 2, 128, 16, 160
    table = U.pages_for([n], pt, 12)
    cache = U.Cache(E, 12, KH, pt, D)
    U.fill_random(cache, table, [n], 3, spread=0)
    for i, p in enumerate(table[0].tolist()):
        cache.vs[p] = 61 + (apart if i % 2 else 0)
    q = A._queries(new, H, D, 0, 5)
    out, lse = A._run(E, attn, cache, U.batch(E, table, [new], [n]), q, H, 0.09, 0, 0)
    A._check(cache, table, [new], [n], q, H, 0.09, 0, 0, out, lse)
