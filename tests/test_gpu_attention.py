"""engram_attention against its definition in 64 bits.

Bounds, from the arithmetic (A = sum_j p_j |v_j| of an output element, B the
row's largest sum |q k| scale): q and the codes enter the products exactly (q
but for 2^-24 of its largest element), the D products of a score are summed in
f32 (error 2^-17 B for D <= 128, taken as 2^-16 B with the exponent's own
rounding); the probabilities are rounded to f16 (2^-11, or 2^-25 of the bound M
under its normal range, where M is at most 8 binary orders over the largest); sums in
f32; the output is rounded to its type.  So
  |out - want| <= u |want| + (2^-10 + 2^-15 B) A + n 2^-23 max|v|,  u = 2^-8 (bf16: 8 significant bits), 2^-11 (f16: 11),
  |lse - want| <= 2^-16 B + 2^-20 (1 + |want|).
"""
import math

import pytest
import torch

import sublayer_glue as U
import sublayer_ref as R

pytestmark = pytest.mark.gpu


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


def _queries(rows, H, D, ty, seed, mag=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mag * torch.randn(rows, H * D, generator=g, device="cuda")).to(U.DTYPES[ty])


def _run(E, attn, cache, plan, q, H, scale, window, ty, rc=0, stream=None):
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    E.engram_attention(attn, cache.desc, plan, ty, q, q.stride(0) if q.shape[0] > 1 else 0, H, scale, window, out, 0, lse,
                       stream=stream)
    assert E.engram_check(stream) == rc
    return out, lse


def _check(cache, table, new, kv, q, H, scale, window, ty, out, lse):
    D, row = cache.D, 0
    u = 2.0 ** -8 if ty == 0 else 2.0 ** -11
    for b, (n, t) in enumerate(zip(new, kv)):
        k, v = U.sequence_tokens(R, cache, table, b, t)
        pos = torch.arange(t - n, t, device="cuda")
        want, wl, mass, reach, big = R.attention(q[row: row + n].double().view(n, H, D), k, v, pos, scale, window)
        got, gl = out[row: row + n].double().view(n, H, D), lse[row: row + n].double()
        tol = (u * want.abs() + (2.0 ** -10 + 2.0 ** -15 * reach)[..., None] * mass + t * 2.0 ** -23 * big[..., None]
               + (2.0 ** -24 if ty == 1 else 0))
        assert ((got - want).abs() <= tol).all(), (b, ((got - want).abs() / tol.clamp(min=1e-30)).max())
        some = torch.isfinite(wl)
        assert (gl[~some] == -math.inf).all() and (got[~some] == 0).all()
        assert ((gl - wl).abs()[some] <= (2.0 ** -16 * reach + 2.0 ** -20 * (1 + wl.abs()))[some]).all()
        row += n


def _case(E, attn, new, kv, H, KH, D, pt, ty, window=0, seed=0, mag=1.0, spread=2, uniform=False):
    n_pages = sum(-(-n // pt) for n in kv) + 3
    table = U.pages_for(kv, pt, n_pages, seed)
    cache = U.Cache(E, n_pages, KH, pt, D)                 # NaN everywhere but in the sequences' tokens
    U.fill_random(cache, table, kv, seed + 1, spread)
    q = _queries(sum(new), H, D, ty, seed + 2, mag)
    plan = U.batch(E, table, new, kv, uniform=uniform)
    scale = D ** -0.5
    out, lse = _run(E, attn, cache, plan, q, H, scale, window, ty)
    _check(cache, table, new, kv, q, H, scale, window, ty, out, lse)


@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 1000, 4097])
@pytest.mark.parametrize("D,pt", [(128, 16), (64, 128)])
def test_one_token(E, attn, kv, D, pt):
    _case(E, attn, [1], [kv], 8, 2, D, pt, 0, seed=kv)


@pytest.mark.parametrize("H,KH", [(1, 1), (4, 4), (5, 1), (16, 1), (17, 1), (40, 2), (64, 1), (24, 8)])
def test_head_layouts(E, attn, H, KH):
    _case(E, attn, [1, 2], [300, 77], H, KH, 128, 32, 1, seed=H)


@pytest.mark.parametrize("new,kv,H,KH,D,pt,ty,window", [
    ([1] * 33, [1 + 40 * i for i in range(33)], 8, 2, 128, 16, 0, 0),
    ([2, 1, 4, 3], [2, 900, 64, 130], 4, 1, 64, 64, 1, 0),
    ([5], [5], 8, 8, 128, 16, 0, 0),
    ([130], [130], 4, 2, 128, 64, 0, 0),                  # a prompt
    ([257], [700], 8, 1, 64, 32, 1, 0),                   # a chunk behind a prefix
    ([300, 1, 64, 17], [301, 500, 64, 1200], 6, 2, 128, 128, 0, 0),
    ([1, 90], [700, 400], 8, 2, 128, 16, 0, 100),         # sliding windows
    ([200], [600], 4, 4, 64, 16, 1, 1),                   # each token sees itself alone
    ([128, 129, 127], [128, 1000, 511], 16, 8, 64, 64, 0, 333),
    ([1] * 3, [5000, 4000, 17], 32, 8, 128, 64, 1, 2048),
    ([600], [2000], 20, 4, 128, 32, 0, 0),
])
def test_batches(E, attn, new, kv, H, KH, D, pt, ty, window):
    _case(E, attn, new, kv, H, KH, D, pt, ty, window, seed=len(new) + kv[0])


def test_uniform_batch_without_row_start(E, attn):
    _case(E, attn, [3] * 5, [3, 40, 64, 200, 1000], 8, 2, 128, 16, 0, uniform=True)


def test_large_scores(E, attn):
    """Scores in the hundreds: one token takes nearly everything, others vanish."""
    _case(E, attn, [1, 70], [800, 300], 8, 2, 128, 16, 0, mag=40.0)
    _case(E, attn, [1], [800], 4, 4, 64, 16, 1, mag=2000.0)


def test_small_and_zero_queries(E, attn):
    _case(E, attn, [1, 20], [100, 50], 8, 2, 128, 16, 0, mag=1e-20)
    _case(E, attn, [1, 20], [100, 50], 8, 2, 128, 16, 0, mag=0.0)


def test_scales_far_apart(E, attn):
    """Blocks of one head 2^40 apart: an output keeps the relative precision of what it attends to."""
    _case(E, attn, [1, 100], [640, 200], 4, 2, 128, 16, 0, spread=20, mag=2.0 ** -12)
    _case(E, attn, [1], [640], 4, 2, 64, 16, 0, spread=20, mag=2.0 ** -12)


def test_blocks_of_zeros_keep_their_weight(E, attn):
    """Values of zero (least scale) beside ordinary ones still count in the sum."""
    KH, H, D, pt, n = 2, 4, 128, 16, 160
    table = U.pages_for([n], pt, 12)
    cache = U.Cache(E, 12, KH, pt, D)
    U.fill_random(cache, table, [n], 3)
    for p in table[0, ::2].tolist():
        cache.v[p], cache.vs[p] = 0, 1
    q = _queries(1, H, D, 0, 5)
    out, lse = _run(E, attn, cache, U.batch(E, table, [1], [n]), q, H, 0.09, 0, 0)
    _check(cache, table, [1], [n], q, H, 0.09, 0, 0, out, lse)


@pytest.mark.parametrize("H,new", [(4, 1), (16, 40)])
def test_rows_that_see_nothing(E, attn, H, new):
    """Idle slots (no tokens, or fewer than rows): zeros and -inf, whatever the cache holds; their neighbours unaffected."""
    KH, D, pt = 2, 64, 16
    kv = [0, 50, new // 2, 0]
    table = U.pages_for(kv, pt, 12, width=4)
    cache = U.Cache(E, 12, KH, pt, D)
    U.fill_random(cache, table, kv, 3)
    news = [new, min(new, 50), new, 0]
    q = _queries(sum(news), H, D, 0, 5)
    out, lse = _run(E, attn, cache, U.batch(E, table, news, kv), q, H, 0.125, 0, 0)
    _check(cache, table, news, kv, q, H, 0.125, 0, 0, out, lse)
    assert (out[:new] == 0).all() and (lse[:new] == -math.inf).all()


@pytest.mark.parametrize("H,new", [(4, 1), (16, 40)])
def test_bad_lengths_and_pages_are_reported(E, attn, H, new):
    """A length past the table or below zero, falling row starts, a page outside the cache: reported, and nothing
    else changes; the tokens of a bad page are not seen."""
    KH, D, pt = 2, 128, 16
    kv = [60, 70, 80]
    news = [new] * 3
    table = U.pages_for(kv, pt, 20, width=5)
    cache = U.Cache(E, 20, KH, pt, D)
    U.fill_random(cache, table, kv, 3)
    q = _queries(3 * new, H, D, 0, 5)
    good = _run(E, attn, cache, U.batch(E, table, news, kv), q, H, 0.1, 0, 0)
    for lens in ([60, 81, 80], [60, -5, 80]):
        out, lse = _run(E, attn, cache, U.batch(E, table, news, lens), q, H, 0.1, 0, 0, rc=-14)
        assert (out[new: 2 * new] == 0).all() and (lse[new: 2 * new] == -math.inf).all()
        for a, b in ((out, good[0]), (lse, good[1])):
            assert torch.equal(a[:new], b[:new]) and torch.equal(a[2 * new:], b[2 * new:])
    plan = U.batch(E, table, news, kv)
    plan.start.copy_(torch.tensor([0, new, 0, 3 * new + 1], dtype=torch.int32))
    out, lse = _run(E, attn, cache, plan, q, H, 0.1, 0, 0, rc=-14)
    assert torch.equal(out[:new], good[0][:new]) and (out[new:] == 7).all()
    # a page in the middle of sequence 1: as if its 16 tokens were not there
    for bad in (-3, 20, 1 << 30):
        tab = table.clone()
        tab[1, 1] = bad
        out, lse = _run(E, attn, cache, U.batch(E, tab, news, kv), q, H, 0.1, 0, 0, rc=-13)
        assert torch.equal(out[:new], good[0][:new]) and torch.equal(out[2 * new:], good[0][2 * new:])
        k, v = U.sequence_tokens(R, cache, table, 1, 70)
        keep = torch.tensor([i for i in range(70) if i // 16 != 1], device="cuda")
        at = torch.arange(70 - new, 70, device="cuda")
        for i in range(new):
            seen = keep[keep <= at[i]]
            want, wl, mass, reach, big = R.attention(q[new + i: new + i + 1].double().view(1, H, D), k[seen], v[seen],
                                                     torch.tensor([10 ** 6], device="cuda"), 0.1, 0)
            got = out[new + i].double().view(1, H, D)
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -15 * reach)[..., None] * mass + 70 * 2.0 ** -23 * big[..., None]
            assert ((got - want).abs() <= tol).all()
            assert ((lse[new + i].double() - wl).abs() <= 2.0 ** -16 * reach + 2.0 ** -20 * (1 + wl.abs())).all()


@pytest.mark.parametrize("H,new", [(4, 1), (16, 40)])
def test_nan_blocks_reach_only_the_rows_that_see_them(E, attn, H, new):
    KH, D, pt, window, n = 2, 64, 16, 24, 96
    table = U.pages_for([n], pt, 8)
    cache = U.Cache(E, 8, KH, pt, D)
    U.fill_random(cache, table, [n], 3)
    q = _queries(new, H, D, 1, 5)
    plan = U.batch(E, table, [new], [n])
    clean = _run(E, attn, cache, plan, q, H, 0.1, window, 1)
    for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
        p = int(table[0, 4])                               # tokens 64..79 of head 1
        keep = codes[p, 1].clone(), scales[p, 1].clone()
        codes[p, 1], scales[p, 1] = 0, 255
        out, lse = _run(E, attn, cache, plan, q, H, 0.1, window, 1)
        pos = torch.arange(n - new, n, device="cuda")
        hit = (pos >= 64) & (pos - window + 1 <= 79)
        o, c = out.view(new, KH, -1), clean[0].view(new, KH, -1)
        assert o[hit, 1].isnan().all() and torch.equal(o[~hit], c[~hit]) and torch.equal(o[:, 0], c[:, 0])
        codes[p, 1], scales[p, 1] = keep


def test_strided_queries_and_outputs(E, attn):
    KH, H, D, pt, n = 2, 8, 128, 32, 90
    table = U.pages_for([n], pt, 4)
    cache = U.Cache(E, 4, KH, pt, D)
    U.fill_random(cache, table, [n], 3)
    plan = U.batch(E, table, [20], [n])
    wide = _queries(20, H + 2 * KH, D, 0, 4)
    q = wide[:, : H * D]
    want = _run(E, attn, cache, plan, q, H, 0.1, 0, 0)
    room = torch.full((20, H * D + 64), 3.0, dtype=q.dtype, device="cuda")
    E.engram_attention(attn, cache.desc, plan, 0, q, wide.stride(0), H, 0.1, 0, room, room.stride(0), None)
    assert E.engram_check() == 0
    assert torch.equal(room[:, : H * D], want[0]) and (room[:, H * D:] == 3).all()


def test_long_caches_and_offsets_past_32_bits(E, attn):
    """Pages 80 MB apart reach past 4 GB; the result is that of the dense cache."""
    KH, H, D, pt, n = 1, 4, 128, 64, 60 * 64 - 5
    a = U.Cache(E, 60, KH, pt, D, page_stride=80 << 20, fill=0)
    b = U.Cache(E, 60, KH, pt, D)
    table = U.pages_for([n], pt, 60)
    U.fill_random(b, table, [n], 3)
    b.clone_into(a)
    for new in (1, 70):
        q = _queries(new, H, D, 0, 5)
        x = _run(E, attn, a, U.batch(E, table, [new], [n]), q, H, 0.1, 0, 0)
        y = _run(E, attn, b, U.batch(E, table, [new], [n]), q, H, 0.1, 0, 0)
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        _check(b, table, [new], [n], q, H, 0.1, 0, 0, *y)


def test_same_bits_every_time_and_on_another_stream(E, attn):
    """Splits join in a fixed order; other calls on the workspace in between leave nothing behind."""
    KH, H, D, pt = 2, 8, 128, 64
    kv = [9000, 5, 300]
    table = U.pages_for(kv, pt, 150)
    cache = U.Cache(E, 150, KH, pt, D)
    U.fill_random(cache, table, kv, 3)
    for news in ([1, 1, 1], [130, 5, 60]):
        q = _queries(sum(news), H, D, 0, 5)
        first = _run(E, attn, cache, U.batch(E, table, news, kv), q, H, 0.1, 0, 0)
        _case(E, attn, [1], [3000], 4, 2, 64, 16, 1)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = _run(E, attn, cache, U.batch(E, table, news, kv), q, H, 0.1, 0, 0, stream=s)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_decode_steps(E, attn):
    """Append and attention in a CUDA graph: replays read the lengths and pages of the moment."""
    KH, H, D, pt = 2, 8, 128, 16
    table = U.pages_for([64, 64], pt, 10)
    cache, other = U.Cache(E, 10, KH, pt, D), U.Cache(E, 10, KH, pt, D)
    plan = U.batch(E, table, [1, 1], [17, 40])
    U.fill_random(cache, table, [16, 39], 3)
    cache.clone_into(other)
    qkv = torch.empty(2, (H + 2 * KH) * D, dtype=torch.bfloat16, device="cuda")
    st = qkv.stride(0)
    q, k, v = qkv[:, : H * D], qkv[:, H * D: (H + KH) * D], qkv[:, (H + KH) * D:]
    out, lse = torch.zeros(2, H * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, H, device="cuda")

    def step(c, o, ls):
        E.engram_kv_append(c.desc, plan, 0, k, st, v, st, None, 0, None, 0, 0)
        E.engram_attention(attn, c.desc, plan, 0, q, st, H, 0.1, 0, o, 0, ls)

    qkv.copy_(_queries(2, H + 2 * KH, D, 0, 1))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cache, out, lse)                              # warm: module load and attributes before the capture
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    other.clone_into(cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out, lse)
    for i in range(5):
        qkv.copy_(_queries(2, H + 2 * KH, D, 0, 10 + i))
        graph.replay()
        o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
        step(other, o2, l2)
        assert E.engram_check() == 0
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert all(torch.equal(x, y) for x, y in zip(cache.tensors(), other.tensors()))
        plan.lens += 1


def test_attn_reset(E, attn):
    E.engram_attn_reset(attn)
    _case(E, attn, [1], [2000], 4, 2, 128, 16, 0)


@pytest.mark.parametrize("n,H", [(16, 1), (17, 1), (128, 1), (129, 1), (256, 1), (257, 1), (4, 4), (32, 8), (33, 8), (51, 5)])
def test_row_tile_edges(E, attn, n, H):
    """Rows of one key/value head around 16, 128 and 256, query groups that do and do not divide them."""
    _case(E, attn, [n], [n + 100], H, 1, 64, 16, 0, seed=n)
    _case(E, attn, [n, n], [n, n + 300], H, 1, 128, 64, 1, window=77, seed=n)


@pytest.mark.parametrize("batch,new", [(33, 1), (300, 1), (40, 30), (300, 9)])
def test_many_sequences(E, attn, batch, new):
    """More sequences than lanes of a warp, some without rows or tokens."""
    news = [0 if b % 11 == 5 else new if b % 3 else max(1, new // 2) for b in range(batch)]
    kv = [0 if b % 13 == 4 else news[b] + (b * 37) % 90 for b in range(batch)]
    _case(E, attn, news, kv, 4, 2, 64, 16, 0, seed=batch)


def test_two_workspaces_at_once(E, attn):
    """Calls that overlap on two streams, each with its own workspace."""
    other = E.Attention()
    KH, H, D, pt, n = 2, 8, 128, 64, 20000
    table = U.pages_for([n], pt, 320)
    cache = U.Cache(E, 320, KH, pt, D)
    U.fill_random(cache, table, [n], 3)
    for new in (1, 40):
        q = _queries(new, H, D, 0, 5)
        plan = U.batch(E, table, [new], [n])
        want = _run(E, attn, cache, plan, q, H, 0.1, 0, 0)
        outs = []
        torch.cuda.synchronize()
        streams = torch.cuda.Stream(), torch.cuda.Stream()
        for i in range(6):
            o = torch.empty_like(q)
            E.engram_attention((attn, other)[i & 1], cache.desc, plan, 0, q, 0, H, 0.1, 0, o, 0, stream=streams[i & 1])
            outs.append(o)
        torch.cuda.synchronize()
        assert E.engram_check() == 0 and all(torch.equal(o, want[0]) for o in outs)
