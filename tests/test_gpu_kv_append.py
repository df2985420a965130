"""engram_kv_append against its definition in 64 bits.

The rotation is two products and one sum in f32 (relative error of an element
under 3 x 2^-24 of the pair's size), so a new code is within half a step of the
64-bit value / scale plus that; scales are equal; earlier codes that are encoded
again come from stored codes and are equal bit for bit.
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


def _table(positions, dim):
    at = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None]
    f = 10000.0 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float64) / (dim // 2))
    return torch.stack([(at * f).cos(), (at * f).sin()], -1).float().contiguous()


def _expect(cache, table, new, kv, k, v, rope, rot, inter):
    """The cache after the append, by the definition, from the cache as it is now."""
    want, tol = [], []
    for which, (codes, scales, x) in enumerate(((cache.k, cache.ks, k), (cache.v, cache.vs, v))):
        codes, scales = codes.clone(), scales.clone().long()
        value = R.e4m3_values().cuda()[codes.long()]
        slack = torch.zeros_like(value)
        row = 0
        for b, (n, total) in enumerate(zip(new, kv)):
            first = max(0, total - n)
            pos = torch.arange(first, total, device="cuda")
            y = x[row + n - (total - first): row + n].double().view(-1, cache.KH, cache.D)
            size = y.abs()
            if not which:
                y = R.rotate(y, rope, pos, rot, inter)
                size = torch.full_like(y, 1) * size.amax(2, keepdim=True) * 2
            row += n
            for p in range(first // cache.pt, (total - 1) // cache.pt + 1 if total > first else 0):
                lo, hi = max(first, p * cache.pt), min(total, (p + 1) * cache.pt)
                page, have = int(table[b, p]), lo - p * cache.pt
                if not 0 <= page < cache.n_pages:
                    continue
                part, sz = y[lo - first: hi - first].transpose(0, 1), size[lo - first: hi - first].transpose(0, 1)
                byte = R.scale_bytes(part.abs().amax((1, 2)).cpu()).cuda()
                old = scales[page].clone()
                if have:
                    byte = torch.maximum(byte, old)
                    down = R.pow2(old - byte)[:, None, None]
                    again = R.e4m3_round(value[page, :, :have] * down)
                    value[page, :, :have] = torch.where((byte == 255)[:, None, None], value[page, :, :have], again)
                scale = R.pow2(byte - 127)[:, None, None]
                put = torch.where((byte == 255)[:, None, None], torch.zeros_like(part), part / scale)
                value[page, :, have: have + hi - lo] = put
                s = 0.5 * R.e4m3_step(put) * (1 + 1e-9) + 3 * 2.0 ** -24 * torch.nan_to_num(sz) / scale
                slack[page, :, have: have + hi - lo] = s
                scales[page] = byte
        want.append((value, scales))
        tol.append(slack)
    return want, tol


def _compare(cache, want, tol):
    for (codes, scales), (value, ws), slack in zip(((cache.k, cache.ks), (cache.v, cache.vs)), want, tol):
        assert torch.equal(scales.long(), ws)
        got = R.e4m3_values().cuda()[codes.long()]
        same = (got == value) | (got.isnan() & value.isnan())
        assert (same | ((got - value).abs() <= slack)).all()


def _data(rows, H, KH, D, dt, seed, stride=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(rows, stride or (H + 2 * KH) * D, generator=g, device="cuda").to(dt)
    return w, w[:, : H * D], w[:, H * D: (H + KH) * D], w[:, (H + KH) * D: (H + 2 * KH) * D]


CASES = [
    # new tokens, tokens with them, H, KH, D, page, type, rot, interleaved
    ([1], [1], 4, 2, 128, 16, 0, 128, 0),
    ([1], [2049], 32, 8, 128, 64, 0, 128, 0),
    ([1, 1, 1, 1, 1], [16, 17, 1, 31, 300], 8, 8, 64, 16, 1, 64, 1),
    ([3, 4, 1, 2], [3, 65, 64, 130], 6, 2, 128, 64, 2, 64, 0),      # inside pages and over their ends
    ([200], [200], 4, 1, 128, 128, 0, 128, 0),                      # a prompt into an empty cache
    ([129, 1, 17, 0, 64], [129, 90, 33, 40, 100], 5, 5, 64, 32, 2, 32, 1),
    ([700, 5], [701, 133], 2, 2, 128, 16, 1, 16, 0),
    ([256], [300], 16, 2, 64, 128, 0, 0, 0),                        # no rotation
    ([33] * 40, [33 + 7 * i for i in range(40)], 2, 1, 64, 16, 0, 48, 0),
    ([1] * 70 + [90], [1 + 3 * i for i in range(71)], 2, 1, 128, 16, 0, 128, 0),   # slots by prefix sum; a short chunk
]


@pytest.mark.parametrize("new,kv,H,KH,D,pt,ty,rot,inter", CASES)
def test_matches_the_definition(E, new, kv, H, KH, D, pt, ty, rot, inter):
    n_pages = sum(-(-n // pt) for n in kv) + 4
    table = U.pages_for(kv, pt, n_pages, seed=len(kv))
    cache = U.Cache(E, n_pages, KH, pt, D)
    U.fill_random(cache, table, [max(0, t - n) for n, t in zip(new, kv)], seed=3, spread=1)
    _, q, k, v = _data(sum(new), H, KH, D, U.DTYPES[ty], seed=11)
    rope = _table(max(kv) + 1, rot) if rot else None
    want, tol = _expect(cache, table, new, kv, k, v, rope, rot, inter)
    qo = torch.full((sum(new), H * D), 9.0, dtype=q.dtype, device="cuda")
    plan = U.batch(E, table, new, kv)
    stride = (H + 2 * KH) * D
    E.engram_kv_append(cache.desc, plan, ty, k, stride, v, stride, q, stride, qo, 0, H,
                       E.Rope(rope, rope.shape[0], rot, inter) if rot else None)
    assert E.engram_check() == 0
    _compare(cache, want, tol)
    row = 0
    for n, t in zip(new, kv):
        first = max(0, t - n)
        skip = n - (t - first)
        assert (qo[row: row + skip] == 0).all()
        x = q[row + skip: row + n].double().view(-1, H, D)
        y = R.rotate(x, rope, torch.arange(first, t, device="cuda"), rot, inter)
        eps = {0: 2.0 ** -8, 1: 2.0 ** -11, 2: 2.0 ** -24}[ty]             # unit roundoffs: 8, 11 and 24 significant bits
        lim = eps * y.abs() + 3 * 2.0 ** -24 * x.abs().amax(2, keepdim=True) * 2 + (2.0 ** -24 if ty == 1 else 0)
        assert ((qo[row + skip: row + n].double().view(-1, H, D) - y).abs() <= lim).all()
        row += n


def test_uniform_batches_need_no_row_start(E):
    KH, D, pt, H = 2, 128, 16, 4
    new, kv = [3] * 6, [3, 18, 19, 40, 64, 100]
    table = U.pages_for(kv, pt, 40)
    _, q, k, v = _data(18, H, KH, D, torch.bfloat16, 1)
    rope = _table(128, 128)
    got = []
    for uniform in (False, True):
        cache = U.Cache(E, 40, KH, pt, D)
        U.fill_random(cache, table, [t - 3 for t in kv], seed=3)
        plan = U.batch(E, table, new, kv, uniform=uniform)
        qo = torch.empty(18, H * D, dtype=q.dtype, device="cuda")
        st = q.stride(0)
        E.engram_kv_append(cache.desc, plan, 0, k, st, v, st, q, st, qo, 0, H, E.Rope(rope, 128, 128))
        assert E.engram_check() == 0
        got.append((*cache.tensors(), qo))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_token_by_token_equals_the_prompt_where_scales_do_not_grow(E):
    """A first token that sets every block's scale: then single appends and one prompt append leave the same bytes."""
    KH, D, pt, n = 2, 64, 32, 70
    table = U.pages_for([n], pt, 5)
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.randn(n, KH * D, generator=g, device="cuda") for _ in "kv")
    k[::pt], v[::pt] = 500.0, -600.0
    a, b = U.Cache(E, 5, KH, pt, D), U.Cache(E, 5, KH, pt, D)
    E.engram_kv_append(a.desc, U.batch(E, table, [n], [n]), 2, k, 0, v, 0, None, 0, None, 0, 0)
    for i in range(n):
        E.engram_kv_append(b.desc, U.batch(E, table, [1], [i + 1]), 2, k[i:], 0, v[i:], 0, None, 0, None, 0, 0)
    assert E.engram_check() == 0
    assert all(torch.equal(x, y) for x, y in zip(a.tensors(), b.tensors()))


@pytest.mark.parametrize("pt,D", [(16, 128), (128, 64), (128, 128)])
def test_growing_scales_encode_the_page_again(E, pt, D):
    """Each token four times its predecessor: every append grows the block's scale, past where the first codes vanish."""
    KH = 3
    table = U.pages_for([14], pt, 3)
    cache = U.Cache(E, 3, KH, pt, D)
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(14):
        k, v = (torch.randn(1, KH * D, generator=g, device="cuda") * 4.0 ** i for _ in "kv")
        want, tol = _expect(cache, table, [1], [i + 1], k, v, None, 0, 0)
        E.engram_kv_append(cache.desc, U.batch(E, table, [1], [i + 1]), 2, k, 0, v, 0, None, 0, None, 0, 0)
        assert E.engram_check() == 0
        _compare(cache, want, tol)


def test_values_that_need_care(E):
    """Zeros (scale 2^-126), the largest and the smallest f32 numbers, and blocks with infinities and NaN."""
    KH, D, pt = 7, 64, 16
    table = U.pages_for([3], pt, 2)
    cache = U.Cache(E, 2, KH, pt, D)
    x = torch.zeros(3, KH, D, device="cuda")
    x[:, 1] = torch.finfo(torch.float32).max
    x[:, 2] = 1e-45
    x[1, 3, 5], x[2, 4, 6], x[0, 5, 1] = math.inf, math.nan, -math.inf
    x[:, 6] = 448.0
    E.engram_kv_append(cache.desc, U.batch(E, table, [3], [3]), 2, x.view(3, -1), 0, -x.view(3, -1), 0, None, 0, None, 0, 0)
    assert E.engram_check() == 0
    p = int(table[0, 0])
    for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
        assert scales[p].tolist() == [1, 247, 1, 255, 255, 255, 127]
        assert (codes[p, [0, 2], :3] & 127 == 0).all() and (codes[p, 3:6, :3] == 0).all()
        assert (codes[p, 6, :3] & 127 == 126).all() and (codes[p, 1, :3] & 127 == 120).all()
        assert (codes[p, :, 3:] == 127).all()
    # a NaN block stays one, its earlier codes as they are
    E.engram_kv_append(cache.desc, U.batch(E, table, [1], [4]), 2, x[0].view(1, -1), 0, x[0].view(1, -1), 0, None, 0, None, 0, 0)
    assert E.engram_check() == 0 and cache.ks[p].tolist() == [1, 247, 1, 255, 255, 255, 127]


def test_queries_in_place(E):
    KH, H, D, pt = 2, 6, 128, 32
    table = U.pages_for([50], pt, 3)
    for inter in (0, 1):
        rope = _table(64, 96)
        w, q, k, v = _data(50, H, KH, D, torch.float16, 4)
        st = w.stride(0)
        outs = []
        for place in (False, True):
            cache = U.Cache(E, 3, KH, pt, D)
            w2 = w.clone()
            q2 = w2[:, : H * D]
            to = q2 if place else torch.zeros(50, H * D, dtype=q.dtype, device="cuda")
            E.engram_kv_append(cache.desc, U.batch(E, table, [50], [50]), 1, k, st, v, st, q2, st, to, to.stride(0), H,
                               E.Rope(rope, 64, 96, inter))
            assert E.engram_check() == 0
            outs.append(to.clone())
            assert torch.equal(w2[:, H * D:], w[:, H * D:])
        assert torch.equal(*outs)


def test_idle_slots_and_bad_arrays(E):
    """Empty rows store nothing and leave zero queries; lengths and pages that do not fit are reported and skipped, the others kept."""
    KH, H, D, pt = 1, 2, 64, 16
    kv = [20, 0, 33]
    table = U.pages_for(kv, pt, 8, width=4)
    _, q, k, v = _data(3, H, KH, D, torch.bfloat16, 5)
    st = q.stride(0)

    def call(lens, tab, start=None, rope=None):
        cache = U.Cache(E, 8, KH, pt, D, fill=1, scale=100)
        plan = U.batch(E, tab, [1, 1, 1], lens)
        if start is not None:
            plan.start.copy_(torch.tensor(start, dtype=torch.int32))
        qo = torch.full((3, H * D), 5.0, dtype=q.dtype, device="cuda")
        E.engram_kv_append(cache.desc, plan, 0, k, st, v, st, q, st, qo, 0, H, rope)
        return E.engram_check(), cache, qo

    rc, cache, qo = call(kv, table)
    assert rc == 0 and (qo[1] == 0).all() and (qo[[0, 2]] != 0).any(1).all()
    assert int((cache.ks != 100).sum()) == 2
    for lens in ([20, 65, 33], [20, -1, 33]):                        # over the table's pages, negative
        rc, c2, qo2 = call(lens, table)
        assert rc == -14 and (qo2[1] == 0).all()
        assert all(torch.equal(a, b) for a, b in zip(cache.tensors(), c2.tensors()))
    bad = table.clone()
    bad[2, 2] = 8                                                    # the page of token 32
    rc, c3, qo3 = call(kv, bad)
    assert rc == -13 and int((c3.ks != 100).sum()) == 1 and torch.equal(qo3, qo)
    rc, c4, _ = call(kv, table, start=[0, 1, 0, 3])                  # falls; then 0..3 holds more than max_rows
    assert rc == -14 and int((c4.ks != 100).sum()) == 1
    rc, c5, qo5 = call(kv, table, rope=E.Rope(_table(32, 64), 32, 64))   # 33 tokens, 32 angles
    assert rc == -14 and (qo5[2] == 0).all() and int((c5.ks != 100).sum()) == 1


def test_offsets_past_32_bits(E):
    """Pages 96 MB apart: the last one lies past 4 GB."""
    KH, D, pt, n_pages, stride = 2, 128, 64, 50, 96 << 20
    cache = U.Cache(E, n_pages, KH, pt, D, page_stride=stride, fill=0)
    table = torch.tensor([[49, 0]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(70, KH * D, generator=g, device="cuda").bfloat16() for _ in "kv")
    want, tol = [], []
    E.engram_kv_append(cache.desc, U.batch(E, table, [70], [70]), 0, k, 0, v, 0, None, 0, None, 0, 0)
    assert E.engram_check() == 0
    small = U.Cache(E, 2, KH, pt, D, fill=0)
    E.engram_kv_append(small.desc, U.batch(E, table.clamp(max=1), [70], [70]), 0, k, 0, v, 0, None, 0, None, 0, 0)
    assert E.engram_check() == 0
    for a, b in zip(cache.tensors(), small.tensors()):
        assert torch.equal(a[49], b[1]) and torch.equal(a[0], b[0])
    assert not cache.raw[0][(KH * pt * D):stride].any()
    del want, tol


@pytest.mark.parametrize("old", [248, 253, 254])
def test_append_under_the_largest_scales(E, old):
    """A page whose scale is the caller's own, past what this library writes (247): new codes are the values at that scale."""
    KH, D, pt = 2, 64, 16
    table = U.pages_for([5], pt, 2)
    cache = U.Cache(E, 2, KH, pt, D)
    p = int(table[0, 0])
    for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
        codes[p, :, :4], scales[p] = 0x38, old
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = ((torch.rand(1, KH * D, generator=g, device="cuda") - 0.5) * 2.0 ** 127 for _ in "kv")
    want, tol = _expect(cache, table, [1], [5], k, v, None, 0, 0)
    E.engram_kv_append(cache.desc, U.batch(E, table, [1], [5]), 2, k, 0, v, 0, None, 0, None, 0, 0)
    assert E.engram_check() == 0
    _compare(cache, want, tol)
    assert (cache.k[p, :, 4] & 127 != 0).any() and (cache.v[p, :, 4] & 127 != 0).any()
