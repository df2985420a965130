"""The attention sub-layer's entry points refuse bad arguments before they
touch the GPU (CPU only: fake addresses, never dereferenced)."""
import ctypes

import pytest

INVALID, NULL, ALIGN, UNSUPPORTED = -1, -2, -3, -11
A, ODD = 1 << 30, (1 << 30) + 2


@pytest.fixture(scope="module")
def E():
    from deepseek_v4_engram_hash_gb300 import build
    build.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    _lib.lib()
    return _lib


def test_error_strings(E):
    assert "page" in E.strerror(-13)
    assert "kv_len" in E.strerror(-14)


def _norm(E, **kw):
    d = dict(x=A, xt=0, xs=0, res=A, rt=2, rs=0, ro=A, w=A, rows=4, dim=256, eps=1e-6, fmt=2, block=32, out=A, sc=A)
    d.update(kw)
    f = E.lib().engram_residual_norm
    return f(d["x"], d["xt"], d["xs"], d["res"], d["rt"], d["rs"], d["ro"], d["w"], d["rows"], d["dim"], d["eps"],
             d["fmt"], d["block"], d["out"], d["sc"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(xt=3), INVALID), (dict(xt=-1), INVALID), (dict(rt=1), INVALID), (dict(rt=3), INVALID), (dict(fmt=1), INVALID),
    (dict(fmt=4), INVALID), (dict(rows=-1), INVALID), (dict(dim=0), INVALID), (dict(dim=252), INVALID),
    (dict(dim=16392), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(block=0), INVALID), (dict(block=24), INVALID), (dict(block=96), INVALID),
    (dict(xs=248), INVALID), (dict(xs=260), INVALID), (dict(rs=8), INVALID), (dict(res=None), NULL),
    (dict(out=None), NULL), (dict(sc=None), NULL), (dict(x=ODD), ALIGN), (dict(res=ODD), ALIGN), (dict(ro=ODD), ALIGN),
    (dict(w=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(fmt=0, sc=ODD), ALIGN), (dict(rows=0, res=None, out=None), 0),
])
def test_residual_norm_refuses(E, kw, code):
    assert _norm(E, **kw) == code


def _kv(E, **kw):
    d = dict(k=A, v=A, ks=A, vs=A, n_pages=8, page_stride=0, KH=2, pt=16, D=128)
    d.update({k: v for k, v in kw.items() if k in d})
    c = E.KvCache(d["k"], d["v"], d["ks"], d["vs"], d["n_pages"], d["KH"], d["pt"], d["D"], d["page_stride"])
    e = dict(table=A, kv_len=A, row_start=None, batch=2, max_pages=4, rows=4, max_rows=2, table_stride=0)
    e.update({k: v for k, v in kw.items() if k in e})
    b = E.KvBatch(e["table"], e["kv_len"], e["row_start"], e["batch"], e["max_pages"], e["rows"], e["max_rows"], e["table_stride"])
    return c, b


KV_REFUSALS = [
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(pt=8), UNSUPPORTED), (dict(pt=48), UNSUPPORTED),
    (dict(KH=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_pages=1 << 31), INVALID), (dict(page_stride=4080), INVALID),
    (dict(page_stride=4104), INVALID), (dict(batch=0), INVALID), (dict(batch=8193), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 27), INVALID), (dict(rows=-2), INVALID), (dict(rows=5), INVALID), (dict(max_rows=1), INVALID),
    (dict(row_start=A, max_rows=0), INVALID), (dict(table_stride=3), INVALID), (dict(k=None), NULL), (dict(vs=None), NULL),
    (dict(table=None), NULL), (dict(kv_len=None), NULL), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN),
    (dict(row_start=ODD - 1), ALIGN), (dict(kv_len=ODD), ALIGN),
]


def _append(E, c, b, type=0, k=A, ks=0, v=A, vs=0, q=A, qs=0, qo=A + 65536, qos=0, heads=4, rope=None):
    return E.lib().engram_kv_append(c.ref if c else None, b.ref if b else None, type, k, ks, v, vs, q, qs, qo, qos, heads,
                                    rope.ref if rope else None, None)


def _attend(E, c, b, attn=A, type=0, q=A, qs=0, heads=4, scale=0.1, window=0, out=A, os=0, lse=A):
    return E.lib().engram_attention(attn, c.ref if c else None, b.ref if b else None, type, q, qs, heads, scale, window,
                                    out, os, lse, None)


@pytest.mark.parametrize("kw,code", KV_REFUSALS)
def test_cache_and_batch_are_checked(E, kw, code):
    c, b = _kv(E, **kw)
    assert _append(E, c, b) == code
    # the workspace handle is only dereferenced after the checks
    assert _attend(E, c, b) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(ks=248), INVALID), (dict(ks=260), INVALID),
    (dict(vs=100), INVALID), (dict(qs=504), INVALID), (dict(qos=520, qo=A), INVALID), (dict(heads=0), INVALID),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(qo=None), NULL), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN),
    (dict(q=ODD), ALIGN), (dict(qo=ODD), ALIGN),
])
def test_append_refuses(E, kw, code):
    c, b = _kv(E)
    assert _append(E, c, b, **kw) == code


@pytest.mark.parametrize("table,positions,dim,code", [
    (A, 64, 24, INVALID), (A, 64, 144, INVALID), (A, 64, -16, INVALID), (A, -1, 64, INVALID), (None, 64, 64, NULL),
    (ODD, 64, 64, ALIGN),
])
def test_append_checks_the_rotation(E, table, positions, dim, code):
    c, b = _kv(E)
    assert _append(E, c, b, rope=E.Rope(table, positions, dim)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(attn=None), NULL), (dict(type=2), INVALID), (dict(type=-1), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(heads=3), INVALID),
    (dict(heads=0), INVALID), (dict(qs=504), INVALID), (dict(os=516), INVALID), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(q=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(lse=ODD), ALIGN),
])
def test_attention_refuses(E, kw, code):
    c, b = _kv(E)
    assert _attend(E, c, b, **kw) == code


def test_null_descriptors_and_empty_calls(E):
    c, b = _kv(E)
    assert _append(E, None, b) == NULL and _append(E, c, None) == NULL
    assert _attend(E, None, b) == NULL and _attend(E, c, None) == NULL
    assert E.lib().engram_attn_create(None) == NULL
    assert E.lib().engram_attn_reset(None, None) == NULL
    E.lib().engram_attn_destroy(None)
    c, b = _kv(E, rows=0, max_rows=0, k=None, v=None, table=None, kv_len=None)
    assert _append(E, c, b, k=None, v=None, q=None) == 0
    assert _attend(E, c, b, q=None, out=None) == 0


def test_refusals_raise_in_the_binding(E):
    c, b = _kv(E, D=96)
    with pytest.raises(E.EngramError) as e:
        E.engram_kv_append(c, b, 0, A, 0, A, 0, None, 0, None, 0, 0, stream=type("S", (), {"cuda_stream": 0}))
    assert e.value.code == UNSUPPORTED
    assert ctypes.sizeof(E.engram_kv_cache) == 64 and ctypes.sizeof(E.engram_kv_batch) == 48


def test_every_source_is_built():
    """No kernel file lies beside the build's lists: a stray one is in no library, and its symbols may be another's."""
    import glob
    import os
    from deepseek_v4_engram_hash_gb300 import build
    have = {os.path.basename(p) for p in glob.glob(os.path.join(build.CSRC, "*.cu"))}
    assert have == set(build.ENGRAM_SRCS) | set(build.SYNTH_SRCS)


def _cache_of(E, k=None, ks=None, n_pages=8, page_stride=0):
    import torch
    k = torch.zeros(8, 2, 16, 64, dtype=torch.uint8) if k is None else k
    ks = torch.zeros(8, 2, dtype=torch.uint8) if ks is None else ks
    return lambda: E.KvCache(k, A, ks, A, n_pages, 2, 16, 64, page_stride)


def test_descriptors_refuse_tensors_that_they_would_misread(E):
    """Element types, strides and sizes that do not fit, and tensors of the CPU: refused where the descriptor is made."""
    import torch
    i32, i64, u8, f32, f64 = torch.int32, torch.int64, torch.uint8, torch.float32, torch.float64

    def batch(table=None, lens=None, start=None, stride=0):
        table = torch.zeros(3, 4, dtype=i32) if table is None else table
        return lambda: E.KvBatch(table, lens, start, 3, 4, 6, 2, stride)

    cases = [
        (_cache_of(E, k=torch.zeros(8, 2, 16, 64, dtype=torch.int16)), "int16"),
        (_cache_of(E, k=torch.zeros(8, 16, 2, 64, dtype=u8).transpose(1, 2)), "strides"),
        (_cache_of(E, k=torch.zeros(16, 2, 16, 64, dtype=u8)[::2]), "strides"),
        (_cache_of(E, n_pages=9), "elements"),
        (_cache_of(E, k=torch.zeros(8 * 4096, dtype=u8), page_stride=8192), "elements"),
        (_cache_of(E, k=A, ks=torch.zeros(8, 2, dtype=f32)), "float32"),
        (_cache_of(E, k=A, ks=torch.zeros(2, 8, dtype=u8).T), "strides"),
        (_cache_of(E, k=A, ks=torch.zeros(15, dtype=u8)), "elements"),
        (_cache_of(E), "cpu"),
        (_cache_of(E, k=torch.zeros(16, 2, 16, 64, dtype=u8)[::2], page_stride=4096), "cpu"),   # its stride is given
        (batch(table=torch.zeros(3, 4, dtype=i64)), "int64"),
        (batch(table=torch.zeros(4, 3, dtype=i32).T), "strides"),
        (batch(table=torch.zeros(3, 8, dtype=i32)[:, :4]), "strides"),
        (batch(table=torch.zeros(2, 4, dtype=i32)), "elements"),
        (batch(table=torch.zeros(3, 8, dtype=i32)[:, :4], stride=8), "cpu"),
        (batch(table=A, lens=torch.zeros(3, dtype=i64)), "int64"),
        (batch(table=A, lens=torch.zeros(6, dtype=i32)[::2]), "strides"),
        (batch(table=A, lens=torch.zeros(2, dtype=i32)), "elements"),
        (batch(table=A, lens=A, start=torch.zeros(3, dtype=i32)), "elements"),
        (batch(table=A, lens=A, start=torch.zeros(4, dtype=i32)), "cpu"),
        (lambda: E.Rope(torch.zeros(64, 32, 2, dtype=f64), 64, 64), "float64"),
        (lambda: E.Rope(torch.zeros(32, 64, 2).transpose(0, 1), 64, 64), "strides"),
        (lambda: E.Rope(torch.zeros(63, 32, 2), 64, 64), "elements"),
        (lambda: E.Rope(torch.zeros(64, 32, 2), 64, 64), "cpu"),
    ]
    for i, (make, why) in enumerate(cases):
        with pytest.raises(E.EngramError) as e:
            make()
        assert e.value.code == INVALID and why in str(e.value), (i, str(e.value))
    E.KvCache(A, A, A, A, 8, 2, 16, 64)                      # addresses are taken as they are
    E.KvBatch(A, A, None, 3, 4, 6, 2)
    E.Rope(A, 64, 64)
