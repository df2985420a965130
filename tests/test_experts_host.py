"""The experts' sub-layer's entry points refuse bad arguments before they touch
the GPU (CPU only: fake addresses, never dereferenced)."""
import ctypes

import pytest

INVALID, NULL, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -5, -11
A, ODD = 1 << 30, (1 << 30) + 1


@pytest.fixture(scope="module")
def E():
    from deepseek_v4_engram_hash_gb300 import build
    build.build()
    from deepseek_v4_engram_hash_gb300 import _lib
    _lib.lib()
    return _lib


def _route(E, **kw):
    d = dict(n=256, k=8, score=0, groups=8, top=4, best=2, renorm=True, scale=1.0, type=2, logits=A, stride=0, bias=A, tokens=100,
             ids=A, w=A, offsets=A, pairs=A, ln=None, lk=None, lt=None, ws=A, ws_bytes=1 << 30, lists=True, router=True)
    d.update(kw)
    r = E.Router(d["n"], d["k"], d["score"], d["groups"], d["top"], d["best"], d["renorm"], d["scale"])
    L = E.ExpertLists(d["offsets"], d["pairs"], d["n"] if d["ln"] is None else d["ln"], d["k"] if d["lk"] is None else d["lk"],
                      d["tokens"] if d["lt"] is None else d["lt"]) if d["lists"] else None
    return E.lib().engram_route(r.ref if d["router"] else None, d["type"], d["logits"], d["stride"], d["bias"], d["tokens"], d["ids"],
                                d["w"], L.ref if L else None, d["ws"], d["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(router=False), NULL), (dict(n=0), INVALID), (dict(n=1025, groups=1, top=1), INVALID), (dict(k=0), INVALID),
    (dict(k=33), INVALID), (dict(k=17, n=32), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID),
    (dict(groups=64, top=8), INVALID), (dict(top=0), INVALID), (dict(top=9), INVALID), (dict(best=0), INVALID),
    (dict(best=3), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(type=3), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=1 << 28), INVALID),
    (dict(stride=255), INVALID), (dict(stride=1 << 40), INVALID), (dict(ln=128), INVALID), (dict(lk=4), INVALID),
    (dict(lt=99), INVALID), (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL), (dict(offsets=None), NULL),
    (dict(pairs=None), NULL), (dict(ws=None), NULL), (dict(ws_bytes=100), WORKSPACE), (dict(logits=ODD), ALIGN),
    (dict(type=0, logits=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(ids=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(offsets=ODD), ALIGN), (dict(pairs=ODD), ALIGN), (dict(ws=ODD), ALIGN),
    (dict(tokens=0, lists=False, logits=None, ids=None, w=None, ws=None), 0),
])
def test_route_refuses(E, kw, code):
    assert _route(E, **kw) == code


def test_route_workspace(E):
    f = E.engram_route_workspace_bytes
    assert f(256, 0) == f(256, 1) == 0 and f(0, 5) == f(1025, 5) == f(8, -1) == 0
    assert f(256, 100000) == f(256, 1 << 24) <= 152 * 256 * 4 and f(256, 100000) % (256 * 4) == 0


def _weight(E, **kw):
    d = dict(codes=A, scales=A, wfmt=2, n_experts=1, n=512, k=256, gated=False)
    d.update({k: v for k, v in kw.items() if k in d})
    return E.Fp8Weight(d["codes"], d["scales"], d["wfmt"], d["n_experts"], d["n"], d["k"], d["gated"])


def _lists(E, kw, n_experts):
    if kw.get("tokens") is None:
        return None
    return E.ExpertLists(kw.get("offsets", A), kw.get("pairs", A), kw.get("ln", n_experts), kw.get("top_k", 4), kw["tokens"])


PRODUCT = [
    (dict(xfmt=1), INVALID), (dict(xfmt=3), INVALID), (dict(wfmt=1), INVALID), (dict(n_experts=0), INVALID),
    (dict(n_experts=1025, tokens=2), INVALID), (dict(n=0), INVALID), (dict(n=(1 << 24) + 16), INVALID), (dict(k=8), INVALID),
    (dict(k=264), INVALID), (dict(k=65552), INVALID), (dict(n=1 << 24, k=65536), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=(1 << 30) + 1), INVALID), (dict(xs=240), INVALID), (dict(xs=264), INVALID), (dict(xs=1 << 40), INVALID),
    (dict(n_experts=4), INVALID), (dict(n_experts=4, tokens=2, ln=5), INVALID), (dict(n_experts=4, tokens=2, top_k=0), INVALID),
    (dict(n_experts=4, tokens=2, top_k=33), INVALID), (dict(n_experts=4, tokens=-1), INVALID),
    (dict(n_experts=4, tokens=7, rows=9), INVALID), (dict(x=None), NULL), (dict(sc=None), NULL), (dict(codes=None), NULL),
    (dict(scales=None), NULL), (dict(out=None), NULL), (dict(weight=False), NULL), (dict(n_experts=4, tokens=2, offsets=None), NULL),
    (dict(n_experts=4, tokens=2, pairs=None), NULL), (dict(x=ODD), ALIGN), (dict(codes=ODD), ALIGN), (dict(xfmt=0, sc=ODD), ALIGN),
    (dict(wfmt=0, scales=ODD), ALIGN), (dict(n_experts=4, tokens=2, offsets=ODD), ALIGN), (dict(n_experts=4, tokens=2, pairs=ODD), ALIGN),
    (dict(rows=0, x=None, sc=None, codes=None, scales=None, out=None), 0),
]


def _project(E, **kw):
    d = dict(x=A, xs=0, sc=A, xfmt=2, rows=None, type=0, out=A, os=0)
    d.update({k: v for k, v in kw.items() if k in d})
    w = _weight(E, **kw)
    L = _lists(E, kw, w.desc.n_experts)
    rows = d["rows"] if d["rows"] is not None else kw["tokens"] * kw.get("top_k", 4) if L else 8
    return E.lib().engram_project_fp8(d["x"], d["xs"], d["sc"], d["xfmt"], rows, w.ref if kw.get("weight", True) else None,
                                      L.ref if L else None, d["type"], d["out"], d["os"], None)


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(gated=True), INVALID), (dict(os=511), INVALID), (dict(os=1 << 40), INVALID),
    (dict(out=ODD), ALIGN), (dict(type=2, out=A + 2), ALIGN),
])
def test_project_refuses(E, kw, code):
    assert _project(E, **kw) == code


def _glu(E, **kw):
    d = dict(x=A, xs=0, sc=A, xfmt=2, rows=None, limit=0.0, fmt=2, out=A, osc=A)
    d.update({k: v for k, v in kw.items() if k in d})
    w = _weight(E, **{"gated": True, **kw})
    L = _lists(E, kw, w.desc.n_experts)
    rows = d["rows"] if d["rows"] is not None else kw["tokens"] if L else 8
    return E.lib().engram_glu_fp8(d["x"], d["xs"], d["sc"], d["xfmt"], rows, w.ref if kw.get("weight", True) else None,
                                  L.ref if L else None, d["limit"], d["fmt"], d["out"], d["osc"], None)


@pytest.mark.parametrize("kw,code", PRODUCT + [
    (dict(gated=False), INVALID), (dict(n=520), INVALID), (dict(limit=-1.0), INVALID), (dict(limit=float("nan")), INVALID),
    (dict(limit=float("inf")), INVALID), (dict(fmt=1), INVALID), (dict(fmt=3), INVALID), (dict(osc=None), NULL), (dict(out=ODD), ALIGN),
    (dict(fmt=0, osc=ODD), ALIGN), (dict(n_experts=4, tokens=1 << 20, xs=1 << 16), UNSUPPORTED),
])
def test_glu_refuses(E, kw, code):
    assert _glu(E, **kw) == code


def _combine(E, **kw):
    d = dict(y=A, yt=0, ys=0, w=A, tokens=4, k=8, dim=256, add=A + 65536, at=0, as_=0, ot=0, out=A + 131072, os=0)
    d.update(kw)
    return E.lib().engram_combine(d["y"], d["yt"], d["ys"], d["w"], d["tokens"], d["k"], d["dim"], d["add"], d["at"], d["as_"], d["ot"],
                                  d["out"], d["os"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(yt=3), INVALID), (dict(at=-1), INVALID), (dict(ot=3), INVALID), (dict(tokens=-1), INVALID), (dict(k=0), INVALID),
    (dict(k=33), INVALID), (dict(dim=0), INVALID), (dict(dim=252), INVALID), (dict(dim=65544), INVALID), (dict(tokens=1 << 28), INVALID),
    (dict(ys=248), INVALID), (dict(ys=260), INVALID), (dict(as_=8), INVALID), (dict(os=12), INVALID),
    (dict(add=A, out=A, at=2), INVALID), (dict(add=A, out=A, os=264), INVALID), (dict(y=None), NULL), (dict(w=None), NULL),
    (dict(out=None), NULL), (dict(y=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(add=ODD), ALIGN), (dict(out=ODD), ALIGN),
    (dict(tokens=0, y=None, w=None, out=None), 0),
])
def test_combine_refuses(E, kw, code):
    assert _combine(E, **kw) == code


def test_refusals_raise_in_the_binding(E):
    with pytest.raises(E.EngramError) as e:
        E.engram_combine(A, 5, 0, A, 4, 8, 256, None, 0, 0, 0, A, 0, stream=type("S", (), {"cuda_stream": 0}))
    assert e.value.code == INVALID
    assert ctypes.sizeof(E.engram_router) == 32 and ctypes.sizeof(E.engram_expert_lists) == 32 and ctypes.sizeof(E.engram_fp8_weight) == 40


def test_descriptors_refuse_tensors_that_they_would_misread(E):
    import torch
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    cases = [
        (lambda: E.ExpertLists(torch.zeros(9, dtype=torch.int64), A, 8, 2, 4), "int64"),
        (lambda: E.ExpertLists(torch.zeros(8, dtype=i32), A, 8, 2, 4), "elements"),
        (lambda: E.ExpertLists(A, torch.zeros(16, dtype=i32)[::2], 8, 2, 4), "strides"),
        (lambda: E.ExpertLists(A, torch.zeros(7, dtype=i32), 8, 2, 4), "elements"),
        (lambda: E.ExpertLists(torch.zeros(9, dtype=i32), A, 8, 2, 4), "cpu"),
        (lambda: E.Fp8Weight(torch.zeros(256, 256, dtype=f32), A, 0, 1, 256, 256), "float32"),
        (lambda: E.Fp8Weight(torch.zeros(256, 256, dtype=u8).T, A, 0, 1, 256, 256), "strides"),
        (lambda: E.Fp8Weight(torch.zeros(256, 256, dtype=u8), A, 0, 1, 256, 256, True), "elements"),
        (lambda: E.Fp8Weight(A, torch.zeros(2, 2, dtype=u8), 0, 1, 256, 256), "uint8"),
        (lambda: E.Fp8Weight(A, torch.zeros(2, 2, dtype=f32), 2, 1, 256, 256), "float32"),
        (lambda: E.Fp8Weight(A, torch.zeros(2, 2, dtype=u8), 2, 1, 257, 256), "elements"),
        (lambda: E.Fp8Weight(A, torch.zeros(2, 2, dtype=f32), 0, 1, 256, 256), "cpu"),
    ]
    for i, (make, why) in enumerate(cases):
        with pytest.raises(E.EngramError) as e:
            make()
        assert e.value.code == INVALID and why in str(e.value), (i, str(e.value))
