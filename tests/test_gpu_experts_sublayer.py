"""The experts' sub-layer as it is used: its operators one behind the other, on other
streams, captured and replayed, two at once; every stage against its definition in
64 bits on what the stage before left."""
import math

import pytest
import torch

import experts_ref as X
from experts_glue import HALF, E, check_codes, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def _sublayer(**kw):
    from examples.experts_sublayer import ExpertsSublayer
    return ExpertsSublayer(**{**dict(dim=512, inter=384, n_experts=32, top_k=4, shared_inter=256, max_tokens=300, seed=3), **kw})


def _rows(E, T, dim, seed, x=None):
    """The norm that the sub-layer starts from."""
    g = rng(seed)
    res = torch.randn((T, dim), generator=g, device="cuda") if x is None else x
    codes, scales = torch.empty((T, dim), dtype=torch.uint8, device="cuda"), torch.empty((T, dim // 128), dtype=torch.uint8, device="cuda")
    E.engram_residual_norm(None, 0, res, 2, None, None, T, dim, 1e-6, E.ENGRAM_FMT_FP8_E8M0, 128, codes, scales)
    return codes, scales


def _near(got, want, mass, K, out):
    rel, least = HALF[out]
    bound = X.sum_error(K) * mass
    assert ((got.double() - want).abs() <= bound + rel * (want.abs() + bound) + least).all()


def _glu(x64, codes, scales, e):
    (g, mg), (u, mu) = (X.product(x64, X.weight64(codes[e, i], scales[e, i])) for i in (0, 1))
    a = X.glu(g, u, 0.0)
    dg, du = (X.sum_error(x64.shape[1]) * m for m in (mg, mu))
    return a, 1.1 * u.abs() * dg + (g * torch.sigmoid(g)).abs() * du + 1.1 * dg * du + 2.0 ** -20 * a.abs()


def _check(s, codes, scales, T):
    x64, k, n = X.rows64(codes, scales), s.top_k, s.n_experts
    _near(s.logits[:T], *X.product(x64, X.weight64(s.gate[1][0, 0], s.gate[2][0, 0])), s.dim, "f32")
    r = s.router.desc
    ids, w = X.route(s.logits[:T], s.bias, k, groups=r.n_groups, top_groups=r.top_groups, scale=r.scale)
    assert torch.equal(s.ids[:T].cpu(), ids)
    assert ((s.weights[:T].double().cpu() - w).abs() <= 2.0 ** -20 * w).all()
    offsets, pairs = X.lists(ids, n)
    assert torch.equal(s.offsets.cpu(), offsets) and torch.equal(s.pairs[: T * k].cpu(), pairs)
    a64 = X.rows64(s.a, s.a_scales)
    for e in range(n):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < hi:
            mine = pairs[lo:hi].long().cuda()
            check_codes(s.a[lo:hi], s.a_scales[lo:hi], *_glu(x64[mine // k], s.up[1], s.up[2], e))
            _near(s.y[mine], *X.product(a64[lo:hi], X.weight64(s.down[1][e, 0], s.down[2][e, 0])), s.inter, "bf16")
    check_codes(s.b[:T], s.b_scales[:T], *_glu(x64, s.shared_up[1], s.shared_up[2], 0))
    shared, mass = X.product(X.rows64(s.b[:T], s.b_scales[:T]), X.weight64(s.shared_down[1][0, 0], s.shared_down[2][0, 0]))
    terms = s.y[: T * k].double().view(T, k, -1) * s.weights[:T].double()[:, :, None]
    # the shared expert's output is rounded to bf16 before it is added, and the sum once more
    want, size = shared + terms.sum(1), shared.abs() + terms.abs().sum(1)
    off = 2.0 ** -8 * (shared.abs() + want.abs()) * (1 + 2.0 ** -7) + X.sum_error(s.shared_inter) * mass * 2 + (k + 2) * 2.0 ** -24 * size
    assert ((s.out[:T].double() - want).abs() <= off + 1e-30).all()


@pytest.mark.parametrize("T", [1, 2, 33, 300])
def test_every_stage(E, T):
    s = _sublayer()
    codes, scales = _rows(E, T, s.dim, T)
    s.forward(codes, scales, T)
    assert E.engram_check() == 0
    _check(s, codes, scales, T)


def test_onto_a_strided_stream(E):
    s = _sublayer()
    h = torch.randn((40, 3, s.dim), generator=rng(1), device="cuda")
    before = h.clone()
    codes, scales = _rows(E, 40, s.dim, 0, h[:, 1].contiguous())
    y = s.forward(codes, scales, 40, h[:, 1]).float()
    assert E.engram_check() == 0
    assert torch.equal(h[:, 1], before[:, 1] + y) and torch.equal(h[:, ::2], before[:, ::2])


def test_graphs_see_new_inputs_and_give_the_same_bits(E):
    """Captured once, replayed with other rows: as eager calls; a second graph of other buffers beside it."""
    subs = [_sublayer(seed=3), _sublayer(seed=4, top_k=6)]
    graphs = []
    side = torch.cuda.Stream()
    for s, T in zip(subs, (1, 120)):
        codes, scales = _rows(E, T, s.dim, 9)
        s.forward(codes, scales, T)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.forward(codes, scales, T)
        graphs.append((s, T, codes, scales, g))
    for turn in range(3):
        streams = [torch.cuda.Stream() for _ in graphs]
        for (s, T, codes, scales, g), st in zip(graphs, streams):
            c, sc = _rows(E, T, s.dim, 50 + turn)
            codes.copy_(c)
            scales.copy_(sc)
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for s, T, codes, scales, g in graphs:
            got = [x.clone() for x in (s.out[:T], s.ids[:T], s.a[: T * s.top_k], s.offsets)]
            s.forward(codes, scales, T)
            assert E.engram_check() == 0
            for x, y in zip(got, (s.out[:T], s.ids[:T], s.a[: T * s.top_k], s.offsets)):
                assert torch.equal(x, y)
    s, T, codes, scales, _ = graphs[1]
    _check(s, codes, scales, T)


def test_captured_behind_copies_and_other_streams(E):
    """A capture in which copies, and a kernel of another stream, come before the calls and behind them."""
    s = _sublayer(seed=7)
    T = 50
    source = [_rows(E, T, s.dim, i) for i in (1, 2)]
    codes, scales = (torch.empty_like(x) for x in source[0])
    kept = torch.empty((T, s.dim), dtype=torch.bfloat16, device="cuda")
    want = []
    for c, sc in source:
        want.append(s.forward(c, sc, T).clone())
    torch.cuda.synchronize()
    staged = [x.clone() for x in source[0]]
    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        codes.copy_(staged[0])
        other.wait_stream(main)
        with torch.cuda.stream(other):
            scales.copy_(staged[1])
        main.wait_stream(other)
        y = s.forward(codes, scales, T)
        kept.copy_(y)
    for (c, sc), w in zip(source, want):
        staged[0].copy_(c)
        staged[1].copy_(sc)
        kept.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert E.engram_check() == 0 and torch.equal(kept, w)


def test_results_do_not_change_with_what_runs_before(E):
    """The calls start beside the end of the kernel before them: one that writes their input late, and one that reads their output."""
    g = rng(8)
    rows, K, N = 96, 2048, 512
    w = E.Fp8Weight(torch.full((1, N, K), 0x38, dtype=torch.uint8, device="cuda"),
                    torch.full((1, N // 128, K // 128), 127, dtype=torch.uint8, device="cuda"), E.ENGRAM_FMT_FP8_E8M0, 1, N, K)
    x = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
    sc = torch.full((rows, K // 128), 127, dtype=torch.uint8, device="cuda")
    y = torch.zeros((rows, N), device="cuda")
    pick = torch.tensor([0x38, 0x40], dtype=torch.uint8, device="cuda")     # 1 and 2
    for turn in range(30):
        big = torch.randn((2048, 2048), generator=g, device="cuda")
        late = (big @ big).abs().argmax() * 0 + turn % 2                    # a value that takes a while to be there
        x.copy_(pick[late].expand(rows, K))
        E.engram_project_fp8(x, 0, sc, E.ENGRAM_FMT_FP8_E8M0, rows, w, None, E.ENGRAM_T_F32, y, 0)
        got = y.clone()
        E.engram_project_fp8(x, 0, sc, E.ENGRAM_FMT_FP8_E8M0, 1, w, None, E.ENGRAM_T_F32, y, 0)
        assert (got == K * (1 + turn % 2)).all() and torch.equal(got, y)
    assert E.engram_check() == 0


def test_two_streams_at_once(E):
    """Calls of unlike sizes that overlap: each with its buffers, both as alone."""
    subs = [_sublayer(seed=5), _sublayer(seed=6)]
    rows = [_rows(E, T, 512, T) for T in (300, 7)]
    alone = []
    for s, r, T in zip(subs, rows, (300, 7)):
        alone.append(s.forward(*r, T).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, r, T, st in zip(subs, rows, (300, 7), streams):
            with torch.cuda.stream(st):
                s.forward(*r, T)
    torch.cuda.synchronize()
    assert E.engram_check() == 0
    for s, want, T in zip(subs, alone, (300, 7)):
        assert torch.equal(s.out[:T], want)


def test_idle_tokens_of_a_padded_batch(E):
    """Tokens whose logits are all masked go nowhere and get the shared expert's output alone."""
    s = _sublayer()
    T, fmt = 64, E.ENGRAM_FMT_FP8_E8M0
    codes, scales = _rows(E, T, s.dim, 2)
    s.forward(codes, scales, T)
    full = s.out[:T].clone()
    idle = torch.arange(T, device="cuda") % 3 == 1
    s.logits[:T][idle] = -math.inf
    s.y.fill_(math.nan)
    lists = E.ExpertLists(s.offsets, s.pairs, s.n_experts, s.top_k, T)
    E.engram_route(s.router, 2, s.logits, 0, s.bias, T, s.ids, s.weights, lists, s.ws, s.ws_bytes)
    E.engram_glu_fp8(codes, 0, scales, fmt, T, s.up[0], lists, 0.0, fmt, s.a, s.a_scales)
    E.engram_project_fp8(s.a, 0, s.a_scales, fmt, T * s.top_k, s.down[0], lists, 0, s.y, 0)
    E.engram_project_fp8(s.b, 0, s.b_scales, fmt, T, s.shared_down[0], None, 0, s.out, 0)
    shared = s.out[:T].clone()
    E.engram_combine(s.y, 0, 0, s.weights, T, s.top_k, s.dim, s.out, 0, 0, 0, s.out, 0)
    assert E.engram_check() == 0
    assert int(s.offsets[-1]) == int((~idle).sum()) * s.top_k and (s.ids[:T][idle] == -1).all()
    assert torch.equal(s.out[:T][~idle], full[~idle]) and torch.equal(s.out[:T][idle], shared[idle])


def test_behind_the_attention(E):
    """The example's chain: engram, attention, experts, for a prompt and a token."""
    import numpy as np
    from deepseek_v4_engram_hash_gb300 import configs, runner, synth
    from examples.attention_sublayer import AttentionSublayer
    cfg = configs.V41_DECODE
    eng = runner.EngramSetup(cfg, batch=1, max_tokens=40)
    attention = AttentionSublayer(cfg.dim, 8, 2, 128, batch=1, max_seq=41, scale_block=128)
    s = _sublayer(dim=cfg.dim, max_tokens=40)
    for T, pos in ((40, 0), (1, 40)):
        d_h = torch.from_numpy(synth.highway(cfg, np.arange(pos, pos + T))).cuda()
        eng.forward(eng.ids_for(f"behind{pos}", T), pos, d_h)
        codes, scales = attention.forward(d_h, 0, T)
        before = d_h.clone()
        y = s.forward(codes, scales, T, d_h[:, 0]).float()
        assert E.engram_check() == 0
        assert torch.equal(d_h[:, 0], before[:, 0] + y) and torch.equal(d_h[:, 1:], before[:, 1:])
        _check(s, codes, scales, T)


