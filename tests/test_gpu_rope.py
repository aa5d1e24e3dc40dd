"""GPU parity of the rotations (la_rope, la_rope_append and its paged form) against the fp64 oracle.

Tolerance. y = s (u cos a -+ w sin a): the angle's fraction of a turn is rounded to 24 bits (2^-25
half turns, pi * 2^-25 of the angle), sincospif is good to 2 units in the last place (2^-22), the
scaling and the two products and the sum round once each (3 * 2^-24). Together less than 2^-20 of
s (|u| + |w|), before the rounding to the result's type (half a step: eps / 2 of the value; fp16's
smallest step is 2^-24). Copied channels and values are exact.
"""
import numpy as np
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCALED = dict(scaling="pairs", factor=8.0, original_max=4096, base=1e6)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def assert_turned(got, x, ref, rotary, layout, out_scale=1.0):
    dtype = got.dtype
    g, x = got.double().cpu().numpy(), x.double().cpu().numpy()
    half = rotary // 2
    mag = np.zeros_like(x)
    if layout == "half":
        m = np.abs(x[..., :half]) + np.abs(x[..., half:rotary])
        mag[..., :half] = mag[..., half:rotary] = m
    else:
        m = np.abs(x[..., 0:rotary:2]) + np.abs(x[..., 1:rotary:2])
        mag[..., 0:rotary:2] = mag[..., 1:rotary:2] = m
    eps = torch.finfo(dtype).eps / 2
    fp32 = 2.0 ** -20 * abs(out_scale) * mag
    tol = (np.abs(ref) + fp32) * eps + fp32 + (2.0 ** -25 if dtype is torch.float16 else 0.0)
    assert np.isfinite(g).all()
    worst = (np.abs(g - ref) - tol).max()
    assert worst <= 0, f"beyond tolerance by {worst:.3e}"
    assert np.array_equal(g[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rotary", [(1, 1, 128, 128), (7, 16, 128, 64), (33, 3, 80, 80), (33, 3, 80, 20),
                                          (5, 2, 66, 66), (3, 1, 2, 2), (600, 2, 256, 256), (257, 5, 64, 32),
                                          (2, 70, 128, 34), (1300, 1, 72, 48)])
def test_rotation(dtype, layout, T, H, D, rotary):
    g = torch.Generator().manual_seed(T * 131 + H * 7 + D + rotary)
    x = torch.randn(T, H, D, generator=g).to(DTYPES[dtype]).cuda()
    pos = torch.randint(-50, 200000, (T,), generator=g, dtype=torch.int32)
    kw = SCALED if rotary == 64 else {}
    plan = bmw.RopePlan.make(rotary, layout=layout, out_scale=1.5, **kw)
    angles = oracle.rope_angles(rotary, **kw)
    for inverse in (False, True):
        out = torch.full_like(x, float("nan"))
        bmw.la_rope(plan, x, pos.cuda(), out, inverse=inverse)
        ref = oracle.rotate(x, pos.numpy(), angles, layout, 1.5, inverse)
        assert_turned(out, x, ref, rotary, layout, 1.5)
    again = x.clone()
    bmw.la_rope(plan, again, pos.cuda(), again, inverse=True)      # in place
    assert torch.equal(again, out)


def test_far_positions():
    """Positions to the ends of int32: the angle is a fraction of a turn of 2^31 positions."""
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    x = torch.randn(7, 2, 128, generator=torch.Generator().manual_seed(0)).cuda()
    out = torch.empty_like(x)
    bmw.la_rope(bmw.RopePlan.make(128), x, pos.cuda(), out)
    # At 2^31 positions the oracle's own angle, and the library's turns, are off by 2^-53 of the
    # angle or of the turns: 2^31 * 2^-52 = 2^-21 radians, 2^-20 for the two, of |u| + |w|.
    ref = oracle.rotate(x, pos.numpy().astype(np.float64), oracle.rope_angles(128))
    g, xx = out.double().cpu().numpy(), x.double().cpu().numpy()
    m = np.abs(xx[..., :64]) + np.abs(xx[..., 64:])
    tol = 2.0 ** -19 * np.concatenate([m, m], -1) + 2.0 ** -24 * np.abs(ref)
    assert (np.abs(g - ref) <= tol).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides(layout):
    """Heads outside tokens, a part of a wider row, an odd offset (no 16-byte chunks), a broadcast
    input; what lies between the output's rows is left as it was."""
    g = torch.Generator().manual_seed(3)
    T, H, D, rotary = 37, 4, 64, 32
    plan, angles = bmw.RopePlan.make(rotary, layout=layout), oracle.rope_angles(rotary)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    wide = torch.randn(T, H * D + 24, generator=g).to(torch.bfloat16).cuda()
    inputs = [torch.randn(H, T, D, generator=g).cuda().transpose(0, 1),
              wide[:, 8:8 + H * D].unflatten(1, (H, D)), wide[:, 3:3 + H * D].unflatten(1, (H, D)),
              torch.randn(T, 1, D, generator=g).half().cuda().expand(T, H, D)]
    for x in inputs:
        ref = oracle.rotate(x, np.arange(T), angles, layout)
        for head_major in (False, True):
            for offset in (0, 1):
                buf = torch.full((2 * T * H * D + 64,), 7.0, dtype=x.dtype, device="cuda")[offset:]
                st = (D + 8, T * (D + 8)) if head_major else (H * D + 16, D)
                out = buf.as_strided((T, H, D), (*st, 1))
                bmw.la_rope(plan, x, pos, out)
                assert_turned(out, x, ref, rotary, layout)
                out.fill_(7.0)
                assert bool((buf == 7.0).all())
    with pytest.raises(bmw.LaError):
        bmw.la_rope(plan, inputs[0], pos, inputs[0].contiguous()[:1].expand(T, H, D))
    with pytest.raises(ValueError):
        bmw.la_rope(plan, inputs[0], pos, torch.empty(T, D, H, device="cuda").transpose(1, 2))


def test_empty_and_large():
    plan = bmw.RopePlan.make(64)
    e = torch.empty(0, 4, 64, device="cuda")
    bmw.la_rope(plan, e, torch.empty(0, dtype=torch.int32, device="cuda"), e)
    # more elements than 2^31, the last rows checked
    T, H, D = 2 ** 15 + 5, 1024, 64
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, H, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    bmw.la_rope(plan, x, pos, out := torch.empty_like(x))
    ref = oracle.rotate(x[-3:], np.arange(T - 3, T), oracle.rope_angles(64))
    assert_turned(out[-3:], x[-3:], ref, 64, "half")
    assert not out[:-3].any()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    """The inverse form is the gradient: against the oracle's transpose and against differences."""
    g = torch.Generator().manual_seed(9)
    T, H, D, rotary = 11, 2, 48, 32
    plan, angles = bmw.RopePlan.make(rotary, layout=layout, out_scale=1.25), oracle.rope_angles(rotary)
    x = torch.randn(T, H, D, generator=g).cuda()
    dy = torch.randn(T, H, D, generator=g).cuda()
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).cuda()
    dx = torch.empty_like(x)
    bmw.la_rope(plan, dy, pos, dx, inverse=True)
    assert_turned(dx, dy, oracle.rotate(dy, pos.cpu().numpy(), angles, layout, 1.25, inverse=True), rotary,
                  layout, 1.25)
    # d/de sum(dy * rope(x + e v)) = sum(dx * v), exactly linear: a difference of the oracle's
    v = np.random.default_rng(0).standard_normal(x.shape)
    p, d = pos.cpu().numpy(), dy.double().cpu().numpy()
    f = lambda y: (d * oracle.rotate(y, p, angles, layout, 1.25)).sum()  # noqa: E731
    diff = f(x.double().cpu().numpy() + v) - f(x.double().cpu().numpy())
    got = (dx.double().cpu().numpy() * v).sum()
    # each dx is off by at most 2^-20 * 1.25 (|u| + |w|) (see above)
    assert abs(got - diff) <= 2.0 ** -19 * 1.25 * np.abs(d).max() * 2 * np.abs(v).sum()


def _append_case(B, T, S, lens, rows, page, packed, Hq=16, Hkv=2, seed=0):
    g = torch.Generator().manual_seed(seed)
    D = 128
    if packed:
        qkv = torch.randn(B, T, (Hq + 2 * Hkv) * D + 8, generator=g).to(torch.bfloat16).cuda()
        parts = qkv[..., 8:].split([Hq * D, Hkv * D, Hkv * D], -1)
        q, kn, vn = (t.unflatten(-1, (-1, D)) for t in parts)
    else:
        q, kn, vn = (torch.randn(B, T, h, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    for b, n in enumerate(rows):           # padding must not be read into anything
        for t in (q, kn, vn):
            t[b, max(n, 0):] = float("nan")
    table = None
    if page:
        per = -(-S // page)
        table = torch.randperm(B * per + 2, generator=g)[:B * per].view(B, per).to(torch.int32).cuda()
        shape = (B * per + 2, Hkv, page, D)
    else:
        shape = (B, Hkv, S, D)
    k, v = (torch.randn(shape, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    return q, kn, vn, k, v, table


@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 96), ("half", 50), ("interleaved", 128),
                                           ("interleaved", 30)])
@pytest.mark.parametrize("page", [0, 64, 192])
@pytest.mark.parametrize("packed", [False, True])
def test_append(layout, rotary, page, packed):
    """Windows that straddle pages, of every length from none, next to invalid sequences; slots,
    positions, padding and the rest of the caches exactly."""
    lens = [0, 60, 127, 376, 5, -1, 380, 10, 383]
    rows = [9, 9, 3, 8, 0, 4, 5, 10, 1]      # sequence 5: P < 0; 6: past the cache; 7: more than T
    B, T, S = len(lens), 9, 384
    q, kn, vn, k, v, table = _append_case(B, T, S, lens, rows, page, packed)
    cfg = bmw.Config.make(B, 16, 2, S)
    plan = bmw.RopePlan.make(rotary, layout=layout, **SCALED)
    angles = oracle.rope_angles(rotary, **SCALED)
    pos0 = torch.tensor([p + 70000 for p in lens], dtype=torch.int32)
    q_out = torch.full((B, T, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    key_pos = torch.full((B, 2, S), -9, dtype=torch.int32, device="cuda")
    k0, v0 = k.clone(), v.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    opt = dict(row_lens=i32(rows), pos0=pos0.cuda(), key_pos=key_pos)
    if page:
        bmw.la_rope_append_paged(cfg, plan, q, kn, vn, table, i32(lens), q_out, k, v, **opt)
    else:
        bmw.la_rope_append(cfg, plan, q, kn, vn, i32(lens), q_out, k, v, **opt)
    for b, (P, n) in enumerate(zip(lens, rows)):
        live = n if P >= 0 and n <= T and P + n <= S else 0
        assert bool((q_out[b, live:] == 7.0).all())
        pos = int(pos0[b]) + np.arange(live)
        if live:
            assert_turned(q_out[b, :live], q[b, :live], oracle.rotate(q[b, :live], pos, angles, layout), rotary,
                          layout)
        want = torch.full((S,), -9, dtype=torch.int32)
        want[P:P + live] = torch.from_numpy(pos.astype(np.int32)) if live else want[P:P]
        assert torch.equal(key_pos[b].cpu(), want.expand(2, S))
        for i in range(live):
            at = (b, slice(None), P + i) if not page else (int(table[b, (P + i) // page]), slice(None), (P + i) % page)
            ref = oracle.rotate(kn[b, i:i + 1], pos[i:i + 1], angles, layout)[0]
            assert_turned(k[at], kn[b, i], ref, rotary, layout)
            assert torch.equal(v[at], vn[b, i])
            k0[at], v0[at] = k[at], v[at]
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_append_prompt_defaults():
    """A whole prompt into an empty cache (no lengths, no positions), more rows than a window may
    have; q in place; equal to the rotation alone."""
    B, T, S = 2, 700, 704
    q, kn, vn, k, v, _ = _append_case(B, T, S, [0, 0], [T, T], 0, False, Hq=8, Hkv=4)
    cfg, plan = bmw.Config.make(B, 8, 4, S), bmw.RopePlan.make(128)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B)
    want_q, want_k = torch.empty_like(q), torch.empty_like(kn)
    bmw.la_rope(plan, q.flatten(0, 1), pos, want_q.view(B * T, 8, 128))
    bmw.la_rope(plan, kn.flatten(0, 1), pos, want_k.view(B * T, 4, 128))
    bmw.la_rope_append(cfg, plan, q, kn, vn, None, q, k, v)
    assert torch.equal(q, want_q)
    assert torch.equal(k[:, :, :T], want_k.transpose(1, 2)) and torch.equal(v[:, :, :T], vn.transpose(1, 2))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (18, 2), (22, 11), (35, 5)])
@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 64), ("half", 50), ("interleaved", 128),
                                           ("interleaved", 48)])
def test_append_in_place_of_any_heads(Hq, Hkv, layout, rotary):
    """Head counts that do not divide over a warp, q in place: the bits of a separate output."""
    B, T, S = 3, 130, 192
    rows = [130, 0, 77]
    q, kn, vn, k, v, _ = _append_case(B, T, S, None, rows, 0, False, Hq=Hq, Hkv=Hkv, seed=Hq)
    cfg, plan = bmw.Config.make(B, Hq, Hkv, S), bmw.RopePlan.make(rotary, layout=layout)
    n = torch.tensor(rows, dtype=torch.int32, device="cuda")
    x, apart, k2, v2 = q.clone(), q.clone(), k.clone(), v.clone()
    bmw.la_rope_append(cfg, plan, q, kn, vn, None, apart, k, v, row_lens=n)
    bmw.la_rope_append(cfg, plan, q, kn, vn, None, q, k2, v2, row_lens=n)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    for b, r in enumerate(rows):
        assert torch.equal(q[b, :r], apart[b, :r])
        assert torch.isnan(q[b, r:]).all()
        ref = oracle.rotate(x[b, :r], np.arange(r), oracle.rope_angles(rotary), layout)
        if r:
            assert_turned(apart[b, :r], x[b, :r], ref, rotary, layout)


def test_append_skips_pages_outside_the_pool():
    B, T, page = 1, 6, 64
    q, kn, vn, k, v, table = _append_case(B, T, 128, [60], [6], page, False)
    table[0, 1] = 1 << 30
    k0 = k.clone()
    cfg, plan = bmw.Config.make(B, 16, 2, 128), bmw.RopePlan.make(128)
    q_out = torch.empty_like(q)
    key_pos = torch.full((1, 2, 128), -9, dtype=torch.int32, device="cuda")
    bmw.la_rope_append_paged(cfg, plan, q, kn, vn, table, torch.tensor([60], dtype=torch.int32, device="cuda"),
                             q_out, k, v, key_pos=key_pos)
    page0 = int(table[0, 0])
    assert not torch.equal(k[page0, :, 60:], k0[page0, :, 60:])
    k[page0, :, 60:] = k0[page0, :, 60:]
    assert torch.equal(k, k0) and torch.isfinite(q_out).all()
    assert key_pos[0, 0, 60:70].tolist() == [60, 61, 62, 63] + [-9] * 6


def test_other_stream_and_graph():
    """On a stream that is not the current one, and captured into a graph and replayed with new
    contents."""
    x = torch.randn(64, 4, 128, generator=torch.Generator().manual_seed(5)).cuda()
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    plan, out, want = bmw.RopePlan.make(128), torch.empty_like(x), torch.empty_like(x)
    bmw.la_rope(plan, x, pos, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bmw.la_rope(plan, x, pos, out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bmw.la_rope(plan, x, pos, out)
        bmw.la_rope(plan, out, pos, out, inverse=True)
    y = torch.randn_like(x)
    x.copy_(y)
    graph.replay()
    # there and back: two rotations of 2^-20 (|u| + |w|) each
    torch.cuda.synchronize()
    m = y.abs()[..., :64] + y.abs()[..., 64:]
    assert bool(((out - y).abs() <= 2.0 ** -18 * torch.cat([m, m], -1)).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("offset", [0, 1])
def test_fp32_rounds_like_fp32(layout, offset):
    """fp32 results are as near to the exact ones as those of the same fp32 arithmetic with exactly
    rounded cosines and sines.

    In units of 2^-24 of |y| (u, w of variance 1): each rounded cosine and sine has a variance of 0.059
    (measured over all angles; ulp^2 / 12), the two products' and the sum's roundings 0.27 together, so
    plain arithmetic's is 0.39. The kernel's angle, an eighth of a turn at most in 24 bits, adds 0.27
    of a rounding's variance, and a function good to one unit, uniform over 3/4 of it to either
    side, has 2.25 of it: 0.059 * 2 * 2.25 * 1.27 + 0.27 = 0.61, a ratio of 1.25 in the norm. (A whole turn
    in 24 bits has 5 times a rounding's variance: 1.49.)
    """
    g = torch.Generator().manual_seed(12)
    T, H, D = 3000, 3, 128
    x = torch.empty(T, H * D + offset)[:, offset:].unflatten(1, (H, D)).copy_(torch.randn(T, H, D, generator=g))
    pos = torch.randint(-2 ** 20, 2 ** 20, (T,), generator=g, dtype=torch.int32)
    a = pos.numpy().astype(np.float64)[:, None, None] * oracle.rope_angles(D)
    c, s = np.cos(a), np.sin(a)
    u, w = ((x[..., :64], x[..., 64:]) if layout == "half" else (x[..., 0::2], x[..., 1::2]))
    u, w = u.numpy(), w.numpy()
    dev = torch.empty(T, H * D + offset, device="cuda")[:, offset:].unflatten(1, (H, D)).copy_(x)
    out = torch.empty_like(dev, memory_format=torch.contiguous_format)
    for inverse in (False, True):
        sn = -s if inverse else s
        exact = np.stack([u * c - w * sn, w * c + u * sn])
        c32, s32 = c.astype(np.float32), sn.astype(np.float32)
        plain = np.stack([(np.float64(u) * c32 - np.float64(w * s32)), (np.float64(w) * c32 + np.float64(u * s32))])
        bmw.la_rope(bmw.RopePlan.make(D, layout=layout), dev, pos.cuda(), out, inverse=inverse)
        y = out.cpu().numpy()
        y = np.stack([y[..., :64], y[..., 64:]] if layout == "half" else [y[..., 0::2], y[..., 1::2]])
        err = [np.linalg.norm(v.astype(np.float32) - exact) / np.linalg.norm(exact) for v in (y, plain)]
        assert err[0] <= 1.25 * err[1], err
