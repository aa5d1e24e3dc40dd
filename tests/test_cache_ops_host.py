"""CPU checks of the operators around the window attention: rotation plans against their
formulas, the oracle's own properties, and every refusal that needs no device."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle


@pytest.fixture(scope="module")
def lib():
    from block_masked_window_b200 import build
    build.build()
    return bmw.load()


def _cfg(**kw):
    base = dict(batch=2, num_q_heads=16, num_kv_heads=2, max_seq=256)
    base.update(kw)
    return bmw.Config.make(**base)


SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=4.0)),
            ("pairs", dict(factor=8.0, original_max=4096)),
            ("turns", dict(factor=8.0, original_max=8192, low_turns=1.0, high_turns=4.0))]


@pytest.mark.parametrize("rotary", [2, 4, 20, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", SCALINGS, ids=[s for s, _ in SCALINGS])
@pytest.mark.parametrize("base", [10000.0, 1000000.0])
def test_plan_formulas(lib, rotary, scaling, kw, base):
    plan = bmw.RopePlan.make(rotary, base=base, layout="interleaved", scaling=scaling, out_scale=1.25, **kw)
    ref = oracle.rope_angles(rotary, base=base, scaling=scaling, **kw) / (2 * math.pi)
    got = np.array(plan.turns[:])
    # pow and exp of 64 bits: a few units in the last place
    np.testing.assert_allclose(got[:rotary // 2], ref, rtol=1e-13)
    assert not got[rotary // 2:].any()
    assert (plan.rotary_dim, plan.layout, plan.out_scale) == (rotary, bmw.LA_ROPE_INTERLEAVED, 1.25)


def test_plan_scalings_differ_where_they_should():
    plain = oracle.rope_angles(128, base=1e6)
    assert np.allclose(oracle.rope_angles(128, base=1e6, scaling="linear", factor=4.0), plain / 4)
    for scaling, kw in SCALINGS[3:]:
        w = oracle.rope_angles(128, base=1e6, scaling=scaling, **kw)
        assert w[0] == pytest.approx(plain[0]) and w[-1] == pytest.approx(plain[-1] / kw["factor"])
        assert np.all((w <= plain * (1 + 1e-12)) & (w >= plain / kw["factor"] * (1 - 1e-12)))


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(layout=2), dict(scaling=5),
    dict(scaling=-1), dict(base=1.0), dict(base=float("nan")), dict(out_scale=float("inf")),
    dict(scaling="linear", factor=0.0), dict(scaling="linear", factor=float("nan")),
    dict(scaling="base", factor=-1.0), dict(scaling="pairs", original_max=0),
    dict(scaling="pairs", original_max=10, low_turns=2.0, high_turns=2.0),
    dict(scaling="turns", original_max=10, low_turns=0.0, high_turns=2.0),
    dict(scaling="turns", original_max=10, low_turns=1.0, high_turns=float("inf")),
])
def test_plan_refusals(lib, kw):
    args = dict(rotary_dim=64)
    args.update(kw)
    with pytest.raises(bmw.LaError) as e:
        bmw.RopePlan.make(**args)
    assert e.value.status == 1
    assert lib.la_rope_plan_init(None, 64, 0, 0, 10000.0, 1.0, 1, 1.0, 32.0, 1.0) == 1


def _rope(lib, plan, dtype=0, x=256, xt=256, xh=128, pos=256, T=4, H=2, D=128, out=512, ot=256, oh=128):
    return lib.la_rope(ctypes.byref(plan) if plan is not None else None, dtype, x, xt, xh, pos, T, H, D, 0,
                       out, ot, oh, None)


def test_rope_refusals(lib):
    plan = bmw.RopePlan.make(64)
    assert _rope(lib, plan, T=0) == 0                    # no work
    assert _rope(lib, None) == 1
    assert _rope(lib, plan, dtype=3) == 1
    assert _rope(lib, plan, T=-1) == 1 and _rope(lib, plan, H=0) == 1 and _rope(lib, plan, D=0) == 1
    assert _rope(lib, plan, D=127) == 2 and _rope(lib, plan, D=258) == 2
    assert _rope(lib, plan, D=62) == 1                   # narrower than the rotation
    assert _rope(lib, plan, x=0) == 1 and _rope(lib, plan, out=0) == 1 and _rope(lib, plan, pos=0) == 1
    assert _rope(lib, plan, x=257) == 1 and _rope(lib, plan, pos=258) == 1
    assert _rope(lib, plan, dtype=2, x=258) == 1
    assert _rope(lib, plan, oh=64) == 1                  # heads of the output overlap
    assert _rope(lib, plan, ot=128) == 1                 # tokens of the output overlap
    assert _rope(lib, plan, ot=0) == 1 and _rope(lib, plan, xt=-256) == 1
    assert _rope(lib, plan, x=512, xt=512) == 1          # in place with other strides
    bad = bmw.RopePlan.make(64)
    bad.rotary_dim = 300
    assert _rope(lib, bad, D=256) == 1
    bad.rotary_dim, bad.layout = 64, 7
    assert _rope(lib, bad) == 1


def _append(lib, cfg, plan, paged=False, **kw):
    a = dict(q=256, sq=2048, k=256, sk=256, v=256, sv=256, table=256, pps=4, size=64, pages=8, lens=256,
             rows=256, pos0=256, T=6, q_out=512, kc=256, vc=256, key_pos=256)
    a.update(kw)
    c = ctypes.byref(cfg) if cfg is not None else None
    p = ctypes.byref(plan) if plan is not None else None
    head = (c, p, a["q"], a["sq"], a["k"], a["sk"], a["v"], a["sv"])
    tail = (a["lens"], a["rows"], a["pos0"], a["T"], a["q_out"], a["kc"], a["vc"], a["key_pos"], None)
    if paged:
        return lib.la_rope_append_paged(*head, a["table"], a["pps"], a["size"], a["pages"], *tail)
    return lib.la_rope_append(*head, *tail)


@pytest.mark.parametrize("paged", [False, True])
def test_rope_append_refusals(lib, paged):
    cfg, plan = _cfg(), bmw.RopePlan.make(128)
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(q_out=0), dict(kc=0), dict(vc=0), dict(T=0), dict(q=264),
               dict(k=264), dict(v=264), dict(q_out=264), dict(kc=264), dict(vc=264), dict(lens=258),
               dict(rows=258), dict(pos0=258), dict(key_pos=258), dict(sq=2040), dict(sk=128),
               dict(sv=252), dict(sq=2052), dict(q=512, sq=2560)):
        assert _append(lib, cfg, plan, paged, **kw) == 1, kw
    assert _append(lib, None, plan, paged) == 1 and _append(lib, cfg, None, paged) == 1
    assert _append(lib, cfg, bmw.RopePlan.make(130), paged) == 1      # wider than a head
    assert _append(lib, _cfg(head_dim=64), plan, paged) == 2
    assert _append(lib, _cfg(batch=4096, max_seq=64), plan, paged, T=1 << 20, pps=1) == 2
    if paged:
        for kw in (dict(table=0), dict(table=258), dict(pps=0), dict(size=32), dict(size=96), dict(pages=0)):
            assert _append(lib, cfg, plan, True, **kw) == 1, kw
        assert _append(lib, cfg, plan, True, pages=1 << 25) == 2


def _evict(lib, cfg, paged=False, **kw):
    need = 1 << 30
    a = dict(w=256, pos=256, table=256, pps=4, size=64, pages=8, lens=256, nxt=256, budget=16, sink=4, recent=8,
             kc=256, vc=256, w_out=256, pos_out=256, kept=256, new=256, ws=256, nb=need)
    a.update(kw)
    c = ctypes.byref(cfg) if cfg is not None else None
    tail = (a["lens"], a["nxt"], a["budget"], a["sink"], a["recent"], a["kc"], a["vc"], a["w_out"],
            a["pos_out"], a["kept"], a["new"], a["ws"], a["nb"], None)
    if paged:
        return lib.la_kv_evict_paged(c, a["w"], a["pos"], a["table"], a["pps"], a["size"], a["pages"], *tail)
    return lib.la_kv_evict(c, a["w"], a["pos"], *tail)


@pytest.mark.parametrize("paged", [False, True])
def test_evict_refusals(lib, paged):
    cfg = _cfg()
    for kw in (dict(w=0), dict(lens=0), dict(kc=0), dict(vc=0), dict(w_out=0), dict(new=0), dict(budget=0),
               dict(budget=257), dict(sink=-1), dict(recent=-1), dict(sink=9, recent=8),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(w=258), dict(pos=258), dict(lens=258),
               dict(nxt=258), dict(kc=264), dict(vc=264), dict(w_out=258), dict(pos_out=258), dict(kept=258),
               dict(new=258), dict(pos_out=0)):
        assert _evict(lib, cfg, paged, **kw) == 1, kw
    assert _evict(lib, None, paged) == 1
    assert _evict(lib, cfg, paged, ws=0) == 3 and _evict(lib, cfg, paged, ws=264) == 3
    assert _evict(lib, cfg, paged, nb=bmw.la_kv_evict_workspace_bytes(cfg) - 1) == 3
    assert bmw.la_kv_evict_workspace_bytes(_cfg(head_dim=64)) == 0
    # the smallest one is still a workspace for la_pbd_workspace_init, which refuses less than this
    least = bmw.la_kv_evict_workspace_bytes(_cfg(batch=1, num_q_heads=1, num_kv_heads=1, max_seq=1))
    assert lib.la_pbd_workspace_init(256 + 1, least, None) == 3 and least >= 16896
    if paged:
        assert _evict(lib, cfg, True, table=0) == 1 and _evict(lib, cfg, True, size=65) == 1
        assert _evict(lib, cfg, True, pages=1 << 25) == 2


def _weights(lib, cfg, W=6, paged=False, **kw):
    a = dict(q=256, kc=256, vc=256, table=256, pps=4, size=64, pages=8, lens=256, wl=256, out=256, win=256,
             decay=1.0, wout=256, ws=256, nb=1 << 30)
    a.update(kw)
    tail = (a["lens"], a["wl"], W, a["out"], a["win"], a["decay"], a["wout"], a["ws"], a["nb"], None)
    c = ctypes.byref(cfg) if cfg is not None else None
    if paged:
        return lib.la_pbd_attn_weights_paged(c, a["q"], a["kc"], a["vc"], a["table"], a["pps"], a["size"],
                                             a["pages"], *tail)
    return lib.la_pbd_attn_weights(c, a["q"], a["kc"], a["vc"], *tail)


@pytest.mark.parametrize("paged", [False, True])
def test_attn_weights_refusals(lib, paged):
    cfg = _cfg()
    assert _weights(lib, None, paged=paged) == 1
    for kw in (dict(q=0), dict(kc=0), dict(vc=0), dict(lens=0), dict(out=0), dict(q=264)):
        assert _weights(lib, cfg, paged=paged, **kw) == 1, kw
    assert _weights(lib, cfg, W=0, paged=paged) == 1 and _weights(lib, cfg, W=17, paged=paged) == 1
    assert _weights(lib, _cfg(head_dim=64), paged=paged) == 2
    assert _weights(lib, cfg, paged=paged, ws=0) == 3
    assert bmw.la_pbd_attn_weights_workspace_bytes(cfg, 17) == 0
    if paged:
        assert _weights(lib, cfg, W=11, paged=True) == 2 and _weights(lib, cfg, paged=True, size=32) == 1


def _verify(lib, dtype=2, **kw):
    a = dict(p=256, pb=6000, pr=1000, q=256, qb=5000, qr=1000, x=256, xl=256, u=256, su=256, B=2, K=5, V=1000,
             tok=256, acc=256, sl=256, slo=256)
    a.update(kw)
    return lib.la_pbd_verify(dtype, a["p"], a["pb"], a["pr"], a["q"], a["qb"], a["qr"], a["x"], a["xl"], a["u"],
                             a["su"], a["B"], a["K"], a["V"], a["tok"], a["acc"], a["sl"], a["slo"], None)


def test_verify_refusals(lib):
    for kw in (dict(dtype=3), dict(p=0), dict(su=0), dict(tok=0), dict(acc=0), dict(x=0), dict(u=0), dict(B=0),
               dict(K=-1), dict(V=0), dict(sl=0), dict(slo=0), dict(p=258), dict(q=258), dict(x=258),
               dict(xl=258), dict(u=258), dict(su=258), dict(tok=258), dict(acc=258), dict(sl=258),
               dict(slo=258), dict(pb=-1), dict(pr=-1), dict(qb=-1), dict(qr=-1)):
        assert _verify(lib, **kw) == 1, kw
    assert _verify(lib, B=4097) == 2 and _verify(lib, K=33) == 2 and _verify(lib, V=(1 << 24) + 1) == 2


def test_binding_refusals(lib):
    cfg, plan = _cfg(), bmw.RopePlan.make(128)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bmw.la_rope(plan, x, torch.zeros(4, dtype=torch.int32), x)       # not on the GPU
    with pytest.raises(TypeError):
        bmw.la_rope(plan, x.double(), torch.zeros(4, dtype=torch.int32), x.double())
    q = torch.zeros(2, 6, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bmw.la_rope_append(cfg, plan, q, q[:, :, :2], q[:, :, :2], None, q, q, q)
    with pytest.raises(ValueError):
        bmw.la_pbd_verify(torch.zeros(1, 2, 8), None, *(torch.zeros(1, 1),) * 5)
    with pytest.raises(TypeError):
        bmw.la_pbd_verify(torch.zeros(1, 2, 8, dtype=torch.float64), None, *(torch.zeros(1, 1),) * 5)
    with pytest.raises(bmw.LaError):
        bmw.EvictWorkspace(_cfg(head_dim=64))
    with pytest.raises(TypeError):
        bmw.la_rope(plan, None, None, None)
    with pytest.raises(TypeError):
        bmw.la_rope_append_paged(cfg, plan, q, q, q, None, None, q, q, q)
    with pytest.raises(TypeError):
        bmw.la_pbd_attn_weights_paged(cfg, q, q, q, None, q, 6, q, q, None)
    with pytest.raises(TypeError):
        bmw.la_kv_evict_paged(cfg, q, None, q, 6, q, q, q, q, None)


def test_oracle_rotation_properties():
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 3, 32))
    w = oracle.rope_angles(16)
    for layout in ("half", "interleaved"):
        y = oracle.rotate(x, [0, 1, 7, 1000, -3], w, layout)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 16:], x[..., 16:])
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
        back = oracle.rotate(y, [0, 1, 7, 1000, -3], w, layout, inverse=True)
        np.testing.assert_allclose(back, x, atol=1e-12)
    # scores depend on the distance of the positions alone
    a = oracle.rotate(x[:1], [10], w)[0] * oracle.rotate(x[1:2], [4], w)[0]
    b = oracle.rotate(x[:1], [106], w)[0] * oracle.rotate(x[1:2], [100], w)[0]
    np.testing.assert_allclose(a.sum(-1), b.sum(-1), atol=1e-12)


def test_oracle_eviction_by_hand():
    # 8 keys, 4 stay: position 0 (sink), 7 (recent), then the heaviest; ties to the lower slot
    w = [0.0, 5.0, 1.0, 5.0, 5.0, float("nan"), 2.0, 0.0]
    assert oracle.evict(w, range(8), 8, 8, 4, 1, 1) == [0, 1, 7, 3]
    assert oracle.evict(w, range(8), 8, 8, 8, 1, 1) == list(range(8))
    assert oracle.evict(w, range(8), 2, 2, 4, 0, 0) == [0, 1]
    assert oracle.evict([1.0] * 5, [4, 3, 2, 1, 0], 5, 5, 2, 1, 1) == [0, 4]


def test_oracle_verification_distribution():
    """The drawn token follows the target whatever the draft: exact by enumeration over a grid of
    uniforms (first draft only)."""
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.25, 0.25, 0.25, 0.25]])
    q = np.array([[0.125, 0.625, 0.125, 0.125]])
    counts = np.zeros(4)
    n = 16
    for x in range(4):
        for i in range(n):
            for j in range(n):
                tokens, _ = oracle.verify(p, q, [x], [(i + 0.5) / n], (j + 0.5) / n)
                counts[tokens[0]] += q[0, x] / (n * n)
    np.testing.assert_allclose(counts, p[0], atol=0.02)
    # a miss and an empty residual: the target row itself
    assert oracle.verify(p[:, :], np.array([[1.0, 1.0, 1.0, 1.0]]), [3], [0.5], 0.6) == ([1], 0)


def test_binding_loads_by_itself(lib):
    """The module over torch tensors is loaded in a process that has not imported torch."""
    code = ("import sys, block_masked_window_b200 as bmw; assert 'torch' not in sys.modules; "
            "assert hasattr(bmw._ext(), 'rope')")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(__file__)))
