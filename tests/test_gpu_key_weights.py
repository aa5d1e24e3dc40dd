"""GPU parity of the window attention with key weights (la_pbd_attn_weights, and its paged form).

The output is the plain call's, bit for bit. Tolerance of the weights: a score is a sum of 128
products accumulated in fp32 (error at most 128 * 2^-24 of sum |q k|, in the score and again in the
row's log-sum-exp), the exponent's argument and the log-sum-exp round at 2^-24 of their size (below
64), 2^x and the sums at a few 2^-23: relative to the probabilities' sum, 2 * 2^-17 * scale * max
sum|q k| + 2^-17. The accumulated part rounds at 2^-23 of the result.
"""
import numpy as np
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def _run(lens, W, Hq=16, Hkv=2, wl=None, mask="pbd", page=0, algo=bmw.LA_ALGO_AUTO, decay=None, seed=0,
         max_seq=None, gain=1.0, alias=False):
    """Weights of one call against the oracle, and its output against the plain call."""
    B = len(lens)
    wi = workloads.random_case(B, [max(0, p) for p in lens], W, num_q_heads=Hq, num_kv_heads=Hkv, seed=seed,
                               max_seq=max_seq, stale_fill=float("nan"))
    li = wi.layers[0]
    S = -(-wi.max_seq // page) * page if page else wi.max_seq
    q, k, v = (li.q * gain).to(torch.bfloat16).cuda(), li.k_cache.cuda(), li.v_cache.cuda()
    if wl is not None:
        for b, w in enumerate(wl):
            q[b, max(w, 0):] = float("nan")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sl, wlt = i32(lens), None if wl is None else i32(wl)
    mode = bmw.LA_MASK_CAUSAL_WINDOW if mask == "causal" else bmw.LA_MASK_PBD
    cfg = bmw.Config.make(B, Hq, Hkv, S, mask_mode=mode, algo=algo)
    g = torch.Generator().manual_seed(seed + 1)
    w_in = None
    if decay is not None:
        w_in = torch.rand(B, Hkv, S, generator=g)
        for b, p in enumerate(lens):
            w_in[b, :, max(p, 0):] = float("nan")     # slots of the window: an earlier occupant's
        w_in = w_in.cuda()
    w_out = w_in if alias else torch.full((B, Hkv, S), 7.0, device="cuda")
    before = w_out.clone()
    out, plain = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    ws = bmw.WeightsWorkspace(cfg, W)
    ws.tensor[256:].fill_(255)                       # nothing but the header needs initialising
    opt = dict(weights_in=w_in, decay=1.0 if decay is None else decay, window_lens=wlt)
    w_ref_in = None if w_in is None else w_in.double().cpu().numpy()
    if page:
        per = S // page
        table = torch.randperm(B * per, generator=g).view(B, per)
        pad = torch.full((B, Hkv, S - wi.max_seq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        kp, vp = torch.empty(B * per, Hkv, page, 128, dtype=torch.bfloat16, device="cuda"), None
        vp = torch.empty_like(kp)
        for src, dst in ((k, kp), (v, vp)):
            full = torch.cat([src, pad], 2).view(B, Hkv, per, page, 128).transpose(1, 2)
            dst[table.flatten().cuda()] = full.reshape(B * per, Hkv, page, 128)
        table = table.to(torch.int32)
        for b, p in enumerate(lens):                 # entries past the sequence are never read
            n = p + (W if wl is None else wl[b])
            table[b, -(-max(n, 0) // page):] = 1 << 29
        table = table.cuda()
        bmw.la_pbd_attn_weights_paged(cfg, q, kp, vp, table, sl, W, out, w_out, ws, **opt)
        if wlt is None:
            bmw.la_pbd_attn_paged(cfg, q, kp, vp, table, sl, W, plain, bmw.Workspace(cfg, W))
        else:
            plain = None
    else:
        bmw.la_pbd_attn_weights(cfg, q, k, v, sl, W, out, w_out, ws, **opt)
        if wlt is None:
            bmw.la_pbd_attn(cfg, q, k, v, sl, W, plain, bmw.Workspace(cfg, W))
        else:
            bmw.la_pbd_attn_varwin(cfg, q, k, v, sl, wlt, W, plain, bmw.Workspace(cfg, W))
    torch.cuda.synchronize()
    status = bmw.la_pbd_check(ws)
    if plain is not None:
        assert torch.equal(out, plain)
    wlens = [W] * B if wl is None else wl
    good = [b for b in range(B) if lens[b] >= 0 and 1 <= wlens[b] <= W and lens[b] + wlens[b] <= S]
    assert status == (0 if len(good) == B else 5)
    got = w_out.double().cpu().numpy()
    if good:
        qc, kc = q.double().cpu().numpy(), k.double().cpu().numpy()
        ref = oracle.key_weights(qc[good], kc[good], [lens[b] for b in good], [wlens[b] for b in good],
                                 cfg.scale, None if w_ref_in is None else w_ref_in[good], opt["decay"], mask)
        G = Hq // Hkv
        for x, b in enumerate(good):
            n = lens[b] + wlens[b]
            mag = max((np.abs(kc[b, h, :n]) @
                       np.abs(qc[b, :wlens[b], h * G:(h + 1) * G]).reshape(-1, 128).T).max()
                      for h in range(Hkv))
            old = np.zeros_like(ref[x][:, :n])
            if w_ref_in is not None:
                old[:, :lens[b]] = np.abs(opt["decay"] * w_ref_in[b, :, :lens[b]])
            new = ref[x][:, :n] - old
            tol = (2 * 2.0 ** -17 * cfg.scale * mag + 2.0 ** -17) * new + 2.0 ** -22 * (new + old) + 1e-37
            diff = np.abs(got[b, :, :n] - ref[x][:, :n])
            assert (diff <= tol).all(), f"b={b}: worst {(diff / tol).max():.2f} of the tolerance"
            # every row's probabilities sum to one
            total = got[b, :, :n].sum(-1) - old.sum(-1)
            np.testing.assert_allclose(total, wlens[b] * G, rtol=3e-4 + 2.0 ** -20 * old.sum() / (wlens[b] * G))
            w_out[b, :, :n] = before[b, :, :n]
    a, b_ = w_out.view(torch.int32), before.view(torch.int32)
    assert torch.equal(a, b_), "entries past the keys, or of a flagged sequence, changed"
    return out


@pytest.mark.parametrize("lens", [[0], [1], [58], [122], [123], [250], [1024], [4096],
                                  [0, 5, 121, 122, 1000, 2047, 300, 64, 1], [700] * 40])
def test_lengths(lens):
    _run(lens, 6)


@pytest.mark.parametrize("W,Hq,Hkv", [(1, 16, 2), (1, 1, 1), (2, 8, 8), (6, 16, 4), (8, 16, 2), (10, 16, 2),
                                      (12, 16, 2), (14, 16, 2), (16, 16, 2), (11, 8, 1)])
@pytest.mark.parametrize("mask", ["pbd", "causal"])
def test_rows_and_masks(W, Hq, Hkv, mask):
    _run([3, 500, 130], W, Hq, Hkv, mask=mask, decay=0.5)


@pytest.mark.parametrize("algo", [bmw.LA_ALGO_TCGEN05, bmw.LA_ALGO_SIMT])
@pytest.mark.parametrize("mask", ["pbd", "causal"])
def test_window_lengths(algo, mask):
    _run([0, 5, 121, 1000, 2047, 300], 8, wl=[1, 8, 6, 7, 2, 8], mask=mask, algo=algo, decay=1.0)


@pytest.mark.parametrize("page", [64, 128, 192])
@pytest.mark.parametrize("mask", ["pbd", "causal"])
@pytest.mark.parametrize("wl", [None, [10, 1, 6, 7, 9]])
def test_paged(page, mask, wl):
    _run([0, 63, 500, 1400, 182], 10, wl=wl, mask=mask, page=page, decay=0.9)


def test_accumulates_in_place():
    _run([70, 900], 6, decay=0.97, alias=True)


@pytest.mark.parametrize("page", [0, 64])
def test_old_weights_over_many_segments(page):
    """Several short sequences to a CTA: the copies of old weights that run past one sequence's keys and
    the first ones of the next use the same slots of shared memory. Every old weight arrives."""
    lens = torch.randint(0, 700, (160,), generator=torch.Generator().manual_seed(5)).tolist()
    wl = [1 + i % 6 for i in range(160)]
    for seed in range(3):
        _run(lens, 6, wl=wl if seed == 2 else None, page=page, decay=0.75, seed=seed, alias=seed == 1)


def test_sharp_rows():
    """Scores of hundreds: all the weight on single keys, the rest vanish without a NaN."""
    _run([300, 2000], 6, gain=40.0)


@pytest.mark.parametrize("algo", [bmw.LA_ALGO_TCGEN05, bmw.LA_ALGO_SIMT])
def test_invalid_sequences_keep_their_weights(algo):
    _run([10, -1, 300, 20], 6, algo=algo, decay=1.0, max_seq=304)
    _run([10, 20, 30], 4, wl=[2, 0, 5], algo=algo, decay=1.0)


def test_long_context():
    """Offsets beyond the first gigabyte and many tiles per CTA: row sums only (no oracle)."""
    B, S = 8, 32832
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(B, 2, S, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(B, 2, S, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(B, 6, 16, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    sl = torch.full((B,), 32768, dtype=torch.int32, device="cuda")
    cfg = bmw.Config.make(B, 16, 2, S)
    out, w = torch.empty_like(q), torch.full((B, 2, S), -1.0, device="cuda")
    bmw.la_pbd_attn_weights(cfg, q, k, v, sl, 6, out, w, bmw.WeightsWorkspace(cfg, 6))
    n = 32774
    assert bool((w[..., n:] == -1).all()) and bool((w[..., :n] >= 0).all())
    np.testing.assert_allclose(w[..., :n].double().sum(-1).cpu().numpy(), 48.0, rtol=2e-4)
    s = torch.einsum("wgd,kd->wgk", q[7, :, 8:].float(), k[7, 1, :n].float()) / 128 ** 0.5
    ref = torch.softmax(s.double(), -1).sum((0, 1))
    assert float(((w[7, 1, :n].double() - ref).abs() / ref).max()) <= 3e-4


def test_two_layers_in_a_graph_and_on_a_stream():
    """Two calls that share a workspace, captured together and replayed with other lengths."""
    B, S, W = 3, 512, 6
    g = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    layers = [(rnd(B, W, 16, 128), rnd(B, 2, S, 128), rnd(B, 2, S, 128)) for _ in range(2)]
    sl = torch.tensor([100, 0, 300], dtype=torch.int32, device="cuda")
    cfg = bmw.Config.make(B, 16, 2, S)
    ws = bmw.WeightsWorkspace(cfg, W)
    outs = [torch.empty_like(q) for q, _, _ in layers]
    sums = [torch.zeros(B, 2, S, device="cuda") for _ in layers]

    def step(ws):
        for (q, k, v), o, w in zip(layers, outs, sums):
            bmw.la_pbd_attn_weights(cfg, q, k, v, sl, W, o, w, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws)
    sl.copy_(torch.tensor([500, 17, 200], dtype=torch.int32))
    for w in sums:
        w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs + sums]
    for t in outs + sums:
        t.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(bmw.WeightsWorkspace(cfg, W))
    s.synchronize()
    for a, b in zip(got, outs + sums):
        assert torch.equal(a, b)
