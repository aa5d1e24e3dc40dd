"""GPU tests of the eviction (la_kv_evict and its paged form): the choice of keys, the moved rows,
weights and positions exactly as the oracle's, everything else untouched."""
import numpy as np
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def _weights(kind, shape, g):
    if kind == "heavy":
        return torch.exp(3 * torch.randn(shape, generator=g))
    if kind == "ties":                       # few distinct values: the slots decide
        return torch.randint(0, 3, shape, generator=g).float()
    if kind == "same":
        return torch.zeros(shape)
    if kind == "signed":                     # every kind of number
        w = torch.randn(shape, generator=g)
        r = torch.rand(shape, generator=g)
        for lo, x in enumerate([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 3e38]):
            w[(r > lo * 0.08) & (r < lo * 0.08 + 0.08)] = x
        return w
    if kind == "close":                      # neighbours in the last bits
        return (torch.randint(0, 1 << 12, shape, generator=g, dtype=torch.int32) + 0x3F800000).view(torch.float32)
    raise KeyError(kind)


def _evict(lens, budget, sink=0, recent=0, kind="heavy", page=0, S=None, Hkv=2, pos="slots", inplace=False,
           kept=True, seed=0, ahead=0):
    B = len(lens)
    g = torch.Generator().manual_seed(seed)
    S = S or -(-max(max(lens), budget) // 8) * 8
    if page:
        S = -(-S // page) * page
    w = _weights(kind, (B, Hkv, S), g)
    table = None
    if page:
        per = S // page
        table = torch.randperm(B * per, generator=g).view(B, per)
        shape = (B * per, Hkv, page, 128)
    else:
        shape = (B, Hkv, S, 128)
    k0, v0 = (torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16) for _ in range(2))
    k, v = k0.cuda().view(torch.bfloat16), v0.cuda().view(torch.bfloat16)
    if pos == "slots":
        p_in, ends = None, list(lens)
        positions = torch.arange(S, dtype=torch.int32).expand(B, Hkv, S).contiguous()
    else:                                    # shuffled, as after earlier evictions
        positions = torch.stack([torch.randperm(S, generator=g) for _ in range(B * Hkv)]).view(B, Hkv, S).int() + ahead
        p_in, ends = positions.cuda(), [S + ahead] * B
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cfg = bmw.Config.make(B, 8 * Hkv, Hkv, S)
    ws = bmw.EvictWorkspace(cfg)
    ws.tensor[256:].fill_(255)
    w_dev, lens_dev = w.cuda(), i32(lens)
    w_out = w_dev if inplace else torch.full((B, Hkv, S), -7.0, device="cuda")
    p_out = p_in if inplace and p_in is not None else torch.full((B, Hkv, S), -7, dtype=torch.int32, device="cuda")
    new = lens_dev if inplace else torch.full((B,), -7, dtype=torch.int32, device="cuda")
    kept_t = torch.full((B, Hkv, budget), -7, dtype=torch.int32, device="cuda") if kept else None
    opt = dict(key_pos=p_in, next_pos=None if pos == "slots" else i32(ends), sink=sink, recent=recent,
               key_pos_out=p_out, kept_slots=kept_t)
    for again in range(1 if inplace else 2):         # separate outputs: repeatable
        if page:
            bmw.la_kv_evict_paged(cfg, w_dev, table.int().cuda(), lens_dev, budget, k, v, w_out, new, ws, **opt)
        else:
            bmw.la_kv_evict(cfg, w_dev, lens_dev, budget, k, v, w_out, new, ws, **opt)
    torch.cuda.synchronize()
    bad = [n < 0 or n > S for n in lens]
    assert bmw.la_pbd_check(ws) == (5 if any(bad) else 0)
    want_w = w.clone() if inplace else torch.full((B, Hkv, S), -7.0)
    want_p = positions.clone() if inplace and p_in is not None else torch.full((B, Hkv, S), -7, dtype=torch.int32)
    want_kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    k_ref, v_ref = k0.clone(), v0.clone()
    for b, n in enumerate(lens):
        keep = 0 if bad[b] else min(n, budget)
        assert int(new[b]) == (n if bad[b] else keep)
        for h in range(Hkv):
            src = [] if bad[b] else oracle.evict(w[b, h].numpy(), positions[b, h].numpy(), n, ends[b], budget, sink,
                                                 recent)
            s = torch.tensor(src, dtype=torch.long)
            want_kept[b, h, :keep] = s.int()
            want_w[b, h, :keep] = w[b, h, s]
            want_p[b, h, :keep] = positions[b, h, s]
            for ref, old in ((k_ref, k0), (v_ref, v0)):
                if not page:
                    ref[b, h, :keep] = old[b, h, s]
                elif keep:
                    j = torch.arange(keep)
                    ref[table[b, j // page], h, j % page] = old[table[b, s // page], h, s % page]
    assert torch.equal(w_out.cpu().view(torch.int32), want_w.view(torch.int32))
    assert torch.equal(p_out.cpu(), want_p)
    if kept:
        assert torch.equal(kept_t.cpu(), want_kept)
    assert torch.equal(k.view(torch.int16).cpu(), k_ref) and torch.equal(v.view(torch.int16).cpu(), v_ref)


@pytest.mark.parametrize("kind", ["heavy", "ties", "same", "signed", "close"])
@pytest.mark.parametrize("page", [0, 64])
def test_choice(kind, page):
    _evict([900, 300, 301, 0, 1, 512, 2048], 300, sink=4, recent=33, kind=kind, page=page)


@pytest.mark.parametrize("lens,budget", [([1], 1), ([2], 1), ([5], 4), ([1023, 1024, 1025], 1000),
                                         ([4096, 4097, 4095], 4095), ([4100], 1), ([9000, 20], 4500),
                                         ([20001], 19999), ([33000], 16384)])
@pytest.mark.parametrize("kind", ["heavy", "ties"])
def test_sizes(lens, budget, kind):
    _evict(lens, budget, kind=kind)


@pytest.mark.parametrize("sink,recent", [(0, 64), (64, 0), (10, 54), (1, 0), (0, 1)])
@pytest.mark.parametrize("kind", ["same", "heavy", "signed"])
def test_protected(sink, recent, kind):
    """Protected keys stay whatever their weight; positions shuffled over the slots."""
    _evict([400, 777], 64, sink=sink, recent=recent, kind=kind)
    _evict([400, 777], 64, sink=sink, recent=recent, kind=kind, pos="shuffled")
    _evict([400, 777], 64, sink=sink, recent=recent, kind=kind, pos="shuffled", ahead=2 ** 31 - 2000)


@pytest.mark.parametrize("pos", ["slots", "shuffled"])
@pytest.mark.parametrize("page", [0, 128])
def test_in_place(pos, page):
    _evict([700, 40, 1500], 256, sink=2, recent=20, inplace=True, pos=pos, page=page, kind="signed")


def test_more_protected_than_the_budget():
    """Positions that repeat can protect more keys than stay: the lower slots win."""
    B, S, budget = 1, 64, 8
    cfg = bmw.Config.make(B, 16, 2, S)
    pos = torch.zeros(B, 2, S, dtype=torch.int32, device="cuda")        # all protected by the sink
    k = torch.randn(B, 2, S, 128, device="cuda").to(torch.bfloat16)
    v, k0 = k.clone(), k.clone()
    w, new = torch.rand(B, 2, S, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    kept = torch.empty(B, 2, budget, dtype=torch.int32, device="cuda")
    bmw.la_kv_evict(cfg, w, torch.tensor([60], dtype=torch.int32, device="cuda"), budget, k, v, w, new,
                    bmw.EvictWorkspace(cfg), key_pos=pos, sink=1, key_pos_out=pos, kept_slots=kept)
    assert kept[0].tolist() == [list(range(8))] * 2 and int(new) == 8 and torch.equal(k, k0)


def test_invalid_sequences_untouched():
    _evict([100, -1, 200, 3000], 64, S=256, kind="heavy")
    _evict([100, -5, 256], 64, S=256, kind="heavy", page=64, inplace=True)


@pytest.mark.parametrize("heads", [1, 8])
def test_heads_without_optional_outputs(heads):
    _evict([777, 500], 250, Hkv=heads, kept=False)


def test_pages_outside_the_pool_are_not_moved():
    """A hole in a page that the table does not name: nothing is written through it, the rest moves."""
    S, page, n, budget = 256, 64, 200, 100
    cfg = bmw.Config.make(1, 16, 2, S)
    pool = torch.randn(4, 2, page, 128, device="cuda").to(torch.bfloat16)
    k, v = pool.clone(), pool.clone()
    w = torch.arange(S, dtype=torch.float32, device="cuda").expand(1, 2, S).contiguous()   # the last 100 stay
    table = torch.tensor([[0, 99, 2, -3]], dtype=torch.int32, device="cuda")
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    bmw.la_kv_evict_paged(cfg, w, table, torch.tensor([n], dtype=torch.int32, device="cuda"), budget, k, v,
                          torch.empty_like(w), new, bmw.EvictWorkspace(cfg))
    assert int(new) == budget
    # holes 0..99 take slots 100..199: holes 0..63 are page 0; slots 128.. (page 2) are sources 28..
    assert torch.equal(k[0, :, 28:], pool[2, :, :36]) and torch.equal(k[0, :, :28], pool[0, :, :28])
    assert torch.equal(k[1:], pool[1:]) and torch.equal(v, k)


def test_very_long_sequence():
    """More keys than a cluster holds in shared memory: the passes read them again."""
    S = n = 400001
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.exp(torch.randn(1, 1, S, generator=g, device="cuda"))
    w[..., ::7] = 0.5                                            # ties around the threshold
    k = torch.arange(S, dtype=torch.int32, device="cuda").view(1, 1, S, 1).expand(1, 1, S, 64).contiguous()
    k = k.view(torch.bfloat16)
    v, k0 = k.clone(), k.clone()
    cfg = bmw.Config.make(1, 8, 1, S)
    for budget in (n // 2, 390000):
        kk, vv = k.clone(), v.clone()
        w_out, new = torch.zeros_like(w), torch.empty(1, dtype=torch.int32, device="cuda")
        kept = torch.empty(1, 1, budget, dtype=torch.int32, device="cuda")
        bmw.la_kv_evict(cfg, w, torch.tensor([n], dtype=torch.int32, device="cuda"), budget, kk, vv, w_out, new,
                        bmw.EvictWorkspace(cfg), kept_slots=kept, sink=10, recent=1000)
        x = w[0, 0].double().cpu().numpy().copy()
        x[:10] = x[-1000:] = np.inf
        order = np.argsort(-x, kind="stable")[:budget]
        stay = np.zeros(n, bool)
        stay[order] = True
        src = np.arange(budget)
        src[~stay[:budget]] = np.nonzero(stay[budget:])[0] + budget
        src = torch.from_numpy(src).cuda()
        assert torch.equal(kept[0, 0].long(), src) and int(new) == budget
        assert torch.equal(kk[0, 0, :budget].view(torch.int16), k0[0, 0, src].view(torch.int16))
        assert torch.equal(vv.view(torch.int16), kk.view(torch.int16))
        assert torch.equal(w_out[0, 0, :budget], w[0, 0, src])


def test_graph_replayed_with_other_lengths():
    B, S, budget = 4, 1024, 500
    g = torch.Generator(device="cuda").manual_seed(6)
    k = torch.randn(B, 2, S, 128, generator=g, device="cuda").to(torch.bfloat16)
    v, w = k.clone(), torch.rand(B, 2, S, generator=g, device="cuda")
    sl = torch.tensor([1000, 400, 600, 501], dtype=torch.int32, device="cuda")
    new, w_out = torch.empty_like(sl), torch.zeros_like(w)
    kept = torch.empty(B, 2, budget, dtype=torch.int32, device="cuda")
    cfg = bmw.Config.make(B, 16, 2, S)
    ws = bmw.EvictWorkspace(cfg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bmw.la_kv_evict(cfg, w, sl, budget, k, v, w_out, new, ws, kept_slots=kept)
    sl.copy_(torch.tensor([500, 1024, 3, 777], dtype=torch.int32))
    k0 = k.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert new.tolist() == [500, 500, 3, 500]
    for b, n in enumerate([500, 1024, 3, 777]):
        for h in range(2):
            src = oracle.evict(w[b, h].cpu().numpy(), range(S), n, n, budget, 0, 0)
            assert kept[b, h, :len(src)].tolist() == src
            assert torch.equal(k[b, h, :len(src)], k0[b, h, torch.tensor(src).cuda()])
