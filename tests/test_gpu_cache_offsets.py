"""Caches whose element offsets pass 2^31: the operators around the attention at the last rows of the
last head of an 8.6 GB cache, against the same rows in a small one."""
import pytest
import torch

import block_masked_window_b200 as bmw

pytestmark = pytest.mark.gpu

B, HQ, HKV, D = 2, 16, 2, 128
S = (1 << 23) + 64                      # B * HKV * S * D = 2^32 elements and more


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield cuda_lib
    torch.cuda.empty_cache()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_rotate_append_and_weights_at_the_far_end():
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    W, small = 6, 640
    q, kn, vn = rnd(B, W, HQ, D), rnd(B, W, HKV, D), rnd(B, W, HKV, D)
    plan, pos0 = bmw.RopePlan.make(128), _i32(5, 123456)
    results = []
    for cap, P in ((small, (small - W, 300)), (S, (small - W, 300))):
        cfg = bmw.Config.make(B, HQ, HKV, cap)
        k = torch.zeros(B, HKV, cap, D, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        g2 = torch.Generator(device="cuda").manual_seed(1)
        k[:, :, :small] = torch.randn(B, HKV, small, D, generator=g2, device="cuda").to(torch.bfloat16)
        v[:, :, :small] = torch.randn(B, HKV, small, D, generator=g2, device="cuda").to(torch.bfloat16)
        sl = _i32(*P)
        q_out, out = torch.empty_like(q), torch.empty_like(q)
        w = torch.zeros(B, HKV, cap, device="cuda")
        bmw.la_rope_append(cfg, plan, q, kn, vn, sl, q_out, k, v, pos0=pos0)
        bmw.la_pbd_attn_weights(cfg, q_out, k, v, sl, W, out, w, bmw.WeightsWorkspace(cfg, W))
        results.append([q_out, k[:, :, :small].clone(), v[:, :, :small].clone(), out, w[:, :, :small].clone()])
        if cap == S:                    # the last slots of the cache
            bmw.la_rope_append(cfg, plan, q, kn, vn, _i32(S - W, S - W), q_out, k, v, pos0=pos0)
            for b in range(B):
                assert torch.equal(k[b, :, S - W:], results[1][1][b, :, P[b]:P[b] + W])
                assert torch.equal(v[b, :, S - W:], vn[b].transpose(0, 1))
        del k, v, w
    # The split of the keys differs with the capacity, so sums are added up in another order: the
    # copies are equal, the output within a step of bf16, the weights within 2^-17 of a row's 48 ones.
    for a, b in zip(results[0][:3], results[1][:3]):
        assert torch.equal(a, b)
    a, b = results[0][3].double(), results[1][3].double()
    assert bool(((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-6).all())
    assert float((results[0][4] - results[1][4]).abs().max()) <= 48 * 2.0 ** -17


def test_evict_at_the_far_end():
    n, budget = 8388000, 8000001
    k = torch.empty(B, HKV, S, D, dtype=torch.bfloat16, device="cuda")
    rows = k.view(torch.int32)          # every row carries its number
    rows[:] = torch.arange(B * HKV * S, dtype=torch.int32, device="cuda").view(B, HKV, S, 1)
    v = k.clone()
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.rand(B, HKV, S, generator=g, device="cuda")
    cfg = bmw.Config.make(B, HQ, HKV, S)
    new, w_out = torch.empty(B, dtype=torch.int32, device="cuda"), torch.zeros_like(w)
    kept = torch.empty(B, HKV, budget, dtype=torch.int32, device="cuda")
    ws = bmw.EvictWorkspace(cfg)
    bmw.la_kv_evict(cfg, w, _i32(100, n), budget, k, v, w_out, new, ws, kept_slots=kept)
    assert bmw.la_pbd_check(ws) == 0 and new.tolist() == [100, budget]
    for h in range(HKV):
        order = w[1, h, :n].sort(descending=True, stable=True).indices[:budget]
        stay = torch.zeros(n, dtype=torch.bool, device="cuda")
        stay[order] = True
        src = torch.arange(budget, device="cuda")
        src[~stay[:budget]] = stay[budget:].nonzero()[:, 0] + budget
        assert torch.equal(kept[1, h].long(), src)
        want = (src + (HKV + h) * S).int()
        for c in (k, v):
            got = c.view(torch.int32)[1, h, :budget]
            assert torch.equal(got[:, 0], want) and torch.equal(got[:, 63], want)
            assert torch.equal(c.view(torch.int32)[0, h, :, 5], torch.arange(S, device="cuda").int() + h * S)
        assert torch.equal(w_out[1, h, :budget], w[1, h, src])
