"""The attention's output inside the decode loop: every step's `out` of la_pbd_attn_weights (contiguous and
paged, eager and captured with the eviction after it) against the fp64 oracle over the cache as the
step's append left it, taken by the same append on copies made before the step.

Tolerance: the acceptance bar of the path and one step of the rounded oracle (gpu_util).
"""
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle
from gpu_util import assert_parity
from test_gpu_decode_loop import D, HKV, HQ, Loop, W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def appended(L, k, v):
    """Rotated queries and the caches [B, Hkv, S, D] after the step's append to the copies k and v."""
    q_rot = torch.zeros_like(L.q)
    if L.page:
        bmw.la_rope_append_paged(L.cfg, L.plan, L.q, L.kn, L.vn, L.table, L.lens, q_rot, k, v, pos0=L.pos)
        k, v = (c[L.table.long()].transpose(1, 2).flatten(2, 3) for c in (k, v))
    else:
        bmw.la_rope_append(L.cfg, L.plan, L.q, L.kn, L.vn, L.lens, q_rot, k, v, pos0=L.pos)
    return q_rot.cpu(), k.cpu(), v.cpu()


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("graphed", [False, True])
def test_out_of_every_step(page, graphed):
    prompt = [100, 0, 37, 150]
    L = Loop(prompt, page, seed=17)
    g = torch.Generator().manual_seed(2)
    qp, kp, vp = (torch.randn(L.B, max(prompt), h, D, generator=g).to(torch.bfloat16).cuda()
                  for h in (HQ, HKV, HKV))
    rows = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    opt = dict(row_lens=rows, key_pos=L.key_pos)
    if page:
        bmw.la_rope_append_paged(L.cfg, L.plan, qp, kp, vp, L.table, None, torch.zeros_like(qp), L.k, L.v, **opt)
    else:
        bmw.la_rope_append(L.cfg, L.plan, qp, kp, vp, None, torch.zeros_like(qp), L.k, L.v, **opt)
    L.lens.copy_(rows)
    L.pos.copy_(rows)
    graph, evicted = None, 0
    for step in range(10):
        L.draw()
        if graphed and graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                L.step()
                L.evict(128)
        q_rot, k, v = appended(L, L.k.clone(), L.v.clone())
        lens = L.lens.cpu()
        L.out.fill_(float("nan"))
        if graphed:
            graph.replay()
        else:
            L.step()
            L.evict(128)
        torch.cuda.synchronize()
        assert torch.equal(L.q_rot.cpu(), q_rot)
        ref = oracle.window_attention(q_rot, k, v, lens, L.cfg.scale)
        assert_parity(L.out.cpu(), ref, f"step {step}")
        evicted += int((lens + L.acc.cpu() + 1 > 128).sum())
    assert evicted > 4
    assert bmw.la_pbd_check(L.ws) == 0 and bmw.la_pbd_check(L.ews) == 0


def test_out_is_checked():
    """The comparison sees a wrong output: planted in the oracle's inputs, one value row changed."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, n, h, D, generator=g).to(torch.bfloat16) for n, h in ((W, HQ), (HKV, 64), (HKV, 64)))
    lens = torch.tensor([40], dtype=torch.int32)
    ref = oracle.window_attention(q, k, v, lens, D ** -0.5)
    out = torch.from_numpy(ref).to(torch.bfloat16)
    assert_parity(out, ref)
    v[0, 1, 44] += 1
    with pytest.raises(AssertionError):
        assert_parity(out, oracle.window_attention(q, k, v, lens, D ** -0.5))


@pytest.mark.parametrize("page", [0, 64])
def test_two_loops_at_once(page):
    """Two loops with buffers and workspaces of their own, their steps queued on two streams without a
    wait between them: the bits of the same loops one after the other."""
    def loops():
        out = []
        for seed, prompt in ((5, [90, 10]), (6, [40, 120, 0])):
            L = Loop(prompt, page, seed)
            for c in (L.k, L.v):
                c.copy_(torch.randn(c.shape, generator=torch.Generator().manual_seed(seed)))
            L.lens.copy_(torch.tensor(prompt, dtype=torch.int32))
            L.pos.copy_(L.lens)
            L.key_pos.copy_(torch.arange(L.S, dtype=torch.int32).expand(L.B, HKV, L.S))
            L.draw()
            out.append(L)
        torch.cuda.synchronize()
        return out

    def state(L):
        torch.cuda.synchronize()
        return [t.clone() for t in (L.k, L.v, L.weights, L.key_pos, L.lens, L.pos, L.q_rot, L.out, L.tokens, L.acc)]

    want = []
    for L in loops():
        for _ in range(40):
            L.step()
            L.evict(128)
        want.append(state(L))
    for _ in range(3):
        both = loops()
        streams = [torch.cuda.Stream() for _ in both]
        for _ in range(40):
            for L, s in zip(both, streams):
                with torch.cuda.stream(s):
                    L.step()
                    L.evict(128)
        for L, w in zip(both, want):
            for a, b in zip(state(L), w):
                assert torch.equal(a, b)
            assert bmw.la_pbd_check(L.ws) == 0 and bmw.la_pbd_check(L.ews) == 0
