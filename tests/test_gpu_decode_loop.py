"""The operators together, as a decode loop uses them: prompt rotated and appended, block-causal
prefill, then steps of rotate + append, window attention with key weights, verification (which sets
the next lengths), and an eviction whenever the cache passes its budget; contiguous and paged,
eager and captured into one graph. The keys, positions and lengths are followed exactly on the CPU,
the attention against the fp64 oracle over the cache as it then is.

Attention: within the acceptance bar of the path (gpu_util). Keys: rotation to bf16, half a step.
"""
import numpy as np
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle
from gpu_util import MAX_ABS, REL_L2, assert_parity, errors

pytestmark = pytest.mark.gpu

HQ, HKV, D, W, V = 16, 2, 128, 6, 997
G = HQ // HKV


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


class Loop:
    """One layer's state on the device."""

    def __init__(self, prompt, page, seed):
        self.B, self.page, self.S = len(prompt), page, 256
        g = self.g = torch.Generator().manual_seed(seed)
        self.plan = bmw.RopePlan.make(128, base=1e6)
        self.cfg = bmw.Config.make(self.B, HQ, HKV, self.S)
        z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
        if page:
            per = self.S // page
            self.table = torch.randperm(self.B * per, generator=g).view(self.B, per).int().cuda()
            shape = (self.B * per, HKV, page, D)
        else:
            self.table, shape = None, (self.B, HKV, self.S, D)
        self.k, self.v = (z(shape, dtype=torch.bfloat16) for _ in range(2))
        self.weights = z(self.B, HKV, self.S)
        self.key_pos = z(self.B, HKV, self.S, dtype=torch.int32)
        self.lens = z(self.B, dtype=torch.int32)
        self.pos = z(self.B, dtype=torch.int32)           # next position
        self.q = z(self.B, W, HQ, D, dtype=torch.bfloat16)
        self.kn, self.vn = (z(self.B, W, HKV, D, dtype=torch.bfloat16) for _ in range(2))
        self.q_rot, self.out = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.p, self.dq = z(self.B, W, V), z(self.B, W - 1, V)
        self.x = z(self.B, W - 1, dtype=torch.int32)
        self.u, self.su = z(self.B, W - 1), z(self.B)
        self.tokens = z(self.B, W, dtype=torch.int32)
        self.acc = z(self.B, dtype=torch.int32)
        self.ws = bmw.WeightsWorkspace(self.cfg, W)
        self.ews = bmw.EvictWorkspace(self.cfg)

    def draw(self):
        """New inputs of a step, in the same buffers."""
        g, r = self.g, lambda t: t.copy_(torch.randn(t.shape, generator=self.g))  # noqa: E731
        for t in (self.q, self.kn, self.vn):
            r(t)
        logits = 2 * torch.randn(self.B, W, V, generator=g)
        self.p.copy_(torch.softmax(logits, -1))
        dq = torch.softmax(logits[:, :-1] + 0.5 * torch.randn(self.B, W - 1, V, generator=g), -1)
        self.dq.copy_(dq)
        self.x.copy_(torch.multinomial(dq.view(-1, V), 1, generator=g).view(self.B, W - 1))
        self.u.copy_(torch.rand(self.B, W - 1, generator=g))
        self.su.copy_(torch.rand(self.B, generator=g))

    def step(self):
        opt = dict(pos0=self.pos, key_pos=self.key_pos)
        paged = (self.table,) if self.page else ()
        append = bmw.la_rope_append_paged if self.page else bmw.la_rope_append
        attend = bmw.la_pbd_attn_weights_paged if self.page else bmw.la_pbd_attn_weights
        append(self.cfg, self.plan, self.q, self.kn, self.vn, *paged, self.lens, self.q_rot, self.k, self.v, **opt)
        attend(self.cfg, self.q_rot, self.k, self.v, *paged, self.lens, W, self.out, self.weights, self.ws,
               weights_in=self.weights)
        bmw.la_pbd_verify(self.p, self.dq, self.x, self.u, self.su, self.tokens, self.acc, seq_lens=self.lens,
                          seq_lens_out=self.lens)
        self.pos.add_(self.acc).add_(1)

    def evict(self, budget):
        paged = (self.table,) if self.page else ()
        fn = bmw.la_kv_evict_paged if self.page else bmw.la_kv_evict
        args = (self.cfg, self.weights, *paged, self.lens, budget, self.k, self.v, self.weights, self.lens, self.ews)
        fn(*args, key_pos=self.key_pos, next_pos=self.pos, sink=2, recent=16, key_pos_out=self.key_pos)

    def cache(self):
        """Caches as [B, Hkv, S, D] on the CPU."""
        torch.cuda.synchronize()
        out = []
        for c in (self.k, self.v):
            if self.page:
                c = c[self.table.long()].transpose(1, 2).flatten(2, 3)
            out.append(c.cpu())
        return out


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("graphed", [False, True])
def test_decode_loop(page, graphed):
    prompt = [100, 37, 150]
    L = Loop(prompt, page, seed=7)
    T = max(prompt)
    angles = oracle.rope_angles(128, base=1e6)
    g = torch.Generator().manual_seed(1)
    qp, kp, vp = (torch.randn(L.B, T, h, D, generator=g).to(torch.bfloat16).cuda() for h in (HQ, HKV, HKV))
    rows = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    q_rot = torch.zeros_like(qp)
    if page:
        bmw.la_rope_append_paged(L.cfg, L.plan, qp, kp, vp, L.table, None, q_rot, L.k, L.v, row_lens=rows,
                                 key_pos=L.key_pos)
    else:
        bmw.la_rope_append(L.cfg, L.plan, qp, kp, vp, None, q_rot, L.k, L.v, row_lens=rows, key_pos=L.key_pos)
        out = torch.empty_like(q_rot)
        bmw.la_block_prefill(L.cfg, q_rot, L.k, L.v, rows, 6, out, bmw.PrefillWorkspace(L.cfg, T))
        k, v = L.cache()
        for b, n in enumerate(prompt):
            ref = oracle.block_prefill_attention(q_rot[b, :n].cpu(), k[b, :, :n].permute(1, 0, 2),
                                                 v[b, :, :n].permute(1, 0, 2), np.arange(n) // 6, L.cfg.scale)
            # The prefill's probabilities are fp16, so its outputs are held to the path's acceptance
            # bar alone (as in its own tests), not to one step of the rounded oracle.
            max_abs, rel = errors(out[b, :n].cpu(), ref)
            assert max_abs <= MAX_ABS and rel <= REL_L2, (b, max_abs, rel)
    L.lens.copy_(rows)
    L.pos.copy_(rows)
    # (position, original key) of every live slot, per sequence and head
    keys = [[[(t, kp[b, t, h].cpu()) for t in range(n)] for h in range(HKV)] for b, n in enumerate(prompt)]
    weights = [[np.zeros(n) for _ in range(HKV)] for n in prompt]
    pos, lens = list(prompt), list(prompt)
    graph = None
    budget = 128
    for step in range(12):
        L.draw()
        if graphed and graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                L.step()
                L.evict(budget)
        if graphed:
            graph.replay()
        else:
            L.step()
            L.evict(budget)
        torch.cuda.synchronize()
        new_lens = L.lens.cpu().tolist()
        k_dev, v_dev = L.cache()
        w_dev, p_dev = L.weights.cpu().double().numpy(), L.key_pos.cpu()
        out, q_in, kn = L.out.cpu(), L.q.cpu(), L.kn.cpu()
        for b in range(L.B):
            want, n_acc = oracle.verify(L.p[b].cpu(), L.dq[b].cpu(), L.x[b].cpu(), L.u[b].cpu(), L.su[b].cpu())
            assert int(L.acc[b]) == n_acc and L.tokens[b].tolist() == want + [-1] * (W - len(want))
            P, n = lens[b], lens[b] + W
            t = pos[b] + np.arange(W)
            qr = oracle.rotate(q_in[b], t, angles)
            for h in range(HKV):
                rows_h = keys[b][h] + [(int(t[i]), kn[b, i, h]) for i in range(W)]
                kk = np.stack([oracle.rotate(x[None, None], [tt], angles)[0, 0] for tt, x in rows_h])
                kk = torch.from_numpy(kk).to(torch.bfloat16).double().numpy()
                qh = torch.from_numpy(qr[:, h * G:(h + 1) * G]).to(torch.bfloat16).double().numpy().reshape(-1, D)
                s = qh @ kk.T * L.cfg.scale
                e = np.exp(s - s.max(-1, keepdims=True))
                total = (e / e.sum(-1, keepdims=True)).sum(0)
                total[:P] += weights[b][h]
                # committed, then evicted by the device's own weights, which are checked below
                live = P + n_acc + 1
                keep = min(live, budget)
                assert new_lens[b] == keep
                have = p_dev[b, h, :keep].tolist()
                by_pos = {tt: j for j, (tt, _) in enumerate(rows_h[:live])}
                assert len(set(have)) == keep and set(have) <= set(by_pos)
                src = [by_pos[tt] for tt in have]
                # kept in place below the new length; protected keys all there
                assert all(j == i for i, j in enumerate(src) if j < keep)
                end = pos[b] + n_acc + 1
                must = {tt for tt, _ in rows_h[:live] if tt < 2 or tt >= end - 16}
                assert must <= set(have)
                # A rounding of q or k to the other side (2^-8) moves a score by up to 2^-7 of
                # sum|q k| scale of one channel; over 128 channels less than 2^-6: 2 % of a weight.
                np.testing.assert_allclose(w_dev[b, h, :keep], total[src], rtol=2.0 ** -5)
                left = sorted(set(range(live)) - set(src))
                if left:
                    safe = [j for j in src if rows_h[j][0] not in must]
                    assert total[left].max() <= min(total[safe], default=np.inf) * (1 + 2.0 ** -4)
                got = k_dev[b, h, :keep].double().numpy()
                assert (np.abs(got - kk[src]) <= 2.0 ** -7 * np.abs(kk[src]) + 2.0 ** -16).all()
                for i, j in enumerate(src):
                    if j >= P:
                        assert torch.equal(v_dev[b, h, i], L.vn[b, j - P, h].cpu())
                keys[b][h] = [rows_h[j] for j in src]
                weights[b][h] = w_dev[b, h, :keep].copy()
            lens[b], pos[b] = keep, end
            assert torch.isfinite(out[b]).all()
        # the attention itself on the cache as it is now, with the last rotated queries
        o = torch.empty_like(L.out)
        if not page:
            bmw.la_pbd_attn(L.cfg, L.q_rot, L.k, L.v, L.lens - W, W, o, bmw.Workspace(L.cfg, W))
            ref = oracle.window_attention(L.q_rot.cpu(), k_dev, v_dev, (L.lens - W).cpu(), L.cfg.scale)
            assert_parity(o.cpu(), ref, f"step {step}")
    assert bmw.la_pbd_check(L.ws) == 0 and bmw.la_pbd_check(L.ews) == 0
    assert max(pos) > budget + W


@pytest.mark.parametrize("attention", ["weights", "attn", "varwin", "step"])
def test_lengths_from_the_kernel_before(attention):
    """Lengths that one kernel writes are read by the next, which may have started before that write:
    a chain of steps in a graph gives the bits of the same calls one at a time."""
    B, S, V, steps, hq = 96, 512, 16, 24, 16
    g = torch.Generator().manual_seed(11)
    r = lambda *n: torch.randn(n, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    i32 = lambda *n, v=0: torch.full(n, v, dtype=torch.int32, device="cuda")  # noqa: E731
    q, kn, vn = r(B, W, hq, 128), r(B, W, HKV, 128), r(B, W, HKV, 128)
    k0, v0 = r(B, HKV, S, 128), r(B, HKV, S, 128)
    p = torch.softmax(torch.randn(B, W, V, generator=g), -1).cuda()
    drafts = torch.randint(V, (steps, B, W - 1), generator=g, dtype=torch.int32).cuda()
    u = (torch.rand(steps, B, W - 1, generator=g) * 0.15).cuda()
    su = torch.rand(steps, B, generator=g).cuda()
    first = torch.randint(0, S - steps * W - W, (B,), generator=g, dtype=torch.int32).cuda()
    wl = i32(B, v=W)
    pos0 = torch.arange(steps, dtype=torch.int32, device="cuda").mul(1000).unsqueeze(1).repeat(1, B)
    cfg, plan = bmw.Config.make(B, hq, HKV, S), bmw.RopePlan.make(128)
    ws, ews = bmw.WeightsWorkspace(cfg, W), bmw.EvictWorkspace(cfg)
    k, v, lens, key_pos = k0.clone(), v0.clone(), first.clone(), i32(B, HKV, S, v=-1)
    weights = torch.zeros(B, HKV, S, device="cuda")
    out = torch.zeros(steps, B, W, hq, 128, dtype=torch.bfloat16, device="cuda")
    q_rot, tokens, acc = torch.empty_like(q), i32(steps, B, W), i32(steps, B)

    def chain(after):
        k.copy_(k0), v.copy_(v0), lens.copy_(first), key_pos.fill_(-1), weights.zero_()
        after()
        for t in range(steps):
            bmw.la_rope_append(cfg, plan, q, kn, vn, lens, q_rot, k, v, pos0=pos0[t], key_pos=key_pos)
            after()
            if attention == "weights":
                bmw.la_pbd_attn_weights(cfg, q_rot, k, v, lens, W, out[t], weights, ws, weights_in=weights)
            elif attention == "attn":
                bmw.la_pbd_attn(cfg, q_rot, k, v, lens, W, out[t], ws)
            elif attention == "varwin":
                bmw.la_pbd_attn_varwin(cfg, q_rot, k, v, lens, wl, W, out[t], ws)
            else:
                bmw.la_pbd_step(cfg, q_rot, kn, vn, k, v, lens, W, out[t], ws)
            after()
            bmw.la_pbd_verify(p, None, drafts[t], u[t], su[t], tokens[t], acc[t], seq_lens=lens, seq_lens_out=lens)
            after()
            if attention == "attn":        # straight from the new lengths to the attention
                bmw.la_pbd_attn(cfg, q_rot, k, v, lens, W, out[t], ws)
                after()
            if t % 8 == 7:
                bmw.la_kv_evict(cfg, weights, lens, S // 2, k, v, weights, lens, ews, key_pos=key_pos,
                                key_pos_out=key_pos)
                after()
        return [x.clone() for x in (k, v, lens, key_pos, weights, out, tokens, acc)]

    want = chain(torch.cuda.synchronize)
    assert int(want[-1].max()) > int(want[-1].min())       # the sequences advance differently
    assert int(want[2].max()) + W <= S
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(10):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
