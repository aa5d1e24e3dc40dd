"""GPU tests of the draft verification (la_pbd_verify): tokens, counts and lengths exactly as the
fp64 oracle's (the library computes in 64 bits too: the accept test is exact, and a border of the
cumulative sum would have to lie within about 1e-16 of the draw to differ)."""
import numpy as np
import pytest
import torch

import block_masked_window_b200 as bmw
import oracle

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def _check(p, q, x, u, su, lens=None, alias=False):
    B, K1, V = p.shape
    K = K1 - 1
    tokens = torch.full((B, K1), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    sl = torch.arange(100, 100 + B, dtype=torch.int32, device="cuda")
    slo = sl if alias else torch.full_like(sl, -9)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    bmw.la_pbd_verify(dev(p), dev(q), dev(x), dev(u), dev(su), tokens, acc, draft_lens=dev(lens), seq_lens=sl,
                      seq_lens_out=slo)
    p, q, x, u, su = (None if t is None else t.cpu() for t in (p, q, x, u, su))
    for b in range(B):
        k = K if lens is None else int(lens[b])
        if k < 0 or k > K:
            assert int(acc[b]) == -1 and tokens[b].tolist() == [-1] * K1 and int(slo[b]) == 100 + b
            continue
        want, n = oracle.verify(p[b, :k + 1], None if q is None else q[b, :k], x[b, :k], u[b], su[b])
        assert int(acc[b]) == n and int(slo[b]) == 100 + b + n + 1, b
        assert tokens[b].tolist() == want + [-1] * (K1 - len(want)), b
    return tokens, acc


def _case(B, K, V, dtype="fp32", certain=False, noise=1.0, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    logits = 3 * torch.randn(B, K + 1, V + pad, generator=g)
    draft = logits[:, :K] + noise * torch.randn(B, K, V + pad, generator=g)
    p = torch.softmax(logits[..., :V], -1)
    q = torch.softmax(draft[..., :V], -1)
    x = torch.multinomial(q.reshape(B * K, V), 1, generator=g).view(B, K).int() if K else torch.empty(B, 0, dtype=torch.int32)
    if pad:                                    # rows of a wider buffer, what follows them not a number
        wide = torch.full((B, K + 1, V + pad), float("nan"))
        wide[..., :V] = p
        p = wide.to(DTYPES[dtype]).cuda()[..., :V]
        wide = torch.full((B, K, V + pad + 3), float("nan"))
        wide[..., :V] = q
        q = wide.to(DTYPES[dtype]).cuda()[..., :V]
    else:
        p, q = p.to(DTYPES[dtype]), q.to(DTYPES[dtype])
    return p, None if certain else q, x, torch.rand(B, K, generator=g), torch.rand(B, generator=g)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("B,K,V", [(1, 5, 152681), (3, 5, 4097), (64, 5, 1000), (700, 1, 33), (5, 32, 777),
                                   (2, 3, 1), (9, 5, 31), (1, 0, 5000), (150, 2, 8191)])
def test_parity(dtype, certain, B, K, V):
    _check(*_case(B, K, V, dtype, certain, seed=B + V), alias=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strided_rows_and_lengths(dtype):
    p, q, x, u, su = _case(12, 5, 1003, dtype, pad=61, noise=0.3)
    lens = torch.tensor([0, 1, 2, 3, 4, 5, 5, 0, -1, 6, 5, 2 ** 30], dtype=torch.int32)
    _check(p, q, x, u, su, lens)
    # the batch a broadcast of one sequence
    _check(p[:1].expand(12, 6, 1003), q[:1].expand(12, 5, 1003), x, u, su, lens)


def test_every_count_of_accepted_drafts():
    B, K, V = 6, 5, 4000
    p, q, x, u, su = _case(B, K, V)
    p = torch.cat([q, p[:, :1]], 1)            # p = q: a draft is accepted whenever u < 1
    u = torch.full((B, K), 0.999)
    for b in range(K):
        p[b, b, int(x[b, b])] = 0.0            # sequence b misses draft b
    _, acc = _check(p, q, x, u, su)
    assert acc.tolist() == [0, 1, 2, 3, 4, 5]


def test_borders_of_the_draw():
    """Exactly representable probabilities: a draw on a border takes the next entry, 0 the first
    with weight, the largest uniform the last with weight."""
    V = 4096
    p = torch.zeros(8, 1, V)
    p[:, 0, 5:4005:1000] = 0.25                # entries 5, 1005, 2005, 3005
    su = torch.tensor([0.0, 0.25, 0.25 - 2.0 ** -25, 0.5, 0.75, 1 - 2.0 ** -24, 0.7499999, 0.2])
    x, u = torch.empty(8, 0, dtype=torch.int32), torch.empty(8, 0)
    tokens, _ = _check(p, None, x, u, su)
    assert tokens[:, 0].tolist() == [5, 1005, 5, 2005, 3005, 3005, 2005, 5]


def test_accept_border_is_strict():
    p = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]]).expand(4, 2, 2).contiguous()
    q = torch.tensor([[[0.5, 0.5]]]).expand(4, 1, 2).contiguous()
    x = torch.tensor([[0], [0], [1], [0]], dtype=torch.int32)
    u = torch.tensor([[0.5], [0.5 - 2.0 ** -25], [0.9999], [0.0]])
    _, acc = _check(p, q, x, u, torch.full((4,), 0.3))
    assert acc.tolist() == [0, 1, 1, 1]


def test_unusual_rows():
    """Empty residual, empty rows, negative, infinite and NaN entries, drafts outside the
    vocabulary, a draft row that is zero at the draft."""
    V, K = 3000, 1
    g = torch.Generator().manual_seed(1)
    p = torch.softmax(torch.randn(10, K + 1, V, generator=g), -1)
    q = torch.softmax(torch.randn(10, K, V, generator=g), -1)
    x = torch.randint(0, V, (10, K), generator=g, dtype=torch.int32)
    u, su = torch.full((10, K), 0.999999), torch.rand(10, generator=g)
    q[0] = 1.0                                  # p - q <= 0 everywhere: drawn from p
    p[1, 0] = 0.0                               # nothing can be drawn
    p[2, 0, 17] = float("inf")
    p[2, 0, int(x[2, 0])] = 0.0
    p[3, 0, ::2] = float("nan")
    p[3, 0, int(x[3, 0])] = 0.0
    p[4, 0] = -p[4, 0]
    x[5, 0], x[6, 0] = -1, V
    q[7, 0, int(x[7, 0])] = 0.0                 # accepted: 0 < p
    p[8, 1] = 0.0
    q[9, 0, 100:200] = float("nan")
    p[9, 0, int(x[9, 0])] = 0.0
    tokens, acc = _check(p, q, x, u, su)
    assert tokens[1].tolist() == [-1, -1] and tokens[2].tolist() == [-1, -1] and tokens[4].tolist() == [-1, -1]
    assert int(acc[7]) == 1
    _check(p, None, x, u, su)


def test_without_lengths_and_distribution():
    """Drawn tokens follow the target: 20000 sequences of one draft, against the multinomial's spread
    (six standard deviations)."""
    B, V = 4000, 8
    g = torch.Generator().manual_seed(3)
    p1 = torch.softmax(torch.randn(1, 2, V, generator=g), -1)
    q1 = torch.softmax(torch.randn(1, 1, V, generator=g), -1)
    counts = np.zeros(V)
    for _ in range(5):
        x = torch.multinomial(q1.view(1, V).expand(B, V), 1, generator=g).int().cuda()
        tokens = torch.empty(B, 2, dtype=torch.int32, device="cuda")
        acc = torch.empty(B, dtype=torch.int32, device="cuda")
        bmw.la_pbd_verify(p1.cuda().expand(B, 2, V), q1.cuda().expand(B, 1, V), x, torch.rand(B, 1, generator=g).cuda(),
                          torch.rand(B, generator=g).cuda(), tokens, acc)
        counts += np.bincount(tokens[:, 0].cpu().numpy(), minlength=V)
    n, want = 5 * B, p1[0, 0].numpy()
    assert (np.abs(counts / n - want) <= 6 * np.sqrt(want * (1 - want) / n)).all()


def test_graph_and_stream():
    p, q, x, u, su = (t.cuda() for t in _case(20, 5, 30000))
    tokens = torch.empty(20, 6, dtype=torch.int32, device="cuda")
    acc = torch.empty(20, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bmw.la_pbd_verify(p, q, x, u, su, tokens, acc)
    su.copy_(torch.rand_like(su))
    graph.replay()
    torch.cuda.synchronize()
    got = tokens.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bmw.la_pbd_verify(p, q, x, u, su, tokens.fill_(0), acc, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, tokens)
    _check(p, q, x, u, su)
