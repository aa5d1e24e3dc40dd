"""Cases, plain forms and exact values of the operators around the window attention.

``run`` makes one pass through an operator: rotary positions (alone, or fused with the append into
the cache), window attention that also accumulates the keys' attention weights, eviction of keys by
those weights, and verification of drafted tokens. With ``own`` false it computes the plain form in
elementary torch operations, otherwise it makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension of the caches
HQ, HKV = 16, 2  # heads of the decoder that the caches belong to
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # Rotation of the queries and keys of one decode window, keys and values appended to the
        # cache: one image, prefix 1024 (the smallest call: latency).
        dict(name="rope_append_window", op="rope_append", batch=1, rows=6, prefix_lo=1024, prefix_hi=1024,
             cap=1088, page=0, packed=False, ragged=False, layout="half", rotary=128,
             scaling="none", far=0),
        # A serving batch on paged caches, windows of 6 to 10 rows, positions beyond the trained
        # length (scaled by a ramp over the pairs) that run ahead of the slots after evictions.
        dict(name="rope_append_ragged_paged", op="rope_append", batch=64, rows=10, prefix_lo=512,
             prefix_hi=4096, cap=4160, page=64, packed=True, ragged=True, layout="half", rotary=128,
             scaling="pairs", far=100000),
        # A prompt of 16384 tokens straight from the fused projection (strided q, k, v).
        dict(name="rope_append_prompt", op="rope_append", batch=1, rows=16384, prefix_lo=0, prefix_hi=0,
             cap=16384, page=0, packed=True, ragged=False, layout="half", rotary=128,
             scaling="turns", far=0),
        # Gradient of a rotation over part of an interleaved head (training), odd token count.
        dict(name="rope_gradient_part", op="rope", tokens=12291, heads=16, dim=128, rotary=64,
             layout="interleaved", scaling="linear", inverse=True, dtype="fp32", span=32768),
        # Window attention with key weights: one image, prefix 1024.
        dict(name="weights_image", op="weights", batch=1, rows=6, prefix_lo=1024, prefix_hi=1024,
             cap=1088, page=0, ragged=False, mask="window", decay=1.0),
        # A ragged serving batch on paged caches, windows of 6 to 10 rows, causal inside.
        dict(name="weights_ragged_paged", op="weights", batch=64, rows=10, prefix_lo=512, prefix_hi=4096,
             cap=4160, page=64, ragged=True, mask="causal", decay=0.97),
        # Eight long prefixes.
        dict(name="weights_long", op="weights", batch=8, rows=6, prefix_lo=32768, prefix_hi=32768,
             cap=32832, page=0, ragged=False, mask="window", decay=1.0),
        # A full 4096-token cache of one sequence, brought down to 2048 keys.
        dict(name="evict_one", op="evict", batch=1, prefix_lo=4096, prefix_hi=4096, cap=4160, page=0,
             budget=2048, sink=4, recent=256),
        # A serving batch on paged caches a few keys over its budget, some sequences below it.
        dict(name="evict_ragged_paged", op="evict", batch=64, prefix_lo=512, prefix_hi=4096, cap=4160,
             page=64, budget=1999, sink=4, recent=128),
        # Eight long prefixes, halved.
        dict(name="evict_long", op="evict", batch=8, prefix_lo=32768, prefix_hi=32768, cap=32832, page=0,
             budget=16384, sink=4, recent=1024),
        # One sequence's window of 5 drafts over the decoder's vocabulary.
        dict(name="verify_one", op="verify", batch=1, drafts=5, vocab=152681, dtype="fp32", certain=False,
             ragged=False, noise=0.5),
        # A serving batch; rows padded to the projection's width.
        dict(name="verify_batch", op="verify", batch=64, drafts=5, vocab=152681, dtype="fp32",
             certain=False, ragged=True, noise=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "rope", "weights", "evict", "verify"])
    if op == "rope":
        dim = rng.choice([64, 80, 128, 256])
        heads = rng.randint(1, 32)
        return dict(op=op, tokens=_log(rng, 1, 12000 * 16 * 128 // (heads * dim)), heads=heads, dim=dim,
                    rotary=rng.choice([dim, dim // 2, dim // 4]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "pairs", "turns"]),
                    inverse=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    span=_log(rng, 64, 1000000))
    if op == "verify":
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, drafts=rng.randint(1, 8), vocab=_log(rng, 1000, 100000),
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), certain=rng.random() < 0.3,
                    ragged=rng.random() < 0.5, noise=rng.uniform(0.1, 2.0))
    if op == "rope_append" and rng.random() < 0.4:  # prompts
        batch = _log(rng, 1, 8)
        rows = _log(rng, 17, 16384 // batch)
        page = rng.choice([0, 64, 128])
        return dict(op=op, batch=batch, rows=rows, prefix_lo=0, prefix_hi=0, cap=-(-rows // 128) * 128,
                    page=page, packed=rng.random() < 0.5, ragged=rng.random() < 0.5,
                    layout=rng.choice(["half", "interleaved"]), rotary=rng.choice([128, 64, 32]),
                    scaling=rng.choice(["none", "linear", "base", "pairs", "turns"]), far=0)
    batch = _log(rng, 1, 64)
    hi = _log(rng, 16, min(32768, 262144 // batch) if op == "evict" else 150000 // batch)
    lo = rng.choice([hi, max(1, hi // 8)])
    page = rng.choice([0, 64, 128])
    cap = -(-(hi + 16) // 128) * 128
    case = dict(op=op, batch=batch, prefix_lo=lo, prefix_hi=hi, cap=cap, page=page)
    if op == "evict":
        budget = rng.randint(max(1, hi // 4), hi)
        recent = rng.randint(0, budget // 2)
        case.update(budget=budget, recent=recent, sink=rng.randint(0, min(8, budget - recent)))
        return case
    case.update(rows=rng.randint(1, 10), ragged=rng.random() < 0.5)
    if op == "rope_append":
        case.update(packed=rng.random() < 0.5, layout=rng.choice(["half", "interleaved"]),
                    rotary=rng.choice([128, 64, 32]), far=rng.choice([0, 250000]),
                    scaling=rng.choice(["none", "linear", "base", "pairs", "turns"]))
    else:
        case.update(mask=rng.choice(["window", "causal"]), decay=rng.choice([1.0, 0.9]))
    return case


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rope_args(case):
    """Arguments of the rotation's plan."""
    s = case["scaling"]
    return dict(rotary_dim=case["rotary"], layout=case["layout"], scaling=s, base=1000000.0,
                factor=1.0 if s == "none" else 4.0, original_max=8192,
                low_turns=1.0, high_turns=32.0 if s == "pairs" else 4.0,
                out_scale=0.1 * math.log(4.0) + 1.0 if s == "pairs" else 1.0)


def _lens(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _caches(case, g):
    """K and V caches [B, Hkv, cap, D], or page pools and a shuffled block table."""
    B, cap, page = case["batch"], case["cap"], case["page"]
    if not page:
        shape, table = (B, HKV, cap, D), None
    else:
        per = -(-cap // page)
        shape = (B * per, HKV, page, D)
        table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return k, v, table


def _slots(case):
    """Key slots of a sequence."""
    return -(-case["cap"] // case["page"]) * case["page"] if case["page"] else case["cap"]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "rope":
        T, H, dim = case["tokens"], case["heads"], case["dim"]
        s["x"] = torch.randn(T, H, dim, generator=g, device="cuda").to(_DT[case["dtype"]])
        s["positions"] = torch.randint(0, case["span"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
    elif op == "verify":
        B, K, V = case["batch"], case["drafts"], case["vocab"]
        dt = _DT[case["dtype"]]
        pad = -(-V // 64) * 64  # the projection's width: rows are padded
        logits = torch.randn(B, K + 1, pad, generator=g, device="cuda") * 3
        draft = logits[:, :K] + case["noise"] * torch.randn(B, K, pad, generator=g, device="cuda")
        s["p"] = torch.zeros(B, K + 1, pad, device="cuda", dtype=dt)[..., :V]
        s["p"].copy_(torch.softmax(logits[..., :V], -1))
        q = torch.softmax(draft[..., :V], -1)
        s["drafts"] = torch.multinomial(q.view(B * K, V), 1, generator=g).view(B, K).to(torch.int32)
        s["q"] = None if case["certain"] else torch.zeros(B, K, pad, device="cuda", dtype=dt)[..., :V].copy_(q)
        s["u"] = torch.rand(B, K, generator=g, device="cuda")
        s["sample_u"] = torch.rand(B, generator=g, device="cuda")
        s["draft_lens"] = _lens(g, 0, K, B) if case["ragged"] else None
        s["seq_lens"] = _lens(g, 64, 4096, B)
        s["tokens"] = torch.empty(B, K + 1, device="cuda", dtype=torch.int32)
        s["accepted"] = torch.empty(B, device="cuda", dtype=torch.int32)
        s["seq_lens_out"] = torch.empty_like(s["seq_lens"])
        del logits, draft, q
    else:
        B, S = case["batch"], _slots(case)
        s["k"], s["v"], s["table"] = _caches(case, g)
        s["seq_lens"] = _lens(g, case["prefix_lo"], case["prefix_hi"], B)
        if op == "evict":
            # Accumulated weights: heavy-tailed, and exactly zero for keys that were never attended.
            w = torch.exp(2 * torch.randn(B, HKV, S, generator=g, device="cuda"))
            s["weights"] = w * (torch.rand(B, HKV, S, generator=g, device="cuda") > 0.02)
            s["key_pos"] = torch.arange(S, device="cuda", dtype=torch.int32).expand(B, HKV, S).contiguous()
            s["next_pos"] = s["seq_lens"].clone()
            s["weights_out"] = torch.zeros_like(s["weights"])
            s["key_pos_out"] = torch.zeros_like(s["key_pos"])
            s["kept"] = torch.empty(B, HKV, case["budget"], device="cuda", dtype=torch.int32)
            s["new_lens"] = torch.empty_like(s["seq_lens"])
        else:
            T = case["rows"]
            s["row_lens"] = _lens(g, max(1, T // 2), T, B) if case["ragged"] else None
            if op == "rope_append":
                if case["packed"]:
                    qkv = torch.randn(B, T, (HQ + 2 * HKV) * D, generator=g, device="cuda", dtype=torch.bfloat16)
                    parts = qkv.split([HQ * D, HKV * D, HKV * D], -1)
                    s["q"], s["kn"], s["vn"] = (x.unflatten(-1, (-1, D)) for x in parts)
                else:
                    s["q"], s["kn"], s["vn"] = (
                        torch.randn(B, T, h, D, generator=g, device="cuda", dtype=torch.bfloat16)
                        for h in (HQ, HKV, HKV))
                s["pos0"] = s["seq_lens"] + case["far"]
                s["q_out"] = torch.zeros(B, T, HQ, D, device="cuda", dtype=torch.bfloat16)
                s["key_pos"] = torch.zeros(B, HKV, S, device="cuda", dtype=torch.int32)
            else:
                s["q"] = torch.randn(B, T, HQ, D, generator=g, device="cuda", dtype=torch.bfloat16)
                s["out"] = torch.empty_like(s["q"])
                s["weights_in"] = torch.exp(2 * torch.randn(B, HKV, S, generator=g, device="cuda"))
                s["weights"] = torch.zeros(B, HKV, S, device="cuda")
    if own:
        # What a program keeps between calls: the configuration, the plan, the workspace.
        import block_masked_window_b200 as bmw
        s["bmw"] = bmw
        if op in ("rope", "rope_append"):
            s["plan"] = bmw.RopePlan.make(**_rope_args(case))
        if op in ("rope_append", "weights", "evict"):
            causal = case.get("mask") == "causal"
            s["cfg"] = bmw.Config.make(case["batch"], HQ, HKV, _slots(case),
                                       mask_mode=bmw.LA_MASK_CAUSAL_WINDOW if causal else bmw.LA_MASK_PBD)
        if op == "weights":
            s["ws"] = bmw.WeightsWorkspace(s["cfg"], case["rows"])
        if op == "evict":
            s["ws"] = bmw.EvictWorkspace(s["cfg"])
    return s


# ------------------------------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rope(s):
    s["bmw"].la_rope(s["plan"], s["x"], s["positions"], s["out"], inverse=s["case"]["inverse"])
    return s["out"]


def _own_rope_append(s):
    bmw = s["bmw"]
    opt = dict(row_lens=s["row_lens"], pos0=s["pos0"], key_pos=s["key_pos"])
    if s["table"] is None:
        bmw.la_rope_append(s["cfg"], s["plan"], s["q"], s["kn"], s["vn"], s["seq_lens"], s["q_out"],
                           s["k"], s["v"], **opt)
    else:
        bmw.la_rope_append_paged(s["cfg"], s["plan"], s["q"], s["kn"], s["vn"], s["table"], s["seq_lens"],
                                 s["q_out"], s["k"], s["v"], **opt)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "key_pos": s["key_pos"]}


def _own_weights(s):
    bmw, c = s["bmw"], s["case"]
    opt = dict(weights_in=s["weights_in"], decay=c["decay"], window_lens=s["row_lens"])
    if s["table"] is None:
        bmw.la_pbd_attn_weights(s["cfg"], s["q"], s["k"], s["v"], s["seq_lens"], c["rows"], s["out"],
                                s["weights"], s["ws"], **opt)
    else:
        bmw.la_pbd_attn_weights_paged(s["cfg"], s["q"], s["k"], s["v"], s["table"], s["seq_lens"], c["rows"],
                                      s["out"], s["weights"], s["ws"], **opt)
    return {"out": s["out"], "weights": s["weights"]}


def _own_evict(s):
    bmw, c = s["bmw"], s["case"]
    opt = dict(key_pos=s["key_pos"], next_pos=s["next_pos"], sink=c["sink"], recent=c["recent"],
               key_pos_out=s["key_pos_out"], kept_slots=s["kept"])
    if s["table"] is None:
        bmw.la_kv_evict(s["cfg"], s["weights"], s["seq_lens"], c["budget"], s["k"], s["v"], s["weights_out"],
                        s["new_lens"], s["ws"], **opt)
    else:
        bmw.la_kv_evict_paged(s["cfg"], s["weights"], s["table"], s["seq_lens"], c["budget"], s["k"], s["v"],
                              s["weights_out"], s["new_lens"], s["ws"], **opt)
    return {"k": s["k"], "v": s["v"], "weights": s["weights_out"], "key_pos": s["key_pos_out"],
            "kept": s["kept"], "new_lens": s["new_lens"]}


def _own_verify(s):
    s["bmw"].la_pbd_verify(s["p"], s["q"], s["drafts"], s["u"], s["sample_u"], s["tokens"], s["accepted"],
                           draft_lens=s["draft_lens"], seq_lens=s["seq_lens"], seq_lens_out=s["seq_lens_out"])
    return {"tokens": s["tokens"], "accepted": s["accepted"], "seq_lens": s["seq_lens_out"]}


# Plain forms.
def _frequencies(a):
    """Angle per position of each pair, in 64 bits."""
    rd, base, factor, L = a["rotary_dim"], a["base"], a["factor"], a["original_max"]
    if a["scaling"] == "base" and rd > 2:
        base = base * factor ** (rd / (rd - 2))
    i = torch.arange(rd // 2, device="cuda", dtype=torch.float64)
    f = base ** (-2 * i / rd)
    if a["scaling"] == "linear":
        f = f / factor
    elif a["scaling"] == "pairs":
        # The pairs that turn `high_turns` and `low_turns` times over the trained length.
        lo = max(math.floor(rd * math.log(L / (a["high_turns"] * 2 * math.pi)) / (2 * math.log(base))), 0)
        hi = min(math.ceil(rd * math.log(L / (a["low_turns"] * 2 * math.pi)) / (2 * math.log(base))), rd - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    elif a["scaling"] == "turns":
        t = ((L * f / (2 * math.pi) - a["low_turns"]) / (a["high_turns"] - a["low_turns"])).clamp(0, 1)
        f = f / factor * (1 - t) + f * t
    return f


def _rotate(x, positions, a, inverse=False):
    """x [..., H, dim] rotated by positions [...], in 32 bits (the angles in 64)."""
    rd = a["rotary_dim"]
    angle = positions.double()[..., None] * _frequencies(a)
    cos = (angle.cos() * a["out_scale"]).float()[..., None, :]
    sin = (angle.sin() * (-a["out_scale"] if inverse else a["out_scale"])).float()[..., None, :]
    y = x.float()
    if a["layout"] == "half":
        x1, x2 = y[..., :rd // 2], y[..., rd // 2:rd]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    else:
        x1, x2 = y[..., 0:rd:2], y[..., 1:rd:2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rd:]], -1).to(x.dtype)


def _plain_rope(s):
    return _rotate(s["x"], s["positions"], _rope_args(s["case"]), s["case"]["inverse"])


def _plain_rope_append(s):
    c, a = s["case"], _rope_args(s["case"])
    B, T = s["q"].shape[:2]
    i = torch.arange(T, device="cuda")
    pos = s["pos0"].long()[:, None] + i
    live = i < (s["row_lens"][:, None] if s["row_lens"] is not None else T)
    live = live.expand(B, T)
    s["q_out"][live] = _rotate(s["q"], pos, a)[live]
    kr = _rotate(s["kn"], pos, a)
    b, r = live.nonzero(as_tuple=True)
    slot = s["seq_lens"].long()[b] + r
    if s["table"] is None:
        s["k"][b, :, slot] = kr[live]
        s["v"][b, :, slot] = s["vn"][live]
    else:
        page = s["table"].long()[b, slot // c["page"]]
        s["k"][page, :, slot % c["page"]] = kr[live]
        s["v"][page, :, slot % c["page"]] = s["vn"][live]
    s["key_pos"][b, :, slot] = pos[live].to(torch.int32)[:, None].expand(-1, HKV)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "key_pos": s["key_pos"]}


def _whole(cache, table):
    """A paged cache as [B, Hkv, slots, D]."""
    if table is None:
        return cache
    x = cache[table.long()]                      # [B, pages, Hkv, page, D]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_weights(s):
    c = s["case"]
    B, W = s["q"].shape[:2]
    G = HQ // HKV
    k, v = _whole(s["k"], s["table"]).float(), _whole(s["v"], s["table"]).float()
    S = k.shape[2]
    q = s["q"].float().view(B, W, HKV, G, D).transpose(1, 2).flatten(2, 3)      # [B, Hkv, W G, D]
    P = s["seq_lens"].long()
    wl = s["row_lens"].long() if s["row_lens"] is not None else torch.full_like(P, W)
    i, j = torch.arange(W, device="cuda"), torch.arange(S, device="cuda")
    limit = P[:, None] + i + 1 if c["mask"] == "causal" else (P + wl)[:, None].expand(B, W)
    limit = torch.where(i < wl[:, None], limit, 0)
    seen = (j < limit[..., None])[:, None, :, None, :].expand(B, 1, W, G, S).flatten(2, 3)
    x = torch.where(seen, q @ k.transpose(-1, -2) / math.sqrt(D), float("-inf"))
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    prob = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    out = (prob @ v).view(B, HKV, W, G, D).transpose(1, 2).flatten(2, 3).to(torch.bfloat16)
    old = torch.where(j < P[:, None, None], c["decay"] * s["weights_in"], 0.0)
    s["weights"].copy_(torch.where(j < (P + wl)[:, None, None], old + prob.sum(2), s["weights"]))
    return {"out": out, "weights": s["weights"]}


def _plain_evict(s):
    c = s["case"]
    B, _, S = s["weights"].shape
    budget = c["budget"]
    P = s["seq_lens"].long()[:, None, None]
    j = torch.arange(S, device="cuda")
    w = s["weights"].double()
    w = torch.where(w.isnan(), float("-inf"), w).clamp(-1e300, 1e300)
    safe = (s["key_pos"] < c["sink"]) | (s["key_pos"] >= s["next_pos"][:, None, None] - c["recent"])
    w = torch.where(safe, float("inf"), w)
    w = torch.where(j < P, w, float("-inf"))
    order = w.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    length = P.clamp(max=budget)
    kept = (rank < length) & (j < P)
    hole, mover = ~kept & (j < length), kept & (j >= length)
    # The k-th mover goes into the k-th hole.
    nth = torch.where(mover, mover.cumsum(-1) - 1, S)
    source = torch.zeros(B, HKV, S + 1, device="cuda", dtype=torch.long).scatter_(-1, nth, j.expand_as(nth).contiguous())
    src = torch.where(hole, source.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), j)
    live = j < length
    s["weights_out"].copy_(torch.where(live, s["weights"].gather(-1, src), s["weights_out"]))
    s["key_pos_out"].copy_(torch.where(live, s["key_pos"].gather(-1, src), s["key_pos_out"]))
    s["kept"].copy_(torch.where(live, src, -1)[..., :budget] if S >= budget else -1)
    s["new_lens"].copy_(length[:, 0, 0])
    b, h, to = hole.nonzero(as_tuple=True)
    frm = src[b, h, to]
    for cache in (s["k"], s["v"]):
        if s["table"] is None:
            cache[b, h, to] = cache[b, h, frm]
        else:
            t, n = s["table"].long(), c["page"]
            cache[t[b, to // n], h, to % n] = cache[t[b, frm // n], h, frm % n]
    return {"k": s["k"], "v": s["v"], "weights": s["weights_out"], "key_pos": s["key_pos_out"],
            "kept": s["kept"], "new_lens": s["new_lens"]}


def _plain_verify(s):
    p, q, x = s["p"], s["q"], s["drafts"].long()
    B, K1, V = p.shape
    K = K1 - 1
    lens = s["draft_lens"].long() if s["draft_lens"] is not None else torch.full((B,), K, device="cuda")
    px = p[:, :K].gather(-1, x[..., None])[..., 0].double()
    qx = q.gather(-1, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    ok = (s["u"].double() * qx < px) & (torch.arange(K, device="cuda") < lens[:, None])
    n = ok.long().cumprod(-1).sum(-1)
    at = torch.arange(B, device="cuda")
    row = p[at, n].double()
    if q is not None:
        less = q[at, n.clamp(max=K - 1)].double()
    else:
        less = torch.zeros_like(row).scatter_(-1, x[at, n.clamp(max=K - 1)][:, None], float("inf"))
    rest = torch.where((n < lens)[:, None], row - less, row).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, row.clamp(min=0))
    cum = rest.cumsum(-1)
    goal = s["sample_u"].double()[:, None] * cum[:, -1:]
    j = torch.arange(V, device="cuda")
    last = torch.where(rest > 0, j, 0).amax(-1)
    token = torch.minimum((cum <= goal).sum(-1), last)
    i = torch.arange(K1, device="cuda")
    drafts = torch.cat([x, x[:, :1]], -1)
    tokens = torch.where(i < n[:, None], drafts, torch.where(i == n[:, None], token[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "accepted": n.to(torch.int32),
            "seq_lens": (s["seq_lens"] + n + 1).to(torch.int32)}


_own = dict(rope=_own_rope, rope_append=_own_rope_append, weights=_own_weights, evict=_own_evict,
            verify=_own_verify)
_plain = dict(rope=_plain_rope, rope_append=_plain_rope_append, weights=_plain_weights, evict=_plain_evict,
              verify=_plain_verify)


# ------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * size + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rotary"]}
    if op == "verify":
        # One row of the target, and of the draft for a sequence with a rejected token (most).
        size = 4 if case["dtype"] == "fp32" else 2
        rows = 1 if case["certain"] else 2
        n = case["batch"] * case["vocab"]
        return {"bytes": n * size * rows, "flops": n * (rows + 1)}
    B, keys = case["batch"], (case["prefix_lo"] + case["prefix_hi"]) / 2
    if op == "evict":
        moved = 0.0
        if keys > case["budget"]:
            moved = B * HKV * case["budget"] * (keys - case["budget"]) / keys
        return {"bytes": B * HKV * keys * 8 + moved * D * 2 * 2 * 2
                + B * HKV * min(keys, case["budget"]) * 12, "flops": B * HKV * keys}
    rows = case["rows"] * (0.75 if case["ragged"] else 1.0)
    if op == "rope_append":
        return {"bytes": B * rows * ((HQ + 2 * HKV) * D * 2 * 2 + HKV * 4),
                "flops": 3 * B * rows * (HQ + HKV) * case["rotary"]}
    return {"bytes": B * HKV * (keys + rows) * (D * 2 * 2 + 8) + 2 * B * rows * HQ * D * 2,
            "flops": 4 * B * HQ * rows * (keys + rows) * D}


# ------------------------------------------------------------------------------------- exact
def _exact_turn(x, positions, c, sign):
    """Rotation as a product of complex numbers, in 64 bits; x [n, H, dim], positions [n]."""
    a = _rope_args(c)
    rd, factor, L = a["rotary_dim"], a["factor"], float(a["original_max"])
    w = []
    for i in range(rd // 2):
        theta = a["base"]
        if c["scaling"] == "base" and rd > 2:
            theta *= factor ** (rd / (rd - 2.0))
        f = math.exp(-2.0 * i / rd * math.log(theta))
        if c["scaling"] == "linear":
            f /= factor
        if c["scaling"] == "turns":
            turns = f * L / (2 * math.pi)
            keep = min(max((turns - a["low_turns"]) / (a["high_turns"] - a["low_turns"]), 0.0), 1.0)
            f = keep * f + (1 - keep) * f / factor
        if c["scaling"] == "pairs":
            at = [rd * math.log(L / (2 * math.pi * n)) / (2 * math.log(theta))
                  for n in (a["high_turns"], a["low_turns"])]
            first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
            share = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            f = (1 - share) * f + share * f / factor
        w.append(f)
    w = torch.tensor(w, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full((), a["out_scale"], dtype=torch.float64, device="cuda").expand(len(positions), rd // 2),
                       sign * torch.outer(positions.double(), w))[:, None]
    y = x.double().clone()
    if c["layout"] == "half":
        z = torch.complex(y[..., :rd // 2].contiguous(), y[..., rd // 2:rd].contiguous()) * turn
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :rd].unflatten(-1, (-1, 2)).contiguous()) * turn
        y[..., :rd] = torch.view_as_real(z).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_turn(s["x"], s["positions"], case, -1.0 if case["inverse"] else 1.0)
    if op == "verify":
        return None  # whole numbers
    B, page, table = case["batch"], case["page"], s["table"]
    lens = s["seq_lens"].tolist()
    rows = s["row_lens"].tolist() if s.get("row_lens") is not None else [case.get("rows", 0)] * B

    def at(b, slots):
        """Where a sequence's slots lie in a cache: (first index, slot index)."""
        slots = torch.as_tensor(slots, device="cuda", dtype=torch.long)
        if table is None:
            return torch.full_like(slots, b), slots
        return table[b].long()[slots // page], slots % page

    if op == "rope_append":
        k, v, q = s["k"].double(), s["v"].double(), s["q_out"].double()
        for b in range(B):
            pos = s["pos0"][b].long() + torch.arange(rows[b], device="cuda")
            x, y = at(b, range(lens[b], lens[b] + rows[b]))
            q[b, :rows[b]] = _exact_turn(s["q"][b, :rows[b]], pos, case, 1.0)
            k[x, :, y] = _exact_turn(s["kn"][b, :rows[b]], pos, case, 1.0)
            v[x, :, y] = s["vn"][b, :rows[b]].double()
        return {"q": q, "k": k, "v": v, "key_pos": None}
    if op == "weights":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        weights = s["weights"].double()
        for b in range(B):
            n = lens[b] + rows[b]
            x, y = at(b, range(n))
            for h in range(HQ):
                kv = h * HKV // HQ
                score = s["q"][b, :rows[b], h].double() @ s["k"][x, kv, y].double().T * D ** -0.5
                if case["mask"] == "causal":
                    score += torch.full((rows[b], n), float("-inf"), dtype=torch.float64, device="cuda").triu(lens[b] + 1)
                prob = torch.softmax(score, -1)
                out[b, :rows[b], h] = prob @ s["v"][x, kv, y].double()
                weights[b, kv, :n] += prob.sum(0)
            weights[b, :, :lens[b]] += case["decay"] * s["weights_in"][b, :, :lens[b]].double()
        return {"out": out, "weights": weights}
    # evict
    k, v = s["k"].double(), s["v"].double()
    weights = s["weights_out"].double()
    w_all, pos_all, ends = s["weights"].cpu().numpy(), s["key_pos"].cpu().numpy(), s["next_pos"].tolist()
    for b in range(B):
        n, keep = lens[b], min(lens[b], case["budget"])
        for h in range(HKV):
            w, pos = w_all[b, h, :n], pos_all[b, h, :n]
            safe = (pos < case["sink"]) | (pos >= ends[b] - case["recent"])
            best = np.lexsort((np.arange(n), -w, ~safe))[:keep]
            chosen = np.zeros(n, bool)
            chosen[best] = True
            src = np.arange(keep)
            src[~chosen[:keep]] = np.nonzero(chosen[keep:])[0] + keep
            weights[b, h, :keep] = torch.from_numpy(w[src]).to("cuda", torch.float64)
            (x, y), (fx, fy) = at(b, range(keep)), at(b, src)
            k[x, h, y] = s["k"][fx, h, fy].double()
            v[x, h, y] = s["v"][fx, h, fy].double()
    return {"k": k, "v": v, "weights": weights, "key_pos": None, "kept": None, "new_lens": None}
