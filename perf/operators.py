"""The prompt-side and cache-keeping operators of the latent cache, as measured cases.

  prefill   attention over whole prompts, causal, packed sequences of different
            lengths, grouped heads, one rotary key shared by all heads
            (mla_prefill): what fills the cache that mla_decode reads.
  weights   the attention weight that every cached token received from a step's
            queries, added into a running score (mla_attn_weights).
  evict     keeping the best-scored tokens of each request within a budget and
            closing the gaps in its pages (mla_cache_evict).

A case names an operator and its sizes. The lengths of its requests are drawn
from the case's own "lens" number, so they are part of the case; the values
are drawn from the seed.
"""
import math

import numpy as np
import torch

own = False

SCALE = 1.0 / math.sqrt(192.0)
ROW_BYTES = {"bf16": 1152, "fp8": 656}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a single short question: what a call costs before any work
        {"name": "prefill_one_short", "op": "prefill", "B": 1, "q_lo": 37, "q_hi": 37, "c_lo": 0, "c_hi": 0, "Hq": 8,
         "Hkv": 8, "causal": True, "lens": 1},
        # an ordinary prefill batch: prompts of very different lengths, none a multiple of a tile, packed
        {"name": "prefill_packed", "op": "prefill", "B": 16, "q_lo": 1, "q_hi": 4100, "c_lo": 0, "c_hi": 0, "Hq": 16,
         "Hkv": 16, "causal": True, "lens": 2},
        # one long document
        {"name": "prefill_long", "op": "prefill", "B": 1, "q_lo": 32768, "q_hi": 32768, "c_lo": 0, "c_hi": 0, "Hq": 16,
         "Hkv": 16, "causal": True, "lens": 3},
        # chunked prefill: a few hundred new tokens over a gathered context, four query heads to a key head
        {"name": "prefill_chunk_grouped", "op": "prefill", "B": 6, "q_lo": 200, "q_hi": 700, "c_lo": 1000, "c_hi": 8192,
         "Hq": 32, "Hkv": 8, "causal": True, "lens": 4},
        # two requests, one step: the latency of keeping scores at all
        {"name": "weights_tiny", "op": "weights", "kind": "bf16", "B": 2, "t_lo": 37, "t_hi": 200, "Hq": 8, "q_len": 1,
         "page": 16, "lens": 5},
        # a serving batch at 16 heads
        {"name": "weights_batched", "op": "weights", "kind": "bf16", "B": 64, "t_lo": 1024, "t_hi": 8192, "Hq": 16,
         "q_len": 1, "page": 16, "lens": 6},
        # very long contexts, a verify step of two tokens
        {"name": "weights_long", "op": "weights", "kind": "bf16", "B": 4, "t_lo": 262144, "t_hi": 262144, "Hq": 32,
         "q_len": 2, "page": 64, "lens": 7},
        # a quantised pool, 64 heads
        {"name": "weights_fp8", "op": "weights", "kind": "fp8", "B": 32, "t_lo": 16384, "t_hi": 32768, "Hq": 64,
         "q_len": 1, "page": 64, "lens": 8},
        # the steady state: every request a few tokens over its budget
        {"name": "evict_step", "op": "evict", "kind": "bf16", "B": 64, "t_lo": 4097, "t_hi": 4160, "budget": 4096,
         "sink": 4, "recent": 64, "page": 16, "lens": 9},
        # after a long prompt: half of a quarter of a million tokens goes, few requests
        {"name": "evict_long", "op": "evict", "kind": "bf16", "B": 4, "t_lo": 262144, "t_hi": 262144, "budget": 131072,
         "sink": 4, "recent": 1024, "page": 64, "lens": 10},
        # a quantised pool after ragged prompts, a quarter kept
        {"name": "evict_fp8", "op": "evict", "kind": "fp8", "B": 32, "t_lo": 1000, "t_hi": 32768, "budget": 6001,
         "sink": 16, "recent": 500, "page": 16, "lens": 11},
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(("prefill", "weights", "evict"))
    case = {"op": op, "lens": rng.randrange(1 << 30)}
    if op == "prefill":
        Hkv = rng.choice((1, 2, 4, 8, 16))
        g = rng.choice([g for g in (1, 2, 3, 4, 8) if g * Hkv <= 32])
        hi = log(1, 12000)
        c_hi = rng.choice((0, 0, log(1, 8192)))
        B = max(1, min(log(1, 48), 16384 // hi, (1 << 28) // (hi * (hi + c_hi))))
        case.update(B=B, q_lo=rng.randint(0, hi) if B > 1 else hi, q_hi=hi, c_lo=c_hi // 3, c_hi=c_hi, Hq=g * Hkv, Hkv=Hkv,
                    causal=rng.random() < 0.8)
        return case
    kind = rng.choice(("bf16", "fp8"))
    B = log(1, 96)
    hi = log(2, min(262144, 1000000 // B))
    case.update(kind=kind, B=B, t_lo=rng.randint(0, hi), t_hi=hi, page=rng.choice((1, 3, 8, 16, 16, 64, 64, 96)))
    if op == "weights":
        q_len = rng.choice((1, 1, 2, 4, 7))
        case.update(Hq=rng.choice((1, 8, 16, 20, 32, 64, 128) if q_len == 1 else (8, 16)), q_len=q_len)
    else:
        budget = rng.randint(0, hi)
        case.update(budget=budget, sink=rng.choice((0, 4, 16)), recent=rng.randint(0, max(0, budget // 2)))
    return case


def _lens(case):
    r = np.random.default_rng(case["lens"])
    if case["op"] == "prefill":
        q = r.integers(case["q_lo"], case["q_hi"], size=case["B"], endpoint=True)
        q[0] = case["q_hi"]
        return q, q + r.integers(case["c_lo"], case["c_hi"], size=case["B"], endpoint=True)
    t = r.integers(case["t_lo"], case["t_hi"], size=case["B"], endpoint=True)
    t[0] = case["t_hi"]
    return t


def _seen(q, k, causal):
    """Pairs of a query and a key that it sees: query t of q sees keys 0 .. k - q + t."""
    return int(sum(int(a) * int(b) - (int(a) * (int(a) - 1) // 2 if causal else 0) for a, b in zip(q, k)))


def work(case):
    if case["op"] == "prefill":
        q, k = _lens(case)
        tq, tk, Hq, Hkv = int(q.sum()), int(k.sum()), case["Hq"], case["Hkv"]
        return {"bytes": 2 * tq * Hq * (192 + 128) + 4 * tq * Hq + 2 * tk * (Hkv * 256 + 64),
                "flops": 2 * (192 + 128) * Hq * _seen(q, k, case["causal"])}
    t = _lens(case)
    n, row = int(t.sum()), ROW_BYTES[case["kind"]]
    if case["op"] == "weights":
        rows = case["Hq"] * case["q_len"]
        return {"bytes": n * (row + 8) + case["B"] * rows * (1152 + 4), "flops": 2 * 576 * rows * n}
    kept = np.minimum(t, case["budget"])
    # a kept token moves if it lies past the budget; scores do not depend on the place, but for the
    # protected ends (the first stay, the last move)
    last = np.minimum(np.minimum(case["recent"], t - kept), kept)
    free_t, free_k = np.maximum(t - case["recent"] - case["sink"], 1), np.maximum(kept - case["recent"] - case["sink"], 0)
    moved = last + (np.maximum(t - kept - last, 0) * free_k) / free_t
    return {"bytes": int(n * 8 + kept.sum() * 8 + moved.sum() * 2 * row), "flops": 0}


# --------------------------------------------------------------- the inputs

def _pages(t, page, gen):
    """Shuffled pages: the table [B, most] (-1 past a request's last page) and the pool's slots."""
    need = -(-t // page)
    ids = torch.randperm(max(1, int(need.sum() * 5 // 4)), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(t), max(1, int(need.max()))), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(table.shape[1], device="cuda")[None] < torch.from_numpy(need).cuda()[:, None]
    table[cols] = ids[:int(need.sum())]
    return table, ids.numel() * page


def _pool(kind, slots, gen):
    """Rows as the cache write leaves them: N(0,1) latents and rotary keys, bf16 or 656-byte quantised."""
    pool = torch.empty((slots, ROW_BYTES[kind]), dtype=torch.uint8, device="cuda")
    step = 1 << 19
    for a in range(0, slots, step):
        n = min(step, slots - a)
        x = torch.randn((n, 576), generator=gen, device="cuda").to(torch.bfloat16)
        if kind == "bf16":
            pool[a:a + n] = x.view(torch.uint8)
            continue
        v = x[:, :512].float().view(n, 4, 128)
        scale = v.abs().amax(2) / 448.0
        pool[a:a + n, :512] = (v / scale[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, 512)
        pool[a:a + n, 512:528] = scale.view(torch.uint8)
        pool[a:a + n, 528:] = x[:, 512:].contiguous().view(torch.uint8)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    randn = lambda *n: torch.randn(n, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if case["op"] == "prefill":
        q, k = _lens(case)
        tq, tk, Hq, Hkv = int(q.sum()), int(k.sum()), case["Hq"], case["Hkv"]
        kv = randn(tk, Hkv, 256)          # what the up-projection of the latents gives: keys, then values
        rows = randn(tk, 576)             # the latent rows; their last 64 values are the shared rotary key
        s.update(q=randn(tq, Hq, 192), k_nope=kv[:, :, :128], v=kv[:, :, 128:], k_pe=rows[:, 512:],
                 cu_q=i32(np.concatenate([[0], np.cumsum(q)])), cu_k=i32(np.concatenate([[0], np.cumsum(k)])),
                 max_q=int(q.max()), max_k=int(k.max()),
                 out=torch.zeros((tq, Hq, 128), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros((tq, Hq), dtype=torch.float32, device="cuda"))
        return s
    t = _lens(case)
    table, slots = _pages(t, case["page"], gen)
    most = max(1, int(t.max()))
    s.update(kind=case["kind"], page=case["page"], table=table, lens=i32(t), cache=_pool(case["kind"], slots, gen))
    if case["op"] == "weights":
        rows = case["Hq"] * case["q_len"]
        s.update(q_lat=randn(case["B"] * case["q_len"], case["Hq"], 512), q_pe=randn(case["B"] * case["q_len"], case["Hq"], 64),
                 weights=torch.rand((case["B"], most), generator=gen, device="cuda") * (2 * rows / most))
        # the decode of the same queries has left their log-sum-exp
        sc, seen = _scores(s)
        s["lse"] = torch.logsumexp(sc.masked_fill(~seen, -math.inf), dim=2).reshape(case["B"] * case["q_len"], case["Hq"])
        return s
    # scores as running sums leave them: a long tail, and many tokens that have decayed to nothing
    w = torch.exp(2 * torch.randn((case["B"], most), generator=gen, device="cuda"))
    w = w * (torch.rand((case["B"], most), generator=gen, device="cuda") > 0.1)
    # positions with the gaps that earlier evictions left, and their order in the older half
    j = torch.arange(most, device="cuda")[None]
    mixed = torch.where(j < s["lens"][:, None] // 2, torch.rand((case["B"], most), generator=gen, device="cuda"), 2.0 + j)
    pos = torch.randint(1, 4, (case["B"], most), generator=gen, device="cuda").cumsum(1).gather(1, mixed.argsort(dim=1))
    s.update(weights=w, positions=pos.to(torch.int32), budgets=torch.full((case["B"],), case["budget"], dtype=torch.int32, device="cuda"),
             new_lens=torch.zeros_like(s["lens"]), new_weights=torch.zeros_like(w),
             new_positions=torch.zeros((case["B"], most), dtype=torch.int32, device="cuda"),
             moves=torch.zeros((case["B"], most + 2), dtype=torch.int32, device="cuda"))
    return s


# ----------------------------------------------------------- the plain forms

def _slots(table, page, most):
    j = torch.arange(most, device=table.device)
    return table.long()[:, j // page].clamp(min=0) * page + j % page


def _rows(cache, kind, slots):
    """Cached rows as fp32 values [..., 576]."""
    raw = cache[slots]
    if kind == "bf16":
        return raw.view(torch.bfloat16).float()
    codes = raw[..., :512].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    scale = raw[..., 512:528].contiguous().view(torch.float32)
    return torch.cat([(codes * scale[..., None]).flatten(-2), raw[..., 528:].contiguous().view(torch.bfloat16).float()], dim=-1)


def _scores(s):
    """Scores [B, rows, most] of a step's queries against their request's tokens, and which of them a query sees."""
    c = s["case"]
    B, most, rows = c["B"], s["weights"].shape[1], c["Hq"] * c["q_len"]
    q = torch.cat([s["q_lat"], s["q_pe"]], dim=-1).float().view(B, rows, 576)
    sc = torch.matmul(q, _rows(s["cache"], s["kind"], _slots(s["table"], s["page"], most)).transpose(1, 2)) * SCALE
    last = s["lens"][:, None] - c["q_len"] + torch.arange(rows, device="cuda")[None] // c["Hq"]
    return sc, torch.arange(most, device="cuda")[None, None] <= last[:, :, None]


def _plain_prefill(s):
    c = s["case"]
    g = c["Hq"] // c["Hkv"]
    q0, k0 = s["cu_q"][:-1, None].long(), s["cu_k"][:-1, None].long()
    nq, nk = s["cu_q"].diff()[:, None], s["cu_k"].diff()[:, None]
    t, j = torch.arange(s["max_q"], device="cuda")[None], torch.arange(s["max_k"], device="cuda")[None]
    qi, ki = (q0 + torch.minimum(t, nq - 1)).clamp(min=0), (k0 + torch.minimum(j, nk - 1)).clamp(min=0)
    real = t < nq
    seen = (j < nk)[:, None, :].expand(-1, s["max_q"], -1)
    if c["causal"]:
        seen = seen & (j[:, None, :] <= (nk - nq + t)[:, :, None])
    rows = qi[real]
    for h in range(c["Hq"]):  # a head at a time: all scores at once do not fit
        k = torch.cat([s["k_nope"][:, h // g].float()[ki], s["k_pe"].float()[ki]], dim=-1)
        sc = torch.matmul(s["q"][:, h].float()[qi] * SCALE, k.transpose(1, 2)).masked_fill_(~seen, -math.inf)
        top = sc.amax(2, keepdim=True).clamp(min=-1e30)
        p = sc.sub_(top).exp_()
        total = p.sum(2, keepdim=True)
        o = torch.matmul(p, s["v"][:, h // g].float()[ki]) / total.clamp(min=1e-30)
        s["out"][rows, h] = o[real].to(torch.bfloat16)
        s["lse"][rows, h] = (top + total.log()).squeeze(2)[real]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weights(s):
    sc, seen = _scores(s)
    got = torch.where(seen, (sc - s["lse"].view(sc.shape[0], -1, 1)).exp(), 0).sum(1)
    cached = torch.arange(s["weights"].shape[1], device="cuda")[None] < s["lens"][:, None]
    s["weights"].copy_(torch.where(cached, 0.875 * s["weights"] + got, s["weights"]))
    return {"weights": s["weights"]}


def _plain_evict(s):
    c, w, pos = s["case"], s["weights"], s["positions"]
    B, most = w.shape
    j = torch.arange(most, device="cuda")[None]
    cached = j < s["lens"][:, None]
    kept_n = torch.minimum(s["lens"], s["budgets"])[:, None]
    end = torch.where(cached, pos, -1).amax(1, keepdim=True) + 1
    safe = (pos < c["sink"]) | (pos >= end - c["recent"])
    key = torch.where(cached, torch.where(safe, math.inf, w), -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices  # equal scores: the lower index first
    kept = torch.zeros_like(cached).scatter_(1, order, j.expand(B, -1) < kept_n) & cached
    hole, mover = ~kept & (j < kept_n), kept & (j >= kept_n)
    at = torch.nonzero(hole)      # the i-th free place of a request takes its i-th kept token past the budget
    frm = torch.nonzero(mover)
    slots = _slots(s["table"], s["page"], most)
    s["cache"][slots[at[:, 0], at[:, 1]]] = s["cache"][slots[frm[:, 0], frm[:, 1]]]
    stay = kept & (j < kept_n)
    for old, new in ((w, s["new_weights"]), (pos, s["new_positions"])):
        new.copy_(torch.where(stay, old, new))
        new[at[:, 0], at[:, 1]] = old[frm[:, 0], frm[:, 1]]
    s["new_lens"].copy_(kept_n.squeeze(1))
    return _evicted(s)


def _evicted(s):
    return {"cache": s["cache"], "lens": s["new_lens"], "weights": s["new_weights"], "positions": s["new_positions"]}


def run(s):
    op, c = s["case"]["op"], s["case"]
    if own:
        import mla_latent_kv_cache_gb300 as mla
        if op == "prefill":
            mla.mla_prefill(s["q"], s["k_nope"], s["k_pe"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], SCALE, s["out"], s["lse"],
                            causal=c["causal"])
            return {"out": s["out"], "lse": s["lse"]}
        kind = mla.MLA_CACHE_BF16_576 if s["kind"] == "bf16" else mla.MLA_CACHE_FP8_DS_MLA_656
        if op == "weights":
            mla.mla_attn_weights(s["q_lat"], s["q_pe"], s["lse"], s["cache"], kind, s["page"], s["table"], s["lens"], c["q_len"],
                                 SCALE, s["weights"], decay=0.875)
            return {"weights": s["weights"]}
        mla.mla_cache_evict(s["cache"], kind, s["page"], s["table"], s["lens"], s["weights"], s["positions"], s["budgets"],
                            c["sink"], c["recent"], s["new_lens"], s["new_weights"], s["new_positions"], s["moves"])
        return _evicted(s)
    return {"prefill": _plain_prefill, "weights": _plain_weights, "evict": _plain_evict}[op](s)


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        host = {k: s[k].cpu().numpy() for k in ("weights", "positions", "new_weights", "new_positions")}
        new_w, new_p, lens = host["new_weights"].astype(np.float64), host["new_positions"], _lens(case)
        for b, n in enumerate(lens.tolist()):
            w, p, kept = host["weights"][b, :n], host["positions"][b, :n], min(n, case["budget"])
            if kept == n:
                new_w[b, :n], new_p[b, :n] = w, p
                continue
            safe = (p < case["sink"]) | (p > p.max() - case["recent"])
            best = np.lexsort((np.arange(n), -w, ~safe))
            best = np.concatenate([np.flatnonzero(safe), best[safe.sum():]])[:kept]  # protected ones count alike
            stay, late = np.zeros(kept, dtype=bool), np.sort(best[best >= kept])
            stay[best[best < kept]] = True
            new_w[b, :kept], new_p[b, :kept] = w[:kept], p[:kept]
            new_w[b, np.flatnonzero(~stay)], new_p[b, np.flatnonzero(~stay)] = w[late], p[late]
        # the pool's bytes are not computed
        return {"cache": None, "lens": np.minimum(lens, case["budget"]).astype(np.int32), "weights": new_w, "positions": new_p}
    if case["op"] == "prefill":
        q, k = _lens(case)
        if _seen(q, k, False) * case["Hq"] > 2e10:
            return None
        g = case["Hq"] // case["Hkv"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        qa = ka = 0
        for a, b in zip(q.tolist(), k.tolist()):
            for h in range(case["Hq"]):
                for t0 in range(0, a, 2048):  # queries in blocks, each against the keys that its last one sees
                    n = min(2048, a - t0)
                    top = min(b, b - a + t0 + n) if case["causal"] else b
                    if top <= 0:
                        continue
                    x = s["q"][qa + t0:qa + t0 + n, h].double()
                    z = x[:, :128] @ s["k_nope"][ka:ka + top, h // g].double().T + x[:, 128:] @ s["k_pe"][ka:ka + top].double().T
                    z *= SCALE
                    if case["causal"]:
                        see = torch.ones((n, top), dtype=torch.bool, device="cuda").tril(b - a + t0)
                        z[~see] = -math.inf
                    l = torch.logsumexp(z, 1)
                    lse[qa + t0:qa + t0 + n, h] = l
                    p = torch.nan_to_num(torch.exp(z - l[:, None]), nan=0.0)
                    out[qa + t0:qa + t0 + n, h] = p @ s["v"][ka:ka + top, h // g].double()
            qa, ka = qa + a, ka + b
        return {"out": out, "lse": lse}
    t, page, Hq, q_len = _lens(case), case["page"], case["Hq"], case["q_len"]
    weights = s["weights"].double()
    for b, n in enumerate(t.tolist()):
        for a in range(0, n, 1 << 16):
            j = torch.arange(a, min(n, a + (1 << 16)), device="cuda")
            raw = s["cache"][s["table"][b].long()[j // page] * page + j % page]
            if case["kind"] == "bf16":
                key = raw.view(torch.bfloat16).double()
            else:
                code = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double()
                key = torch.cat([code * raw[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, dim=1),
                                 raw[:, 528:].contiguous().view(torch.bfloat16).double()], dim=1)
            got = torch.zeros(len(j), dtype=torch.float64, device="cuda")
            for i in range(q_len):
                r = b * q_len + i
                z = (torch.cat([s["q_lat"][r], s["q_pe"][r]], dim=1).double() @ key.T) * SCALE - s["lse"][r].double()[:, None]
                got += torch.where(j <= n - q_len + i, z.exp().sum(0), 0.0)
            weights[b, a:a + len(j)] = 0.875 * weights[b, a:a + len(j)] + got
    return {"weights": weights}
