"""Plain 64-bit forms of the calls that keep the cache (mla_attn_weights,
mla_cache_evict) in numpy, written from their definitions, for the tests."""
import numpy as np
import torch


def rows_f64(cache, kind, lat_dim=512):
    """Every row of a pool as fp64 values [num_slots, lat_dim + 64]."""
    raw = cache.cpu()
    if kind == 0:
        return raw.view(torch.bfloat16).reshape(-1, lat_dim + 64).double().numpy()
    codes = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double().numpy()
    scale = raw[:, 512:528].contiguous().view(torch.float32).double().numpy()
    rope = raw[:, 528:].contiguous().view(torch.bfloat16).double().numpy()
    return np.concatenate([codes * np.repeat(scale, 128, axis=1), rope], axis=1)


def request_slots(block_table, b, T, page_size, num_slots):
    """Slots of request b's tokens; a page outside the pool reads as page 0."""
    j = np.arange(T)
    table = block_table[b].astype(np.int64)
    page = np.where(j // page_size < len(table), table[np.minimum(j // page_size, len(table) - 1)], -1)
    bad = (page < 0) | ((page + 1) * page_size > num_slots)
    return np.where(bad, 0, page) * page_size + j % page_size, bad.any()


def scores(wl, cache, lat_dim=512):
    """Per request: scores [rows, T] fp64 (-inf where a row does not see the
    token), and a bound on the magnitude of the products summed in a score."""
    x = rows_f64(cache, wl.kind, lat_dim)
    q = np.concatenate([wl.q_lat.cpu().double().numpy(), wl.q_pe.cpu().double().numpy()], axis=2)
    bt, sl = wl.block_table.cpu().numpy(), wl.seq_lens.cpu().numpy()
    out, mag = [], 0.0
    for b in range(wl.B):
        T = int(sl[b])
        slots, _ = request_slots(bt, b, T, wl.page_size, x.shape[0])
        k = x[slots]
        qb = q[b * wl.Qt:(b + 1) * wl.Qt].reshape(wl.Qt * wl.Hq, -1)
        s = wl.scale * (qb @ k.T)
        last = T - wl.Qt + np.arange(wl.Qt * wl.Hq) // wl.Hq
        s[np.arange(T)[None, :] > last[:, None]] = -np.inf
        out.append(s)
        if T:
            m = wl.scale * (np.abs(qb) @ np.abs(k).T)
            mag = max(mag, float(m[np.isfinite(m)].max(initial=0.0)))
    return out, mag


def lse_of(sc):
    """Natural log-sum-exp of each row; -inf for a row that sees nothing."""
    res = []
    for s in sc:
        m = s.max(axis=1, initial=-np.inf)
        safe = np.where(np.isfinite(m), m, 0.0)
        with np.errstate(divide="ignore"):
            res.append(safe + np.log(np.exp(s - safe[:, None]).sum(axis=1)))
    return np.concatenate(res) if res else np.zeros(0)


def attn_weights(sc, lse, rows, old, decay):
    """The new scores: `old` [B, max_len] fp64 with each request's entries replaced."""
    new = old.copy()
    for b, s in enumerate(sc):
        L = lse[b * rows:(b + 1) * rows]
        use = L > -np.inf
        got = np.exp(s[use] - L[use][:, None]).sum(axis=0)
        n = min(s.shape[1], old.shape[1])
        new[b, :n] = (decay * old[b, :n] if decay != 0 else 0.0) + got[:n]
    return new


def evict(cache, block_table, lens, weights, positions, budgets, n_sink, n_recent, page_size):
    """Returns (cache, new_lens, kept scores per request, kept positions, moves [n, 2]) of one call."""
    cache = cache.copy()
    B, max_len = weights.shape
    new_lens, kept_w, kept_p, moves = [], [], [], []
    for b in range(B):
        T = max(min(int(lens[b]), max_len, block_table.shape[1] * page_size), 0)
        K = min(max(int(budgets[b]), 0), T)
        w, p = weights[b, :T].astype(np.float64), positions[b, :T].astype(np.int64)
        # rank: protected first, then scores from the top, NaN last; equal ones by place
        safe = np.zeros(T, bool) if T == 0 else (p < n_sink) | (p > p.max() - n_recent)
        cls = np.where(safe, 0, np.where(np.isnan(w), 2, 1))
        val = np.where(cls == 1, -w, 0.0)
        order = np.lexsort((np.arange(T), val, cls))
        keep = np.zeros(T, bool)
        keep[order[:K]] = True
        hole = np.flatnonzero(~keep[:K])
        src = np.flatnonzero(keep[K:]) + K
        nw, npos = weights[b, :K].copy(), positions[b, :K].copy()
        for d, s in zip(hole, src):
            nw[d], npos[d] = weights[b, s], positions[b, s]
            pd, ps = int(block_table[b, d // page_size]), int(block_table[b, s // page_size])
            ds, ss = pd * page_size + d % page_size, ps * page_size + s % page_size
            if min(pd, ps) >= 0 and max(ds, ss) < len(cache):
                cache[ds] = cache[ss]
        new_lens.append(K)
        kept_w.append(nw)
        kept_p.append(npos)
        moves.append(np.stack([src, hole], axis=1))
    return cache, np.array(new_lens), kept_w, kept_p, moves
