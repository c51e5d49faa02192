"""From a prompt to a bounded cache, as a serving loop runs it: attention over
the packed prompts (mla_prefill), their latents written into pages
(mla_cache_write), the attention that the prompt's last queries gave every token
(mla_decode for their log-sum-exp, mla_attn_weights), eviction down to a budget
(mla_cache_evict), then steps that append a token, decode over what was kept,
score again and evict the one token over. Every stage is held to 64-bit
arithmetic on the values that it was given. Also: calls on two streams at once,
and pools whose offsets pass 32 bits."""
import math

import numpy as np
import pytest
import torch

import keep_ref
import mla_latent_kv_cache_gb300 as m
import oracle
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 1 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    oracle.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


class _Loop:
    """Requests with pages of their own; Hq heads with up-projections W_UK, W_UV."""

    def __init__(self, kind, lens, Hq=8, page=16, window=4, seed=0):
        self.kind, self.lens, self.Hq, self.page, self.window = kind, list(lens), Hq, page, window
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.rand = lambda *n: torch.randn(n, generator=g, device=DEV).to(torch.bfloat16)
        self.B, T = len(lens), sum(lens)
        self.w_uk, self.w_uv = self.rand(Hq, 128, 512) / 22, self.rand(Hq, 128, 512) / 22
        self.most = max(lens) + 8
        pages = -(-self.most // page)
        perm = np.random.default_rng(seed).permutation(self.B * pages)
        self.bt = torch.from_numpy(perm.reshape(self.B, pages).astype(np.int32)).to(DEV)
        self.cache = torch.zeros((self.B * pages * page, m.mla_row_bytes(kind)), dtype=torch.uint8, device=DEV)
        self.sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.weights = torch.zeros((self.B, self.most), device=DEV)
        self.positions = torch.zeros((self.B, self.most), dtype=torch.int32, device=DEV)
        for b, n in enumerate(lens):
            self.positions[b, :n] = torch.arange(n, device=DEV)
        self.moves = torch.zeros((self.B, self.most + 2), dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def slots(self, b, j):
        j = torch.as_tensor(j, device=DEV)
        return self.bt[b].long()[j // self.page] * self.page + j % self.page

    def absorbed(self, q):  # [n, Hq, 192] -> q_lat, q_pe
        q_lat = torch.einsum("nhd,hdc->nhc", q[:, :, :128].float(), self.w_uk.float()).to(torch.bfloat16)
        return q_lat.contiguous(), q[:, :, 128:].contiguous()

    def decode(self, q_lat, q_pe, q_len):
        out, lse, ws = m.decode(q_lat, q_pe, self.cache, self.kind, self.page, self.bt, self.sl, q_len, SCALE,
                                out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert m.device_status(ws) == 0
        ref_o, ref_l = oracle.decode(q_lat.cpu(), q_pe.cpu(), self.cache.cpu().numpy(), self.kind, self.page,
                                     self.bt.cpu().numpy(), self.sl.cpu().numpy(), self.B, q_len, self.Hq, SCALE)
        tol = 1e-2 + 2e-2 * np.abs(ref_o) if self.kind == 0 else 5e-2  # the decode's own bar
        assert np.all(np.abs(out.double().cpu().numpy().reshape(ref_o.shape) - ref_o) <= tol)
        assert np.abs(lse.double().cpu().numpy().reshape(ref_l.shape) - ref_l).max() <= (1e-3 if self.kind == 0 else 5e-2)
        return lse

    def score(self, q_lat, q_pe, lse, q_len, decay):
        old = self.weights.clone()
        m.mla_attn_weights(q_lat, q_pe, lse, self.cache, self.kind, self.page, self.bt, self.sl, q_len, SCALE,
                           self.weights, decay=decay, status=self.status)
        x = keep_ref.rows_f64(self.cache, self.kind)
        q = torch.cat([q_lat, q_pe], dim=2).double().cpu().numpy()
        got, L = self.weights.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(self.B):
            T = int(self.sl[b])
            k = x[self.slots(b, torch.arange(T)).cpu().numpy()]
            want = np.zeros(T)
            for t in range(q_len):
                s = SCALE * (q[b * q_len + t] @ k.T) - L[b * q_len + t][:, None]
                want += np.where(np.arange(T) <= T - q_len + t, np.exp(s).sum(axis=0), 0)
            want += decay * old[b, :T].double().cpu().numpy()
            # |products| up to about 40 after scaling: see the bound in the scores' own test
            assert np.all(np.abs(got[b, :T] - want) <= 1e-3 * want + 1e-30)

    def evict(self, budget, n_sink, n_recent):
        before = [t.cpu().numpy().copy() for t in (self.cache, self.bt, self.sl, self.weights, self.positions)]
        m.mla_cache_evict(self.cache, self.kind, self.page, self.bt, self.sl, self.weights, self.positions,
                          torch.full((self.B,), budget, dtype=torch.int32, device=DEV), n_sink, n_recent, self.sl,
                          self.weights, self.positions, self.moves, status=self.status)
        torch.cuda.synchronize()
        assert int(self.status) == 0
        ref = keep_ref.evict(*before, np.full(self.B, budget), n_sink, n_recent, self.page)
        assert np.array_equal(self.cache.cpu().numpy(), ref[0]) and np.array_equal(self.sl.cpu().numpy(), ref[1])
        for b in range(self.B):
            n = int(ref[1][b])
            assert np.array_equal(self.weights[b, :n].cpu().numpy(), ref[2][b])
            assert np.array_equal(self.positions[b, :n].cpu().numpy(), ref[3][b])


@pytest.mark.parametrize("kind", [0, 1])
def test_prompt_to_bounded_cache(kind):
    r = _Loop(kind, [5, 300, 129, 64])
    T = sum(r.lens)
    latent, k_pe, q = r.rand(T, 512), r.rand(T, 64), r.rand(T, r.Hq, 192)
    # the prompt: keys and values from the latents, attention over all of it
    k_nope = torch.einsum("tc,hdc->thd", latent.float(), r.w_uk.float()).to(torch.bfloat16)
    v = torch.einsum("tc,hdc->thd", latent.float(), r.w_uv.float()).to(torch.bfloat16)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(r.lens)]), dtype=torch.int32, device=DEV)
    out = torch.empty((T, r.Hq, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((T, r.Hq), device=DEV)
    m.mla_prefill(q, k_nope, k_pe, v, cu, cu, max(r.lens), SCALE, out, lse, status=r.status)
    # its latents into the pages
    slots = torch.cat([r.slots(b, torch.arange(n)) for b, n in enumerate(r.lens)])
    m.mla_cache_write(latent, k_pe, slots, r.cache, kind)
    # the last `window` queries of every prompt (requests are longer than that)
    last = torch.cat([torch.arange(int(cu[b + 1]) - r.window, int(cu[b + 1])) for b in range(r.B)]).to(DEV)
    q_lat, q_pe = r.absorbed(q[last])
    lse_w = r.decode(q_lat, q_pe, r.window)
    # the absorbed form and the prompt's own are the same scores, up to the bf16
    # rounding of keys and absorbed queries (and of the codes): a score is a sum
    # of 192 products of N(0,1) values, each off by 2^-8 twice at most; their
    # root-sum-square times the scale is about 0.01, 20 times that the worst
    assert float((lse_w - lse[last]).abs().max()) < (0.2 if kind == 0 else 0.5)
    r.score(q_lat, q_pe, lse_w, r.window, 0.0)
    r.evict(100, 4, 16)
    assert r.sl.tolist() == [5, 100, 100, 64]
    for step in range(3):
        # a new token: its row at the next place, its position after the newest
        rows, pe, qn = r.rand(r.B, 512), r.rand(r.B, 64), r.rand(r.B, r.Hq, 192)
        at = r.sl.long()
        m.mla_cache_write(rows, pe, torch.stack([r.slots(b, at[b]) for b in range(r.B)]).reshape(-1), r.cache, kind)
        for b in range(r.B):
            r.positions[b, at[b]] = r.lens[b] + step
            r.weights[b, at[b]] = 0
        r.sl += 1
        q_lat, q_pe = r.absorbed(qn)
        r.score(q_lat, q_pe, r.decode(q_lat, q_pe, 1), 1, 0.9)
        r.evict(100, 4, 16)
    assert r.sl.tolist() == [8, 100, 100, 67]
    for b, n in enumerate(r.lens):  # the protected ends are there, each position once
        kept = r.positions[b, :int(r.sl[b])].tolist()
        assert len(set(kept)) == len(kept)
        assert set(range(min(4, n))) <= set(kept) and set(range(max(0, n + 3 - 16), n + 3)) <= set(kept)


def test_calls_without_work():
    e = lambda *n, dt=torch.bfloat16: torch.empty(n, dtype=dt, device=DEV)
    i32 = torch.int32
    m.mla_prefill(e(0, 8, 192), e(0, 2, 128), e(0, 64), e(0, 2, 128), torch.zeros(4, dtype=i32, device=DEV),
                  torch.zeros(4, dtype=i32, device=DEV), 0, SCALE, e(0, 8, 128), e(0, 8, dt=torch.float32))
    cache = torch.zeros((64, 1152), dtype=torch.uint8, device=DEV)
    none = (e(0, 4, dt=i32), e(0, dt=i32))
    m.mla_attn_weights(e(0, 8, 512), e(0, 8, 64), e(0, 8, dt=torch.float32), cache, 0, 16, *none, 1, SCALE,
                       e(0, 50, dt=torch.float32))
    m.mla_cache_evict(cache, 0, 16, *none, e(0, 50, dt=torch.float32), e(0, 50, dt=i32), e(0, dt=i32), 0, 0, e(0, dt=i32),
                      e(0, 50, dt=torch.float32), e(0, 50, dt=i32), e(0, 52, dt=i32))
    # requests without tokens, and score rows of no length
    bt, sl = torch.zeros((2, 4), dtype=i32, device=DEV), torch.zeros(2, dtype=i32, device=DEV)
    w, pos = torch.ones((2, 5), device=DEV), torch.ones((2, 5), dtype=i32, device=DEV)
    m.mla_attn_weights(e(2, 8, 512), e(2, 8, 64), torch.zeros((2, 8), device=DEV), cache, 0, 16, bt, sl, 1, SCALE, w)
    nl, mv = sl + 9, torch.full((2, 7), -1, dtype=i32, device=DEV)
    m.mla_cache_evict(cache, 0, 16, bt, sl, w, pos, sl + 3, 0, 0, nl, w, pos, mv)
    assert bool((w == 1).all()) and nl.tolist() == [0, 0] and mv[:, :2].tolist() == [[0, 0], [0, 0]]
    m.mla_cache_evict(cache, 0, 16, bt, sl + 6, w[:, :0], pos[:, :0], sl + 3, 0, 0, nl, w[:, :0], pos[:, :0], mv)
    torch.cuda.synchronize()
    assert nl.tolist() == [0, 0] and not bool(cache.any())


def test_two_streams_at_once():
    # the same kernels twice at the same time share nothing
    r = _Loop(0, [700, 900])
    q, kv, pe = r.rand(1600, 8, 192), r.rand(1600, 8, 256), r.rand(1600, 64)
    cu = torch.tensor([0, 700, 1600], dtype=torch.int32, device=DEV)
    m.mla_cache_write(r.rand(1600, 512), pe, torch.cat([r.slots(0, torch.arange(700)), r.slots(1, torch.arange(900))]),
                      r.cache, 0)
    q_lat, q_pe = r.absorbed(q[:2])
    lse_d = r.decode(q_lat, q_pe, 1)

    def work():
        out = torch.empty((1600, 8, 128), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((1600, 8), device=DEV)
        w = torch.zeros((2, r.most), device=DEV)
        cache, sl, wp = r.cache.clone(), r.sl.clone(), r.positions.clone()
        nw, mv = torch.zeros_like(w), torch.zeros_like(r.moves)
        bud = torch.tensor([333, 444], dtype=torch.int32, device=DEV)

        def go():
            for _ in range(5):
                m.mla_prefill(q, kv[:, :, :128], pe, kv[:, :, 128:], cu, cu, 900, SCALE, out, lse)
                m.mla_attn_weights(q_lat, q_pe, lse_d, r.cache, 0, 16, r.bt, r.sl, 1, SCALE, w, decay=0.5)
                m.mla_cache_evict(cache, 0, 16, r.bt, r.sl, w, r.positions, bud, 4, 8, sl, nw, wp, mv)
        return go, (out, lse, w, cache, sl, nw, wp)

    alone, want = work()
    alone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = [work() for _ in streams]
    torch.cuda.synchronize()
    for s, (go, _) in zip(streams, runs):
        with torch.cuda.stream(s):
            go()
    torch.cuda.synchronize()
    for _, got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", [0, 1])
def test_pool_past_32_bit_offsets(kind):
    # rows above slot 2^31 / 576 and byte offsets past 2^32
    page, row = 64, m.mla_row_bytes(kind)
    pages = (5 << 30) // (row * page)
    cache = torch.empty((pages * page, row), dtype=torch.uint8, device=DEV)
    lens = [500, 77]
    ids = [pages - 1 - i for i in range(8)] + [pages - 9, pages - 10]
    bt = torch.tensor([ids[:8], ids[8:] + [-1] * 6], dtype=torch.int32, device=DEV)
    small = _Loop(kind, lens, page=page)
    rows, pe = small.rand(577, 512), small.rand(577, 64)
    big_slots = torch.cat([bt[b].long()[torch.arange(n, device=DEV) // page] * page + torch.arange(n, device=DEV) % page
                           for b, n in enumerate(lens)])
    low_slots = torch.cat([small.slots(b, torch.arange(n)) for b, n in enumerate(lens)])
    m.mla_cache_write(rows, pe, big_slots, cache, kind)
    m.mla_cache_write(rows, pe, low_slots, small.cache, kind)
    q_lat, q_pe = small.absorbed(small.rand(2, 8, 192))
    lse = small.decode(q_lat, q_pe, 1)
    got, want = torch.zeros_like(small.weights), torch.zeros_like(small.weights)
    m.mla_attn_weights(q_lat, q_pe, lse, cache, kind, page, bt, small.sl, 1, SCALE, got)
    m.mla_attn_weights(q_lat, q_pe, lse, small.cache, kind, page, small.bt, small.sl, 1, SCALE, want)
    assert torch.equal(got, want)
    bud = torch.tensor([200, 50], dtype=torch.int32, device=DEV)
    for c, table in ((cache, bt), (small.cache, small.bt)):
        nl = torch.zeros(2, dtype=torch.int32, device=DEV)
        m.mla_cache_evict(c, kind, page, table, small.sl, want, small.positions, bud, 4, 8, nl, torch.zeros_like(want),
                          torch.zeros_like(small.positions), small.moves, status=small.status)
        assert nl.tolist() == [200, 50] and int(small.status) == 0
    for b, n in ((0, 200), (1, 50)):
        j = torch.arange(n, device=DEV)
        big = cache[bt[b].long()[j // page] * page + j % page]
        assert torch.equal(big, small.cache[small.slots(b, j)])


def test_a_length_far_past_the_scores_costs_nothing():
    # tokens past the score rows are not read: a length that nothing backs ends at once
    r = _Loop(0, [100, 40])
    m.mla_cache_write(r.rand(140, 512), r.rand(140, 64),
                      torch.cat([r.slots(0, torch.arange(100)), r.slots(1, torch.arange(40))]), r.cache, 0)
    q_lat, q_pe = r.absorbed(r.rand(2, 8, 192))
    lse = r.decode(q_lat, q_pe, 1)
    want = torch.zeros((2, 90), device=DEV)
    m.mla_attn_weights(q_lat, q_pe, lse, r.cache, 0, 16, r.bt, r.sl, 1, SCALE, want)
    got = torch.zeros_like(want)
    sl = torch.tensor([2 ** 31 - 1, 40], dtype=torch.int32, device=DEV)
    m.mla_attn_weights(q_lat, q_pe, lse, r.cache, 0, 16, r.bt, sl, 1, SCALE, got, status=r.status)
    assert torch.equal(got, want) and int(r.status) == 0
