"""mla_cache_evict on the GPU against its definition in numpy: bytes, lengths,
scores, positions and moves have to be equal."""
import numpy as np
import pytest
import torch

import keep_ref
import mla_latent_kv_cache_gb300 as m
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


def _row_bytes(kind, lat_dim):
    return 656 if kind else 2 * (lat_dim + 64)


def _case(lens, page, kind=0, lat_dim=512, seed=0, extra=7, scores="ties"):
    r = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    most = int(max(1, lens.max())) + extra
    need = -(-np.maximum(lens, 0).astype(np.int64) // page)
    ids = r.permutation(int(need.sum()) + 3)
    bt = np.full((len(lens), max(1, int(need.max()))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    cache = r.integers(0, 256, size=(len(ids) * page, _row_bytes(kind, lat_dim)), dtype=np.uint8)
    w = r.random((len(lens), most)).astype(np.float32)
    if scores == "ties":
        w = np.floor(w * 16) / 16
    elif scores == "equal":
        w[:] = 0.0
    elif scores == "wild":
        pool = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, -3.0, 3.4e38, 1.0], dtype=np.float32)
        w = pool[r.integers(0, len(pool), size=w.shape)]
    pos = np.cumsum(r.integers(1, 4, size=w.shape), axis=1).astype(np.int32)
    return lens, bt, cache, w.astype(np.float32), pos


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _go(lens, bt, cache, w, pos, budgets, n_sink, n_recent, page, kind=0, lat_dim=512, alias=False, want_status=0):
    budgets = np.broadcast_to(np.asarray(budgets, dtype=np.int32), lens.shape).copy()
    d = dict(cache=_t(cache), bt=_t(bt), lens=_t(lens), w=_t(w), pos=_t(pos), bud=_t(budgets))
    if alias:
        nl, nw, npos = d["lens"], d["w"], d["pos"]
    else:
        nl = torch.full_like(d["lens"], -7)
        nw, npos = torch.full_like(d["w"], 123.0), torch.full_like(d["pos"], -9)
    moves = torch.full((len(lens), w.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ref_c, ref_l, ref_w, ref_p, ref_m = keep_ref.evict(cache, bt, lens, w, pos, budgets, n_sink, n_recent, page)
    for rep in range(1 if alias else 2):  # the call can be repeated
        m.mla_cache_evict(d["cache"], kind, page, d["bt"], d["lens"], d["w"], d["pos"], d["bud"], n_sink, n_recent, nl,
                          nw, npos, moves, lat_dim=lat_dim, status=st)
        torch.cuda.synchronize()
        assert int(st) == want_status
        assert np.array_equal(nl.cpu().numpy(), ref_l)
        mv, got_w, got_p = moves.cpu().numpy(), nw.cpu().numpy(), npos.cpu().numpy()
        for b in range(len(lens)):
            K = int(ref_l[b])
            n = len(ref_m[b])
            assert mv[b, 0] == n and mv[b, 1] == K
            assert np.array_equal(mv[b, 2:2 + 2 * n].reshape(n, 2), ref_m[b])
            assert (mv[b, 2 + 2 * n:] == -1).all()
            assert np.array_equal(got_w[b, :K].view(np.uint32), ref_w[b].view(np.uint32))
            assert np.array_equal(got_p[b, :K], ref_p[b])
            if alias:
                assert np.array_equal(got_w[b, K:].view(np.uint32), w[b, K:].view(np.uint32))
            else:
                assert (got_w[b, K:] == 123.0).all() and (got_p[b, K:] == -9).all()
        assert np.array_equal(d["cache"].cpu().numpy(), ref_c)


LENS = [0, 1, 2, 31, 32, 33, 500, 1000, 1023, 1024, 1025, 3000]


@pytest.mark.parametrize("kind,lat_dim", [(0, 512), (1, 512), (0, 256), (0, 768), (0, 1792)])
@pytest.mark.parametrize("scores", ["ties", "distinct", "equal", "wild"])
def test_against_the_definition(kind, lat_dim, scores):
    c = _case(LENS, 16, kind, lat_dim, seed=len(scores) + kind, scores=scores)
    _go(*c, budgets=400, n_sink=5, n_recent=50, page=16, kind=kind, lat_dim=lat_dim)


@pytest.mark.parametrize("budget", [0, 1, 2, 31, 32, 500, 999, 1024, 2999, 3000, 10 ** 9, -5])
def test_budgets(budget):
    _go(*_case(LENS, 16, seed=budget % 97), budgets=budget, n_sink=0, n_recent=3, page=16)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 64, 784])
@pytest.mark.parametrize("alias", [False, True])
def test_page_sizes_and_in_place(page, alias):
    _go(*_case(LENS, page, seed=page), budgets=[0, 1, 1, 30, 32, 7, 499, 100, 1023, 512, 1000, 2000], n_sink=4,
        n_recent=16, page=page, alias=alias)


@pytest.mark.parametrize("n_sink,n_recent", [(0, 0), (10 ** 6, 0), (0, 10 ** 6), (300, 300), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_protected_ends(n_sink, n_recent):
    # more protected tokens than the budget holds: the first of them stay
    _go(*_case(LENS, 16, seed=3), budgets=333, n_sink=n_sink, n_recent=n_recent, page=16)


@pytest.mark.parametrize("most", [4097, 9000, 20000, 40000, 100000, 200000])
def test_requests_that_several_ctas_share(most):
    r = np.random.default_rng(most)
    lens = [most, most // 2, 1, 0, most - 1]
    for scores in ("ties", "distinct"):
        _go(*_case(lens, 64, 1, seed=most, scores=scores), budgets=r.integers(0, most, size=5), n_sink=4,
            n_recent=100, page=64, kind=1)


def test_many_requests_that_fewer_ctas_share_each():
    r = np.random.default_rng(6)
    lens = r.integers(0, 20000, size=100)
    _go(*_case(lens, 16, 0, 256, seed=6), budgets=r.integers(0, 20000, size=100), n_sink=4, n_recent=64, page=16, lat_dim=256)


@pytest.mark.parametrize("row_bytes", [16, 48, 9216, 9232, 20000, 65536])
def test_any_row_size(row_bytes):
    lens, bt, cache, w, pos = _case([300, 0, 77], 16, seed=row_bytes)
    cache = np.random.default_rng(1).integers(0, 256, size=(len(cache), row_bytes), dtype=np.uint8)
    ref_c, ref_l, _, _, _ = keep_ref.evict(cache, bt, lens, w, pos, np.array([100, 5, 40]), 2, 8, 16)
    d = [_t(x) for x in (cache, bt, lens, w, pos, np.array([100, 5, 40], np.int32))]
    nl, nw, npos = torch.zeros_like(d[2]), torch.zeros_like(d[3]), torch.zeros_like(d[4])
    mv = torch.zeros((3, w.shape[1] + 2), dtype=torch.int32, device=DEV)
    st = m.load().mla_cache_evict(d[0].data_ptr(), row_bytes, len(cache), 16, d[1].data_ptr(), bt.shape[1], d[2].data_ptr(),
                                  d[3].data_ptr(), d[4].data_ptr(), w.shape[1], w.shape[1], d[5].data_ptr(), 3, 2, 8,
                                  nl.data_ptr(), nw.data_ptr(), npos.data_ptr(), mv.data_ptr(), mv.shape[1], None, None)
    torch.cuda.synchronize()
    assert st == m.MLA_OK
    assert np.array_equal(nl.cpu().numpy(), ref_l) and np.array_equal(d[0].cpu().numpy(), ref_c)


def test_more_tokens_than_shared_memory_holds_keys():
    # 16 CTAs keep 524,288 keys in registers; past that 8 keep 393,216 in shared
    # memory and form the rest again on every pass
    for n in (400000, 600000):
        _go(*_case([n, 5], 784, 0, 256, seed=1), budgets=[170001, 3], n_sink=4, n_recent=1000, page=784, lat_dim=256)


def test_more_requests_than_a_cta_counts_at_once():
    r = np.random.default_rng(5)
    lens = r.integers(0, 40, size=2500)
    _go(*_case(lens, 8, 1, seed=2), budgets=r.integers(0, 40, size=2500), n_sink=1, n_recent=2, page=8, kind=1)


def test_lengths_past_the_score_rows_or_the_table_row_flag():
    lens, bt, cache, w, pos = _case([100, 200, 50], 16, seed=4, extra=0)
    _go(np.array([100, 300, 50], np.int32), bt, cache, w, pos, 30, 2, 5, 16, want_status=m.STATUS_BAD_BLOCK)
    _go(lens, bt[:, :5].copy(), cache, w, pos, 30, 2, 5, 16, want_status=m.STATUS_BAD_BLOCK)


def test_pages_outside_the_pool_are_not_copied_and_flag():
    lens, bt, cache, w, pos = _case([300], 16, seed=6)
    bt[0, 1] = 10 ** 6   # holes there
    bt[0, 17] = -3       # kept tokens there
    w[0, 16:32] = 0
    w[0, 272:288] = 1
    _go(lens, bt, cache, w, pos, 100, 0, 0, 16, want_status=m.STATUS_BAD_BLOCK)


def test_negative_and_repeated_positions():
    lens, bt, cache, w, pos = _case([500, 40], 16, seed=7)
    pos = (pos % 13 - 6).astype(np.int32)
    _go(lens, bt, cache, w, pos, 77, 2, 3, 16)


def test_graph_replay_and_rows_of_wider_buffers():
    lens, bt, cache, w, pos = _case([500, 900, 64], 16, seed=8)
    ref_c, ref_l, ref_w, ref_p, _ = keep_ref.evict(cache, bt, lens, w, pos, np.array([100] * 3), 4, 8, 16)
    c, b_, l = _t(cache), _t(bt), _t(lens)
    wide_w, wide_p = torch.zeros((3, 2000), device=DEV), torch.zeros((3, 2000), dtype=torch.int32, device=DEV)
    n = w.shape[1]
    wide_w[:, :n], wide_p[:, :n] = _t(w), _t(pos)
    nw, npos = torch.zeros_like(wide_w), torch.zeros_like(wide_p)
    nl = torch.zeros(3, dtype=torch.int32, device=DEV)
    mv = torch.zeros((3, n + 2), dtype=torch.int32, device=DEV)
    bud = torch.full((3,), 100, dtype=torch.int32, device=DEV)
    args = (c, 0, 16, b_, l, wide_w[:, :n], wide_p[:, :n], bud, 4, 8, nl, nw[:, :n], npos[:, :n], mv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.mla_cache_evict(*args)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_cache_evict(*args)
    for _ in range(2):
        c.copy_(_t(cache))
        nw.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(c.cpu().numpy(), ref_c) and np.array_equal(nl.cpu().numpy(), ref_l)
        for b in range(3):
            assert np.array_equal(nw[b, :ref_l[b]].cpu().numpy(), ref_w[b])
            assert np.array_equal(npos[b, :ref_l[b]].cpu().numpy(), ref_p[b])
            assert not bool(nw[b, n:].any())


@pytest.mark.parametrize("ctas", [1, 2, 4, 8])
@pytest.mark.parametrize("most", [5000, 40000, 300000])
def test_where_no_large_cluster_fits(ctas, most):
    # a part of a GPU may hold fewer than 16 CTAs of a cluster: fewer share a request, or the
    # keys that no longer fit registers go to shared memory (and past that are formed again)
    lens, bt, cache, w, pos = _case([most, most // 3, 7], 64, 1, seed=most + ctas)
    bud = np.array([most // 2, most // 3, 3], dtype=np.int32)
    ref_c, ref_l, ref_w, ref_p, ref_m = keep_ref.evict(cache, bt, lens, w, pos, bud, 4, 100, 64)
    d = [_t(x) for x in (cache, bt, lens, w, pos, bud)]
    nl, nw, npos = torch.zeros_like(d[2]), torch.zeros_like(d[3]), torch.zeros_like(d[4])
    moves = torch.zeros((3, w.shape[1] + 2), dtype=torch.int32, device=DEV)
    m.test_limit_next_evict(ctas)
    m.mla_cache_evict(d[0], 1, 64, d[1], d[2], d[3], d[4], d[5], 4, 100, nl, nw, npos, moves)
    torch.cuda.synchronize()
    assert np.array_equal(nl.cpu().numpy(), ref_l) and np.array_equal(d[0].cpu().numpy(), ref_c)
    for b in range(3):
        n, K = len(ref_m[b]), int(ref_l[b])
        mv = moves[b].cpu().numpy()
        assert mv[0] == n and mv[1] == K and np.array_equal(mv[2:2 + 2 * n].reshape(n, 2), ref_m[b])
        assert np.array_equal(nw[b, :K].cpu().numpy(), ref_w[b]) and np.array_equal(npos[b, :K].cpu().numpy(), ref_p[b])
