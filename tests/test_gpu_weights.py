"""mla_attn_weights on the GPU against the 64-bit form of its definition.

Tolerance. A score is a sum of exact products in fp32: the tensor core adds
16 or 32 products at a time to the running sum, each addition off by at most
one unit of 2^-23 of the magnitudes summed so far, so with n additions the
score is off by at most n 2^-23 M (M the largest sum of |products| times the
scale; n = (D + 64) / 16, and twice (D / 32) + 4 for fp8 rows, whose query is
in two parts and whose 4 block sums are joined by 5 more). The exponent
s - L is rounded once to fp32 (|s| + |L| <= 2 M + |L|, 2^-24 of it), the log2
scaling of s and L once each, and exp2 is off by 2^-22. So a term is off by a
factor 1 + eps, eps = (n + 4) 2^-23 (2 M + |L|) + 2^-22, and a sum of positive
terms by the same factor plus one rounding (2^-24) per term added. fp8 rows:
query elements under 2^-14 of their row's largest may be off by 2^-21 of it."""
import numpy as np
import pytest
import torch

import keep_ref
import mla_latent_kv_cache_gb300 as m
from mla_latent_kv_cache_gb300 import build as mbuild
from mla_latent_kv_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


def _workload(kind, Hq, Qt, page, lens, seed=0, lat_dim=512, **kw):
    wl = W.make("weights", B=len(lens), Hq=Hq, Qt=Qt, page_size=page, seq_lens=lens, kind=kind, seed=seed, device=DEV,
                write_all=kind == 1, lat_dim=lat_dim, **kw)
    if kind == 1:
        m.mla_cache_write(wl.w_latent, wl.w_k_pe, wl.w_slots, wl.pool, kind)
    torch.cuda.synchronize()
    return wl


def _eps(mag, L, D, kind, rows):
    n = (D + 64) / 16 if kind == 0 else 2 * (D / 32) + 4 + 5
    big = np.abs(L[np.isfinite(L)]).max(initial=0.0)
    return (n + 4) * 2.0 ** -23 * (2 * mag + big) + 2.0 ** -22 + rows * 2.0 ** -24 + (2.0 ** -21 * mag if kind else 0)


def _run(wl, lse, old, decay, **kw):
    w = old.clone()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mla_attn_weights(wl.q_lat, wl.q_pe, lse, wl.pool, wl.kind, wl.page_size, wl.block_table, wl.seq_lens, wl.Qt,
                       wl.scale, w, decay=decay, lat_dim=wl.lat_dim, status=st, **kw)
    torch.cuda.synchronize()
    return w, int(st)


def _lse(wl, sc):
    L = keep_ref.lse_of(sc)
    return L, torch.from_numpy(L.astype(np.float32)).to(DEV).reshape(wl.B * wl.Qt, wl.Hq)


def _check(wl, decay=0.875, extra=9, **kw):
    sc, mag = keep_ref.scores(wl, wl.pool, wl.lat_dim)
    rows = wl.Hq * wl.Qt
    L, lse = _lse(wl, sc)
    most = int(wl.seq_lens.max()) + extra
    g = torch.Generator().manual_seed(3)
    old = torch.rand((wl.B, most), generator=g)
    got, st = _run(wl, lse, old.to(DEV), decay, **kw)
    assert st == 0
    want = keep_ref.attn_weights(sc, lse.reshape(-1).double().cpu().numpy(), rows, old.double().numpy(), decay)
    got = got.cpu().double().numpy()
    eps = _eps(mag, L, wl.lat_dim, wl.kind, rows)
    assert eps < 5e-3  # the bound must still tell a rounded score from an exact one
    assert np.all(np.abs(got - want) <= eps * np.abs(want) + 2.0 ** -126), np.abs(got - want).max()
    for b in range(wl.B):  # past a request's tokens nothing is written
        T = int(wl.seq_lens[b])
        assert np.array_equal(got[b, T:], old.double().numpy()[b, T:])
    return got


LENS = [37, 0, 200, 1, 127, 128, 129, 640]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("Hq,Qt", [(8, 1), (16, 1), (1, 1), (20, 2), (32, 1), (16, 4), (16, 8), (40, 5)])
def test_rows(kind, Hq, Qt):
    _check(_workload(kind, Hq, Qt, 16, LENS, seed=Hq + Qt))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("page", [1, 3, 5, 7, 8, 16, 24, 64, 96, 128, 784])
def test_page_sizes(kind, page):
    _check(_workload(kind, 16, 2, page, LENS, seed=page))


@pytest.mark.parametrize("kind,page,Hq,Qt", [(0, 7, 128, 1), (0, 3, 100, 3), (1, 5, 96, 1), (1, 1, 64, 4)])
def test_odd_pages_with_a_short_ring(kind, page, Hq, Qt):
    # many query rows leave four blocks to the four warps that read odd pages
    _check(_workload(kind, Hq, Qt, page, LENS + [1100], seed=page))


def test_odd_pages_of_a_wide_row():
    _check(_workload(0, 40, 1, 7, LENS, seed=3, lat_dim=1792))


@pytest.mark.parametrize("lat_dim,Hq", [(256, 16), (256, 40), (768, 16), (768, 100), (1792, 8), (1792, 40)])
def test_other_latent_widths(lat_dim, Hq):
    _check(_workload(0, Hq, 1, 16, LENS, seed=lat_dim, lat_dim=lat_dim))


@pytest.mark.parametrize("kind", [0, 1])
def test_many_rows_take_several_groups(kind):
    # 1,000 rows: groups over chunks of tiles, a request of many chunks
    _check(_workload(kind, 125, 8, 64, [1500, 9, 300], seed=5))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("ctas", [1, 2, 7, 400])
def test_result_does_not_depend_on_the_grid(kind, ctas):
    wl = _workload(kind, 16, 2, 16, LENS + [1000], seed=11)
    assert np.array_equal(_check(wl, num_ctas=ctas), _check(wl))


@pytest.mark.parametrize("decay", [0.0, 1.0])
def test_decay(decay):
    wl = _workload(0, 16, 1, 16, LENS, seed=2)
    _check(wl, decay=decay)
    if decay == 0:  # the old values are not read: NaN does not spread
        sc, _ = keep_ref.scores(wl, wl.pool)
        w, _ = _run(wl, _lse(wl, sc)[1], torch.full((wl.B, 640), float("nan"), device=DEV), 0.0)
        for b in range(wl.B):
            T = int(wl.seq_lens[b])
            assert bool(torch.isfinite(w[b, :T]).all()) and bool(torch.isnan(w[b, T:]).all())


def test_many_short_requests():
    _check(_workload(0, 16, 1, 16, list(range(0, 300, 2)), seed=4))
    _check(_workload(1, 32, 2, 64, list(range(0, 300, 2)), seed=4))


def test_row_stride_and_a_buffer_shorter_than_the_requests():
    wl = _workload(0, 16, 1, 16, [300, 70], seed=6)
    sc, _ = keep_ref.scores(wl, wl.pool)
    lse = _lse(wl, sc)[1]
    full, _ = _run(wl, lse, torch.zeros((2, 300), device=DEV), 1.0)
    wide = torch.zeros((2, 999), device=DEV)
    m.mla_attn_weights(wl.q_lat, wl.q_pe, lse, wl.pool, 0, 16, wl.block_table, wl.seq_lens, 1, wl.scale, wide[:, :250],
                       decay=1.0)
    assert torch.equal(wide[:, :250], full[:, :250]) and not bool(wide[:, 250:].any())


def test_bad_pages_read_page_0_and_flag():
    for kind in (0, 1):
        wl = _workload(kind, 16, 1, 16, [300, 100, 50], seed=8, force_block=0)
        wl.block_table[0, 3] = 10 ** 6
        wl.block_table[1, 0] = -5
        sc, mag = keep_ref.scores(wl, wl.pool)
        L, lse = _lse(wl, sc)
        got, st = _run(wl, lse, torch.zeros((3, 300), device=DEV), 1.0)
        assert st == m.STATUS_BAD_BLOCK
        want = keep_ref.attn_weights(sc, lse.reshape(-1).double().cpu().numpy(), 16, np.zeros((3, 300)), 1.0)
        assert np.all(np.abs(got.cpu().numpy() - want) <= _eps(mag, L, 512, kind, 16) * np.abs(want) + 1e-30)


def test_rows_without_visible_tokens_and_extreme_lse():
    wl = _workload(0, 8, 4, 16, [2, 100], seed=9)  # the first two queries of request 0 see nothing
    got = _check(wl)
    assert np.all(np.isfinite(got))
    lse = torch.full((8, 8), float("-inf"), device=DEV)
    w, _ = _run(wl, lse, torch.ones((2, 100), device=DEV), 1.0)
    assert bool((w == 1).all())
    w, _ = _run(wl, torch.full((8, 8), float("inf"), device=DEV), torch.ones((2, 100), device=DEV), 1.0)
    assert bool((w == 1).all())


@pytest.mark.parametrize("kind", [0, 1])
def test_nan_in_one_token_stays_in_it(kind):
    wl = _workload(kind, 20, 1, 16, [200], seed=10)
    sc, mag = keep_ref.scores(wl, wl.pool)
    lse = _lse(wl, sc)[1]
    clean, _ = _run(wl, lse, torch.zeros((1, 200), device=DEV), 0.0)
    slot = int(wl.block_table[0, 4]) * 16 + 6  # token 70
    wl.pool[slot] = 0xFF  # NaN in every field of either kind
    got, st = _run(wl, lse, torch.zeros((1, 200), device=DEV), 0.0)
    assert st == 0 and bool(torch.isnan(got[0, 70]))
    keep = torch.arange(200, device=DEV) != 70
    assert torch.equal(got[0, keep], clean[0, keep])


@pytest.mark.parametrize("kind", [0, 1])
def test_rows_that_add_nothing_add_nothing_to_a_nan_token(kind):
    wl = _workload(kind, 20, 2, 16, [200], seed=10)
    lse = _lse(wl, keep_ref.scores(wl, wl.pool)[0])[1]
    wl.pool[int(wl.block_table[0, 4]) * 16 + 6] = 0xFF  # token 70, NaN in every field of either kind
    none = torch.full_like(lse, float("-inf"))
    w, _ = _run(wl, none, torch.ones((1, 200), device=DEV), 1.0)
    assert bool((w == 1).all())
    some = none.clone()
    some.view(-1)[7] = lse.view(-1)[7]
    w, _ = _run(wl, some, torch.ones((1, 200), device=DEV), 1.0)
    assert torch.isnan(w[0]).nonzero().view(-1).tolist() == [70]


def test_fp8_queries_of_any_magnitude():
    # rows whose values span many powers of two, tiny rows, a zero row
    wl = _workload(1, 16, 1, 16, [200], seed=12)
    f = torch.exp2(torch.arange(16, device=DEV).float() * 2 - 30).to(torch.bfloat16)
    f[3] = 0
    wl.q_lat *= f[None, :, None]
    wl.q_lat[0, 5, ::7] *= 2.0 ** -9
    _check(wl)


def test_after_decode_the_weights_of_a_step_sum_to_one_per_row():
    wl = _workload(0, 16, 2, 16, [37, 500, 1200], seed=13)
    m.mla_cache_write(wl.w_latent, wl.w_k_pe, wl.w_slots, wl.pool, 0)
    out, lse, ws = m.decode(wl.q_lat, wl.q_pe, wl.pool, 0, 16, wl.block_table, wl.seq_lens, 2, wl.scale)
    w, st = _run(wl, lse, torch.zeros((3, 1200), device=DEV), 0.0)
    assert st == 0 and m.device_status(ws) == 0
    # the decode's lse is held to 1e-3, so each row's terms sum to 1 within that
    assert float((w.sum(1) - 32).abs().max()) <= 32 * 1.1e-3


def test_graph_replay_and_side_stream():
    wl = _workload(0, 16, 1, 16, LENS, seed=14)
    sc, _ = keep_ref.scores(wl, wl.pool)
    lse = _lse(wl, sc)[1]
    want, _ = _run(wl, lse, torch.ones((8, 640), device=DEV), 0.5)
    w = torch.ones((8, 640), device=DEV)
    args = (wl.q_lat, wl.q_pe, lse, wl.pool, 0, 16, wl.block_table, wl.seq_lens, 1, wl.scale, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.mla_attn_weights(*args, decay=0.5)
    side.synchronize()
    assert torch.equal(w, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_attn_weights(*args, decay=0.5)
    for _ in range(2):
        w.fill_(1.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, want)


# fp8 rows multiply a query in two parts, e4m3 and e5m2, of its values times the power of
# two that brings the row's largest, mx, into [128, 256). A scaled value x >= 2^-6 is held
# exactly: in e4m3's normal range the rest is at most 8 units of the value's last place,
# 3 bits, and those are e5m2's. Below 2^-6 (2^-13 of 128) e4m3's step stays at 2^-9, so the
# rest is up to 2^-10 and may have more bits than e5m2 holds: it is off by at most half a
# step of e5m2 in [2^-11, 2^-10], 2^-14 = 2^-21 of 128. So a score is off by at most
# scale 2^-21 mx sum |k_d| over the values under 2^-13 mx (all of them at worst).

def _wide_rows(seed):
    """Rows of one large value (in each of the four blocks in turn) and small ones from 2^-10 to 2^-20 of it."""
    wl = _workload(1, 16, 1, 16, [200, 37], seed=seed)
    g = torch.Generator().manual_seed(seed)
    shape = tuple(wl.q_lat.shape)
    x = torch.exp2(-10 - 10 * torch.rand(shape, generator=g)) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    for r in range(shape[0]):
        for h in range(shape[1]):
            x[r, h, (h * 32 + 7 * r) % 512] = 1 + float(torch.rand((), generator=g))
    x *= torch.exp2(torch.arange(16).float() % 5 - 2)[None, :, None]
    wl.q_lat.copy_(x.to(torch.bfloat16))
    return wl


def _split(q):
    """The two parts of a row's values added up (bf16 rows, CPU), in fp64."""
    x = q.double()
    e = torch.floor(torch.log2(x.abs().amax(-1, keepdim=True)))
    up = torch.exp2(7 - e)
    s = (x * up).float()
    h = s.to(torch.float8_e4m3fn).float()
    lo = (s - h).to(torch.float8_e5m2).float()
    return (h.double() + lo.double()) / up


@pytest.mark.parametrize("seed", [21, 22])
def test_fp8_queries_whose_values_span_many_powers_of_two(seed):
    wl = _wide_rows(seed)
    q = wl.q_lat.cpu()
    held, mx = _split(q), q.double().abs().amax(-1, keepdim=True)
    off = (held - q.double()).abs()
    assert bool((off <= 2.0 ** -21 * mx).all()) and bool((off[q.double().abs() >= 2.0 ** -13 * mx] == 0).all())
    assert bool((off > 0).any())  # the rounded range is exercised

    # against the definition: the bound above
    sc, mag = keep_ref.scores(wl, wl.pool)
    L, lse = _lse(wl, sc)
    got, st = _run(wl, lse, torch.zeros((2, 200), device=DEV), 0.0)
    assert st == 0
    got = got.cpu().double().numpy()
    lse64 = lse.reshape(-1).double().cpu().numpy()
    want = keep_ref.attn_weights(sc, lse64, 16, np.zeros((2, 200)), 0.0)
    ksum = np.abs(keep_ref.rows_f64(wl.pool, 1)[:, :512]).sum(axis=1)
    ksum = ksum[np.isfinite(ksum)].max()
    n = 2 * (512 // 32) + 4 + 5
    eps = (n + 4) * 2.0 ** -23 * (2 * mag + np.abs(L).max()) + 2.0 ** -22 + 16 * 2.0 ** -24
    split = wl.scale * 2.0 ** -21 * float(mx.max()) * ksum
    assert eps + split < 5e-3
    assert np.all(np.abs(got - want) <= (eps + split) * want + 2.0 ** -126)

    # and against the two parts as they are held, without any allowance for the rounding
    wl.q_lat = held.to(DEV)
    sc, _ = keep_ref.scores(wl, wl.pool)
    want = keep_ref.attn_weights(sc, lse64, 16, np.zeros((2, 200)), 0.0)
    assert np.all(np.abs(got - want) <= eps * want + 2.0 ** -126)
