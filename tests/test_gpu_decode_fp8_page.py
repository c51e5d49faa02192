"""mla_decode_fp8_page on the GPU against its definition in 64 bits.

Tolerances, per query row. Scores: a query value is off by at most 2^-22 of its
row's largest, and a sum of 576 exact products in fp32 by 2^-19 of the sum of
their magnitudes (18 steps of truncating additions); ds is the largest of these over the
row's tokens. lse is off by ds and 2^-20 of itself. Output: a weight times its page's
scale is rounded by 2^-8 of itself or 2^-16 of the largest, its exponential follows
ds, and the sum of fp32 additions adds 2^-18; then half a step of the type."""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
import step_ref as R
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


class Batch:
    def __init__(self, lens, Hq, q_len=1, page=16, seed=0, q_lens=None, loud=1.0, spread=True, peaked=False, f32=True, extra=2):
        r = np.random.default_rng(seed)
        self.lens, self.Hq, self.q_len, self.page = np.array(lens), Hq, q_len, page
        B = len(lens)
        need = -(-self.lens // page)
        ids = r.permutation(int(need.sum()) + extra)
        self.bt = np.full((B, max(1, int(need.max()))), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = ids[at:at + n]
            at += n
        pages = len(ids)
        # every code but NaN; free slots all NaN
        x = r.standard_normal((pages * page, 576)).astype(np.float32) * 60
        self.codes = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
        used = np.zeros(pages * page, dtype=bool)
        for b, n in enumerate(self.lens):
            used[self.slots(b, np.arange(n))] = True
        self.codes[~used] = 0x7F
        base = 2.0 ** -6
        self.scales = (base * loud * 2.0 ** (r.integers(-3, 3, size=pages) if spread else np.zeros(pages))).astype(np.float32)
        self.q_lens = np.full(B, q_len) if q_lens is None else np.array(q_lens)
        self.cu = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        tokens = int(self.cu[-1])
        q = r.standard_normal((tokens, Hq, 576)) * np.exp(r.standard_normal((tokens, Hq, 1)) * 0.5)
        if peaked:  # one token per request matches the queries
            for b, n in enumerate(self.lens):
                if n:
                    v = self.value(b, int(r.integers(n)))
                    q[self.cu[b]:self.cu[b + 1]] += 3 * v / max(1e-9, np.sqrt((v * v).mean()))
        self.q = torch.from_numpy(q).to(torch.bfloat16)
        self.varlen = q_lens is not None
        self.odt = torch.float32 if f32 else torch.bfloat16
        self.dev = {}

    def slots(self, b, j):
        return self.bt[b, j // self.page].astype(np.int64) * self.page + j % self.page

    def value(self, b, j):
        s = self.slots(b, np.array([j]))
        return self.code_values(s)[0] * float(self.scales[s[0] // self.page])

    def code_values(self, slots):
        return torch.from_numpy(self.codes[slots]).view(torch.float8_e4m3fn).double().numpy()

    def upload(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        tokens = self.q.shape[0]
        self.dev = dict(q_lat=self.q[..., :512].contiguous().to(DEV), q_pe=self.q[..., 512:].contiguous().to(DEV),
                        cache=t(self.codes), scales=t(self.scales), table=t(self.bt), lens=t(self.lens.astype(np.int32)),
                        cu=t(self.cu), out=torch.full((tokens, self.Hq, 512), 7.0, dtype=self.odt, device=DEV),
                        lse=torch.full((tokens, self.Hq), 7.0, device=DEV))
        return self.dev

    def go(self, num_ctas=0, ws=None, **over):
        d = self.dev or self.upload()
        if ws is None:
            ws = torch.empty(m.mla_decode_workspace_bytes(len(self.lens), self.q_len, self.Hq, num_ctas), dtype=torch.uint8, device=DEV)
        kw = dict(cu_q_lens=d["cu"] if self.varlen else None, num_ctas=num_ctas)
        kw.update(over)
        m.mla_decode_fp8_page(d["q_lat"], d["q_pe"], d["cache"], d["scales"], self.page, d["table"], d["lens"], self.q_len, SCALE,
                              d["out"], d["lse"], ws, **kw)
        return d["out"], d["lse"], ws

    def check(self, out, lse, requests=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        half = torch.finfo(self.odt).eps / 2
        worst = 0.0
        for b in range(len(self.lens)) if requests is None else requests:
            n, a, e = int(self.lens[b]), self.cu[b], self.cu[b + 1]
            slots = self.slots(b, np.arange(n)) if n else np.zeros(0, dtype=np.int64)
            code, s = self.code_values(slots), self.scales[slots // self.page].astype(np.float64)[:, None]
            q = self.q[a:e].double().numpy().reshape(-1, 576)
            want_o, want_l = R.decode_page(q, code * s, SCALE, e - a, self.Hq)
            got_o, got_l = out[a:e].reshape(-1, 512), lse[a:e].reshape(-1)
            for r in range(len(q)):
                see = n - (e - a) + r // self.Hq + 1
                if see <= 0:
                    assert (got_o[r] == 0).all() and got_l[r] == -np.inf
                    continue
                c, sc = code[:see], s[:see, 0]
                ds = SCALE * (sc * (2.0 ** -22 * np.abs(q[r]).max() * np.abs(c).sum(1) + 2.0 ** -19 * np.abs(c) @ np.abs(q[r]))).max()
                p = np.exp((c * s[:see]) @ q[r] * SCALE - want_l[r])
                w = p * sc
                mag = w @ np.abs(c[:, :512])
                room = mag * (2.0 ** -8 + 2 * ds + 2.0 ** -18) + 2.0 ** -16 * w.max() * np.abs(c[:, :512]).sum(0)
                off = np.abs(got_o[r] - want_o[r])
                assert (off <= room + half * np.abs(want_o[r])).all(), (b, r, (off / np.maximum(room, 1e-300)).max())
                assert abs(got_l[r] - want_l[r]) <= ds + 2.0 ** -20 * abs(want_l[r]) + 2.0 ** -20, (b, r, got_l[r], want_l[r], ds)
                worst = max(worst, (off / np.maximum(room, 1e-300)).max())
        return worst


RAGGED = [0, 1, 127, 128, 129, 300, 5, 1000]


def run(batch, num_ctas=0):
    out, lse, ws = batch.go(num_ctas)
    torch.cuda.synchronize()
    assert m.device_status(ws) == 0, m.device_status_words(ws)
    return batch.check(out, lse)


@pytest.mark.parametrize("Hq,q_len", [(1, 1), (8, 1), (16, 1)])
def test_few_rows(Hq, q_len):
    run(Batch([37, 200], Hq, q_len, 16, seed=Hq))
    run(Batch(RAGGED, Hq, q_len, 16, seed=Hq))


@pytest.mark.parametrize("Hq,q_len", [(20, 1), (32, 1), (33, 1), (64, 1), (80, 1), (128, 1), (16, 4), (8, 3), (16, 8), (48, 3)])
def test_more_rows_and_verify_steps(Hq, q_len):
    run(Batch(RAGGED, Hq, q_len, 64, seed=Hq + q_len))


@pytest.mark.parametrize("page", [8, 24, 32, 96, 128, 200, 784, 1, 3, 5, 12, 100])
@pytest.mark.parametrize("Hq,q_len", [(16, 1), (16, 2), (16, 4), (20, 4)])
def test_page_sizes(page, Hq, q_len):
    run(Batch(RAGGED, Hq, q_len, page, seed=page))


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 40, 400])
@pytest.mark.parametrize("Hq,q_len", [(16, 1), (64, 1), (16, 8)])
def test_any_number_of_ctas(num_ctas, Hq, q_len):
    run(Batch([700, 0, 3, 1500], Hq, q_len, 16, seed=1), num_ctas)
    run(Batch([2, 5], Hq, q_len, 16, seed=1), num_ctas)


@pytest.mark.parametrize("Hq,q_len", [(8, 1), (16, 2), (32, 2), (16, 8)])
@pytest.mark.parametrize("loud,peaked", [(1.0, True), (2.0 ** -10, False), (16.0, False), (2.0 ** 3, True), (2.0 ** -30, False)])
def test_peaked_flat_and_loud(Hq, q_len, loud, peaked):
    """Softmaxes from a single token to all alike, scales far apart."""
    run(Batch([400, 64, 2000], Hq, q_len, 16, seed=4, loud=loud, peaked=peaked))


@pytest.mark.parametrize("q_lens", [[1, 4, 0, 2, 4, 3], [4, 4, 4, 4, 4, 4], [0, 0, 1, 0, 0, 0]])
@pytest.mark.parametrize("Hq", [8, 16, 32])
def test_verify_lengths_of_their_own(Hq, q_lens):
    run(Batch([300, 2, 50, 1, 129, 0], Hq, 4, 16, seed=Hq, q_lens=q_lens))


def test_bf16_output():
    run(Batch(RAGGED, 16, 1, 16, seed=2, f32=False))


def test_rising_scores():
    """The maximum moves in every tile."""
    b = Batch([1500], 16, 1, 64, seed=3, spread=False)
    v = b.q[0, 0].double().numpy()
    for j in range(1500):
        s = b.slots(0, np.array([j]))
        row = torch.from_numpy(v * (j / 1500) * 30).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        b.codes[s] = row
    run(b)


def test_pages_of_extreme_scales():
    """Pages of zeros (scale 2^-40) among others, and pages far louder than others."""
    b = Batch([640, 640], 16, 1, 64, seed=5)
    for pi, e in ((0, -40), (3, -30), (5, 2), (9, -40)):
        b.scales[b.bt[0, pi]] = 2.0 ** e
    for pi in (0, 9):
        b.codes[b.bt[0, pi] * 64:(b.bt[0, pi] + 1) * 64] = 0
    b.scales[b.bt[1]] = 2.0 ** -40
    run(b)


@pytest.mark.parametrize("Hq,q_len,page", [(8, 4, 16), (16, 4, 64), (16, 8, 64), (16, 4, 3)])
def test_nan_rows_reach_only_the_queries_that_see_them(Hq, q_len, page):
    n = 300
    for j, at in ((n - 1, 5), (n - 2, 511), (n - 2, 530), (n - q_len, 0)):
        b, c = Batch([n, 40], Hq, q_len, page, seed=6), Batch([n, 40], Hq, q_len, page, seed=6)
        b.codes[b.slots(0, np.array([j])), at] = 0xFF
        out, lse, _ = b.go()
        want, want_l, _ = c.go()
        torch.cuda.synchronize()
        first = j - (n - q_len)  # the first query that sees token j
        assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_l[:first])
        assert torch.equal(out[q_len:], want[q_len:])
        assert bool(lse[first:q_len].isnan().all()) and bool(out[first:q_len].isnan().all())


def test_queries_that_are_not_finite():
    b = Batch([200, 50], 16, 1, 16, seed=7)
    b.upload()
    want = b.go()[0].clone()
    b.dev["q_lat"][0, 3, 5] = float("nan")
    b.dev["q_pe"][1, 7, 9] = float("inf")
    out = b.go()[0]
    keep = torch.ones((2, 16), dtype=torch.bool, device=DEV)
    keep[0, 3] = keep[1, 7] = False
    assert torch.equal(out[keep], want[keep]) and bool(out[~keep].isnan().all())


def test_small_queries_beside_large_ones():
    """Values 2^-15 of the row's largest still count in full."""
    b = Batch([129], 8, 1, 16, seed=8)
    q = b.q.float()
    q[..., ::2] *= 2.0 ** -12
    q[..., 0] = 40.0
    b.q = q.to(torch.bfloat16)
    run(b)


@pytest.mark.parametrize("page", [16, 3])
def test_pages_outside_the_pool_are_reported(page):
    b = Batch([200, 100], 16, 1, page, seed=9)
    b.codes[np.arange(page)] = 0  # (page 0 is read in their place)
    b.upload()
    want = b.go()[0].clone()
    b.dev["table"][0, 1] = 10 ** 6
    out, _, ws = b.go()
    assert m.device_status(ws) == 2
    if 0 not in b.bt[1]:
        assert torch.equal(out[1], want[1])
    # a request longer than its table row
    b.upload()
    b.dev["lens"][0] = b.bt.shape[1] * page + 1
    ws = b.go()[2]
    assert m.device_status(ws) == 2
    # columns of a wider table
    b.upload()
    wide = torch.full((2, b.bt.shape[1] + 9), -1, dtype=torch.int32, device=DEV)
    wide[:, 4:4 + b.bt.shape[1]] = b.dev["table"]
    b.dev["table"] = wide[:, 4:4 + b.bt.shape[1]]
    out, _, ws = b.go()
    assert m.device_status(ws) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("Hq,q_len", [(16, 1), (32, 1), (16, 4), (16, 8)])
def test_the_same_bits_every_time_and_from_a_graph(Hq, q_len):
    b = Batch([900, 0, 3000, 1, 257], Hq, q_len, 16, seed=10)
    out, lse, ws = b.go()
    first, first_l = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.go(ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(lse, first_l)


def test_two_streams_with_workspaces_of_their_own():
    a, b = Batch([5000] * 3, 16, 1, 16, seed=11), Batch([4000] * 5, 64, 1, 64, seed=12)
    wa, wb = a.go()[0].clone(), b.go()[0].clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = [torch.empty(m.mla_decode_workspace_bytes(8, 1, 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    for _ in range(10):
        a.go(ws=ws[0], stream=s1)
        b.go(ws=ws[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a.dev["out"], wa) and torch.equal(b.dev["out"], wb)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, its used pages at the end."""
    page = 64
    a = Batch([500, 130], 16, 1, page, seed=13)
    out = a.go()[0].clone()
    pages = (1 << 32) // (576 * page) + 5
    shift = pages - len(a.scales)
    big = torch.empty((pages * page, 576), dtype=torch.uint8, device=DEV)
    big[shift * page:] = a.dev["cache"]
    a.dev["scales"] = torch.cat([torch.ones(shift, device=DEV), a.dev["scales"]])
    a.dev["table"] = torch.where(a.dev["table"] >= 0, a.dev["table"] + shift, a.dev["table"])
    a.dev["cache"] = big
    assert torch.equal(a.go()[0], out)


@pytest.mark.parametrize("B", [319, 321, 700])
@pytest.mark.parametrize("Hq,q_len", [(16, 1), (64, 1)])
def test_many_requests(B, Hq, q_len):
    """More requests than a CTA has threads, and as many."""
    r = np.random.default_rng(B)
    run(Batch(list(r.choice([0, 1, 5, 130, 300], size=B)), Hq, q_len, 16, seed=B))


def test_rows_that_no_request_names_are_left_as_they_were():
    b = Batch([300, 2, 129], 16, 4, 16, seed=15, q_lens=[1, 4, 2])
    d = b.upload()
    pad = 5
    for name in ("q_lat", "q_pe", "out", "lse"):
        t = d[name]
        d[name] = torch.cat([t, torch.full((pad, *t.shape[1:]), 7.0, dtype=t.dtype, device=DEV)])
    out, lse, ws = b.go()
    torch.cuda.synchronize()
    assert m.device_status(ws) == 0
    b.check(out, lse)
    assert bool((out[-pad:] == 7.0).all()) and bool((lse[-pad:] == 7.0).all())


def test_a_workspace_that_is_too_small_is_refused():
    b = Batch([300], 16, 1, 16, seed=16)
    need = m.mla_decode_workspace_bytes(1, 1, 16)
    with pytest.raises(m.MlaError) as e:
        b.go(ws=torch.empty(need - 256, dtype=torch.uint8, device=DEV))
    assert e.value.status == m.MLA_ERR_WORKSPACE


@pytest.mark.parametrize("Hq,page", [(16, 16), (32, 16), (64, 64), (16, 3)])
def test_a_wait_that_runs_out_is_reported(Hq, page):
    """A hand-off that never comes: the call ends after about a second with status bit 1,
    and the next one is right."""
    b = Batch([3000, 700], Hq, 1, page, seed=17)
    want = b.go()[0].clone()
    m.test_hold_next_decode()
    ws = b.go()[2]
    torch.cuda.synchronize()
    assert m.device_status(ws) & 1
    out, _, ws = b.go()
    torch.cuda.synchronize()
    assert m.device_status(ws) == 0 and torch.equal(out, want)


def test_one_long_request():
    b = Batch([100003], 16, 1, 64, seed=14)
    run(b)


class Sink:
    """One token far above a long tail. Rotary codes alone make the scores (the latent part
    of the queries is 0), so a token's value may be anything: the tail's is 8 in dims 0 .. 127,
    random in the rest, the sink's is 0 in dims 0 .. 127. Head h puts the sink nats[h] above
    the tail's middle; `wide` is the tail's width in nats (0: all alike)."""

    def __init__(self, lens, at, Hq, q_len, nats, wide, seed=0, page=64):
        r = np.random.default_rng(seed)
        self.lens, self.Hq, self.q_len, self.page = lens, Hq, q_len, page
        T, rows, B = max(lens), Hq * q_len, len(lens)
        need = -(-T // page)
        self.table = np.arange(B * need, dtype=np.int32).reshape(B, need)
        x = np.zeros((B * need * page, 576), dtype=np.float32)
        x[:, 128:512] = r.standard_normal((len(x), 384)) * 60
        x[:, :128] = 8.0
        x[:, 513:517] = r.standard_normal((len(x), 4)) * 60
        for b in range(B):
            j = b * need * page + at
            x[j, :128], x[j, 512], x[j, 513:517] = 0.0, 448.0, 0.0
        self.codes = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn)
        q = np.zeros((B * q_len, Hq, 576), dtype=np.float32)
        q[..., 512] = np.resize(nats, Hq)[None] / 448.0
        q[..., 513:517] = wide / 120.0
        self.q = torch.from_numpy(q).to(torch.bfloat16)

    def bounds(self, cache, q):
        """For each row: the output in 64 bits and how far each value may be off, lse and its room."""
        fine = self.Hq * self.q_len <= 32  # the codes of small weights (include/mla.h)
        need, page = self.table.shape[1], self.page
        for b, n in enumerate(self.lens):
            code = cache[b * need * page:b * need * page + n].view(torch.float8_e4m3fn).double()
            mag = code[:, :512].abs()
            sq = mag * mag
            for r in range(self.q_len * self.Hq):
                see = n - self.q_len + r // self.Hq + 1
                c, a, a2 = code[:see], mag[:see], sq[:see]
                qr = q[b * self.q_len + r // self.Hq, r % self.Hq].double()
                z = c[:, 512:] @ qr[512:]
                top = z.max()
                e = torch.exp(z - top)
                want = (e @ c[:, :512]) / e.sum()
                # in units of the weights as they are held, the largest of them 2^kTop or more
                # (where it is more, every step below is smaller beside it)
                P = e * (64.0 if fine else 8.0)
                Pa = P @ a
                # f16, and codes above 2^-6 (2^-8 where the largest may be held as 2^8)
                big = torch.where(e * 256.0 >= 2.0 ** -6, P, 0.0)
                room = 2.0 ** -11 * Pa + 2.0 ** -8 * (big @ a)
                # below: a rounding of mean 0 within a step. Over tokens of equal weight the
                # positions that are rounded up are evenly spread (a dozen steps at most); over
                # others the roundings are independent, of deviation half a step at most.
                step = torch.full_like(P, 2.0 ** -14) if fine else torch.clamp(P * 0.25, 2.0 ** -16, 2.0 ** -13)
                step = torch.where(P < 2.0 ** -6, step, 0.0)
                room = room + 7 * 0.5 * torch.sqrt((step * step) @ a2) + 12 * 448 * step.max()
                # scores, fp32 sums of a CTA's tiles (32 tokens a step, truncated) and of its weights
                ds = 2.0 ** -22 * qr.abs().max() * c[:, 512:].abs().sum(1).max() + 2.0 ** -19 * (c[:, 512:].abs() @ qr[512:].abs()).max()
                room = room + (2 * ds + n / 32 * 2.0 ** -23 + 2.0 ** -13) * Pa
                yield want, room / P.sum(), top + torch.log(e.sum()), ds + 2.0 ** -13

    def check(self, *num_ctas):
        B, page, Hq, q_len = len(self.lens), self.page, self.Hq, self.q_len
        pages = len(self.codes) // page
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        cache, q = self.codes.view(torch.uint8).to(DEV), self.q.to(DEV)
        want, room, want_l, room_l = (torch.stack(x) for x in zip(*self.bounds(cache, q)))
        for n in num_ctas:
            out = torch.empty((B * q_len, Hq, 512), dtype=torch.float32, device=DEV)
            lse = torch.empty((B * q_len, Hq), device=DEV)
            ws = torch.empty(m.mla_decode_workspace_bytes(B, q_len, Hq, n), dtype=torch.uint8, device=DEV)
            m.mla_decode_fp8_page(q[..., :512].contiguous(), q[..., 512:].contiguous(), cache, torch.ones(pages, device=DEV), page,
                                  t(self.table), t(np.array(self.lens, dtype=np.int32)), q_len, 1.0, out, lse, ws, num_ctas=n)
            assert m.device_status(ws) == 0
            off = (out.double().reshape(-1, 512) - want).abs()
            assert bool((off <= room).all()), (n, float((off / room).max()))
            assert bool(((lse.double().reshape(-1) - want_l).abs() <= room_l).all()), n


@pytest.mark.parametrize("wide", [0.0, 1.0])
@pytest.mark.parametrize("Hq,q_len", [(16, 1), (32, 1), (16, 4), (32, 4)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_token_far_above_a_long_tail(Hq, q_len, wide, where):
    """The tail's share counts although each of its weights is 2^-9 to 2^-23 of the largest."""
    T = 65536
    at = {"first": 3, "middle": T // 2 + 77, "last": T - q_len - 2}[where]
    nats = [6.5, 8.0, 9.3, 10.0, 10.7, 11.4, 12.1, 12.5, 12.9, 13.3, 13.7, 14.1, 14.5, 15.0, 15.5, 16.0]
    Sink([T], at, Hq, q_len, nats, wide, seed=31).check(1)


@pytest.mark.parametrize("Hq,q_len", [(16, 1), (32, 1), (16, 4)])
@pytest.mark.parametrize("wide", [0.0, 1.0])
def test_a_token_above_a_tail_of_the_longest_contexts(Hq, q_len, wide):
    """262,144 tokens, whole and cut between CTAs."""
    Sink([262144, 262001], 131000, Hq, q_len, [10.0, 11.0, 12.0, 12.54, 13.0, 14.0, 15.0, 17.0], wide, seed=32).check(1, 5, 0)


@pytest.mark.parametrize("Hq,q_len", [(16, 2), (16, 4), (16, 8)])
def test_weights_of_nothing_stay_nothing(Hq, q_len):
    """Rounding small weights gives none to a token that a query does not see: its value may be anything."""
    b, c = Batch([700, 300], Hq, q_len, 16, seed=33), Batch([700, 300], Hq, q_len, 16, seed=33)
    for x in range(2):
        n = int(b.lens[x])
        b.codes[b.slots(x, np.arange(n - q_len + 1, n)), :512] = 0x7E  # 448, in tokens that query 0 does not see
    out, lse, _ = b.go()
    want, want_l, _ = c.go()
    torch.cuda.synchronize()
    for x in range(2):
        assert torch.equal(out[x * q_len], want[x * q_len]) and torch.equal(lse[x * q_len], want_l[x * q_len])


@pytest.mark.parametrize("Hq,q_len,page", [(8, 4, 16), (16, 4, 16), (16, 8, 16), (16, 4, 3)])
def test_a_page_scale_that_is_not_a_number_reaches_only_the_queries_that_see_the_page(Hq, q_len, page):
    n = 18 * 16 * 3 + 1
    b, c = Batch([n, 40], Hq, q_len, page, seed=34), Batch([n, 40], Hq, q_len, page, seed=34)
    b.scales[b.bt[0, n // page]] = np.nan  # the page of the last token alone
    out, lse, _ = b.go()
    want, want_l, _ = c.go()
    torch.cuda.synchronize()
    last = q_len - 1
    assert torch.equal(out[:last], want[:last]) and torch.equal(lse[:last], want_l[:last])
    assert torch.equal(out[q_len:], want[q_len:]) and torch.equal(lse[q_len:], want_l[q_len:])
    assert bool(lse[last].isnan().all()) and bool(out[last].isnan().all())
