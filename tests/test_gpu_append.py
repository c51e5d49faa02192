"""mla_cache_append on the GPU against its definition in 64 bits.

Tolerances, relative to a value x before its last rounding: the sum of squares
has at most 64 additions in a row and each lane, 1 / sqrt two units, two products:
under 2^-19 in all; a turned pair as in test_gpu_rope. bf16 adds 2^-8, e4m3 half
a step (2^-4, or half the smallest step of the scale)."""
import numpy as np
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
import step_ref as R
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP8, PAGE = m.MLA_CACHE_BF16_576, m.MLA_CACHE_FP8_DS_MLA_656, m.MLA_CACHE_FP8_PAGE_576
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


class Case:
    """A batch: request b holds before[b] tokens and gets new[b]."""

    def __init__(self, new, before, page, kind, D=512, seed=0, pad=0, norm=True, turn=True, inter=False, given=False, dense=True,
                 loud=1.0):
        r = np.random.default_rng(seed)
        self.new, self.before, self.page, self.kind, self.D = np.array(new), np.array(before), page, kind, D
        self.inter = inter
        lens = self.new + self.before
        need = -(-lens // page)
        ids = r.permutation(int(need.sum()) + 3)
        bt = np.full((len(lens), max(1, int(need.max())) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            bt[b, :n] = ids[at:at + n]
            at += n
        self.bt, self.pages = bt, len(ids)
        total = int(self.new.sum()) + pad
        gen = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
        self.proj = (rnd(total, D + 64) * torch.exp(rnd(total, 1)) * loud).to(torch.bfloat16)
        rb = {BF16: 2 * (D + 64), FP8: 656, PAGE: 576}[kind]
        self.cache = torch.from_numpy(r.integers(0, 256, size=(self.pages * page, rb), dtype=np.uint8)).to(DEV)
        self.scales = torch.from_numpy((2.0 ** r.integers(-12, 2, size=self.pages)).astype(np.float32)).to(DEV) if kind == PAGE else None
        self.w = (1 + 0.2 * rnd(D)).to(torch.bfloat16) if norm else None
        self.steps, self.ms = m.rope_steps(64, scaling="yarn", factor=40.0, device=DEV) if turn else (None, 1.0)
        self.cu = torch.from_numpy(np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)).to(DEV)
        self.lens = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        self.table = torch.from_numpy(bt).to(DEV)
        self.pos = torch.from_numpy(r.integers(0, 1 << 21, size=total).astype(np.int32)).to(DEV) if given else None
        self.rows = torch.full((total, D + 64), 7.0, dtype=torch.bfloat16, device=DEV) if dense else None
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def go(self, **over):
        kw = dict(steps=self.steps, positions=self.pos, interleaved=self.inter, mscale=self.ms, norm_weight=self.w, eps=EPS,
                  scales=self.scales, rows=self.rows, lat_dim=self.D, status=self.status)
        kw.update(over)
        m.mla_cache_append(self.proj[:, :self.D], self.proj[:, self.D:], self.cu, self.lens, self.table, self.page, self.cache,
                           self.kind, **kw)

    def want(self):
        """Rows in 64 bits, and how far each value may be off before its last rounding."""
        x = self.proj.double().cpu().numpy()
        lat, pe = x[:, :self.D], x[:, self.D:]
        place = np.concatenate([np.arange(b, b + n) for b, n in zip(self.before, self.new)] + [np.zeros(len(x) - self.new.sum(), int)])
        if self.w is not None:
            lat = R.norm(lat, self.w.double().cpu().numpy(), EPS)
        off = np.abs(lat) * 2.0 ** -19 if self.w is not None else np.zeros_like(lat)
        if self.steps is not None:
            pos = place if self.pos is None else self.pos.cpu().numpy()
            half = np.abs(pe[:, 0::2]) + np.abs(pe[:, 1::2]) if self.inter else np.abs(pe[:, :32]) + np.abs(pe[:, 32:])
            pair = np.repeat(half, 2, axis=1) if self.inter else np.concatenate([half, half], axis=1)
            pe = R.rope(pe[:, None], pos, self.steps.cpu().numpy(), self.inter, self.ms)[:, 0]
            off_pe = pair * 2.0 ** -20 * self.ms
        else:
            off_pe = np.zeros_like(pe)
        return np.concatenate([lat, pe], axis=1), np.concatenate([off, off_pe], axis=1), place

    def slots(self, b, place):
        return self.bt[b, place // self.page].astype(np.int64) * self.page + place % self.page


def _bf16(raw):
    return torch.from_numpy(np.ascontiguousarray(raw)).view(torch.bfloat16).double().numpy()


def _e4m3(raw):
    return torch.from_numpy(np.ascontiguousarray(raw)).view(torch.float8_e4m3fn).double().numpy()


def check(c, cache0, scales0):
    torch.cuda.synchronize()
    rows, off, place = c.want()
    got, t = c.cache.cpu().numpy(), 0
    expect = cache0.copy()      # what must not change
    scales = None if scales0 is None else scales0.copy()
    if c.rows is not None:
        n = int(c.new.sum())
        d = c.rows.double().cpu().numpy()
        assert (np.abs(d[:n] - rows[:n]) <= np.abs(rows[:n]) * 2.0 ** -8 + off[:n] * 1.01).all()
        assert (d[n:] == 7.0).all()
    for b, n in enumerate(c.new):
        if n == 0:
            continue
        y, o, pl = rows[t:t + n], off[t:t + n] * 1.01, place[t:t + n]
        at = c.slots(b, pl)
        if c.kind == BF16:
            assert (np.abs(_bf16(got[at]) - y) <= np.abs(y) * 2.0 ** -8 + o).all()
        elif c.kind == FP8:
            sc = np.ascontiguousarray(got[at][:, 512:528]).view(np.float32).astype(np.float64)
            top = np.abs(y[:, :512]).reshape(n, 4, 128).max(2)
            want = np.where(top > 0, top / 448, 1.0)  # (a block of zeros has scale 1)
            assert (np.abs(sc - want) <= want * 2.0 ** -18).all()
            s = np.repeat(sc, 128, axis=1)
            v = _e4m3(got[at][:, :512]) * s
            assert (np.abs(v - y[:, :512]) <= R.e4m3_off(y[:, :512], s) * (1 + 2.0 ** -17) + o[:, :512]).all()
            assert (np.abs(_bf16(got[at][:, 528:]) - y[:, 512:]) <= np.abs(y[:, 512:]) * 2.0 ** -8 + o[:, 512:]).all()
        else:
            for pi in range(pl[0] // c.page, pl[-1] // c.page + 1):
                mine = pl // c.page == pi
                pid = c.bt[b, pi]
                first = max(pl[0] - pi * c.page, 0)
                top = np.abs(y[mine]).max()
                # (a largest value next to the border may fall on either side of it)
                fits = {R.page_scale(top * (1 + k * 2.0 ** -18)) for k in (-1, 1)}
                old = float(scales[pid])
                s = float(c.scales[pid])
                assert s in ({max(old, f) for f in fits} if first else fits), (s, fits, old, first)
                if first and s > old:
                    at0 = pid * c.page + np.arange(first)
                    was = torch.from_numpy(expect[at0]).view(torch.float8_e4m3fn).float()
                    expect[at0] = (was * (old / s)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                    nan = was.isnan().numpy()
                    assert ((got[at0] & 0x7F) == 0x7F)[nan].all()
                    expect[at0] = np.where(nan, got[at0], expect[at0])  # NaN stays NaN, of either sign
                scales[pid] = s
                v = _e4m3(got[at[mine]]) * s
                assert (np.abs(v - y[mine]) <= R.e4m3_off(y[mine], s) + o[mine]).all()
        expect[at] = got[at]
        t += n
    assert np.array_equal(got, expect)
    if scales is not None:
        assert np.array_equal(c.scales.cpu().numpy(), scales)


def run(c, **over):
    cache0 = c.cache.cpu().numpy().copy()
    scales0 = None if c.scales is None else c.scales.cpu().numpy().copy()
    c.go(**over)
    check(c, cache0, scales0)
    assert int(c.status) == 0


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 96, 200])
def test_ragged_batches(kind, page):
    run(Case([1, 0, 130, 37, 0, 1, 300], [0, 5, 3, 64, 0, 199, 400], page, kind, seed=page, pad=5, inter=page % 2 == 0))


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
@pytest.mark.parametrize("n", [1, 4])
def test_a_step_of_many_requests(kind, n):
    run(Case([n] * 150, list(range(150)), 64, kind, seed=n, given=True, dense=False))


@pytest.mark.parametrize("kind,D", [(BF16, 512), (FP8, 512), (PAGE, 512), (BF16, 256), (BF16, 768), (BF16, 1792)])
def test_long_prompts(kind, D):
    """Enough tokens for every kernel's form for prompts, odd numbers of them, one request without any."""
    run(Case([20001, 0, 3, 14999, 1], [0, 9, 100, 7, 0], 64, kind, D=D, seed=D + kind, pad=3, dense=kind != FP8))


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_long_prompts_without_norm_equal_the_separate_calls(kind):
    c = Case([30011, 77], [0, 60], 16, kind, norm=False, turn=False, seed=12)
    other = c.cache.clone()
    c.go()
    slots = np.concatenate([c.slots(b, np.arange(p, p + n)) for b, (n, p) in enumerate(zip(c.new, c.before))])
    m.mla_cache_write(c.proj[:, :512], c.proj[:, 512:], torch.from_numpy(slots).to(DEV), other, kind)
    assert torch.equal(c.cache, other)


@pytest.mark.parametrize("kind,D", [(BF16, 256), (BF16, 512), (BF16, 768), (FP8, 512)])
def test_a_very_long_call_equals_short_ones(kind, D):
    """Tokens are independent of each other in these rows: one call for 130,000 of them
    and calls for pieces give the same bits (positions that do not follow each
    other, so every angle is formed for itself). Rows behind the last token stay."""
    c = Case([90001, 0, 39000, 17], [5, 9, 0, 300], 64, kind, D=D, seed=13, pad=700, given=True)
    other, rows = c.cache.clone(), c.rows.clone()
    c.go()
    t = 0
    for b, (n, p) in enumerate(zip(c.new.tolist(), c.before.tolist())):
        for i in range(0, n, 9000):
            k = min(9000, n - i)
            cu = torch.tensor([0, k], dtype=torch.int32, device=DEV)
            lens = torch.tensor([p + i + k], dtype=torch.int32, device=DEV)
            at = slice(t + i, t + i + k)
            m.mla_cache_append(c.proj[at, :D], c.proj[at, D:], cu, lens, c.table[b:b + 1], 64, other, kind, steps=c.steps,
                               positions=c.pos[at], mscale=c.ms, norm_weight=c.w, eps=EPS, rows=rows[at], lat_dim=D,
                               status=c.status)
        t += n
    assert torch.equal(c.cache, other) and torch.equal(c.rows, rows) and int(c.status) == 0
    assert bool((rows[t:] == 7.0).all())


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_a_very_long_call_with_pages_outside_the_pool(kind):
    """The tokens of a bad page are left out and reported, the others are written."""
    c = Case([40000], [0], 64, kind, seed=17, given=True)
    good = Case([40000], [0], 64, kind, seed=17, given=True)
    good.go()
    cache0 = c.cache.clone()
    bad = [3, 77, 400, 624]
    for i, pi in enumerate(bad):
        c.table[0, pi] = [-1, c.pages, 1 << 30, -(1 << 31)][i]
    c.go()
    assert int(c.status) == 2 and int(good.status) == 0
    hit = torch.zeros(c.pages, dtype=torch.bool, device=DEV)
    hit[torch.from_numpy(c.bt[0, bad].astype(np.int64)).to(DEV)] = True
    slots = hit.repeat_interleave(64)
    assert torch.equal(c.cache[slots], cache0[slots]) and torch.equal(c.cache[~slots], good.cache[~slots])
    assert torch.equal(c.rows, good.rows)


@pytest.mark.parametrize("D", [256, 768, 1792])
def test_other_latent_widths(D):
    run(Case([5, 70, 1], [0, 9, 100], 16, BF16, D=D, seed=D))


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
@pytest.mark.parametrize("norm,turn", [(False, False), (True, False), (False, True)])
def test_without_norm_or_rotation(kind, norm, turn):
    run(Case([20, 3], [7, 0], 16, kind, seed=3, norm=norm, turn=turn))


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_equals_the_separate_calls(kind):
    """Without a norm and rotation the rows are mla_cache_write's bit for bit; with
    a rotation, bf16 rows are mla_rope's and then mla_cache_write's."""
    for turn in (False, True) if kind == BF16 else (False,):
        c = Case([33, 0, 90], [0, 4, 60], 16, kind, norm=False, turn=turn, seed=11, inter=True)
        other = c.cache.clone()
        c.go()
        slots = np.concatenate([c.slots(b, np.arange(p, p + n)) for b, (n, p) in enumerate(zip(c.new, c.before)) if n])
        pe = c.proj[:, 512:].clone()
        if turn:
            pos = torch.from_numpy(c.want()[2].astype(np.int32)).to(DEV)
            m.mla_rope(pe[:, None], pos, c.steps, pe[:, None], interleaved=True, mscale=c.ms)
        m.mla_cache_write(c.proj[:, :512], pe, torch.from_numpy(slots).to(DEV), other, kind)
        assert torch.equal(c.cache, other)


@pytest.mark.parametrize("page", [5, 16, 64, 150])
def test_a_page_filled_step_by_step(page):
    """Scales that grow again and again: after every step each earlier code is the
    one before times a power of two, rounded."""
    c = Case([1], [0], page, PAGE, seed=2, dense=False, norm=False)
    r = np.random.default_rng(5)
    for i in range(2 * page + 3):
        c.new, c.before = np.array([1]), np.array([i])
        need = i // page + 1
        if need > c.bt.shape[1] or c.bt[0, need - 1] < 0:
            break
        c.lens.fill_(i + 1)
        c.proj = (torch.randn((1, 576), device=DEV) * float(2.0 ** r.integers(-6, 12))).to(torch.bfloat16)
        run(c)


def test_steps_and_a_prompt_at_once_agree_up_to_the_rounding():
    """The same tokens one by one: the same scales, and codes off by one more rounding."""
    one, many = Case([100], [0], 64, PAGE, seed=9), Case([100], [0], 64, PAGE, seed=9)
    one.go()
    rows = many.proj.clone()
    for i in range(100):
        many.proj = rows[i:i + 1]
        many.rows = None
        many.cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        many.lens.fill_(i + 1)
        many.go()
    ids = one.bt[0, :2]
    assert torch.equal(one.scales[ids], many.scales[ids])
    at = one.slots(0, np.arange(100))
    s = np.repeat(one.scales.cpu().numpy()[ids], 64)[:100, None]
    a, b = (_e4m3(x.cache.cpu().numpy()[at]) * s for x in (one, many))
    # the code before is within half a step of its own, smaller or equal scale, so within half a step here as well
    assert (np.abs(a - b) <= 2.0 ** -3 * np.abs(a) + 2.0 ** -9 * s).all()


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
def test_dense_rows_over_the_projection_itself(kind):
    c = Case([50, 3, 200], [10, 0, 100], 64, kind, seed=4)
    d = Case([50, 3, 200], [10, 0, 100], 64, kind, seed=4)
    c.go()
    d.go(rows=d.proj)
    assert torch.equal(c.cache, d.cache) and torch.equal(c.rows, d.proj)
    if kind == PAGE:
        assert torch.equal(c.scales, d.scales)


def test_values_that_are_not_finite():
    """They stay what they are (an infinity saturates in 8 bits), and do not enter the page's scale."""
    c = Case([70], [0], 64, PAGE, norm=False, turn=False, seed=6)
    c.proj[3, 5], c.proj[4, 6], c.proj[66, 515], c.proj[5, 530] = float("nan"), float("inf"), float("-inf"), float("nan")
    c.go()
    x = c.proj.double().cpu().numpy()
    fin = np.where(np.isfinite(x), np.abs(x), 0)
    at = c.slots(0, np.arange(70))
    got = _e4m3(c.cache.cpu().numpy()[at])
    for pi, sel in ((0, slice(0, 64)), (1, slice(64, 70))):
        assert float(c.scales[c.bt[0, pi]]) == R.page_scale(fin[sel].max())
    assert np.array_equal(np.isnan(got), np.isnan(x))
    assert got[4, 6] == 448 and got[66, 515] == -448


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
def test_zeros_and_extremes(kind):
    """Rows of zeros, the smallest and the largest values of a trained layer."""
    for loud in (0.0, 2.0 ** -110, 2.0 ** -75, 2.0 ** -30, 2.0 ** 30):
        run(Case([40, 1], [0, 3], 16, kind, norm=False, turn=False, seed=8, loud=loud))
    run(Case([40, 1], [0, 3], 16, kind, norm=True, seed=8, loud=0.0))


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
def test_tokens_without_a_place(kind):
    """A request shorter than its new tokens, a page outside the pool, a table that
    is too short: those tokens are not cached, the status says so, nothing else changes."""
    for what in ("short", "outside", "negative", "columns"):
        c = Case([30, 12], [0, 5], 8, kind, seed=12)
        cache0, scales0 = c.cache.clone(), None if c.scales is None else c.scales.clone()
        rows, _, place = c.want()
        table = c.table
        lost = np.zeros(42, dtype=bool)
        if what == "short":
            c.lens[0] = 20          # places -10 .. 19
            lost[:10] = True
            place[:30] -= 10
        elif what == "columns":
            table = c.table[:, :2]  # places below 16
            lost = place >= 16
        else:
            c.table[0, 1] = c.pages if what == "outside" else -1
            lost[:30] = place[:30] // 8 == 1
        keep = c.table
        c.table = table
        c.go(positions=torch.from_numpy(place.astype(np.int32)).to(DEV))
        c.table = keep
        assert int(c.status) == 2
        b = np.repeat([0, 1], [30, 12])
        ok = ~lost
        slots = np.array([c.bt[b[i], place[i] // 8].astype(np.int64) * 8 + place[i] % 8 for i in range(42) if ok[i]])
        mask = np.ones(c.cache.shape[0], dtype=bool)
        mask[slots] = False
        if kind == PAGE:  # request 1's rows before, which may be rescaled
            mask[c.bt[1, 0] * 8 + np.arange(5)] = False
        assert torch.equal(c.cache[torch.from_numpy(mask).to(DEV)], cache0[torch.from_numpy(mask).to(DEV)])
        d = c.rows.double().cpu().numpy()  # the dense rows are there for every token
        if what != "short":
            rows2 = rows
            assert (np.abs(d - rows2) <= np.abs(rows2) * 2.0 ** -8 + c.want()[1] * 1.01).all()
        s = c.cache.cpu().numpy()[slots]
        if kind == BF16:
            assert np.array_equal(_bf16(s), d[ok])
        if kind == PAGE:
            touched = np.unique(slots // 8)
            other = np.setdiff1d(np.arange(c.pages), touched)
            assert np.array_equal(c.scales.cpu().numpy()[other], scales0.cpu().numpy()[other])


@pytest.mark.parametrize("n,length", [(1, 0), (1, -3), (20, 0), (20, -1), (70, 0)])
@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
def test_requests_without_any_place_leave_the_pages_their_table_names(kind, n, length):
    """A padding request of a batch of fixed size: new tokens, no length, and a table row that
    names pages of other requests. Page and scale of those stay, and what a live request
    appends to them in the same call is there, whichever comes first."""
    for live in (False, True):
        c = Case([n, 3, n], [0, 5, 0], 16, kind, seed=21)
        if not live:
            c.cu = torch.tensor([0, n, n, 2 * n], dtype=torch.int32, device=DEV)
        c.table[0] = c.table[1]
        c.table[2] = c.table[1]
        c.lens[0] = c.lens[2] = length
        cache0, scales0 = c.cache.clone(), None if c.scales is None else c.scales.clone()
        c.go()
        torch.cuda.synchronize()
        assert int(c.status) == 2
        cache1, scales1 = cache0.clone(), None if scales0 is None else scales0.clone()
        if live:  # the same tokens alone
            d = Case([n, 3, n], [0, 5, 0], 16, kind, seed=21)
            d.cache, d.scales = cache1, scales1
            d.cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
            d.proj, d.rows = c.proj[n:n + 3], None
            d.lens, d.table = c.lens[1:2].clone(), c.table[1:2].clone()
            d.go()
            torch.cuda.synchronize()
            assert int(d.status) == 0
        assert torch.equal(c.cache, cache1)
        if kind == PAGE:
            assert torch.equal(c.scales, scales1)
        # the dense rows are there all the same
        assert not bool((c.rows[:n] == 7.0).all(1).any())


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
def test_thousands_of_requests(kind):
    """More of them than one round of probes looks at, most without a token."""
    r = np.random.default_rng(7)
    new = r.choice([0, 0, 0, 1, 2, 17], size=2500)
    run(Case(list(new), list(r.integers(0, 40, size=2500)), 16, kind, seed=7, dense=False))


@pytest.mark.parametrize("norm", [True, False])
def test_small_and_large_blocks_of_one_row(norm):
    """656-byte rows whose blocks lie hundreds of powers of two apart, zeros of both signs among them."""
    c = Case([40], [0], 16, FP8, norm=norm, turn=False, seed=13)
    x = torch.randn((40, 4, 128), device=DEV) * torch.tensor([2.0 ** -118, 2.0 ** -84, 1.0, 2.0 ** 50], device=DEV)[:, None]
    if norm:
        x = x[:, [0, 1, 1, 1]]
    x[3, 1, 7], x[4, 2, 9] = -0.0, 0.0
    c.proj[:, :512] = x.reshape(40, 512).to(torch.bfloat16)
    if norm:
        run(c)
        return
    other = c.cache.clone()
    c.go()
    m.mla_cache_write(c.proj[:, :512], c.proj[:, 512:], torch.from_numpy(c.slots(0, np.arange(40))).to(DEV), other, FP8)
    assert torch.equal(c.cache, other)


def test_padded_batches_and_empty_calls():
    """Prefix sums that end early leave the other rows out; no tokens, no requests: nothing happens."""
    c = Case([4, 4], [0, 10], 16, PAGE, seed=1, pad=120)
    run(c)
    before = c.cache.clone()
    c.cu.zero_()
    c.rows.fill_(7.0)
    c.go()
    assert torch.equal(c.cache, before) and bool((c.rows == 7.0).all())
    c.proj, c.rows = c.proj[:0], None
    c.pos = None
    c.go()
    assert torch.equal(c.cache, before)


@pytest.mark.parametrize("kind", [BF16, FP8, PAGE])
def test_replayed_graph_and_another_stream(kind):
    new, before = [1] * 20, list(range(0, 200, 10))
    a, b = Case(new, before, 16, kind, seed=3), Case(new, before, 16, kind, seed=3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.go()
    s = torch.cuda.Stream()
    for step in range(4):
        x = torch.randn_like(a.proj.float()).to(torch.bfloat16)
        for c in (a, b):
            c.proj.copy_(x)
            c.lens += 1 if step else 0
        # (the 20th request's table ends where its pages do: a step more stays inside it)
        g.replay()
        s.wait_stream(torch.cuda.current_stream())
        b.go(stream=s)
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(a.cache, b.cache) and torch.equal(a.rows, b.rows)
    if kind == PAGE:
        assert torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("kind", [FP8, PAGE])
def test_offsets_past_32_bits(kind):
    """A pool of more than 2^31 bytes: pages at its end."""
    rb, page = (656, 64) if kind == FP8 else (576, 64)
    pages = (1 << 32) // (rb * page) + 10
    c = Case([70, 3], [10, 64], page, kind, seed=5)
    old = {int(p): c.cache[int(p) * page:(int(p) + 1) * page].clone() for p in np.unique(c.bt) if p >= 0}
    shift = pages - c.pages
    big = torch.empty((pages * page, rb), dtype=torch.uint8, device=DEV)
    for p, v in old.items():
        big[(p + shift) * page:(p + shift + 1) * page] = v
    d = Case([70, 3], [10, 64], page, kind, seed=5)
    d.table = torch.where(d.table >= 0, d.table + shift, d.table)
    d.cache = big
    if kind == PAGE:
        d.scales = torch.cat([torch.ones(shift, device=DEV), c.scales])
    c.go()
    d.go()
    for p in old:
        assert torch.equal(big[(p + shift) * page:(p + shift + 1) * page], c.cache[p * page:(p + 1) * page])
    if kind == PAGE:
        assert torch.equal(d.scales[shift:], c.scales)
