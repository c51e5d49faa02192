"""Rotation, appending and attention as a serving loop uses them together: a prompt
(append with its dense rows, mla_prefill over them), then steps of one or more
tokens (mla_rope on the queries, append, decode), some of whose tokens are taken
back, with the cached rows and the attention checked in 64 bits all along."""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
import step_ref as R
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP8, PAGE = m.MLA_CACHE_BF16_576, m.MLA_CACHE_FP8_DS_MLA_656, m.MLA_CACHE_FP8_PAGE_576
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


class Server:
    """B requests with pages of their own; what a layer of a program would hold."""

    def __init__(self, B, pages_each, page, kind, Hq, q_len, seed=0):
        self.B, self.page, self.kind, self.Hq, self.q_len = B, page, kind, Hq, q_len
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16)
        self.table = torch.randperm(B * pages_each, generator=gen, device=DEV).to(torch.int32).view(B, pages_each)
        self.cache = torch.zeros((B * pages_each * page, m.mla_row_bytes(kind)), dtype=torch.uint8, device=DEV)
        self.scales = torch.ones(B * pages_each, device=DEV) if kind == PAGE else None
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.steps, self.ms = m.rope_steps(64, scaling="yarn", factor=40.0, device=DEV)
        self.w = (1 + 0.1 * self.rnd(512).float()).to(torch.bfloat16)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(m.mla_decode_workspace_bytes(B, q_len, Hq), dtype=torch.uint8, device=DEV)
        n = B * q_len
        self.q = self.rnd(n, Hq, 576 + 64)  # absorbed latent queries, then rotary ones before their rotation
        self.q_lat = torch.zeros((n, Hq, 512), dtype=torch.bfloat16, device=DEV)
        self.q_pe = torch.zeros((n, Hq, 64), dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros((n, Hq, 512), dtype=torch.float32, device=DEV)
        self.lse = torch.zeros((n, Hq), device=DEV)
        self.proj = self.rnd(n, 576)
        self.cu = torch.arange(B + 1, dtype=torch.int32, device=DEV) * q_len
        self.pos = torch.zeros(n, dtype=torch.int32, device=DEV)

    def append(self, proj, cu, rows=None):
        m.mla_cache_append(proj[:, :512], proj[:, 512:], cu, self.lens, self.table, self.page, self.cache, self.kind,
                           steps=self.steps, interleaved=True, mscale=self.ms, norm_weight=self.w, scales=self.scales, rows=rows,
                           status=self.status)

    def step(self):
        """One step's calls, on buffers that stay where they are."""
        self.lens += self.q_len
        self.append(self.proj, self.cu)
        torch.sub(self.lens.repeat_interleave(self.q_len), self.q_len, out=self.pos)
        self.pos += torch.arange(self.q_len, device=DEV, dtype=torch.int32).repeat(self.B)
        m.mla_rope(self.q[..., 576:], self.pos, self.steps, self.q_pe, interleaved=True, mscale=self.ms)
        self.q_lat.copy_(self.q[..., :512])
        if self.kind == PAGE:
            m.mla_decode_fp8_page(self.q_lat, self.q_pe, self.cache, self.scales, self.page, self.table, self.lens, self.q_len,
                                  SCALE, self.out, self.lse, self.ws)
        else:
            m.mla_decode(self.q_lat, self.q_pe, self.cache, self.kind, self.page, self.table, self.lens, self.q_len, SCALE,
                         self.out, self.lse, self.ws)

    def rows_of(self, b):
        """Request b's cached rows, as the values they stand for."""
        n = int(self.lens[b])
        j = torch.arange(n, device=DEV)
        ids = self.table[b].long()[j // self.page]
        raw = self.cache[ids * self.page + j % self.page]
        if self.kind == BF16:
            return raw.view(torch.bfloat16).double().cpu().numpy()
        if self.kind == PAGE:
            return (raw.view(torch.float8_e4m3fn).double() * self.scales[ids].double()[:, None]).cpu().numpy()
        lat = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double() * raw[:, 512:528].contiguous().view(
            torch.float32).double().repeat_interleave(128, dim=1)
        return torch.cat([lat, raw[:, 528:].contiguous().view(torch.bfloat16).double()], dim=1).cpu().numpy()

    def expected(self, proj, first):
        x = proj.double().cpu().numpy()
        lat = R.norm(x[:, :512], self.w.double().cpu().numpy(), 1e-6)
        pe = R.rope(x[:, None, 512:], np.arange(first, first + len(x)), self.steps.cpu().numpy(), True, self.ms)[:, 0]
        return np.concatenate([lat, pe], axis=1)


def _near(kind, got, want, page, first=0):
    """Rows against their 64-bit values: bf16 half a step, 8 bits half a step of the row's
    block or twice that where the page's scale grew later (the codes were rounded again)."""
    if kind == BF16:
        return (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -16).all()
    if kind == FP8:
        top = np.abs(want[:, :512]).reshape(len(want), 4, 128).max(2).repeat(128, axis=1) / 448
        lat = np.abs(got[:, :512] - want[:, :512]) <= R.e4m3_off(want[:, :512], top) * 1.001 + 2.0 ** -16
        return lat.all() and (np.abs(got[:, 512:] - want[:, 512:]) <= np.abs(want[:, 512:]) * 2.0 ** -8 + 2.0 ** -16).all()
    ok = True
    for a in range(0, len(want), page):
        rows = slice(a, a + page)
        s = R.page_scale(np.abs(want[rows]).max() * (1 + 2.0 ** -16))
        ok = ok and (np.abs(got[rows] - want[rows]) <= 2 * R.e4m3_off(want[rows], s) + 2.0 ** -16).all()
    return ok


@pytest.mark.parametrize("kind", [PAGE, FP8, BF16])
@pytest.mark.parametrize("page,Hq,q_len", [(16, 16, 1), (64, 16, 4), (24, 8, 2)])
def test_a_prompt_and_then_steps(kind, page, Hq, q_len):
    prompt = [70, 1, 133]
    s = Server(3, -(-300 // page), page, kind, Hq, q_len, seed=page + Hq)
    history = [s.rnd(n, 576) for n in prompt]
    # the prompt, in two chunks: the second behind rows that are there already
    for part in (lambda n: (0, n // 2), lambda n: (n // 2, n)):
        cut = [part(n) for n in prompt]
        proj = torch.cat([h[a:e] for h, (a, e) in zip(history, cut)])
        cu = torch.tensor(np.concatenate([[0], np.cumsum([e - a for a, e in cut])]), dtype=torch.int32, device=DEV)
        s.lens.copy_(torch.tensor([e for _, e in cut], dtype=torch.int32))
        rows = torch.zeros((len(proj), 576), dtype=torch.bfloat16, device=DEV)
        s.append(proj, cu, rows)
        want = np.concatenate([s.expected(h, 0)[a:e] for h, (a, e) in zip(history, cut)])
        assert (np.abs(rows.double().cpu().numpy() - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -16).all()
    # attention over the prompt's dense rows as mla_prefill takes them: the rotated key is a column of theirs
    n = prompt[0]
    rows = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV)
    t = Server(1, -(-n // page), page, kind, Hq, q_len, seed=1)
    t.w, t.lens = s.w, torch.tensor([n], dtype=torch.int32, device=DEV)
    t.append(history[0], torch.tensor([0, n], dtype=torch.int32, device=DEV), rows)
    q, kv = s.rnd(n, 2, 192), s.rnd(n, 2, 256)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out, lse = torch.zeros((n, 2, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((n, 2), device=DEV)
    m.mla_rope(q[..., 128:], torch.arange(n, dtype=torch.int32, device=DEV), s.steps, q[..., 128:], interleaved=True, mscale=s.ms)
    m.mla_prefill(q, kv[..., :128], rows[:, 512:], kv[..., 128:], cu, cu, n, SCALE, out, lse)
    key = torch.cat([kv[..., :128].double(), rows[:, None, 512:].double().expand(-1, 2, -1)], dim=2)
    z = torch.einsum("qhd,khd->hqk", q.double(), key) * SCALE
    z = z.masked_fill(~torch.ones((n, n), dtype=torch.bool, device=DEV).tril(), -math.inf)
    want = torch.einsum("hqk,khd->qhd", z.softmax(2), kv[..., 128:].double())
    assert bool(((out.double() - want).abs() <= 1e-2 + 2e-2 * want.abs()).all())
    # steps; every third one's last token is taken back (a draft that was refused)
    for i in range(7):
        s.q.copy_(s.rnd(*s.q.shape))
        s.proj.copy_(s.rnd(*s.proj.shape))
        s.step()
        history = [torch.cat([h, s.proj[b * q_len:(b + 1) * q_len]]) for b, h in enumerate(history)]
        torch.cuda.synchronize()
        assert int(s.status) == 0 and m.device_status(s.ws) == 0
        for b in range(3):
            got = s.rows_of(b)
            assert _near(kind, got, s.expected(history[b], 0), page)
            q = torch.cat([s.q_lat, s.q_pe], dim=2)[b * q_len:(b + 1) * q_len].double().cpu().numpy().reshape(-1, 576)
            want_o, want_l = R.decode_page(q, got, SCALE, q_len, Hq)
            o = s.out[b * q_len:(b + 1) * q_len].double().cpu().numpy().reshape(-1, 512)
            l = s.lse[b * q_len:(b + 1) * q_len].double().cpu().numpy().reshape(-1)
            assert (np.abs(o - want_o) <= 1e-2 + 2e-2 * np.abs(want_o)).all()
            assert (np.abs(l - want_l) <= (1e-3 if kind != FP8 else 5e-2)).all()
        pe = R.rope(s.q[..., 576:].double().cpu().numpy(), s.pos.cpu().numpy(), s.steps.cpu().numpy(), True, s.ms)
        assert (np.abs(s.q_pe.double().cpu().numpy() - pe) <= np.abs(pe) * 2.0 ** -8 + 2.0 ** -12).all()
        if i % 3 == 2:
            s.lens -= 1
            history = [h[:-1] for h in history]


@pytest.mark.parametrize("kind", [PAGE, BF16])
def test_a_captured_step_is_replayed(kind):
    """The whole step in a graph, replayed, against eager steps; two layers' graphs in turn on one workspace."""
    a, b = Server(4, 8, 16, kind, 16, 2, seed=3), Server(4, 8, 16, kind, 16, 2, seed=3)
    layers = []
    for s in (a, b):
        other = Server(4, 8, 16, kind, 16, 2, seed=4)
        other.ws = s.ws
        layers.append((s, other))
    for s in layers[0] + layers[1]:
        s.step()
    torch.cuda.synchronize()
    graphs = []
    for s in layers[0]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        s.lens.fill_(2)  # (the capture itself ran nothing, but the host added to no tensor either)
        graphs.append(g)
    for i in range(5):
        x, q = a.rnd(*a.proj.shape), a.rnd(*a.q.shape)
        for s in layers[0] + layers[1]:
            s.proj.copy_(x)
            s.q.copy_(q)
        for g in graphs:
            g.replay()
        for s in layers[1]:
            s.step()
        torch.cuda.synchronize()
        for s, e in zip(*layers):
            assert torch.equal(s.out, e.out) and torch.equal(s.lse, e.lse) and torch.equal(s.cache, e.cache)
