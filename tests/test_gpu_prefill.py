"""mla_prefill on the GPU against the 64-bit form of its definition.

Tolerance. A score is a sum of 192 exact products added 16 at a time in fp32,
each addition off by at most 2^-23 of the magnitudes summed so far: with M the
largest sum of |products| times the scale it is off by 12 2^-23 M, and the
exponent's fp32 arithmetic adds 4 2^-23 (2 M + |lse|) more at most: eps. The
log-sum-exp is off by eps plus the rounding of fp32 sums of positive terms
(2^-24 a term, of Lk terms at worst) and of the result. A probability is then
off by a factor 1 + 2 eps, and its rounding to bf16 by 2^-8; so with
A = sum_j p_j |v_j| the output is off by (2^-8 + 2 eps + Lk 2^-23) A before its own
rounding, which is 2^-8 of it."""
import numpy as np
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.empty_cache()


def _inputs(q_lens, k_lens, Hq, Hkv, seed=0, amp=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *n: (amp * torch.randn(n, generator=g, device=DEV)).to(torch.bfloat16)
    tq, tk = sum(q_lens), sum(k_lens)
    kv, rows = r(tk, Hkv, 256), r(tk, 576)
    cu = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV)
    return dict(q=r(tq, Hq, 192), k_nope=kv[:, :, :128], v=kv[:, :, 128:], k_pe=rows[:, 512:], cu_q=cu(q_lens), cu_k=cu(k_lens),
                q_lens=list(q_lens), k_lens=list(k_lens), Hq=Hq, Hkv=Hkv)


def _call(a, causal=True, scale=SCALE, **kw):
    tq = a["q"].shape[0]
    out = torch.full((tq, a["Hq"], 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((tq, a["Hq"]), 7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mla_prefill(a["q"], a["k_nope"], a["k_pe"], a["v"], a["cu_q"], a["cu_k"], max(a["q_lens"] + [1]), scale, out, lse,
                  causal=causal, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return out, lse


def _want(a, causal=True, scale=SCALE):
    """(out, lse, A, M) in fp64, of finite inputs."""
    f = {k: a[k].double().cpu().numpy() for k in ("q", "k_nope", "k_pe", "v")}
    tq, Hq, g = f["q"].shape[0], a["Hq"], a["Hq"] // a["Hkv"]
    out, A = np.zeros((tq, Hq, 128)), np.zeros((tq, Hq, 128))
    lse, M = np.full((tq, Hq), -np.inf), 0.0
    q0 = k0 = 0
    for lq, lk in zip(a["q_lens"], a["k_lens"]):
        for h in range(Hq if lq and lk else 0):
            k = np.concatenate([f["k_nope"][k0:k0 + lk, h // g], f["k_pe"][k0:k0 + lk]], axis=1)
            q, v = f["q"][q0:q0 + lq, h], f["v"][k0:k0 + lk, h // g]
            s = scale * (q @ k.T)
            M = max(M, scale * (np.abs(q) @ np.abs(k).T).max())
            if causal:
                s[np.arange(lk)[None] > (lk - lq + np.arange(lq))[:, None]] = -np.inf
            top = s.max(axis=1, keepdims=True)
            top[top == -np.inf] = 0
            p = np.exp(s - top)
            tot = p.sum(axis=1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[q0:q0 + lq, h] = (top + np.log(tot))[:, 0]
            p = p / np.where(tot > 0, tot, 1)
            out[q0:q0 + lq, h] = p @ v
            A[q0:q0 + lq, h] = p @ np.abs(v)
        q0, k0 = q0 + lq, k0 + lk
    return out, lse, A, M


def _check(a, causal=True, scale=SCALE):
    got, glse = _call(a, causal, scale)
    out, lse, A, M = _want(a, causal, scale)
    fin = np.isfinite(lse)
    big = np.abs(lse[fin]).max(initial=0.0)
    eps = 12 * 2.0 ** -23 * M + 4 * 2.0 ** -23 * (2 * M + big)
    lk = max(a["k_lens"] + [1])
    assert eps < 1e-3
    got, glse = got.double().cpu().numpy(), glse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(glse), ~fin)
    assert np.all(got[~fin] == 0)
    assert np.all(np.abs(glse[fin] - lse[fin]) <= eps + lk * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(lse[fin])))
    tol = (2.0 ** -8 + 2 * eps + lk * 2.0 ** -23) * A + 2.0 ** -8 * np.abs(out) + 1e-30
    assert np.all(np.abs(got - out) <= tol), np.abs(got - out).max()
    return got, glse


LENS = [1, 0, 37, 127, 128, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 2), (6, 2), (3, 1), (16, 1)])
def test_packed_prompts(Hq, Hkv, causal):
    _check(_inputs(LENS, LENS, Hq, Hkv, seed=Hq), causal)


@pytest.mark.parametrize("causal", [True, False])
def test_contexts_longer_and_shorter_than_the_queries(causal):
    q = [1, 5, 64, 130, 300, 200, 10, 0, 90]
    k = [1000, 5, 191, 513, 301, 50, 0, 77, 129]  # 200 over 50 and 10 over 0 leave queries without keys
    _check(_inputs(q, k, 4, 2, seed=1), causal)


@pytest.mark.parametrize("n", [1, 2, 31, 128, 256, 384, 1000, 2049])
def test_one_sequence(n):
    _check(_inputs([n], [n], 2, 2, seed=n))


@pytest.mark.parametrize("Hq,Hkv", [(5, 1), (14, 2), (48, 1), (130, 1), (256, 2)])
def test_group_sizes_that_do_not_divide_a_tile(Hq, Hkv):
    # heads of a group share tiles of 128 rows: whole tokens of 5, 7, ... heads
    q, k = [1, 40, 130, 0, 9], [1, 40, 150, 10, 300]
    for causal in (True, False):
        _check(_inputs(q, k, Hq, Hkv, seed=Hq), causal)


def test_no_keys_at_all():
    a = _inputs([3, 300], [0, 0], 2, 1, seed=2)
    for causal in (True, False):
        out, lse = _call(a, causal)
        assert not bool(out.any()) and bool(torch.isneginf(lse).all())


def test_many_short_sequences():
    r = np.random.default_rng(0)
    lens = r.integers(0, 40, size=150).tolist()
    _check(_inputs(lens, lens, 2, 1, seed=3))
    lens = r.integers(0, 600, size=70).tolist()
    _check(_inputs(lens, lens, 1, 1, seed=3))


def test_single_tokens_over_contexts():
    _check(_inputs([1] * 40, list(range(1, 801, 20)), 4, 4, seed=4))


def test_large_scores_and_scales():
    a = _inputs([300], [300], 2, 2, seed=5, amp=3.0)
    _check(a)
    _check(a, scale=1e-6)
    # scores that keep rising along the keys: the running maximum moves every tile
    a = _inputs([500], [500], 1, 1, seed=6)
    a["k_nope"] *= torch.linspace(0.1, 3, 500, device=DEV)[:, None, None].to(torch.bfloat16)
    _check(a)


def test_strides():
    a = _inputs([70, 200], [70, 200], 4, 2, seed=7)
    want, wl = _call(a)
    b = dict(a)
    wide = torch.full((270, 4 + 1, 200), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :4, :192] = a["q"]
    b["q"] = wide[:, :4, :192]
    heads = torch.full((2, 270, 136), float("nan"), dtype=torch.bfloat16, device=DEV)  # head-major keys
    heads[:, :, :128] = a["k_nope"].transpose(0, 1)
    b["k_nope"] = heads[:, :, :128].transpose(0, 1)
    b["v"] = a["v"].contiguous()
    b["k_pe"] = a["k_pe"].contiguous()
    got, gl = _call(b)
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_grouped_heads_equal_repeated_ones():
    a = _inputs(LENS, LENS, 6, 2, seed=8)
    b = dict(a, Hkv=6, k_nope=a["k_nope"].repeat_interleave(3, dim=1), v=a["v"].repeat_interleave(3, dim=1))
    x, y = _call(a), _call(b)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_a_chunk_equals_the_tail_of_the_whole_prompt():
    # the last 300 queries over all the keys: both are within the bound of the same values
    a = _inputs([1000], [1000], 2, 2, seed=9)
    _check(a)
    _check(dict(a, q=a["q"][700:].contiguous(), q_lens=[300], cu_q=torch.tensor([0, 300], dtype=torch.int32, device=DEV)))


@pytest.mark.parametrize("where", ["k_nope", "k_pe", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_query_does_not_see_does_not_reach_it(where, bad):
    # a bad value in the middle of the first sequence, at the start of the second
    # and in the last token of the third: earlier queries and other sequences are as before
    q = [200, 130, 140, 60]
    a = _inputs(q, q, 2, 1, seed=10)
    clean, cl = _call(a)
    tokens = [150, 200, 469]
    x = a[where].clone()
    for t in tokens:
        x[t, ..., 3] = bad
    got, gl = _call(dict(a, **{where: x}))
    start = np.concatenate([[0], np.cumsum(q)])
    sees = torch.zeros(sum(q), dtype=torch.bool, device=DEV)
    for t in tokens:
        s = int(np.searchsorted(start, t, side="right"))
        sees[t:start[s]] = True
    assert torch.equal(gl[~sees], cl[~sees])
    # rows formed again differ by the rounding of the probabilities, 2^-8 of sum p |v| at most twice
    A = torch.from_numpy(_want(a)[2]).to(DEV).float()
    tol = 2.0 ** -7 * A + 2.0 ** -7 * clean.float().abs() + 1e-6
    near = (got.float() - clean.float()).abs() <= tol
    assert bool(near[~sees].all())
    if where == "v":
        assert torch.equal(gl, cl)
        hit = got[sees][:, :, 3].float()
        assert bool(torch.isnan(hit).all() if bad != bad else (hit == bad).all())
        other = [d for d in range(128) if d != 3]
        assert bool(near[:, :, other].all())


def test_rows_formed_again_over_a_long_context():
    # the last key's value is not finite and lies in the last key tile of every query:
    # all but the last are formed again, for longer than the kernel's own waits
    # last; heads of one group make more items than SMs, so that others wait for these
    Lq, Lk, Hq = 127, 200063, 320
    a = _inputs([Lq], [Lk], Hq, 1, seed=21)
    clean, cl = _call(a)
    a["v"][Lk - 1, 0, 5] = float("nan")
    got, gl = _call(a)
    assert torch.equal(gl, cl)
    assert bool(torch.isnan(got[-1, :, 5]).all()) and int(torch.isnan(got).sum()) == Hq
    k = torch.cat([a["k_nope"][:, 0], a["k_pe"]], 1).double()
    for t, h in ((0, 0), (63, 177), (125, 319)):
        n = Lk - Lq + t + 1
        s = SCALE * (k[:n] @ a["q"][t, h].double())
        A = torch.softmax(s, 0) @ a["v"][:n, 0].double().abs()
        # rounded probabilities on one side, fp32 additions on both, and both outputs' rounding
        tol = (2.0 ** -8 + 2 * n * 2.0 ** -24) * A + 2.0 ** -8 * (got[t, h].double().abs() + clean[t, h].double().abs())
        assert bool(((got[t, h].double() - clean[t, h].double()).abs() <= tol).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (16, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_lies_behind_a_sequence_changes_nothing(Hq, Hkv, bad, causal):
    # rows of no sequence at the end of longer buffers, and those of the next sequence
    q, k = [130, 1, 64, 300, 77], [130, 257, 63, 449, 640]
    a = _inputs(q + [0], k + [200], Hq, Hkv, seed=22)
    T = sum(k)
    a["cu_q"], a["cu_k"] = a["cu_q"][:-1].contiguous(), a["cu_k"][:-1].contiguous()
    clean, cl = _call(a, causal=causal)
    for x in ("v", "k_nope", "k_pe"):
        a[x][T:] = bad
    got, gl = _call(a, causal=causal)
    assert torch.equal(got, clean) and torch.equal(gl, cl)
    a["v"][sum(k[:3]):] = bad  # the last two sequences' values
    got, gl = _call(a, causal=causal)
    n = sum(q[:3])
    assert torch.equal(got[:n], clean[:n]) and torch.equal(gl, cl)
    assert not bool(torch.isfinite(got[n:]).any())


def test_values_whose_sum_passes_the_range():
    # 2^127 under hundreds of weights near 1: past fp32, while their mean is not; the
    # probabilities' rounding and the output's are off by 2^-8 at most each
    a = _inputs([200], [600], 2, 1, seed=23)
    a["v"].fill_(2.0 ** 127)
    out, _ = _call(a)
    assert bool(((out.double() / 2.0 ** 127 - 1).abs() <= 2.0 ** -7).all())


def test_prefix_sums_past_the_rows_are_clamped():
    a = _inputs([100, 60], [100, 60], 2, 2, seed=11)
    want, wl = _call(a)
    a["cu_q"] = torch.tensor([0, 100, 10 ** 9], dtype=torch.int32, device=DEV)
    a["cu_k"] = torch.tensor([0, 100, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    got, gl = _call(a)
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_rows_that_no_sequence_names_are_left():
    a = _inputs([100, 60], [100, 60], 2, 2, seed=12)
    a["cu_q"] = torch.tensor([0, 100, 130], dtype=torch.int32, device=DEV)
    out, lse = _call(a)
    assert bool((out[130:] == 7).all()) and bool((lse[130:] == 7).all()) and not bool((lse[:130] == 7).any())


def test_repeats_bit_for_bit_on_a_side_stream_and_from_a_graph():
    a = _inputs(LENS, LENS, 4, 2, seed=13)
    want, wl = _call(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, gl = _call(a)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_prefill(a["q"], a["k_nope"], a["k_pe"], a["v"], a["cu_q"], a["cu_k"], 700, SCALE, out, lse)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_a_query_whose_keys_take_longer_than_a_wait():
    # one query over 120 million keys: 1.5 s of one CTA, whose other tile and scheduler have
    # nothing to do until the next item. Two keys, at both ends, hold all the weight but 5e-10.
    Lk = 120_000_000
    k = torch.zeros((Lk, 1, 128), dtype=torch.bfloat16, device=DEV)  # 31 GB; the values and rotary keys are views of it
    q = torch.zeros((1, 1, 192), dtype=torch.bfloat16, device=DEV)
    q[0, 0, 0] = 8
    k[5, 0, 0] = k[Lk - 10, 0, 0] = 5
    k[5, 0, 70], k[Lk - 10, 0, 9] = 3, 1
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)
    a = dict(q=q, k_nope=k, k_pe=k[:, 0, 64:], v=k, cu_q=cu(1), cu_k=cu(Lk), q_lens=[1], k_lens=[Lk], Hq=1, Hkv=1)
    out, lse = _call(a, scale=1.0)
    want = torch.zeros(128, dtype=torch.bfloat16)
    want[0], want[70], want[9] = 5, 1.5, 0.5
    assert torch.equal(out[0, 0].cpu(), want)  # probabilities of 1 and 2^-58: no rounding is left
    L = 40 + np.log(2.0)
    assert abs(float(lse) - L) <= 4 * 2.0 ** -23 * (2 * 40 + L) + 2.0 ** -22 * (1 + L)


def test_scores_of_any_magnitude_that_is_allowed():
    # multiples of 2^24 up to 2^30: a row is the mean of the values with the largest it sees
    n, H = 300, 2
    a = _inputs([n], [n], H, 1, seed=31)
    g = torch.Generator().manual_seed(31)
    r = torch.randint(-64, 65, (n,), generator=g)
    for x in ("q", "k_nope", "k_pe"):
        a[x] = torch.zeros_like(a[x])
    a["q"][:, :, 3] = 2.0 ** 15
    a["k_nope"][:, 0, 3] = (r * 2.0 ** 9).to(torch.bfloat16).to(DEV)  # (at most 7 bits)
    out, lse = _call(a, scale=1.0)
    out, lse, v = out.double().cpu(), lse.double().cpu(), a["v"][:, 0].double().cpu()
    for t in range(n):
        top = int(r[:t + 1].max())
        best = (r[:t + 1] == top).nonzero()[:, 0]
        want, A = v[best].mean(0), v[best].abs().mean(0)
        tol = 2.0 ** -8 * A + 2.0 ** -8 * want.abs() + n * 2.0 ** -23 * A
        assert bool(((out[t] - want).abs() <= tol).all())
        L = top * 2.0 ** 24 + np.log(len(best))
        M = 2.0 ** 30
        assert bool(((lse[t] - L).abs() <= 4 * 2.0 ** -23 * (2 * M + abs(L)) + 2.0 ** -22 * (1 + abs(L))).all())
