"""mla_rope on the GPU against its definition in 64 bits.

Tolerance, an element of a pair (a, b): the angle is off by at most 2^-25 pi,
sincospif by a few units of 2^-24, the two products and their sum by three
roundings, in all under 2^-20 (|a| + |b|) mscale; then half a step of the type."""
import numpy as np
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
import step_ref as R
from mla_latent_kv_cache_gb300 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()
    m.load()
    torch.cuda.set_device(DEV)
    yield


def _steps(dim, scaling="none", **kw):
    return m.rope_steps(dim, scaling=scaling, device=DEV, **kw)


def _within(got, x, pos, steps, inter, mscale):
    xd = x.double().cpu().numpy()
    want = R.rope(xd, pos.cpu().numpy(), steps.cpu().numpy(), inter, mscale)
    h = xd.shape[-1] // 2
    pair = np.abs(xd[..., 0::2]) + np.abs(xd[..., 1::2]) if inter else np.abs(xd[..., :h]) + np.abs(xd[..., h:])
    pair = np.repeat(pair, 2, axis=-1) if inter else np.concatenate([pair, pair], axis=-1)
    half = torch.finfo(got.dtype).eps / 2
    off = np.abs(got.double().cpu().numpy() - want)
    room = half * np.abs(want) + 2.0 ** -20 * pair * abs(mscale)
    assert (off <= room).all(), (off - room).max()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,R_", [(1, 1, 64), (1, 128, 64), (3, 16, 64), (65, 20, 64), (700, 3, 128), (5, 7, 16),
                                    (9, 5, 24), (33, 2, 2), (4, 3, 256), (2, 3, 258), (2500, 16, 64)])
def test_matches_the_definition(T, H, R_, dt, inter):
    gen = torch.Generator(device=DEV).manual_seed(T * 7 + H)
    x = torch.randn((T, H, R_), generator=gen, device=DEV).to(dt)
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen, device=DEV, dtype=torch.int32)
    pos[-1] = 2 ** 31 - 1
    pos[0] = 0
    steps, ms = _steps(R_, "yarn", factor=40.0)
    out = torch.full_like(x, float("nan"))
    m.mla_rope(x, pos, steps, out, interleaved=inter, mscale=ms)
    _within(out, x, pos, steps, inter, ms)
    assert torch.equal(out[0], (x[0].float() * ms).to(dt)) if T > 1 else True  # position 0 turns nothing


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R_,lead,tail", [(64, 128, 0), (64, 0, 8), (64, 3, 0), (32, 1, 1), (10, 6, 0)])
def test_part_of_the_head_in_place_and_apart(R_, lead, tail, dt, inter):
    gen = torch.Generator(device=DEV).manual_seed(R_ + lead)
    T, H = 37, 6
    heads = torch.randn((T, H, lead + R_ + tail), generator=gen, device=DEV).to(dt)
    before = heads.clone()
    pos = torch.arange(T, device=DEV, dtype=torch.int32) * 1000
    steps, _ = _steps(R_)
    out = torch.empty((T, H, R_), dtype=dt, device=DEV)
    part = slice(lead, lead + R_)
    m.mla_rope(heads[..., part], pos, steps, out, interleaved=inter)
    assert torch.equal(heads, before)
    _within(out, before[..., part], pos, steps, inter, 1.0)
    m.mla_rope(heads[..., part], pos, steps, heads[..., part], interleaved=inter)
    assert torch.equal(heads[..., part], out)
    assert torch.equal(heads[..., :lead], before[..., :lead]) and torch.equal(heads[..., lead + R_:], before[..., lead + R_:])


def test_from_one_part_of_the_heads_into_another():
    x = torch.randn((11, 4, 192), device=DEV).to(torch.bfloat16)
    steps, _ = _steps(64)
    pos = torch.arange(11, device=DEV, dtype=torch.int32)
    want = torch.empty((11, 4, 64), dtype=torch.bfloat16, device=DEV)
    m.mla_rope(x[..., 128:], pos, steps, want)
    m.mla_rope(x[..., 128:], pos, steps, x[..., 64:128])
    assert torch.equal(x[..., 64:128], want)


def test_heads_before_tokens():
    """[H, T, R] memory seen as [T, H, R]."""
    x = torch.randn((4, 50, 64), device=DEV).to(torch.bfloat16).transpose(0, 1)
    steps, _ = _steps(64)
    pos = torch.arange(50, device=DEV, dtype=torch.int32)
    out = torch.empty_like(x)
    m.mla_rope(x, pos, steps, out, interleaved=True)
    _within(out, x, pos, steps, True, 1.0)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_is_the_call_with_negated_steps(inter):
    """The rotation is linear: <g, rope(x)> = <rope with -steps (g), x>, and the
    difference of two outputs along a direction is the output of the direction."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    T, H = 19, 5
    x, g, d = (torch.randn((T, H, 64), generator=gen, device=DEV) for _ in range(3))
    pos = torch.randint(0, 200000, (T,), generator=gen, device=DEV, dtype=torch.int32)
    steps, ms = _steps(64, "yarn", factor=8.0)
    back, y, y2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    m.mla_rope(g, pos, -steps, back, interleaved=inter, mscale=ms)
    _within(back, g, pos, -steps, inter, ms)
    m.mla_rope(x, pos, steps, y, interleaved=inter, mscale=ms)
    # both sums have n = T H 64 terms, each off by at most 2^-20 (|a| + |b|) mscale times the other factor
    room = 2.0 ** -19 * ms * float((g.abs().double().sum(-1) * x.abs().double().amax(-1)).sum())
    lhs, rhs = float((g.double() * y.double()).sum()), float((back.double() * x.double()).sum())
    assert abs(lhs - rhs) <= room
    h = 2.0 ** -3
    m.mla_rope(x + h * d, pos, steps, y2, interleaved=inter, mscale=ms)
    slope = ((y2.double() - y.double()) * g.double()).sum() / h
    want = (back.double() * ((x + h * d).double() - x.double())).sum() / h
    assert abs(float(slope - want)) <= 2 * room / h + room


def test_empty_calls_and_streams():
    steps, _ = _steps(64)
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    m.mla_rope(e, torch.empty(0, dtype=torch.int32, device=DEV), steps, e)
    x = torch.randn((300, 8, 64), device=DEV)
    pos = torch.arange(300, device=DEV, dtype=torch.int32)
    want, out = torch.empty_like(x), torch.zeros_like(x)
    m.mla_rope(x, pos, steps, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.mla_rope(x, pos, steps, out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        m.mla_rope(x, pos, steps, out)
        m.mla_rope(out, pos, -steps, out)
    x.copy_(torch.randn_like(x))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    m.mla_rope(x, pos, steps, want)
    m.mla_rope(want, pos, -steps, want)
    assert torch.equal(out, want)
    assert (out - x).abs().max() <= 2.0 ** -17 * x.abs().max()  # there and back: two calls' 2^-20 of at most 4 max


def test_offsets_past_32_bits():
    """Tokens that lie past 2^31 elements; wider strides than the call takes are refused."""
    T, H, st = 3, 2, (1 << 30) + 64
    buf = torch.empty((T - 1) * st + H * 64, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((T, H, 64), (st, 64, 1))
    steps, _ = _steps(64)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    out = torch.empty((T, H, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(m.MlaError) as e:
        m.mla_rope(x, pos, steps, out)
    assert e.value.status == m.MLA_ERR_UNSUPPORTED
    x = buf.as_strided((T, H, 64), (1 << 30, 64, 1))
    x.copy_(torch.randn((T, H, 64), device=DEV))
    m.mla_rope(x, pos, steps, out)
    _within(out, x, pos, steps, False, 1.0)
