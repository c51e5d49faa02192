"""Refusals of mla_rope, mla_cache_append and mla_decode_fp8_page, and the table of angles (no GPU
needed): the library's host checks, which come before any CUDA call, and the
binding's own checks with a stand-in library."""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
import step_ref
from mla_latent_kv_cache_gb300 import build as mbuild
from test_prompt_and_keep_checks import _Recorder, _refused, _with, bf, f32, i32

INVALID, UNSUPPORTED, OK = m.MLA_ERR_INVALID_ARG, m.MLA_ERR_UNSUPPORTED, m.MLA_OK
i64 = lambda *n: torch.zeros(n, dtype=torch.int64)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load()


@pytest.fixture
def fake(monkeypatch, lib):
    rec = _Recorder(lib)
    monkeypatch.setattr(m, "_is_cuda", lambda t: isinstance(t, torch.Tensor))
    monkeypatch.setattr(m, "_current_device", lambda: -1)  # what a host tensor gives as its device
    monkeypatch.setattr(m, "load", lambda: rec)
    monkeypatch.setattr(m, "_stream", lambda s: 0)
    monkeypatch.setattr(m, "_device", -1)
    monkeypatch.setattr(m, "_addresses", {n: getattr(rec, n) for n in ("mla_rope", "mla_cache_append", "mla_decode_fp8_page")})
    return rec


# ------------------------------------------------------------ rope_steps

@pytest.mark.parametrize("dim", [2, 24, 64, 128])
def test_steps_hold_the_frequencies(dim):
    for base in (10000.0, 500000.0):
        s, ms = m.rope_steps(dim, base, device="cpu")
        want = step_ref.steps_of([base ** (-2.0 * i / dim) for i in range(dim // 2)])
        assert ms == 1.0 and s.dtype == torch.int64
        # a double holds 53 bits of f / (2 pi)
        assert (np.abs(s.numpy() - want) <= np.abs(want) * 2.0 ** -50 + 1).all()


def test_scaled_steps():
    f = np.array([10000.0 ** (-2.0 * i / 64) for i in range(32)])
    as_f = lambda s: s.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi  # noqa: E731
    near = lambda a, b: np.allclose(a, b, rtol=1e-12, atol=0)  # noqa: E731
    s, ms = m.rope_steps(64, scaling="linear", factor=8.0, device="cpu")
    assert near(as_f(s), f / 8) and ms == 1.0
    s, ms = m.rope_steps(64, scaling="ntk", factor=8.0, device="cpu")
    got = as_f(s)
    assert ms == 1.0 and near(got[0], f[0]) and near(got[-1], f[-1] / 8) and (np.diff(f / got) > 0).all()
    s, ms = m.rope_steps(64, scaling="yarn", factor=40.0, original_max=4096, device="cpu")
    got, turns = as_f(s), 4096 * f / (2 * math.pi)
    assert ms == pytest.approx(0.1 * math.log(40) + 1)
    # the ramp goes from the whole index below that of 32 turns to the one above that of one turn
    fast, slow = turns > 32 * f[0] / f[1], turns < f[1] / f[0]
    assert fast.any() and slow.any() and near(got[fast], f[fast]) and near(got[slow], f[slow] / 40)
    # (steps are whole: the least, 9.8e12, is off by 1, so a ratio of 40 by 5e-12)
    assert (np.diff(f / got) >= -1e-11).all()
    assert m.rope_steps(64, scaling="yarn", factor=1.0, device="cpu")[1] == 1.0


@pytest.mark.parametrize("bad", [dict(dim=3), dict(dim=0), dict(base=0.0), dict(factor=0.0), dict(scaling="other"),
                                 dict(original_max=0), dict(scaling="yarn", base=1.0), dict(scaling="yarn", beta_slow=0.0),
                                 dict(scaling="yarn", beta_fast=0.5), dict(dim=2, scaling="ntk", factor=2.0)], ids=str)
def test_bad_steps_are_refused(bad):
    with pytest.raises(ValueError):
        m.rope_steps(**{"device": "cpu", **bad})


# ------------------------------------------------------------ the library

ROPE = [("x", 4096), ("x_t", 512), ("x_h", 64), ("pos", 16), ("steps", 16), ("T", 10), ("H", 8), ("R", 64), ("f32", 0),
        ("inter", 0), ("ms", 1.0), ("out", 65536), ("o_t", 512), ("o_h", 64), ("stream", None)]

ROPE_BAD = [
    dict(T=-1), dict(H=-1), dict(R=0), dict(R=63), dict(R=-2), dict(ms=float("nan")), dict(ms=float("inf")), dict(x=None),
    dict(pos=None), dict(steps=None), dict(out=None), dict(x=4097), dict(out=65537), dict(x=4098, f32=1), dict(pos=18),
    dict(steps=20), dict(x_h=63), dict(o_h=0), dict(x_t=63), dict(o_t=-512), dict(x_t=500),   # tokens that share values
    dict(out=4096 + 64), dict(out=4096 + 128), dict(out=4096, o_h=128, o_t=1024),             # overlaps its input
    dict(out=4096 + 2 * 65, x_h=192, o_h=192, x_t=1536, o_t=1536, R=66),
    dict(out=4096 + 2 * 150, x_h=192, o_h=192, x_t=1536, o_t=1536),                            # runs into the next head
    dict(out=4096 + 2 * 64, x_h=192, o_h=192, x_t=1408, o_t=1408),                             # or a token's last into the next token
    dict(out=4096 + 2 * 64, x_h=1792, o_h=1792, x_t=192, o_t=192),                             # (heads outermost)
]


@pytest.mark.parametrize("over", ROPE_BAD, ids=str)
def test_rope_refuses(lib, over):
    assert lib.mla_rope(*_with(ROPE, **over)) == INVALID


def test_rope_limits_and_empty_calls(lib):
    assert lib.mla_rope(*_with(ROPE, T=0, x=None)) == OK
    assert lib.mla_rope(*_with(ROPE, H=0, x=None)) == OK
    for over in (dict(T=1 << 31), dict(R=(1 << 20) + 2), dict(H=(1 << 20) + 1), dict(x_t=(1 << 30) + 8), dict(T=1 << 30, H=1 << 10), dict(T=1, H=1 << 20, R=1 << 12)):
        assert lib.mla_rope(*_with(ROPE, **over)) == UNSUPPORTED


APPEND = [("lat", 1 << 20), ("lat_st", 576), ("pe", (1 << 20) + 1024), ("pe_st", 576), ("cu", 16), ("sl", 16), ("bt", 16),
          ("bts", 4), ("btc", 4), ("B", 2), ("total", 10), ("page", 16), ("pos", 16), ("steps", 16), ("inter", 0), ("ms", 1.0),
          ("norm", 16), ("eps", 1e-6), ("cache", 16), ("kind", 0), ("D", 512), ("slots", 64), ("scales", None), ("rows", None),
          ("rows_st", 0), ("st", None), ("stream", None)]

APPEND_BAD = [
    dict(B=-1), dict(total=-1), dict(page=0), dict(slots=-1), dict(kind=3), dict(kind=-1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(ms=float("nan")), dict(lat=None), dict(pe=None), dict(cu=None), dict(sl=None), dict(bt=None),
    dict(cache=None), dict(lat=8), dict(pe=8), dict(cache=24), dict(norm=2), dict(cu=18), dict(sl=1), dict(bt=2), dict(pos=2),
    dict(steps=12), dict(st=2), dict(lat_st=504), dict(lat_st=580), dict(pe_st=56), dict(pe_st=68), dict(bts=3), dict(btc=-1),
    dict(scales=16), dict(kind=2), dict(kind=2, scales=18), dict(kind=1, scales=16),
    dict(rows=1 << 24, rows_st=568), dict(rows=1 << 24, rows_st=580), dict(rows=(1 << 24) + 8, rows_st=576),
    dict(rows=(1 << 20) + 16, rows_st=576), dict(rows=1 << 20, rows_st=584), dict(rows=1 << 20, rows_st=576, pe=(1 << 20) + 1040),
]


@pytest.mark.parametrize("over", APPEND_BAD, ids=str)
def test_append_refuses(lib, over):
    assert lib.mla_cache_append(*_with(APPEND, **over)) == INVALID


def test_append_limits_and_empty_calls(lib):
    assert lib.mla_cache_append(*_with(APPEND, B=0, lat=None)) == OK
    assert lib.mla_cache_append(*_with(APPEND, total=0, lat=None)) == OK
    for over in (dict(D=384), dict(D=256, kind=1), dict(D=768, kind=2, scales=16), dict(total=1 << 31), dict(lat_st=1 << 31),
                 dict(B=1 << 29)):
        assert lib.mla_cache_append(*_with(APPEND, **over)) == UNSUPPORTED


def test_page_rows_are_refused_by_the_other_calls(lib):
    assert m.mla_row_bytes(m.MLA_CACHE_FP8_PAGE_576) == 576
    assert lib.mla_cache_write(16, 512, 16, 64, 16, 4, 16, 10, 2, None, None) == INVALID
    assert lib.mla_decode(16, 16, 16, 2, 100, 16, 16, 4, 16, 2, 1, 8, 0.1, 16, 0, 16, 256, 1 << 24, 0, None) == INVALID


# ------------------------------------------------------------ the binding

def _rope(**over):
    a = dict(x=bf(10, 4, 192)[..., 128:], positions=i32(10), steps=i64(32), out=bf(10, 4, 64))
    a.update(over)
    return m.mla_rope(**a)


def _append(**over):
    proj = bf(10, 576)
    a = dict(latent=proj[:, :512], k_pe=proj[:, 512:], cu_new_lens=i32(3), seq_lens=i32(2), block_table=i32(2, 4), page_size=16,
             cache=torch.zeros((64, 1152), dtype=torch.uint8), cache_kind=0)
    a.update(over)
    return m.mla_cache_append(**a)


PAGE = dict(cache_kind=2, cache=torch.zeros((64, 576), dtype=torch.uint8), scales=torch.zeros(4))


DECODE = [("ql", 16), ("qp", 16), ("tokens", 2), ("cache", 16), ("scales", 16), ("slots", 100), ("page", 16), ("bt", 16),
          ("bts", 4), ("btc", 4), ("sl", 16), ("cu", None), ("B", 2), ("q_len", 1), ("Hq", 8), ("scale", 0.1), ("out", 16),
          ("odt", 0), ("lse", 16), ("ws", 256), ("wsb", 1 << 24), ("ctas", 0), ("stream", None)]

DECODE_BAD = [
    dict(B=0), dict(q_len=0), dict(Hq=0), dict(page=0), dict(slots=0), dict(ctas=-1), dict(tokens=0), dict(tokens=3), dict(odt=2),
    dict(ql=None), dict(qp=None), dict(cache=None), dict(scales=None), dict(bt=None), dict(sl=None), dict(out=None), dict(lse=None),
    dict(ws=None), dict(ql=8), dict(qp=24), dict(cache=8), dict(out=2), dict(ws=128), dict(scales=2), dict(bt=1), dict(sl=2),
    dict(cu=3), dict(lse=2), dict(btc=-1), dict(bts=3), dict(scale=float("nan")),
]


@pytest.mark.parametrize("over", DECODE_BAD, ids=str)
def test_decode_refuses(lib, over):
    assert lib.mla_decode_fp8_page(*_with(DECODE, **over)) == INVALID


def test_decode_limits(lib):
    for over in (dict(slots=1 << 31), dict(Hq=1 << 21), dict(tokens=1 << 29, cu=16)):
        assert lib.mla_decode_fp8_page(*_with(DECODE, **over)) == UNSUPPORTED


def _decode(**over):
    a = dict(q_lat=bf(4, 8, 512), q_pe=bf(4, 8, 64), cache=torch.zeros((64, 576), dtype=torch.uint8), scales=torch.zeros(4), page_size=16,
             block_table=i32(2, 4), seq_lens=i32(2), q_len=2, scale=0.1, out=bf(4, 8, 512), lse=f32(4, 8),
             workspace=torch.zeros(1024, dtype=torch.uint8))
    a.update(over)
    return m.mla_decode_fp8_page(**a)


@pytest.mark.parametrize("over,words", [
    (dict(q_lat=bf(4, 8, 256)), "q_lat must be"), (dict(q_lat=f32(4, 8, 512)), "bf16"), (dict(q_pe=bf(4, 8, 32)), "q_pe"),
    (dict(q_pe=bf(4, 64, 8).transpose(1, 2)), "contiguous"), (dict(q_len=1), "expected"), (dict(out=bf(4, 8, 256)), "out must be"),
    (dict(out=bf(4, 8, 512).half()), "out must be"), (dict(lse=f32(4, 7)), "lse must be"), (dict(lse=bf(4, 8)), "lse must be"),
    (dict(scales=torch.zeros(3)), "scales"), (dict(scales=bf(4)), "scales"), (dict(page_size=0), "page_size"),
    (dict(page_size=1 << 40), "page_size"), (dict(block_table=i32(1, 4)), "block_table"), (dict(block_table=i32(4, 2).t()), "block_table"),
    (dict(block_table=i32(8).as_strided((2, 4), (3, 1))), "overlap"), (dict(seq_lens=f32(2)), "seq_lens"),
    (dict(cu_q_lens=i32(2)), "cu_q_lens"), (dict(cu_q_lens=f32(3)), "cu_q_lens"), (dict(cache=torch.zeros((576, 64), dtype=torch.uint8).t()), "cache"),
], ids=str)
def test_decode_binding_refuses(fake, over, words):
    _refused(lambda: _decode(**over), words)
    assert fake.calls == []


def test_good_decodes_pass_their_arguments_through(fake):
    _decode()
    c = fake.calls[-1][1]
    assert c[2] == 4 and c[5:7] == (64, 16) and c[8:10] == (4, 4) and c[11] is None and c[12:15] == (2, 2, 8) and c[17] == 0 and c[20:22] == (1024, 0)
    _decode(cu_q_lens=i32(3), out=f32(4, 8, 512), num_ctas=7, q_lat=bf(4, 8, 512))
    c = fake.calls[-1][1]
    assert c[11] and c[17] == 1 and c[21] == 7


def test_arguments_of_other_types_are_errors(fake):
    for call, over in ((_rope, dict(mscale="x")), (_append, dict(eps=None)), (_append, dict(page_size=2.5)), (_decode, dict(q_len=None)),
                       (_decode, dict(scale=[]))):
        with pytest.raises(TypeError):
            call(**over)
    assert fake.calls == []


def test_host_tensors_are_refused():
    for call in (_rope, _append, _decode):
        _refused(call, "must be a CUDA tensor")


def test_missing_tensors_and_other_devices_are_refused(fake, monkeypatch):
    for name in ("x", "positions", "steps", "out"):
        _refused(lambda: _rope(**{name: None}), f"{name} must be a CUDA tensor")
    for name in ("latent", "k_pe", "cu_new_lens", "seq_lens", "block_table", "cache"):
        _refused(lambda: _append(**{name: None}), f"{name} must be a CUDA tensor")
    for name in ("steps", "positions", "norm_weight", "scales", "rows", "status"):
        _refused(lambda: _append(**{name: 5}), f"{name} must be a CUDA tensor")
    for name in ("q_lat", "scales", "block_table", "lse", "workspace"):
        _refused(lambda: _decode(**{name: None}), f"{name} must be a CUDA tensor")
    _refused(lambda: _decode(cu_q_lens=5), "CUDA tensor")
    monkeypatch.setattr(m, "_current_device", lambda: 1)
    monkeypatch.setattr(m, "_device", 1)
    for call in (_rope, _append, _decode):
        _refused(call, "the current device is cuda:1")
    assert fake.calls == []


def test_good_calls_pass_strides_through(fake):
    _rope()
    assert fake.calls[-1][1][1:3] == (768, 192) and fake.calls[-1][1][5:11] == (10, 4, 64, 0, 0, 1.0)
    _rope(x=f32(10, 4, 64), out=f32(10, 4, 64), interleaved=True, mscale=2.0)
    assert fake.calls[-1][1][8:11] == (1, 1, 2.0)
    _append()
    c = fake.calls[-1][1]
    assert (c[1], c[3]) == (576, 576) and c[7:12] == (4, 4, 2, 10, 16) and c[19:22] == (0, 512, 64)
    _append(**PAGE, rows=bf(10, 600), steps=i64(32), positions=i32(10), norm_weight=bf(512), status=i32(1))
    c = fake.calls[-1][1]
    assert c[19:22] == (2, 512, 64) and c[24] == 600 and all(c[i] for i in (12, 13, 16, 22, 23, 25))
    _append(block_table=i32(2, 8)[:, 4:])
    assert fake.calls[-1][1][7:9] == (8, 4)
    _append(seq_lens=i32(1), cu_new_lens=i32(2), block_table=i32(1, 8)[:, 2:5])
    assert fake.calls[-1][1][7:9] == (3, 3)


@pytest.mark.parametrize("over,words", [
    (dict(x=bf(40, 64)), "x must be"), (dict(x=bf(10, 4, 64).half()), "bf16 or fp32"), (dict(out=bf(10, 4, 62)), "out must be"),
    (dict(out=f32(10, 4, 64)), "out must be"), (dict(x=bf(10, 4, 63), out=bf(10, 4, 63)), "even"), (dict(positions=i32(9)), "positions"),
    (dict(positions=i64(10)), "positions"), (dict(steps=i64(31)), "steps"), (dict(steps=f32(32)), "steps"),
    (dict(positions=i32(20)[::2]), "positions"), (dict(x=bf(10, 64, 4).transpose(1, 2)), "contiguous last"),
    (dict(out=bf(10, 64, 4).transpose(1, 2)), "contiguous last"),
], ids=str)
def test_rope_binding_refuses(fake, over, words):
    _refused(lambda: _rope(**over), words)
    assert fake.calls == []


@pytest.mark.parametrize("over,words", [
    (dict(latent=bf(10, 256)), "latent must be"), (dict(latent=f32(10, 512)), "latent must be"), (dict(latent=bf(512, 10).t()), "latent must be"),
    (dict(k_pe=bf(9, 64)), "k_pe must be"), (dict(k_pe=bf(10, 32)), "k_pe must be"), (dict(page_size=0), "page_size"),
    (dict(cache=torch.zeros((1152, 64), dtype=torch.uint8).t()), "cache"), (dict(cache_kind=3), "cache kind"),
    (dict(cache_kind=1, lat_dim=256, latent=bf(10, 256)), "lat_dim 512"), (dict(**PAGE, lat_dim=256, latent=bf(10, 256)), "lat_dim 512"),
    (dict(block_table=i32(1, 4)), "block_table"), (dict(block_table=i32(4)), "block_table"), (dict(block_table=i32(8).as_strided((2, 4), (3, 1))), "overlap"),
    (dict(seq_lens=f32(2)), "seq_lens"), (dict(cu_new_lens=i32(4)), "cu_new_lens"), (dict(steps=i64(16)), "steps"),
    (dict(positions=i32(9)), "positions"), (dict(norm_weight=bf(256)), "norm_weight"), (dict(norm_weight=f32(512)), "norm_weight"),
    (dict(PAGE, scales=torch.zeros(3)), "scales"), (dict(PAGE, scales=None), "scales"), (dict(PAGE, scales=bf(4)), "scales"),
    (dict(scales=torch.zeros(4)), "scales"), (dict(rows=bf(9, 576)), "rows must be"), (dict(rows=bf(10, 512)), "rows must be"),
    (dict(rows=f32(10, 576)), "rows must be"), (dict(status=f32(1)), "status"),
], ids=str)
def test_append_binding_refuses(fake, over, words):
    _refused(lambda: _append(**over), words)
    assert fake.calls == []


def test_evicting_page_rows_is_refused(fake):
    """Rows that move between pages would need their codes changed to the other page's scale."""
    _refused(lambda: m.mla_cache_evict(
        torch.zeros((64, 576), dtype=torch.uint8), 2, 16, i32(2, 4), i32(2), f32(2, 50), i32(2, 50), i32(2), 1, 2, i32(2), f32(2, 50),
        i32(2, 50), i32(2, 52)), "cache kind")
    assert fake.calls == []


# ------------------------------------------------------------ the compiled checks

def _three_calls():
    lens, cu, table = i32(2), i32(3), i32(2, 4)
    x = bf(4, 2, 64)
    return (lambda: m.mla_rope(x, i32(4), i64(32), torch.empty_like(x)),
            lambda: m.mla_cache_append(bf(4, 512), bf(4, 64), cu, lens, table, 16, torch.zeros((64, 576), dtype=torch.uint8),
                                       m.MLA_CACHE_FP8_PAGE_576, scales=f32(4)),
            lambda: m.mla_decode_fp8_page(bf(2, 8, 512), bf(2, 8, 64), torch.zeros((64, 576), dtype=torch.uint8), f32(4), 16,
                                          table, lens, 1, 0.1, f32(2, 8, 512), f32(2, 8), torch.zeros(1 << 16, dtype=torch.uint8)))


@pytest.mark.parametrize("what", ["missing", "another PyTorch", "no record"])
def test_only_the_calls_that_need_the_compiled_checks_go_without_them(monkeypatch, tmp_path, lib, what):
    """The library loads and answers; the three calls name what is wrong."""
    monkeypatch.setattr(m, "_bind", None)
    monkeypatch.setattr(m, "_lib", None)
    key = tmp_path / "key"
    if what == "missing":
        monkeypatch.setattr(m, "BIND_PATH", str(tmp_path / "_mla_bind.so"))
    else:
        if what == "another PyTorch":
            key.write_text("torch 1.0 other\n")
        monkeypatch.setattr(mbuild, "BIND_KEY", str(key))
    assert m.mla_row_bytes(m.MLA_CACHE_BF16_576) == 1152
    with pytest.raises(m.MlaError):  # an earlier call's own checks
        m.mla_merge_lse(f32(1, 1, 512), f32(1, 1), f32(1, 512))
    for call in _three_calls():
        with pytest.raises(ImportError, match="missing" if what == "missing" else "built against"):
            call()


def test_the_compiled_checks_load_with_the_first_call(monkeypatch, lib):
    for call in _three_calls():
        monkeypatch.setattr(m, "_bind", None)
        with pytest.raises(m.MlaError):  # (host tensors)
            call()
        assert m._bind is not None


def test_the_compiled_checks_are_built_anew_for_another_pytorch(monkeypatch, tmp_path):
    """A record of another PyTorch has them built again, and the library not; where that fails,
    the library stands, and the old ones do not."""
    mbuild.build()
    at, key = tmp_path / "bind.so", tmp_path / "key"
    at.write_bytes(b"")
    key.write_text(mbuild.bind_key() + "\n")
    monkeypatch.setattr(mbuild, "BIND", str(at))
    monkeypatch.setattr(mbuild, "BIND_KEY", str(key))
    made = []
    monkeypatch.setattr(mbuild, "_bind_command", lambda out: made.append(out) or ["cp", mbuild.LIB, out])
    monkeypatch.setattr(mbuild, "nvcc", lambda: pytest.fail("the library is as it should be"))
    mbuild.build()
    assert not made
    key.write_text("torch 1.0 other\n")
    mbuild.build()
    assert len(made) == 1 and at.stat().st_size > 0 and key.read_text().strip() == mbuild.bind_key()
    key.write_text("torch 1.0 other\n")
    monkeypatch.setattr(mbuild, "_bind_command", lambda out: ["false"])
    with pytest.warns(UserWarning, match="cannot be called"):
        assert mbuild.build() == mbuild.LIB
    assert not at.exists() and not key.exists()
