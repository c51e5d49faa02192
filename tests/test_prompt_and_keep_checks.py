"""Refusals of mla_prefill, mla_attn_weights and mla_cache_evict (no GPU
needed): the library's host checks, which come before any CUDA call, and the
binding's own checks with a stand-in library."""
import pytest
import torch

import mla_latent_kv_cache_gb300 as m
from mla_latent_kv_cache_gb300 import build as mbuild

INVALID, UNSUPPORTED, OK = m.MLA_ERR_INVALID_ARG, m.MLA_ERR_UNSUPPORTED, m.MLA_OK


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load()


def _with(args, **over):
    """`args` (name, value) with some replaced, as a positional list."""
    d = dict(args)
    assert set(over) <= set(d)
    d.update(over)
    return list(d.values())


PREFILL = [("q", 16), ("q_st", 1536), ("q_sh", 192), ("kn", 16), ("k_st", 2048), ("k_sh", 256), ("kp", 16), ("kp_st", 576),
           ("v", 16), ("v_st", 2048), ("v_sh", 256), ("cq", 16), ("ck", 16), ("B", 2), ("tq", 40), ("tk", 50), ("mq", 30),
           ("Hq", 8), ("Hkv", 8), ("causal", 1), ("scale", 0.1), ("out", 16), ("lse", 16), ("st", None), ("stream", None)]

PREFILL_BAD = [
    dict(B=-1), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(mq=0), dict(Hq=0), dict(Hkv=0), dict(Hq=8, Hkv=3),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=None), dict(kn=None), dict(kp=None), dict(v=None), dict(cq=None), dict(ck=None), dict(out=None), dict(lse=None),
    dict(q=24), dict(kn=8), dict(kp=20), dict(v=2), dict(out=8), dict(lse=18), dict(cq=17), dict(ck=2), dict(st=6),
    dict(q_st=1540), dict(q_sh=184), dict(k_st=100), dict(k_sh=0), dict(kp_st=56), dict(v_st=-2048), dict(v_sh=132),
]


@pytest.mark.parametrize("over", PREFILL_BAD, ids=str)
def test_prefill_refuses(lib, over):
    assert lib.mla_prefill(*_with(PREFILL, **over)) == INVALID


def test_prefill_limits_and_empty_calls(lib):
    assert lib.mla_prefill(*_with(PREFILL, B=0)) == OK
    assert lib.mla_prefill(*_with(PREFILL, tq=0, mq=0, q=None)) == OK
    assert lib.mla_prefill(*_with(PREFILL, tq=2 ** 31)) == UNSUPPORTED
    assert lib.mla_prefill(*_with(PREFILL, tk=2 ** 31)) == UNSUPPORTED
    assert lib.mla_prefill(*_with(PREFILL, Hq=2 ** 30, Hkv=2 ** 30)) == UNSUPPORTED
    assert lib.mla_prefill(*_with(PREFILL, k_st=1 << 38)) == UNSUPPORTED


WEIGHTS = [("ql", 16), ("qp", 16), ("lse", 16), ("cache", 16), ("kind", 0), ("D", 512), ("slots", 100), ("page", 16),
           ("bt", 16), ("bts", 4), ("sl", 16), ("B", 2), ("q_len", 1), ("Hq", 8), ("scale", 0.1), ("decay", 1.0), ("w", 16),
           ("ws", 64), ("ml", 64), ("st", None), ("ctas", 0), ("stream", None)]

WEIGHTS_BAD = [
    dict(B=-1), dict(q_len=0), dict(Hq=0), dict(page=0), dict(slots=0), dict(ml=-1), dict(ctas=-1), dict(kind=2),
    dict(decay=-0.5), dict(decay=float("nan")), dict(decay=float("inf")), dict(scale=float("nan")), dict(ql=None),
    dict(qp=None), dict(lse=None), dict(cache=None), dict(bt=None), dict(sl=None), dict(w=None), dict(ql=8), dict(qp=24),
    dict(cache=8), dict(lse=2), dict(w=17), dict(bt=18), dict(sl=1), dict(st=3), dict(bts=0), dict(ws=63),
]


@pytest.mark.parametrize("over", WEIGHTS_BAD, ids=str)
def test_weights_refuse(lib, over):
    assert lib.mla_attn_weights(*_with(WEIGHTS, **over)) == INVALID


def test_weights_limits_and_empty_calls(lib):
    assert lib.mla_attn_weights(*_with(WEIGHTS, B=0, ql=None)) == OK
    assert lib.mla_attn_weights(*_with(WEIGHTS, ml=0, w=None)) == OK
    for over in (dict(D=384), dict(D=256, kind=1), dict(slots=2 ** 31), dict(Hq=1 << 21)):
        assert lib.mla_attn_weights(*_with(WEIGHTS, **over)) == UNSUPPORTED


EVICT = [("cache", 16), ("rb", 1152), ("slots", 100), ("page", 16), ("bt", 16), ("bts", 4), ("sl", 16), ("w", 4096),
         ("pos", 8192), ("stride", 64), ("ml", 64), ("bud", 16), ("B", 2), ("sink", 4), ("recent", 8), ("nl", 16),
         ("nw", 12288), ("np", 16384), ("mv", 16), ("mvs", 66), ("st", None), ("stream", None)]

EVICT_BAD = [
    dict(B=-1), dict(page=0), dict(slots=0), dict(ml=-1), dict(sink=-1), dict(recent=-1), dict(rb=0), dict(rb=1160),
    dict(rb=65552), dict(bts=0), dict(stride=63), dict(mvs=65), dict(cache=None), dict(bt=None), dict(sl=None), dict(w=None),
    dict(pos=None), dict(bud=None), dict(nl=None), dict(nw=None), dict(np=None), dict(mv=None), dict(cache=8), dict(bt=2),
    dict(sl=2), dict(w=4098), dict(pos=8193), dict(bud=3), dict(nl=5), dict(nw=12289), dict(np=2), dict(mv=6), dict(st=1),
    dict(nw=4096 + 256), dict(nw=4096 - 4), dict(np=8192 + 508),  # overlaps its input
]


@pytest.mark.parametrize("over", EVICT_BAD, ids=str)
def test_evict_refuses(lib, over):
    assert lib.mla_cache_evict(*_with(EVICT, **over)) == INVALID


def test_evict_limits_and_empty_calls(lib):
    assert lib.mla_cache_evict(*_with(EVICT, B=0, cache=None)) == OK
    assert lib.mla_cache_evict(*_with(EVICT, ml=(1 << 30) + 1, stride=1 << 31, mvs=1 << 31)) == UNSUPPORTED


# ------------------------------------------------------------- the binding

class _Recorder:
    def __init__(self, real):
        self.calls, self.real = [], real

    def __getattr__(self, name):
        if name in ("mla_row_bytes", "mla_status_string"):
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or m.MLA_OK


@pytest.fixture
def fake(monkeypatch, lib):
    rec = _Recorder(lib)
    monkeypatch.setattr(m, "_is_cuda", lambda t: isinstance(t, torch.Tensor))
    monkeypatch.setattr(m, "_current_device", lambda: -1)  # what a host tensor gives as its device
    monkeypatch.setattr(m, "load", lambda: rec)
    monkeypatch.setattr(m, "_stream", lambda s: 0)
    return rec


def _refused(fn, words):
    with pytest.raises(m.MlaError) as e:
        fn()
    assert e.value.status == INVALID and words in str(e.value), str(e.value)


bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)
i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
f32 = lambda *n: torch.zeros(n)


def _prefill(**over):
    a = dict(q=bf(10, 4, 192), k_nope=bf(12, 2, 256)[:, :, :128], k_pe=bf(12, 576)[:, 512:], v=bf(12, 2, 256)[:, :, 128:],
             cu_q_lens=i32(3), cu_k_lens=i32(3), max_q_len=6, scale=0.1, out=bf(10, 4, 128), lse=f32(10, 4))
    a.update(over)
    return m.mla_prefill(**a)


def _weights(**over):
    a = dict(q_lat=bf(4, 8, 512), q_pe=bf(4, 8, 64), lse=f32(4, 8), cache=torch.zeros((64, 1152), dtype=torch.uint8),
             cache_kind=0, page_size=16, block_table=i32(2, 4), seq_lens=i32(2), q_len=2, scale=0.1, weights=f32(2, 50))
    a.update(over)
    return m.mla_attn_weights(**a)


def _evict(**over):
    a = dict(cache=torch.zeros((64, 1152), dtype=torch.uint8), cache_kind=0, page_size=16, block_table=i32(2, 4),
             seq_lens=i32(2), weights=f32(2, 50), positions=i32(2, 50), budgets=i32(2), n_sink=1, n_recent=2,
             new_seq_lens=i32(2), new_weights=f32(2, 50), new_positions=i32(2, 50), moves=i32(2, 52))
    a.update(over)
    return m.mla_cache_evict(**a)


def test_host_tensors_are_refused():
    for call in (_prefill, _weights, _evict):
        _refused(call, "must be a CUDA tensor")


def test_missing_tensors_are_refused(fake):
    for name in ("q", "k_nope", "k_pe", "v", "cu_q_lens", "cu_k_lens", "out", "lse"):
        _refused(lambda: _prefill(**{name: None}), f"{name} must be a CUDA tensor")
    for name in ("q_lat", "lse", "cache", "block_table", "seq_lens", "weights"):
        _refused(lambda: _weights(**{name: None}), f"{name} must be a CUDA tensor")
    for name in ("cache", "positions", "budgets", "new_seq_lens", "new_weights", "moves"):
        _refused(lambda: _evict(**{name: None}), f"{name} must be a CUDA tensor")
    assert fake.calls == []


def test_tensors_on_another_device_than_the_current_one_are_refused(fake, monkeypatch):
    monkeypatch.setattr(m, "_current_device", lambda: 1)
    for call in (_prefill, _weights, _evict):
        _refused(call, "the current device is cuda:1")
    assert fake.calls == []


def test_good_calls_pass_strides_through(fake):
    _prefill()
    _weights()
    _evict()
    names = [n for n, _ in fake.calls]
    assert names == ["mla_prefill", "mla_attn_weights", "mla_cache_evict"]
    p = fake.calls[0][1]
    assert p[1:3] == (768, 192) and p[4:6] == (512, 256) and p[7] == 576 and p[9:11] == (512, 256)
    assert p[13:19] == (2, 10, 12, 6, 4, 2)
    _weights(weights=f32(2, 99)[:, :50])
    assert fake.calls[-1][1][17:19] == (99, 50)
    w, x = f32(2, 99)[:, :50], i32(2, 99)[:, :50]
    _evict(weights=w, positions=x, new_weights=w, new_positions=x)
    assert fake.calls[-1][1][9:11] == (99, 50)


@pytest.mark.parametrize("over,words", [
    (dict(q=bf(10, 4, 128)), "q must be"), (dict(q=bf(40, 192)), "q must be"), (dict(q=f32(10, 4, 192)), "q must be bf16"),
    (dict(k_nope=bf(12, 2, 192)), "k_nope must be"), (dict(v=bf(12, 4, 128)), "v must have"), (dict(v=bf(13, 2, 128)), "v must have"),
    (dict(k_pe=bf(11, 64)), "k_pe must be"), (dict(k_pe=bf(12, 32)), "k_pe must be"),
    (dict(k_nope=bf(2, 128, 12).transpose(0, 2).transpose(1, 2)), "contiguous last dimension"),
    (dict(out=bf(10, 4, 192)), "out must be"), (dict(out=f32(10, 4, 128)), "out must be"), (dict(lse=f32(10, 3)), "lse must be"),
    (dict(lse=bf(10, 4)), "lse must be"), (dict(cu_k_lens=i32(4)), "cu_k_lens"), (dict(cu_q_lens=torch.zeros(3)), "cu_q_lens"),
    (dict(status=f32(1)), "status"),
], ids=str)
def test_prefill_binding_refuses(fake, over, words):
    _refused(lambda: _prefill(**over), words)
    assert fake.calls == []


@pytest.mark.parametrize("over,words", [
    (dict(q_lat=bf(4, 8, 256)), "expected"), (dict(q_lat=f32(4, 8, 512)), "bf16"), (dict(q_pe=bf(4, 8, 32)), "expected"),
    (dict(q_len=1), "expected"), (dict(lse=f32(4, 7)), "lse"), (dict(lse=bf(4, 8)), "lse"), (dict(weights=f32(1, 50)), "weights"),
    (dict(weights=f32(1, 50).expand(2, 50)), "weights"), (dict(weights=f32(50, 2).t()), "weights"), (dict(weights=bf(2, 50)), "weights"),
    (dict(block_table=i32(1, 4)), "block_table"), (dict(seq_lens=f32(2)), "seq_lens"), (dict(cache_kind=3), "cache kind"),
    (dict(cache_kind=1, lat_dim=256, q_lat=bf(4, 8, 256)), "lat_dim 512"), (dict(status=f32(1)), "status"),
], ids=str)
def test_weights_binding_refuses(fake, over, words):
    _refused(lambda: _weights(**over), words)
    assert fake.calls == []


@pytest.mark.parametrize("over,words", [
    (dict(weights=f32(1, 50)), "weights"), (dict(weights=f32(1, 50).expand(2, 50)), "weights"), (dict(positions=f32(2, 50)), "positions"),
    (dict(positions=i32(2, 49)), "positions"), (dict(new_weights=f32(2, 60)[:, :50]), "new_weights"), (dict(new_positions=i32(2, 51)), "new_positions"),
    (dict(new_weights=f32(1, 50).expand(2, 50)), "new_weights"), (dict(budgets=i32(1)), "budgets"), (dict(new_seq_lens=f32(2)), "new_seq_lens"),
    (dict(moves=i32(2, 51)), "moves"), (dict(moves=i32(1, 52)), "moves"), (dict(moves=i32(1, 52).expand(2, 52)), "moves"),
    (dict(block_table=i32(2, 4).t()), "block_table"), (dict(cache=torch.zeros((1152, 64), dtype=torch.uint8).t()), "cache"),
], ids=str)
def test_evict_binding_refuses(fake, over, words):
    _refused(lambda: _evict(**over), words)
    assert fake.calls == []


def test_columns_of_a_wider_table(fake):
    table = i32(2, 8)[:, 4:]  # the last row ends four pages of 16 after it begins
    _weights(block_table=table, weights=f32(2, 64))
    _evict(block_table=table)
    _weights(block_table=i32(2, 8)[:, :4], weights=f32(2, 999))
    assert len(fake.calls) == 3
    _refused(lambda: _weights(block_table=table, weights=f32(2, 65)), "block_table")
    _refused(lambda: _evict(block_table=table, weights=f32(2, 65), positions=i32(2, 65), new_weights=f32(2, 65),
                            new_positions=i32(2, 65), moves=i32(2, 67)), "block_table")
    assert len(fake.calls) == 3


# One row: its stride says nothing, but the elements inside the row still have
# to follow each other (the kernels walk a row as contiguous values).
ONE_ROW = dict(block_table=i32(1, 4), seq_lens=i32(1), weights=f32(1, 50), positions=i32(1, 50), budgets=i32(1),
               new_seq_lens=i32(1), new_weights=f32(1, 50), new_positions=i32(1, 50), moves=i32(1, 52))


@pytest.mark.parametrize("name,view", [
    (name, view(make))
    for name, make in (("weights", f32), ("positions", i32), ("new_weights", f32), ("new_positions", i32))
    for view in (lambda t: t(1, 100)[:, ::2], lambda t: t(50, 2).t()[:1], lambda t: t(1, 1).expand(1, 50))
], ids=lambda x: x if isinstance(x, str) else f"strides{x.stride()}")
def test_evict_refuses_one_row_whose_values_lie_apart(fake, name, view):
    _refused(lambda: _evict(**{**ONE_ROW, name: view}), name)
    assert fake.calls == []


def test_evict_takes_one_row_of_any_row_stride(fake):
    wide = lambda make: make(3, 99)[1:2, :50]
    tall = lambda make: make(50, 1).t()  # strides (1, 1)
    for view in (wide, tall):
        _evict(**{**ONE_ROW, "weights": view(f32), "positions": view(i32), "new_weights": f32(1, 50), "new_positions": view(i32)})
    _evict(**{**ONE_ROW, "weights": wide(f32), "positions": i32(1, 50)})
    assert [c[1][9] >= 50 and c[1][10] == 50 for c in fake.calls] == [True] * 3
    one = dict(weights=f32(1, 2)[:, ::2], positions=i32(1, 2)[:, ::2], new_weights=f32(1, 1), new_positions=i32(1, 1))
    _evict(**{**ONE_ROW, **one})  # one value: its stride says nothing either
    assert len(fake.calls) == 4


def test_a_one_row_table_reaches_as_far_as_its_columns(fake):
    # torch leaves the stride of a dimension of one entry as it comes: 1 here, and 0 for
    # an expanded view
    table = torch.arange(4, dtype=torch.int32).view(4, 1).t()
    assert table.stride() == (1, 1) and table.is_contiguous()
    narrow = (table, i32(4).as_strided((1, 4), (0, 1)), i32(4).as_strided((1, 4), (3, 1)))
    for t in narrow:
        _weights(block_table=t, seq_lens=i32(1), q_lat=bf(2, 8, 512), q_pe=bf(2, 8, 64), lse=f32(2, 8), weights=f32(1, 50))
        assert fake.calls[-1][1][9] == 4
        _evict(**{**ONE_ROW, "block_table": t})
        assert fake.calls[-1][1][5] == 4
    # columns of a wider row go on to its end, however large a stride the view has
    _evict(**{**ONE_ROW, "block_table": i32(1, 8)[:, :4]})
    assert fake.calls[-1][1][5] == 8
    _evict(**{**ONE_ROW, "block_table": i32(6).as_strided((1, 4), (10 ** 6, 1), 1)})
    assert fake.calls[-1][1][5] == 5


@pytest.mark.parametrize("stride", [0, 1, 3])
def test_tables_whose_rows_overlap_are_refused(fake, stride):
    table = i32(8).as_strided((2, 4), (stride, 1))
    _refused(lambda: _weights(block_table=table), "block_table")
    _refused(lambda: _evict(block_table=table), "block_table")
    assert fake.calls == []


def test_tables_without_columns(fake):
    # nothing is cached and nothing can be: the lengths still go over
    for n in (1, 2):
        empty = dict(seq_lens=i32(n), budgets=i32(n), weights=f32(n, 0), positions=i32(n, 0), new_weights=f32(n, 0),
                     new_positions=i32(n, 0), new_seq_lens=i32(n), moves=i32(n, 2))
        _evict(**{**empty, "block_table": i32(n, 0)})
        assert fake.calls[-1][1][5] >= 1 and fake.calls[-1][1][10] == 0
    # room for tokens but no table entry for them (one row: the library refuses a stride of 0)
    _evict(**{**ONE_ROW, "block_table": i32(1, 0)})
    assert fake.calls[-1][1][5] == 0
    _refused(lambda: _evict(block_table=i32(2, 0)), "block_table")


@pytest.mark.parametrize("scale", [2.0 ** 127, 3e38])
def test_prefill_refuses_a_scale_that_log2_units_cannot_hold(lib, scale):
    assert lib.mla_prefill(*_with(PREFILL, scale=scale)) == INVALID
