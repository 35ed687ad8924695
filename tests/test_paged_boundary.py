"""The paged calls reject bad arguments before they touch a device (CPU only), and the
tests' own pools read back what was written to them."""
import dataclasses

import numpy as np
import pytest

import factorised_kv_attention_b200 as kpa
import paged_util as pu
from workloads import Shape

S = Shape(h1=4, h2=4, d1=8, d2=16, r_k=2, r_v=2)
CFG = kpa.make_config(S, "bf16")
A = 1 << 20                      # a 16-byte (and 256-byte) aligned address that is never followed


def _pages(**kw):
    return kpa.make_pages(**{"page_size": 64, "n_pages": 10, "table_stride": 4, "format": "e4m3", **kw})


def _append(cfg=CFG, pages=None, **kw):
    a = dict(batch=2, n_rows=5, k_factors=A, v_factors=A, cu_rows=A, start_pos=A, page_table=A, kpool=A, vpool=A, stream=0)
    kpa.kpa_paged_append_factors(cfg, pages or _pages(), **{**a, **kw})


def _read(cfg=CFG, pages=None, **kw):
    a = dict(batch=2, n_rows=5, k_factors=A, v_factors=A, cu_rows=A, start_pos=A, page_table=A, kpool=A, vpool=A, stream=0)
    kpa.kpa_paged_read_factors(cfg, pages or _pages(), **{**a, **kw})


def _prefill(cfg=CFG, pages=None, **kw):
    a = dict(batch=2, n_rows=5, q=A, cu_rows=A, start_pos=A, page_table=A, kpool=A, vpool=A, max_len=256, window=0,
             sinks=0, sm_scale=1.0, out=A, workspace=A, ws_bytes=1 << 40, stream=0)
    kpa.kpa_paged_prefill(cfg, pages or _pages(), **{**a, **kw})


def _decode(cfg=CFG, pages=None, **kw):
    a = dict(batch=2, q=A, seq_len=A, page_table=A, kpool=A, vpool=A, max_len=256, window=0, sinks=0, sm_scale=1.0,
             out=A, workspace=A, ws_bytes=1 << 40, stream=0)
    kpa.kpa_paged_decode(cfg, pages or _pages(), **{**a, **kw})


CALLS = {"append": _append, "read": _read, "prefill": _prefill, "decode": _decode}


def _refused(call, status, **kw):
    with pytest.raises(kpa.KpaError) as e:
        call(**kw)
    assert e.value.status == status


def test_page_bytes():
    e = S.e_k
    assert kpa.kpa_paged_page_bytes(CFG, _pages()) == (64 * (e + 2), 64 * (e + 2))
    assert kpa.kpa_paged_page_bytes(CFG, _pages(format="bf16")) == (64 * e * 2, 64 * e * 2)
    uneven = kpa.make_config(dataclasses.replace(S, r_k=3, r_v=1), "bf16")
    assert kpa.kpa_paged_page_bytes(uneven, _pages(page_size=16)) == (16 * (3 * e // 2 + 2), 16 * (e // 2 + 2))


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("bad", [{"page_size": 0}, {"page_size": 24}, {"page_size": 8192}, {"page_size": -16},
                                 {"n_pages": 0}, {"table_stride": 0}, {"table_stride": 1 << 26}], ids=str)
def test_bad_pool(name, bad):
    _refused(CALLS[name], kpa.KPA_ERR_INVALID_ARG, pages=_pages(**bad))


def test_bad_format():
    with pytest.raises(KeyError):
        _pages(format="int8")
    for call in CALLS.values():
        _refused(call, kpa.KPA_ERR_INVALID_ARG, pages=kpa.kpa_pages(64, 10, 4, 2))


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("cfg", [kpa.make_config(S, "f32"), kpa.make_config(dataclasses.replace(S, shared_b=1), "bf16"),
                                 kpa.make_config(Shape(h1=16, h2=1, d1=8, d2=8, r_k=2, r_v=2, order=3), "bf16")],
                         ids=["f32", "shared_b", "order3"])
def test_unsupported_config(name, cfg):
    _refused(CALLS[name], kpa.KPA_ERR_UNSUPPORTED, cfg=cfg)


@pytest.mark.parametrize("name", ["prefill", "decode"])
def test_wide_heads_are_refused(name):
    wide = kpa.make_config(dataclasses.replace(S, d1=16, d2=16), "bf16")
    _refused(CALLS[name], kpa.KPA_ERR_UNSUPPORTED, cfg=wide)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_negative_sizes(name):
    _refused(CALLS[name], kpa.KPA_ERR_INVALID_ARG, batch=-1)
    if name != "decode":
        _refused(CALLS[name], kpa.KPA_ERR_INVALID_ARG, n_rows=-1)


@pytest.mark.parametrize("name", ["prefill", "decode"])
@pytest.mark.parametrize("bad", [{"window": -1}, {"sinks": -1}, {"max_len": -1}, {"max_len": 257},
                                 {"sm_scale": float("nan")}, {"sm_scale": float("inf")}], ids=str)
def test_bad_mask_or_length(name, bad):
    _refused(CALLS[name], kpa.KPA_ERR_INVALID_ARG, **bad)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_pointers(name):
    call = CALLS[name]
    ptr = {"append": ["k_factors", "v_factors", "cu_rows", "start_pos", "page_table", "kpool", "vpool"],
           "read": ["k_factors", "v_factors", "cu_rows", "start_pos", "page_table", "kpool", "vpool"],
           "prefill": ["q", "cu_rows", "start_pos", "page_table", "kpool", "vpool", "out"],
           "decode": ["q", "seq_len", "page_table", "kpool", "vpool", "out"]}[name]
    for p in ptr:
        _refused(call, kpa.KPA_ERR_INVALID_ARG, **{p: None})
        _refused(call, kpa.KPA_ERR_INVALID_ARG, **{p: A + 2})
        if p not in ("cu_rows", "start_pos", "page_table", "seq_len"):
            _refused(call, kpa.KPA_ERR_INVALID_ARG, **{p: A + 8})


@pytest.mark.parametrize("name", sorted(CALLS))
def test_nothing_to_do(name):
    none = {"batch": 0}
    CALLS[name](**none)
    if name != "decode":
        CALLS[name](n_rows=0)


def test_workspace_size_of_nothing():
    assert kpa.kpa_paged_decode_workspace_size(CFG, _pages(), 0, 256) == 0
    assert kpa.kpa_paged_prefill_workspace_size(CFG, _pages(), 3, 0, 256) == 0
    for bad in ((3, 257, 0, 0), (-1, 10, 0, 0), (3, 10, -1, 0), (3, 10, 0, -1)):
        with pytest.raises(kpa.KpaError):
            kpa.kpa_paged_decode_workspace_size(CFG, _pages(), *bad)


def test_null_descriptors():
    import ctypes
    lib = ctypes.CDLL(kpa.LIB_PATH)
    assert lib.kpa_paged_page_bytes(None, None, None, None) == kpa.KPA_ERR_INVALID_ARG
    assert lib.kpa_paged_page_bytes(ctypes.byref(CFG), None, None, None) == kpa.KPA_ERR_INVALID_ARG


def test_the_tests_pool_reads_back():
    """Quantising moves a value by at most half a step: 2^-4 of it, or 2^-10 of its scale."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, S.e_k)) * np.exp2(rng.integers(-8, 9, (40, 1)))
    x[3], x[4, 0], x[5, -1] = 0.0, np.nan, np.inf
    a = S.r_k * S.h1 * S.d1
    p = pu.planes(S, "e4m3", 3, 32)[0]
    pool = p.empty()
    slots = np.arange(40)
    p.write(pool, slots // 32, slots % 32, x)
    y = p.read(pool, slots // 32, slots % 32)
    assert np.isnan(y[4, 0]) and np.isnan(y[5, -1]) and (y[3] == 0).all()
    fine = np.isfinite(x)
    e = np.where(np.arange(S.e_k) < a, pu.exponents(x[:, :a])[:, None], pu.exponents(x[:, a:])[:, None])
    step = np.maximum(2.0 ** -4 * np.abs(np.where(fine, x, 0)), np.exp2(e - 10.0))
    assert (np.abs(y - x)[fine] <= step[fine]).all()
