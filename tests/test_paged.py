"""The paged factor cache on the GPU, against the definition in 64 bits.

Every pool starts with each byte a NaN, and page table entries that no row may look at lead
outside it, so a read past a length, of a masked slot or of a wrong page shows."""
import dataclasses

import numpy as np
import pytest
import torch

import paged_util as pu
from gpu_util import kpa
from workloads import Shape

pytestmark = pytest.mark.gpu

SPLITS = {
    "kpa_4x4_8x16_r2": Shape(h1=4, h2=4, d1=8, d2=16, r_k=2, r_v=2),
    "kpa_4x8_8x16_r4": Shape(h1=4, h2=8, d1=8, d2=16, r_k=4, r_v=4),
    "kpa_4x8_8x16_r2": Shape(h1=4, h2=8, d1=8, d2=16, r_k=2, r_v=2),
    "kpa_4x4_8x8_r2": Shape(h1=4, h2=4, d1=8, d2=8, r_k=2, r_v=2),
    "kpa_2x8_8x8_r2": Shape(h1=2, h2=8, d1=8, d2=8, r_k=2, r_v=2),
    "kpa_8x2_8x8_r2": Shape(h1=8, h2=2, d1=8, d2=8, r_k=2, r_v=2),
    "tpa_16_64_r2": Shape(h1=16, h2=1, d1=1, d2=64, r_k=2, r_v=2),
    "tpa_32_64_r1": Shape(h1=32, h2=1, d1=1, d2=64, r_k=1, r_v=1),
    "tpa_16_128_r2": Shape(h1=16, h2=1, d1=1, d2=128, r_k=2, r_v=2),
    "tpa_61_64_r1": Shape(h1=61, h2=1, d1=1, d2=64, r_k=1, r_v=1),          # odd records
    "kpa_3x2_4x6_r2": Shape(h1=3, h2=2, d1=4, d2=6, r_k=2, r_v=2),
    "kpa_4x4_8x16_rk3_rv1": Shape(h1=4, h2=4, d1=8, d2=16, r_k=3, r_v=1),
}
NAMES = sorted(SPLITS)
FORMATS = ["bf16", "e4m3"]
I32 = {"dtype": torch.int32, "device": "cuda"}


def _i32(x):
    return torch.tensor(x, **I32)


def _no_error(lib):
    torch.cuda.synchronize()
    assert lib.kpa_read_device_error() == 0


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


# ------------------------------------------------------------------ writing and reading
def _append(lib, s, fmt, page, start, new, seed, scale=1.0, tail=0, poke=None):
    rng = np.random.default_rng(seed)
    total = [a + n for a, n in zip(start, new)]
    c = pu.Cache(s, fmt, page, [0] * len(start), seed, stride=max(-(-t // page) for t in total) + 1)
    # a pool with room for every sequence, all bytes NaN
    need = [-(-t // page) for t in total]
    n_pages = sum(need) + 2
    order = rng.permutation(n_pages).astype(np.int32)
    c.n_pages = n_pages
    c.kp, c.vp = pu.planes(s, fmt, n_pages, page)
    k, v = c.kp.empty().cuda(), c.vp.empty().cuda()
    at = 0
    for b, n in enumerate(need):
        c.table[b, :n] = torch.from_numpy(order[at:at + n])
        at += n
    cu = _cu(new)
    rows = int(cu[-1]) + tail
    kf = torch.from_numpy(rng.standard_normal((rows, s.e_k)) * scale).to(torch.bfloat16)
    vf = torch.from_numpy(rng.standard_normal((rows, s.e_v)) * scale).to(torch.bfloat16)
    if poke:
        poke(kf, vf)
    lib.kpa_paged_append_factors(lib.make_config(s, "bf16"), c.descriptor(lib), len(start), rows, kf.cuda(), vf.cuda(),
                                 _i32(cu), _i32(start), c.table.cuda(), k, v)
    return c, k, v, kf, vf, cu


def _check_records(c, k, v, kf, vf, cu, start):
    """Every row against its records rotated in 64 bits, every other byte still a NaN."""
    s = c.s
    seen = {"k": c.kp.empty(), "v": c.vp.empty()}
    for b in range(len(start)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        pos = np.arange(start[b], start[b] + n)
        pages, inside = c.where(b, pos)
        for name, plane, pool, want, e0, r in (
                ("k", c.kp, k, pu.rotate(pu.f64(kf[cu[b]:cu[b + 1]]), s, pos), s.e_k, s.r_k),
                ("v", c.vp, v, pu.f64(vf[cu[b]:cu[b + 1]]), s.e_v, s.r_v)):
            raw, got = plane.raw(pool, pages, inside), plane.read(pool, pages, inside)
            view = plane._view(seen[name])
            if plane.fmt == "bf16":
                # the rotation in fp32 is off by a few 2^-24 of the pair, then one rounding
                pair = np.abs(want).max(1, keepdims=True)
                tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * pair
                view[torch.as_tensor(pages).long(), torch.as_tensor(inside) // 8, :, torch.as_tensor(inside) % 8] = raw
            else:
                a = plane.a
                ex = raw[:, e0:].numpy().astype(int) - 127
                for i, part in enumerate((want[:, :a], want[:, a:])):
                    top = np.abs(part).max(1)
                    lo, hi = pu.exponents(part * (1 - 2.0 ** -20)), pu.exponents(part * (1 + 2.0 ** -20))
                    assert ((ex[:, i] == lo) | (ex[:, i] == hi)).all(), (name, b, i, top)
                step = np.exp2(np.where(np.arange(e0) < a, ex[:, :1], ex[:, 1:]) - 10.0)
                tol = np.maximum(2.0 ** -4 * np.abs(want), step) + 2.0 ** -21 * np.abs(want).max(1, keepdims=True)
                view[torch.as_tensor(pages).long(), torch.as_tensor(inside) // 16, :,
                     torch.tensor(pu.BYTE)[torch.as_tensor(inside) % 16]] = raw
            pu.assert_within(torch.from_numpy(got), want, tol, f"{name} of sequence {b}")
    for name, pool in (("k", k), ("v", v)):
        assert torch.equal(pool.cpu().view(torch.uint8), seen[name].view(torch.uint8)), f"{name}: a byte of no row changed"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
def test_append(name, fmt):
    lib = kpa()
    start, new = [0, 5, 16, 31, 7, 3], [1, 40, 16, 1, 0, 130]
    r = _append(lib, SPLITS[name], fmt, 32, start, new, 1)
    _no_error(lib)
    _check_records(*r, start)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 48, 256])
def test_append_pages_and_far_positions(page, fmt):
    lib = kpa()
    start, new = [100003, 0, 77], [35, 513, 1]
    r = _append(lib, SPLITS["kpa_4x4_8x16_r2"], fmt, page, start, new, 2, tail=9)   # 9 rows of no sequence
    _no_error(lib)
    _check_records(*r, start)


def test_append_many_sequences():
    """More sequences than one scan step of the block takes, most of them with one row."""
    lib = kpa()
    rng = np.random.default_rng(3)
    start = [int(x) for x in rng.integers(0, 90, 700)]
    new = [int(x) for x in rng.integers(0, 3, 700)]
    r = _append(lib, SPLITS["kpa_4x4_8x8_r2"], "e4m3", 16, start, new, 3)
    _no_error(lib)
    _check_records(*r, start)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -90, 2.0 ** 50, 1.0])
def test_quantised_extremes(scale):
    """Zero records, tiny and huge ones, values on a scale's border, infinities and NaN."""
    lib = kpa()
    s = SPLITS["kpa_4x4_8x16_r2"]

    def poke(kf, vf):
        vf[0] = 0
        vf[1, :] = 448 * 2.0 ** -7
        vf[2, 3] = 449 * 2.0 ** -7
        vf[3, 0], vf[3, -1], vf[3, 5] = float("inf"), float("nan"), float("-inf")
        vf[4] = float("nan")

    c, k, v, kf, vf, cu = _append(lib, s, "e4m3", 16, [3], [40], 4, scale=scale, poke=poke)
    _no_error(lib)
    pages, inside = c.where(0, np.arange(3, 43))
    x = pu.f64(vf)
    assert np.array_equal(c.vp.raw(v, pages, inside).numpy()[:, s.e_v:], pu.quantise(x, c.vp.a)[:, s.e_v:])
    want = pu.quantise(x, c.vp.a)
    got = c.vp.raw(v, pages, inside).numpy()
    nan = ~np.isfinite(x)
    assert ((got[:, :s.e_v] & 0x7F) == 0x7F)[nan].all()
    same = (got[:, :s.e_v] == want[:, :s.e_v]) | ((got[:, :s.e_v] & 0x7F) + (want[:, :s.e_v] & 0x7F) == 0)
    assert same[~nan].all()                                   # values are not rotated: equal bytes


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
def test_read(name, fmt):
    lib = kpa()
    s = SPLITS[name]
    c = pu.Cache(s, fmt, 48, [77, 5, 300, 0], 5)
    start, new = [3, 0, 250, 0], [70, 5, 50, 0]
    cu = _cu(new) + 2
    rows = int(cu[-1]) + 3
    kf = torch.full((rows, s.e_k), 7.0, dtype=torch.bfloat16, device="cuda")
    vf = torch.full((rows, s.e_v), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.kpa_paged_read_factors(lib.make_config(s, "bf16"), c.descriptor(lib), 4, rows, _i32(cu), _i32(start),
                               c.table.cuda(), c.k.cuda(), c.v.cuda(), kf, vf)
    _no_error(lib)
    for b in range(3):
        wk, wv = c.records(b, np.arange(start[b], start[b] + new[b]))
        assert np.array_equal(pu.f64(kf[cu[b]:cu[b + 1]]), wk) and np.array_equal(pu.f64(vf[cu[b]:cu[b + 1]]), wv)
    for x in (kf, vf):
        assert (x[:2] == 7).all() and (x[rows - 3:] == 7).all()


# ------------------------------------------------------------------ attention
def _q(rng, n, s):
    return torch.from_numpy(rng.standard_normal((n, s.h, s.dh)) * 0.3).to(torch.bfloat16)


def _seen_from(past, window):
    """First slot of the window of the first row (or of the query) of each sequence."""
    return [max(0, p - window + 1) if window else 0 for p in past]


def _prefill(lib, s, fmt, page, past, new, window, sinks, seed, tail=2, max_len=None):
    total = [p + n for p, n in zip(past, new)]
    c = pu.Cache(s, fmt, page, total, seed, first_seen=_seen_from(past, window), sinks=sinks)
    rng = np.random.default_rng(seed + 1)
    cu = _cu(new) + 1                                             # one row before, `tail` rows behind
    rows = int(cu[-1]) + tail
    q = _q(rng, rows, s)
    max_len = max(total) if max_len is None else max_len
    cfg, pages = lib.make_config(s, "bf16"), c.descriptor(lib)
    ws = torch.full((max(256, lib.kpa_paged_prefill_workspace_size(cfg, pages, len(past), rows, max_len, window, sinks)),),
                    255, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, s.h, s.dh), 5.0, dtype=torch.bfloat16, device="cuda")
    scale = 1.0 / np.sqrt(s.dh)
    lib.kpa_paged_prefill(cfg, pages, len(past), rows, q.cuda(), _i32(cu), _i32(past), c.table.cuda(), c.k.cuda(),
                          c.v.cuda(), max_len, window, sinks, scale, out, ws)
    _no_error(lib)
    assert (out[:1] == 5).all() and (out[rows - tail:] == 5).all()
    for b in range(len(past)):
        if new[b]:
            pick = np.unique(np.concatenate([[0, new[b] - 1], rng.integers(0, new[b], 6)]))
            want, tol = pu.attention(c, b, pu.f64(q[cu[b]:cu[b + 1]])[pick], past[b] + pick, window, sinks, scale)
            pu.assert_within(out[cu[b]:cu[b + 1]][torch.from_numpy(pick).cuda()], want, tol, f"sequence {b}")


def _decode(lib, s, fmt, page, length, window, sinks, seed, max_len=None):
    c = pu.Cache(s, fmt, page, length, seed, first_seen=_seen_from([n - 1 for n in length], window), sinks=sinks,
                 stride=None if max_len is None else -(-max_len // page) + 1)
    rng = np.random.default_rng(seed + 1)
    B = len(length)
    q = _q(rng, B, s)
    max_len = max(length) if max_len is None else max_len
    cfg, pages = lib.make_config(s, "bf16"), c.descriptor(lib)
    ws = torch.full((max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, B, max_len, window, sinks)),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full((B, s.h, s.dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    scale = 1.0 / np.sqrt(s.dh)
    lib.kpa_paged_decode(cfg, pages, B, q.cuda(), _i32(length), c.table.cuda(), c.k.cuda(), c.v.cuda(), max_len, window,
                         sinks, scale, out, ws)
    _no_error(lib)
    for b in range(B):
        if length[b] == 0:
            assert (out[b] == 0).all()
            continue
        want, tol = pu.attention(c, b, pu.f64(q[b:b + 1]), [length[b] - 1], window, sinks, scale, factored=True)
        pu.assert_within(out[b:b + 1], want, tol, f"sequence {b}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
def test_prefill(name, fmt):
    _prefill(kpa(), SPLITS[name], fmt, 32, [0, 77, 0, 300, 9], [1, 129, 0, 1, 64], 0, 0, 10)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["kpa_4x4_8x16_r2", "kpa_4x8_8x16_r4", "kpa_4x4_8x8_r2", "tpa_16_128_r2", "tpa_32_64_r1", "kpa_3x2_4x6_r2"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 70), (130, 1), (5000, 9), (64, 1000)])
def test_prefill_window(name, fmt, window, sinks):
    _prefill(kpa(), SPLITS[name], fmt, 48, [0, 290, 701, 64], [140, 130, 3, 260], window, sinks, 11)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 112, 1024])
def test_prefill_long_past(page, fmt):
    """Few rows over a long cache: the key range is split and its parts joined."""
    _prefill(kpa(), SPLITS["kpa_4x4_8x16_r2"], fmt, page, [4001], [17], 0, 0, 12)
    _prefill(kpa(), SPLITS["tpa_16_64_r2"], fmt, page, [2999, 0], [1, 5], 900, 20, 13)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("new,past,window,sinks", [
    ([1, 127, 128, 129], [0, 1, 0, 0], 0, 0),                 # one or two key tiles
    ([1, 1, 1, 1, 1], [127, 128, 255, 256, 383], 0, 0),       # an odd and an even number of them
    ([3, 128, 64, 256 + 1, 256 + 128, 256 + 129], [700, 333, 512, 450, 100, 0], 0, 0),
    ([1, 2, 300], [5000, 4000, 2500], 0, 0),                  # split over the keys
    ([1, 100, 128, 270], [3000, 2000, 1030, 900], 200, 130)], ids=["one", "tiles", "short", "split", "window"])
def test_prefill_few_rows(name, fmt, new, past, window, sinks):
    _prefill(kpa(), SPLITS[name], fmt, 64, past, new, window, sinks, 67)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
def test_decode(name, fmt):
    _decode(kpa(), SPLITS[name], fmt, 32, [1, 77, 0, 301, 16, 1000], 0, 0, 20)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["kpa_4x8_8x16_r2", "kpa_4x8_8x16_r4", "kpa_4x4_8x8_r2", "tpa_32_64_r1", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (100, 70), (777, 17), (5000, 9)])
def test_decode_window(name, fmt, window, sinks):
    _decode(kpa(), SPLITS[name], fmt, 48, [1, 290, 2003, 64, 0], window, sinks, 21)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["kpa_4x8_8x16_r2", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
def test_decode_long(name, fmt):
    _decode(kpa(), SPLITS[name], fmt, 64, [20011], 0, 0, 22)
    _decode(kpa(), SPLITS[name], fmt, 16, [9000, 1], 0, 0, 23, max_len=9007)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_large_batch(fmt):
    rng = np.random.default_rng(24)
    _decode(kpa(), SPLITS["kpa_4x4_8x16_r2"], fmt, 16, [int(x) for x in rng.integers(0, 200, 333)], 90, 2, 24)


@pytest.mark.parametrize("fmt", FORMATS)
def test_several_b_heads_at_d1_one(fmt):
    """A split of TPA's d1 and d2 whose B factors are not shared by every head."""
    s = Shape(h1=8, h2=2, d1=1, d2=64, r_k=2, r_v=2)
    cfg, pages = kpa().make_config(s, "bf16"), kpa().make_pages(32, 1, 1, fmt)
    assert kpa().kpa_paged_prefill_kernel_kind(cfg, pages) == "chunks"
    _prefill(kpa(), s, fmt, 32, [0, 77, 300], [130, 1, 40], 0, 0, 68)
    _prefill(kpa(), s, fmt, 48, [290, 64], [3, 260], 100, 20, 69)
    _decode(kpa(), s, fmt, 32, [1, 77, 0, 301], 0, 0, 70)


@pytest.mark.parametrize("name", ["kpa_4x4_8x16_r2", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
def test_prefill_many_sequences(name):
    """More sequences than the ordered search of a row tile holds."""
    rng = np.random.default_rng(25)
    past, new = [int(x) for x in rng.integers(0, 60, 300)], [int(x) for x in rng.integers(0, 4, 300)]
    new[7], new[250] = 300, 131
    _prefill(kpa(), SPLITS[name], "e4m3", 16, past, new, 40, 3, 25)


def test_every_kernel_is_reached():
    """The splits of these tests reach each kernel of both attentions."""
    lib = kpa()
    pages = lib.make_pages(16, 10, 10)
    kinds = {n: (lib.kpa_paged_decode_kernel_kind(lib.make_config(s, "bf16"), pages),
                 lib.kpa_paged_prefill_kernel_kind(lib.make_config(s, "bf16"), pages)) for n, s in SPLITS.items()}
    assert kinds["kpa_3x2_4x6_r2"] == kinds["kpa_4x4_8x16_rk3_rv1"] == ("chunks", "chunks")
    assert kinds["tpa_61_64_r1"] == ("chunks", "tcgen05")
    assert all(kinds[n] == ("factors", "tcgen05") for n in NAMES if n not in
               ("kpa_3x2_4x6_r2", "kpa_4x4_8x16_rk3_rv1", "tpa_61_64_r1"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["kpa_4x4_8x16_r2", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_other_scales(name, fmt, scale):
    """No scale, a negative one, and one that leaves a softmax of few tokens."""
    lib = kpa()
    s = SPLITS[name]
    c = pu.Cache(s, fmt, 16, [90, 33], 70)
    cfg, pages = lib.make_config(s, "bf16"), c.descriptor(lib)
    q = _q(np.random.default_rng(71), 2, s)
    t, k, v = c.table.cuda(), c.k.cuda(), c.v.cuda()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
    for decode in (True, False):
        if decode:
            lib.kpa_paged_decode(cfg, pages, 2, q.cuda(), _i32([90, 33]), t, k, v, 90, 0, 0, scale, out, ws)
        else:
            lib.kpa_paged_prefill(cfg, pages, 2, 2, q.cuda(), _i32([0, 1, 2]), _i32([89, 32]), t, k, v, 90, 0, 0, scale, out, ws)
        _no_error(lib)
        for b, n in enumerate((90, 33)):
            want, tol = pu.attention(c, b, pu.f64(q[b:b + 1]), [n - 1], 0, 0, scale, factored=decode)
            pu.assert_within(out[b:b + 1], want, tol, f"sequence {b}, decode {decode}")


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_of_many_magnitudes(fmt):
    """Tokens whose factors differ by powers of two up to 2^12, and tiny ones throughout."""
    lib = kpa()
    s = SPLITS["kpa_4x8_8x16_r2"]
    for level in (0, -10):
        c = pu.Cache(s, fmt, 32, [0, 0], 72, spare=8, stride=4)
        rng = np.random.default_rng(73)
        c.table[:, :4] = torch.arange(8, dtype=torch.int32).view(2, 4)
        for plane, pool, e in ((c.kp, c.k, s.e_k), (c.vp, c.v, s.e_v)):
            x = rng.standard_normal((256, e)) * np.exp2(rng.integers(-6, 7, (256, 1)) / 2 + level)
            plane.write(pool, np.arange(256) // 32, np.arange(256) % 32, x)
        cfg, pages = lib.make_config(s, "bf16"), c.descriptor(lib)
        q = _q(rng, 2, s)
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        out = torch.empty(2, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
        args = (c.table.cuda(), c.k.cuda(), c.v.cuda(), 128, 0, 0, 0.05, out, ws)
        for decode in (True, False):
            if decode:
                lib.kpa_paged_decode(cfg, pages, 2, q.cuda(), _i32([128, 117]), *args)
            else:
                lib.kpa_paged_prefill(cfg, pages, 2, 2, q.cuda(), _i32([0, 1, 2]), _i32([127, 116]), *args)
            _no_error(lib)
            for b, n in enumerate((128, 117)):
                want, tol = pu.attention(c, b, pu.f64(q[b:b + 1]), [n - 1], 0, 0, 0.05, factored=decode)
                pu.assert_within(out[b:b + 1], want, tol, f"level {level}, sequence {b}, decode {decode}")


def test_shared_pages():
    """Two sequences that share the pages of a common prefix."""
    lib = kpa()
    s = SPLITS["kpa_4x4_8x16_r2"]
    c = pu.Cache(s, "e4m3", 16, [64, 60], 74)
    c.table[1, :2] = c.table[0, :2]
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    q = _q(np.random.default_rng(75), 12, s)
    out = torch.empty(12, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    lib.kpa_paged_prefill(cfg, pages, 2, 12, q.cuda(), _i32([0, 4, 12]), _i32([60, 52]), c.table.cuda(), c.k.cuda(), c.v.cuda(),
                          64, 0, 0, scale, out, ws)
    _no_error(lib)
    for b, (lo, hi, p) in enumerate(((0, 4, 60), (4, 12, 52))):
        want, tol = pu.attention(c, b, pu.f64(q[lo:hi]), p + np.arange(hi - lo), 0, 0, scale)
        pu.assert_within(out[lo:hi], want, tol)


@pytest.mark.parametrize("name", ["kpa_4x4_8x16_r2", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
def test_positions_near_the_end_of_the_range(name):
    """Slots just below 2^31, reached through a window."""
    lib = kpa()
    s = SPLITS[name]
    page, stride = 4096, (1 << 19) - 1
    cfg, pages = lib.make_config(s, "bf16"), lib.make_pages(page, 3, stride, "e4m3")
    last = page * stride
    n, window = 70, 50
    start = last - n
    kb, vb = lib.kpa_paged_page_bytes(cfg, pages)
    k, v = (torch.full((3 * b,), 255, dtype=torch.uint8, device="cuda") for b in (kb, vb))
    table = torch.full((1, stride), -1, **I32)
    table[0, -1] = 1
    rng = np.random.default_rng(76)
    kf, vf = (torch.from_numpy(rng.standard_normal((n, e)) * 0.7).to(torch.bfloat16).cuda() for e in (s.e_k, s.e_v))
    lib.kpa_paged_append_factors(cfg, pages, 1, n, kf, vf, _i32([0, n]), _i32([start]), table, k, v)
    rk, rv = torch.empty_like(kf), torch.empty_like(vf)
    lib.kpa_paged_read_factors(cfg, pages, 1, n, _i32([0, n]), _i32([start]), table, k, v, rk, rv)
    _no_error(lib)
    want = pu.rotate(pu.f64(kf), s, start + np.arange(n))
    assert np.abs(pu.f64(rk) - want).max() <= 2.0 ** -4 * np.abs(want).max()
    c = pu.Cache(s, "e4m3", page, [0], 0, stride=2)
    c.records = lambda b, slots, *_: (pu.f64(rk)[slots], pu.f64(rv)[slots])
    rows, scale = 15, 1.0 / np.sqrt(s.dh)
    q = _q(rng, rows, s)
    out = torch.empty(rows, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    lib.kpa_paged_prefill(cfg, pages, 1, rows, q.cuda(), _i32([0, rows]), _i32([last - rows]), table, k, v, last, window, 0, scale,
                          out, ws)
    _no_error(lib)
    want, tol = pu.attention(c, 0, pu.f64(q), n - rows + np.arange(rows), window, 0, scale)
    pu.assert_within(out, want, tol, "prefill")
    lib.kpa_paged_decode(cfg, pages, 1, q[:1].cuda(), _i32([last]), table, k, v, last, window, 0, scale, out, ws)
    _no_error(lib)
    want, tol = pu.attention(c, 0, pu.f64(q[:1]), [n - 1], window, 0, scale, factored=True)
    pu.assert_within(out[:1], want, tol, "decode")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["kpa_4x8_8x16_r4", "kpa_4x4_8x8_r2", "tpa_32_64_r1"])
@pytest.mark.parametrize("length,window", [([3000, 1, 0, 17, 4001, 16], 0), ([9000, 1, 0, 17], 5000), ([0, 0, 0], 0),
                                           (list(range(0, 400, 2)), 0)], ids=["ragged", "window", "empty", "many"])
def test_decode_ragged(name, fmt, length, window):
    """One long sequence among short ones, empty batches, and more sequences than SMs: the
    blocks size the splits themselves."""
    _decode(kpa(), SPLITS[name], fmt, 64, length, window, 5 if window else 0, 26, max_len=max(max(length), 30000))


def test_bad_lengths_of_a_long_batch():
    lib = kpa()
    s = SPLITS["kpa_4x4_8x8_r2"]
    c = pu.Cache(s, "bf16", 64, [40, 40, 0], 27, stride=400)
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    q = _q(np.random.default_rng(28), 3, s)
    ws = torch.empty(max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, 3, 25600)), dtype=torch.uint8, device="cuda")
    args = (c.table.cuda(), c.k.cuda(), c.v.cuda(), 25600, 0, 0, scale)
    for bad in (-1, -2 ** 31):
        out = torch.full((3, s.h, s.dh), 5.0, dtype=torch.bfloat16, device="cuda")
        lib.kpa_paged_decode(cfg, pages, 3, q.cuda(), _i32([40, bad, 0]), *args, out, ws)
        assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
        want, tol = pu.attention(c, 0, pu.f64(q[:1]), [39], 0, 0, scale, factored=True)
        pu.assert_within(out[:1], want, tol)
        assert (out[1:] == 0).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("name", ["kpa_4x4_8x16_r2", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_served_requests(name, fmt, window, sinks):
    """Requests as a server runs them: prompts in chunks, then single tokens, each step's
    attention against the pool as it stands; pages that fall out of the window are given to
    another sequence."""
    lib = kpa()
    s = SPLITS[name]
    rng = np.random.default_rng(30)
    page, B, scale = 16, 3, 1.0 / np.sqrt(s.dh)
    steps = [[40, 7, 0], [33, 60, 1], [1, 1, 1], [1, 1, 50], [1, 1, 1], [1, 0, 1]]
    cfg = lib.make_config(s, "bf16")
    n_pages, stride, max_len = 30, 12, 192
    c = pu.Cache(s, fmt, page, [0] * B, 30, stride=stride)
    c.n_pages = n_pages
    c.kp, c.vp = pu.planes(s, fmt, n_pages, page)
    k, v = c.kp.empty().cuda(), c.vp.empty().cuda()
    pages = c.descriptor(lib)
    free, length = list(rng.permutation(n_pages)), [0] * B
    c.table[:] = -1
    for new in steps:
        for b in range(B):
            for i in range(-(-(length[b] + new[b]) // page)):
                first = max(0, length[b] - window + 1) if window else 0
                dead = window and (i + 1) * page <= first and i * page >= sinks
                if dead and c.table[b, i] >= 0:
                    free.insert(0, int(c.table[b, i]))
                    c.table[b, i] = -1
                if not dead and c.table[b, i] < 0:
                    c.table[b, i] = int(free.pop())
        cu = _cu(new)
        n = int(cu[-1])
        kf, vf = (torch.from_numpy(rng.standard_normal((n, e)) * 0.7).to(torch.bfloat16) for e in (s.e_k, s.e_v))
        q = _q(rng, n, s)
        table, start = c.table.cuda(), _i32(length)
        lib.kpa_paged_append_factors(cfg, pages, B, n, kf.cuda(), vf.cuda(), _i32(cu), start, table, k, v)
        out = torch.full((n, s.h, s.dh), float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(256, lib.kpa_paged_prefill_workspace_size(cfg, pages, B, n, max_len, window, sinks)),
                         dtype=torch.uint8, device="cuda")
        lib.kpa_paged_prefill(cfg, pages, B, n, q.cuda(), _i32(cu), start, table, k, v, max_len, window, sinks, scale,
                              out, ws)
        if max(new) == 1:                                         # the same rows through the decode
            rows = [cu[b] for b in range(B) if new[b]]
            alive = [b for b in range(B) if new[b]]
            qd, lens = q[rows].cuda(), _i32([length[b] + 1 for b in alive])
            od = torch.full_like(out, float("nan"))
            ws = torch.empty(max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, len(alive), max_len, window, sinks)),
                             dtype=torch.uint8, device="cuda")
            lib.kpa_paged_decode(cfg, pages, len(alive), qd, lens, table[alive].contiguous(), k, v, max_len, window, sinks,
                                 scale, od, ws)
        _no_error(lib)
        rk, rv = torch.empty(n, s.e_k, dtype=torch.bfloat16, device="cuda"), torch.empty(n, s.e_v, dtype=torch.bfloat16, device="cuda")
        lib.kpa_paged_read_factors(cfg, pages, B, n, _i32(cu), start, table, k, v, rk, rv)
        _no_error(lib)
        kc, vc = k.cpu(), v.cpu()
        for b in range(B):
            if new[b] == 0:
                continue
            pos = np.arange(length[b], length[b] + new[b])
            gk, gv = c.records(b, pos, kc, vc)
            assert np.array_equal(pu.f64(rk[cu[b]:cu[b + 1]]), gk) and np.array_equal(pu.f64(rv[cu[b]:cu[b + 1]]), gv)
            qb = pu.f64(q[cu[b]:cu[b + 1]])
            want, tol = pu.attention(c, b, qb, pos, window, sinks, scale, kc, vc)
            pu.assert_within(out[cu[b]:cu[b + 1]], want, tol, f"prefill of sequence {b}")
            if max(new) == 1:
                want, tol = pu.attention(c, b, qb, pos, window, sinks, scale, kc, vc, factored=True)
                pu.assert_within(od[alive.index(b)][None], want, tol, f"decode of sequence {b}")
            length[b] += new[b]


# ------------------------------------------------------------------ what the device checks
def _two(lib, fmt="bf16", page=16):
    s = SPLITS["kpa_4x4_8x16_r2"]
    c = pu.Cache(s, fmt, page, [40, 40], 40)
    return s, c, lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("entry", [-1, 10 ** 9, -2 ** 31])
def test_bad_page_is_reported(fmt, entry):
    """A page outside the pool: reported, nothing written there, other sequences right."""
    lib = kpa()
    s, c, cfg, pages, scale = _two(lib, fmt)
    table = c.table.clone()
    table[1, 1] = entry
    q = _q(np.random.default_rng(1), 2, s)
    want, tol = pu.attention(c, 0, pu.f64(q[:1]), [39], 0, 0, scale)
    k, v, t = c.k.cuda(), c.v.cuda(), table.cuda()
    out = torch.zeros(2, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    lib.kpa_paged_decode(cfg, pages, 2, q.cuda(), _i32([40, 40]), t, k, v, 40, 0, 0, scale, out, ws)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    pu.assert_within(out[:1], want, tol)
    lib.kpa_paged_prefill(cfg, pages, 2, 2, q.cuda(), _i32([0, 1, 2]), _i32([39, 39]), t, k, v, 40, 0, 0, scale, out, ws)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    pu.assert_within(out[:1], want, tol)
    rk = torch.full((80, s.e_k), 7.0, dtype=torch.bfloat16, device="cuda")
    rv = torch.full((80, s.e_v), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.kpa_paged_read_factors(cfg, pages, 2, 80, _i32([0, 40, 80]), _i32([0, 0]), t, k, v, rk, rv)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    wk, _ = c.records(0, np.arange(40))
    assert np.array_equal(pu.f64(rk[:40]), wk)
    assert (rk[56:72] == 0).all() and (rv[56:72] == 0).all()      # slots 16 .. 31 of sequence 1
    before = k.clone(), v.clone()
    kf, vf = rk[:32].clone().fill_(1.0), rv[:32].clone().fill_(1.0)
    lib.kpa_paged_append_factors(cfg, pages, 2, 16, kf, vf, _i32([0, 0, 16]), _i32([0, 16]), t, k, v)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    assert torch.equal(before[0].view(torch.uint8), k.view(torch.uint8))
    assert torch.equal(before[1].view(torch.uint8), v.view(torch.uint8))


@pytest.mark.parametrize("cu,start", [([0, 5, 3], [0, 0]), ([0, 2, 900], [0, 0]), ([-4, 2, 4], [0, 0]), ([0, 2, 4], [0, -3]),
                                      ([0, 2, 4], [0, 10 ** 6]), ([0, 2, 4], [0, 2 ** 31 - 1])], ids=str)
def test_bad_rows_are_reported(cu, start):
    lib = kpa()
    s, c, cfg, pages, scale = _two(lib)
    q = _q(np.random.default_rng(2), 4, s)
    k, v, t = c.k.cuda(), c.v.cuda(), c.table.cuda()
    out = torch.full((4, s.h, s.dh), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    lib.kpa_paged_prefill(cfg, pages, 2, 4, q.cuda(), _i32(cu), _i32(start), t, k, v, 40, 0, 0, scale, out, ws)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    if start[1] != 0:                                             # rows without a slot: zeros
        want, tol = pu.attention(c, 0, pu.f64(q[:2]), [0, 1], 0, 0, scale)
        pu.assert_within(out[:2], want, tol)
        assert (out[2:] == 0).all()
    rk = torch.full((4, s.e_k), 7.0, dtype=torch.bfloat16, device="cuda")
    rv = torch.full((4, s.e_v), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.kpa_paged_read_factors(cfg, pages, 2, 4, _i32(cu), _i32(start), t, k, v, rk, rv)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    if start[1] != 0:
        assert (rk[2:] == 0).all() and np.array_equal(pu.f64(rv[:2]), c.records(0, np.arange(2))[1])
    before = k.clone()
    lib.kpa_paged_append_factors(cfg, pages, 2, 4, rk, rv, _i32(cu), _i32(start), t, k, v)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    bad = 0 if cu[0] < 0 else 1                                   # the sequence that is skipped
    where, inside = c.where(bad, np.arange(40))
    assert torch.equal(c.kp.raw(before, where, inside), c.kp.raw(k, where, inside))


def test_bad_lengths_are_reported():
    lib = kpa()
    s, c, cfg, pages, scale = _two(lib)
    q = _q(np.random.default_rng(3), 2, s)
    out = torch.full((2, s.h, s.dh), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    lib.kpa_paged_decode(cfg, pages, 2, q.cuda(), _i32([41, -1]), c.table.cuda(), c.k.cuda(), c.v.cuda(), 40, 0, 0, scale,
                         out, ws)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    want, tol = pu.attention(c, 0, pu.f64(q[:1]), [39], 0, 0, scale)
    pu.assert_within(out[:1], want, tol)
    assert (out[1] == 0).all()


def test_nonfinite_values_are_reported():
    lib = kpa()
    s, c, cfg, pages, scale = _two(lib)
    pg, inside = c.where(1, np.arange(40))
    c.vp._view(c.v)[int(pg[7]), int(inside[7]) // 8, 0, int(inside[7]) % 8] = float("inf")
    q = _q(np.random.default_rng(4), 2, s)
    out = torch.zeros(2, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    want, tol = pu.attention(c, 0, pu.f64(q[:1]), [39], 0, 0, scale)
    args = (c.table.cuda(), c.k.cuda(), c.v.cuda(), 40, 0, 0, scale, out, ws)
    lib.kpa_paged_decode(cfg, pages, 2, q.cuda(), _i32([40, 40]), *args)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    pu.assert_within(out[:1], want, tol)
    lib.kpa_paged_prefill(cfg, pages, 2, 2, q.cuda(), _i32([0, 1, 2]), _i32([39, 39]), *args)
    assert lib.kpa_read_device_error() == lib.KPA_ERR_DEVICE_CHECK
    pu.assert_within(out[:1], want, tol)
    # and out of the window it changes nothing
    lib.kpa_paged_decode(cfg, pages, 2, q.cuda(), _i32([40, 40]), *args[:4], 32, 0, scale, out, ws)
    _no_error(lib)
    want, tol = pu.attention(c, 1, pu.f64(q[1:]), [39], 32, 0, scale)
    pu.assert_within(out[1:], want, tol)


def test_short_workspace_is_refused():
    lib = kpa()
    s, c, cfg, pages, scale = _two(lib)
    big = dataclasses.replace(s)
    pages = lib.make_pages(16, 4000, 4000, "bf16")
    need = lib.kpa_paged_decode_workspace_size(lib.make_config(big, "bf16"), pages, 1, 64000)
    assert need > 256
    x = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    for ws, size in ((None, 0), (x, 256)):
        with pytest.raises(lib.KpaError) as e:
            lib.kpa_paged_decode(cfg, pages, 1, x, x, x, x, x, 64000, 0, 0, scale, x, ws, size)
        assert e.value.status == lib.KPA_ERR_WORKSPACE


# ------------------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("fmt", FORMATS)
def test_other_stream_and_graph(fmt):
    """Two captured steps that share one workspace, replayed with new lengths and queries on a
    stream of their own, give what eager calls give, bit for bit."""
    lib = kpa()
    s = SPLITS["kpa_4x8_8x16_r2"]
    c = pu.Cache(s, fmt, 32, [3000, 700], 50)
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    k, v, t = c.k.cuda(), c.v.cuda(), c.table.cuda()
    rng = np.random.default_rng(51)
    q, lens = _q(rng, 2, s).cuda(), _i32([2990, 650])
    ws = torch.empty(max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, 2, 3000),
                         lib.kpa_paged_decode_workspace_size(cfg, pages, 2, 3000, 64, 4)), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(2, s.h, s.dh, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(out, window, sinks):
        lib.kpa_paged_decode(cfg, pages, 2, q, lens, t, k, v, 3000, window, sinks, scale, out, ws)

    step(outs[0], 0, 0)
    _no_error(lib)
    graphs = []
    for out, mask in zip(outs, ((0, 0), (64, 4))):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(out, *mask)
        graphs.append(g)
    side = torch.cuda.Stream()
    for length in ([2999, 700], [1, 64], [3000, 0]):
        lens.copy_(_i32(length))
        q.copy_(_q(rng, 2, s).cuda())
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
        side.synchronize()
        got = [o.clone() for o in outs]
        step(outs[0], 0, 0)
        step(outs[1], 64, 4)
        _no_error(lib)
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace and output."""
    lib = kpa()
    s = SPLITS["tpa_16_64_r2"]
    c = pu.Cache(s, "bf16", 64, [5000, 4000], 52)
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    k, v, t = c.k.cuda(), c.v.cuda(), c.table.cuda()
    q, cu, start, lens = _q(np.random.default_rng(53), 40, s).cuda(), _i32([0, 20, 40]), _i32([4980, 3980]), _i32([5000, 4000])
    runs = []
    for i in range(2):
        out = torch.empty(40, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
        od = torch.empty(2, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(256, lib.kpa_paged_prefill_workspace_size(cfg, pages, 2, 40, 5000),
                             lib.kpa_paged_decode_workspace_size(cfg, pages, 2, 5000)), dtype=torch.uint8, device="cuda")
        runs.append((torch.cuda.Stream(), out, od, ws))
    torch.cuda.synchronize()
    for _ in range(10):
        for stream, out, od, ws in runs:
            lib.kpa_paged_prefill(cfg, pages, 2, 40, q, cu, start, t, k, v, 5000, 0, 0, scale, out, ws, stream=stream)
            lib.kpa_paged_decode(cfg, pages, 2, q, lens, t, k, v, 5000, 0, 0, scale, od, ws, stream=stream)
    _no_error(lib)
    assert torch.equal(runs[0][1], runs[1][1]) and torch.equal(runs[0][2], runs[1][2])
    want, tol = pu.attention(c, 0, pu.f64(q[19:20]), [4999], 0, 0, scale)
    pu.assert_within(runs[0][1][19:20], want, tol)


def test_far_page_offsets():
    """A pool plane above 2^32 bytes, with the sequence in its last pages."""
    lib = kpa()
    s = SPLITS["kpa_4x8_8x16_r4"]
    page = 4096
    kb, vb = lib.kpa_paged_page_bytes(lib.make_config(s, "bf16"), lib.make_pages(page, 1, 1, "bf16"))
    n_pages = (1 << 32) // kb + 3
    k = torch.empty(n_pages * kb // 2, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(n_pages * vb // 2, dtype=torch.bfloat16, device="cuda")
    cfg, pages = lib.make_config(s, "bf16"), lib.make_pages(page, n_pages, 2, "bf16")
    rng = np.random.default_rng(60)
    n = 50
    kf = torch.from_numpy(rng.standard_normal((n, s.e_k)) * 0.7).to(torch.bfloat16).cuda()
    vf = torch.from_numpy(rng.standard_normal((n, s.e_v)) * 0.7).to(torch.bfloat16).cuda()
    table = _i32([[n_pages - 1, n_pages - 2]])
    start = page - 20
    lib.kpa_paged_append_factors(cfg, pages, 1, n, kf, vf, _i32([0, n]), _i32([start]), table, k, v)
    rk, rv = torch.empty_like(kf), torch.empty_like(vf)
    lib.kpa_paged_read_factors(cfg, pages, 1, n, _i32([0, n]), _i32([start]), table, k, v, rk, rv)
    q = _q(rng, 1, s)
    out = torch.empty(1, s.h, s.dh, dtype=torch.bfloat16, device="cuda")
    scale = 1.0 / np.sqrt(s.dh)
    ws = torch.empty(max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, 1, 8192, n, 0)), dtype=torch.uint8, device="cuda")
    lib.kpa_paged_decode(cfg, pages, 1, q.cuda(), _i32([start + n]), table, k, v, 8192, n, 0, scale, out, ws)
    _no_error(lib)
    assert torch.equal(rv, vf)
    c = pu.Cache(s, "bf16", page, [0], 0, stride=2)
    c.records = lambda b, slots, *_: (pu.f64(rk)[slots - start], pu.f64(rv)[slots - start])
    want, tol = pu.attention(c, 0, pu.f64(q), [start + n - 1], n, 0, scale)
    pu.assert_within(out, want, tol)
