"""Paged attention on the GPU over magnitudes, against the definition in 64 bits: factors whose A
and B differ by powers of two, values near fp16's largest, small ones, and queries far from 1."""
import numpy as np
import pytest
import torch

import paged_marks as pm
import paged_util as pu
from gpu_util import kpa
from workloads import Shape

pytestmark = pytest.mark.gpu

# every split of the single-token kernel of its own, and two that run on the chunk kernel
SPLITS = {
    "kpa_4x4_8x16_r2": Shape(h1=4, h2=4, d1=8, d2=16, r_k=2, r_v=2),
    "kpa_4x8_8x16_r4": Shape(h1=4, h2=8, d1=8, d2=16, r_k=4, r_v=4),
    "kpa_4x4_8x16_r4": Shape(h1=4, h2=4, d1=8, d2=16, r_k=4, r_v=4),
    "kpa_4x8_8x16_r2": Shape(h1=4, h2=8, d1=8, d2=16, r_k=2, r_v=2),
    "kpa_4x4_8x8_r2": Shape(h1=4, h2=4, d1=8, d2=8, r_k=2, r_v=2),
    "kpa_2x8_8x8_r2": Shape(h1=2, h2=8, d1=8, d2=8, r_k=2, r_v=2),
    "kpa_8x2_8x8_r2": Shape(h1=8, h2=2, d1=8, d2=8, r_k=2, r_v=2),
    "tpa_16_64_r2": Shape(h1=16, h2=1, d1=1, d2=64, r_k=2, r_v=2),
    "tpa_32_64_r1": Shape(h1=32, h2=1, d1=1, d2=64, r_k=1, r_v=1),
    "tpa_16_128_r2": Shape(h1=16, h2=1, d1=1, d2=128, r_k=2, r_v=2),
    "kpa_3x2_4x6_r2": Shape(h1=3, h2=2, d1=4, d2=6, r_k=2, r_v=2),
    "kpa_4x4_8x16_rk3_rv1": Shape(h1=4, h2=4, d1=8, d2=16, r_k=3, r_v=1),
}
NAMES = sorted(SPLITS)
FORMATS = ["bf16", "e4m3"]
N = 45                                  # tokens: two whole groups of 16 and part of one


def _cache(s, fmt, seed, scale_k=(1.0, 1.0), scale_v=(1.0, 1.0), fill=None):
    """One sequence of N records whose A and B factors are scaled as given (or what `fill` makes of
    them)."""
    c = pu.Cache(s, fmt, 32, [0], seed, spare=2, stride=2)
    c.table[0, :2] = torch.tensor([1, 0], dtype=torch.int32)
    rng = np.random.default_rng(seed)
    slots = np.arange(N)
    for plane, pool, e, (fa, fb) in ((c.kp, c.k, s.e_k, scale_k), (c.vp, c.v, s.e_v, scale_v)):
        x = rng.standard_normal((N, e)) * 0.7
        x[:, :plane.a] *= fa
        x[:, plane.a:] *= fb
        if fill:
            fill(plane, x, pool is c.v)
        plane.write(pool, c.table[0].numpy()[slots // 32], slots % 32, x)
    return c


def _attend(lib, c, q, scale, decode, error=0):
    s = c.s
    cfg, pages = lib.make_config(s, "bf16"), c.descriptor(lib)
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    out = torch.full((1, s.h, s.dh), 7.0, dtype=torch.bfloat16, device="cuda")
    t, k, v = c.table.cuda(), c.k.cuda(), c.v.cuda()
    if decode:
        lib.kpa_paged_decode(cfg, pages, 1, q.cuda(), torch.tensor([N], **i32), t, k, v, N, 0, 0, scale, out, ws)
    else:
        lib.kpa_paged_prefill(cfg, pages, 1, 1, q.cuda(), torch.tensor([0, 1], **i32), torch.tensor([N - 1], **i32), t, k, v, N, 0, 0,
                              scale, out, ws)
    torch.cuda.synchronize()
    assert lib.kpa_read_device_error() == error
    return out.cpu()


def _check(lib, c, q, scale, decode, floor):
    want, tol, _ = pm.attention(q, [N - 1], *pm.planes(c, 0, N, "cpu"), 0, 0, scale, floor=floor)
    got = _attend(lib, c, q, scale, decode)
    pu.assert_within(got, want.numpy(), tol.numpy(), "decode" if decode else "prefill")


def _q(s, seed, scale=0.3):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((1, s.h, s.dh)) * scale).to(torch.bfloat16)


def _factors(lib, s, fmt):
    """Whether the single-token kernel of its own takes this split."""
    return lib.kpa_paged_decode_kernel_kind(lib.make_config(s, "bf16"), lib.make_pages(16, 1, 1, fmt)) == "factors"


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("power", [-30, -14, 16, 24])
def test_unbalanced_factors(power, name, fmt, decode):
    """Keys and values of ordinary size from A factors 2^power as large and B factors 2^-power."""
    lib, s = kpa(), SPLITS[name]
    f = (2.0 ** power, 2.0 ** -power)
    c = _cache(s, fmt, 1, f, f)
    _check(lib, c, _q(s, 2), 1.0 / np.sqrt(s.dh), decode, floor=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
def test_unbalanced_tokens(name, fmt):
    """Each token's factors unbalanced by a power of its own."""
    lib, s = kpa(), SPLITS[name]
    power = np.random.default_rng(3).integers(-28, 29, (N, 1)).astype(np.float64)

    def fill(plane, x, _):
        x[:, :plane.a] *= np.exp2(power)
        x[:, plane.a:] *= np.exp2(-power)

    c = _cache(s, fmt, 4, fill=fill)
    for decode in (True, False):
        _check(lib, c, _q(s, 5), 1.0 / np.sqrt(s.dh), decode, floor=True)


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("a,b", [(240.0, 260.0), (2.0 ** 12, 15.0), (15.0, 2.0 ** 12)])
def test_values_near_the_largest(a, b, name, fmt, decode):
    """Rebuilt values just inside fp16's range (65504): right, and no error reported."""
    lib, s = kpa(), SPLITS[name]
    rng = np.random.default_rng(6)

    def fill(plane, x, values):
        if not values:
            return
        ea = s.h1 * s.d1
        sign = rng.choice([-1.0, 1.0], x.shape)
        x[:, :plane.a] = a * sign[:, :plane.a]
        x[:, ea:plane.a] = 0.0                                     # one rank: the rebuilt sum is a b
        x[:, plane.a:] = b * sign[:, plane.a:]

    c = _cache(s, fmt, 7, fill=fill)
    _check(lib, c, _q(s, 8), 1.0 / np.sqrt(s.dh), decode, floor=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("power", [-5, -10])
def test_small_values(power, name, fmt):
    """Factors of 2^power: the single-token kernel keeps its relative precision (values to 2^-20)."""
    lib, s = kpa(), SPLITS[name]
    if not _factors(lib, s, fmt):
        pytest.skip("the chunk kernels round a rebuilt value to fp16")
    c = _cache(s, fmt, 9, scale_v=(2.0 ** power, 2.0 ** power))
    _check(lib, c, _q(s, 10), 1.0 / np.sqrt(s.dh), True, floor=False)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("power", [-16, -30, -50])
def test_tiny_bf16_values(power, name):
    """Over a bf16 pool the single-token kernel has no smallest value of its own."""
    lib, s = kpa(), SPLITS[name]
    if not _factors(lib, s, "bf16"):
        pytest.skip("the chunk kernels round a rebuilt value to fp16")
    c = _cache(s, "bf16", 11, scale_v=(2.0 ** power, 2.0 ** power))
    _check(lib, c, _q(s, 12), 1.0 / np.sqrt(s.dh), True, floor=False)


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("power", [-100, -20, 18, 100])
def test_queries_far_from_one(power, name, fmt, decode):
    """A query of any size whose scores are ordinary, as sm_scale takes its size back."""
    lib, s = kpa(), SPLITS[name]
    c = _cache(s, fmt, 13)
    q = _q(s, 14, 0.3 * 2.0 ** power)
    _check(lib, c, q, 4.0 / np.sqrt(s.dh) * 2.0 ** -power, decode, floor=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
def test_query_elements_of_many_sizes(name, fmt):
    """Elements of one query that differ by powers of two up to 2^16, and a head of zeros."""
    lib, s = kpa(), SPLITS[name]
    c = _cache(s, fmt, 15)
    rng = np.random.default_rng(16)
    q = _q(s, 17).double() * torch.from_numpy(np.exp2(rng.integers(-16, 1, (1, s.h, s.dh))))
    q[0, s.h // 2] = 0
    _check(lib, c, q.to(torch.bfloat16), 8.0 / np.sqrt(s.dh), True, floor=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_bad_query_element_stays_in_its_head(bad, name, fmt):
    """A query element that is not finite: reported, and the other heads are right."""
    lib, s = kpa(), SPLITS[name]
    c = _cache(s, fmt, 18)
    q, scale = _q(s, 19), 4.0 / np.sqrt(s.dh)
    want, tol, _ = pm.attention(q, [N - 1], *pm.planes(c, 0, N, "cpu"), 0, 0, scale)
    q[0, 1, 3] = bad
    for decode in (True, False):
        got = _attend(lib, c, q, scale, decode, lib.KPA_ERR_DEVICE_CHECK)
        rest = [h for h in range(s.h) if h != 1]
        pu.assert_within(got[:, rest], want[:, rest].numpy(), tol[:, rest].numpy(), "decode" if decode else "prefill")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("plane", ["k", "v"])
@pytest.mark.parametrize("part", ["A", "B"])
def test_a_bad_value_of_any_slot_is_reported(part, plane, name, fmt):
    """A NaN in any place of a 16-slot group, in the first factor or the last, and an infinity among
    the values (a key's may give a score of -inf, whose weight is 0)."""
    lib, s = kpa(), SPLITS[name]
    q, scale = _q(s, 20), 1.0 / np.sqrt(s.dh)
    for slot in range(13, 34):
        def fill(p, x, values):
            if values == (plane == "v"):
                bad = np.nan if plane == "k" or slot % 2 else (np.inf if slot % 3 else -np.inf)
                x[slot, p.a - 1 if part == "A" else p.a] = bad
        c = _cache(s, fmt, 21, fill=fill)
        for decode in (True, False):
            _attend(lib, c, q, scale, decode, lib.KPA_ERR_DEVICE_CHECK)


@pytest.mark.parametrize("bits", [0x7FC00000, 0x7FFFFFFF, -0x400000, -1], ids=hex)
def test_the_polynomial_exponential_of_a_nan_is_no_fp16(bits):
    """So a score that is NaN does not give a weight of 0."""
    lib = kpa()
    x = torch.tensor([bits] * 4, dtype=torch.int32, device="cuda").view(torch.float32)
    y = torch.zeros_like(x)
    lib.kpa_test_exp2_poly(x, y)
    assert not y.to(torch.float16).isfinite().any()
