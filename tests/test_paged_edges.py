"""The paged cache at the ends of its arguments: records longer than a block, the largest windows
and sink counts."""
import numpy as np
import pytest
import torch

import paged_marks as pm
import paged_util as pu
from gpu_util import kpa
from test_paged import FORMATS, SPLITS, _append, _check_records, _cu, _i32, _no_error
from workloads import Shape

pytestmark = pytest.mark.gpu

# more than 1024 elements a record, so that a block takes it in pieces; an odd A part in the second
LONG = {"kpa_4x8_8x16_r9": Shape(h1=4, h2=8, d1=8, d2=16, r_k=9, r_v=7),
        "tpa_61_64_r17": Shape(h1=61, h2=1, d1=1, d2=64, r_k=17, r_v=9),
        "kpa_2x2_8x64_r32": Shape(h1=2, h2=2, d1=8, d2=64, r_k=32, r_v=1)}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(LONG))
def test_append_long_records(name, fmt):
    lib = kpa()
    assert LONG[name].e_k > 1024
    start, new = [0, 5, 16, 31], [1, 40, 16, 3]
    r = _append(lib, LONG[name], fmt, 32, start, new, 80)
    _no_error(lib)
    _check_records(*r, start)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(LONG))
def test_read_long_records(name, fmt):
    lib, s = kpa(), LONG[name]
    c = pu.Cache(s, fmt, 48, [77, 5], 81)
    start, new = [3, 0], [70, 5]
    cu = _cu(new) + 2
    rows = int(cu[-1]) + 3
    kf = torch.full((rows, s.e_k), 7.0, dtype=torch.bfloat16, device="cuda")
    vf = torch.full((rows, s.e_v), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.kpa_paged_read_factors(lib.make_config(s, "bf16"), c.descriptor(lib), 2, rows, _i32(cu), _i32(start), c.table.cuda(),
                               c.k.cuda(), c.v.cuda(), kf, vf)
    _no_error(lib)
    for b in range(2):
        wk, wv = c.records(b, np.arange(start[b], start[b] + new[b]))
        assert np.array_equal(pu.f64(kf[cu[b]:cu[b + 1]]), wk) and np.array_equal(pu.f64(vf[cu[b]:cu[b + 1]]), wv)
    for x in (kf, vf):
        assert (x[:2] == 7).all() and (x[rows - 3:] == 7).all()


def test_tiles_of_a_batch_past_32_bits():
    """The blocks of a long batch size its parts from a 32-bit sum of tiles: a batch that may have
    more (pages shared, so that it fits) takes one part a sequence, which needs no workspace."""
    lib, page = kpa(), 4096
    pages = lib.make_pages(page, 10, (1 << 19) - 1, "bf16")
    for name in ("kpa_4x4_8x16_r2", "tpa_16_64_r2"):
        cfg = lib.make_config(SPLITS[name], "bf16")
        assert lib.kpa_paged_decode_workspace_size(cfg, pages, 200, 1 << 20) > 0
        assert lib.kpa_paged_decode_workspace_size(cfg, pages, 256, page * ((1 << 19) - 1)) == 0
        assert lib.kpa_paged_decode_workspace_size(cfg, pages, 256, page * ((1 << 19) - 1), 5000, 4) > 0


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["kpa_4x4_8x16_r2", "tpa_16_64_r2", "kpa_3x2_4x6_r2"])
@pytest.mark.parametrize("window,sinks", [(16, TOP), (TOP, TOP), (TOP, 0), (1, 700), (16, 5000)], ids=str)
def test_largest_windows_and_sinks(window, sinks, name, fmt):
    """Sink counts and windows beyond the cache, up to the type's largest: every earlier slot is
    seen."""
    lib, n, rows = kpa(), 700, 40
    s = SPLITS[name]
    c = pu.Cache(s, fmt, 48, [n], 82)
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    K, V, VA = pm.planes(c, 0, n, "cpu")
    t = pm.groups(n - rows)[:rows]
    q = pm.select(K, t, scale)
    assert len(t) == rows
    pos = n - rows + np.arange(rows)
    want, tol, _ = pm.attention(q, pos, K, V, VA, 0, 0, scale)     # every slot up to the row's own
    tab, k, v = c.table.cuda(), c.k.cuda(), c.v.cuda()
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, s.h, s.dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.kpa_paged_prefill(cfg, pages, 1, rows, q.cuda(), _i32([0, rows]), _i32([n - rows]), tab, k, v, n, window, sinks, scale, out, ws)
    _no_error(lib)
    pu.assert_within(out, want.numpy(), tol.numpy(), "prefill")
    for i in (0, rows - 1):
        lib.kpa_paged_decode(cfg, pages, 1, q[i:i + 1].cuda(), _i32([int(pos[i]) + 1]), tab, k, v, n, window, sinks, scale, out[:1], ws)
        _no_error(lib)
        pu.assert_within(out[:1], want[i:i + 1].numpy(), tol[i:i + 1].numpy(), "decode")
