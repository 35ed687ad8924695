"""Long paged caches, slot by slot: for each 16-slot group a query that selects one slot of it, so
that a group, a page or a split left out, met twice or taken from elsewhere shows."""
import numpy as np
import pytest
import torch

import paged_marks as pm
import paged_util as pu
from gpu_util import kpa
from workloads import Shape

SPLITS = {
    "kpa_4x8_8x16_r2": Shape(h1=4, h2=8, d1=8, d2=16, r_k=2, r_v=2),
    "kpa_4x8_8x16_r4": Shape(h1=4, h2=8, d1=8, d2=16, r_k=4, r_v=4),
    "kpa_4x4_8x8_r2": Shape(h1=4, h2=4, d1=8, d2=8, r_k=2, r_v=2),
    "tpa_16_64_r2": Shape(h1=16, h2=1, d1=1, d2=64, r_k=2, r_v=2),
    "tpa_32_64_r1": Shape(h1=32, h2=1, d1=1, d2=64, r_k=1, r_v=1),
    "kpa_3x2_4x6_r2": Shape(h1=3, h2=2, d1=4, d2=6, r_k=2, r_v=2),          # the kernel of every split
}
FORMATS = ["bf16", "e4m3"]
MARKED = 0.99                      # a query that selects its slot gives it this weight


def _assert_marked(weight, ranges):
    """Every row gives its slot the weight in some head (elsewhere a larger key may win)."""
    marked = (weight > MARKED).any(-1)
    assert marked.all(), f"rows of {ranges[(~marked).cpu().numpy()]} select nothing"


def _check(got, q, pos, K, V, VA, window, sinks, scale, targets):
    for i in range(0, len(q), 32):
        j = slice(i, i + 32)
        want, tol, weight = pm.attention(q[j], pos[j], K, V, VA, window, sinks, scale)
        _assert_marked(weight, targets[j])
        over = (got[j].double() - want).abs() - tol
        worst = over.flatten(1).amax(-1)
        assert got[j].isfinite().all() and (worst <= 0).all(), \
            f"slots {targets[j][(worst > 0).cpu().numpy()]}: {worst.max()} past the bound"


# ------------------------------------------------------------------ the bound, on the CPU
@pytest.mark.parametrize("name", sorted(SPLITS))
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_lost_group_fails_the_bound(name, fmt):
    """The definition itself with one 16-slot group left out, a page read twice, or a slot taken
    from elsewhere: past the bound for the queries whose slots it touches."""
    s, n, scale = SPLITS[name], 1003, 1.0 / np.sqrt(SPLITS[name].dh)
    c = pu.Cache(s, fmt, 64, [n], 1)
    K, V, VA = pm.planes(c, 0, n, "cpu")
    targets = pm.groups(n)[::3]
    q = pm.select(K, targets, scale)
    pos = np.full(len(targets), n - 1)
    want, tol, weight = pm.attention(q, pos, K, V, VA, 0, 0, scale)
    _assert_marked(weight, targets)
    slots = torch.arange(n)
    for m in range(0, len(targets), 5):
        hit, t = slice(m, m + 1), int(targets[m][0])
        lost, _, _ = pm.attention(q[hit], pos[hit], K, V, VA, 0, 0, scale, hidden=slots // 16 == t // 16)
        assert ((lost - want[hit]).abs() > 4 * tol[hit]).any()
        page = t // 64 * 64
        other = 0 if page else 64
        take = slots.clone()
        take[page:page + 64] = (torch.arange(other, other + 64))[:min(64, n - page)]      # another page in its place
        wrong, _, _ = pm.attention(q[hit], pos[hit], K[:, take], V[:, take], VA[:, take], 0, 0, scale)
        assert ((wrong - want[hit]).abs() > 4 * tol[hit]).any()


# ------------------------------------------------------------------ the kernels
def _cache(name, fmt, page, n, seed, batch, stride):
    """A cache of one sequence whose pages `batch` sequences share, on the GPU."""
    s = SPLITS[name]
    c = pu.Cache(s, fmt, page, [n], seed, stride=stride)
    table = c.table[:1].clone()
    table[0, -(-n // page):] = -1
    return c, c.k.cuda(), c.v.cuda(), table.expand(batch, -1).contiguous().cuda(), pm.planes(c, 0, n, "cuda")


# how the parts of a sequence are merged depends on the batch and the lengths: one sequence over every
# SM and a second kernel; a cluster per sequence; blocks that size the parts themselves; a window
DECODES = {"parts": dict(batch=1, n=9003, max_len=9003, window=0, sinks=0),
           "cluster": dict(batch=8, n=1027, max_len=1027, window=0, sinks=0),
           "sized": dict(batch=16, n=5003, max_len=60000, window=0, sinks=0),
           "window": dict(batch=2, n=9003, max_len=9003, window=2500, sinks=200),
           "one part": dict(batch=300, n=700, max_len=700, window=0, sinks=0)}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(SPLITS))
@pytest.mark.parametrize("how", sorted(DECODES))
def test_decode_meets_every_group(how, name, fmt):
    lib = kpa()
    s, page, p = SPLITS[name], 48, DECODES[how]
    batch, n, window, sinks = p["batch"], p["n"], p["window"], p["sinks"]
    stride = -(-p["max_len"] // page)
    c, k, v, table, (K, V, VA) = _cache(name, fmt, page, n, 3, batch, stride)
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    t = pm.groups(n, pu.visible(n - 1, n, window, sinks))
    t = np.resize(t, (-(-len(t) // batch) * batch, 2))
    q = pm.select(K, t, scale)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    ws = torch.full((max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, batch, p["max_len"], window, sinks)),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full((len(t), s.h, s.dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i in range(0, len(t), batch):
        lib.kpa_paged_decode(cfg, pages, batch, q[i:i + batch].contiguous(), lens, table, k, v, p["max_len"], window, sinks, scale,
                             out[i:i + batch], ws)
    torch.cuda.synchronize()
    assert lib.kpa_read_device_error() == 0
    _check(out, q, np.full(len(t), n - 1), K, V, VA, window, sinks, scale, t)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["kpa_4x8_8x16_r2", "tpa_16_64_r2"])
def test_decode_merges_differ(name):
    """The calls above take different ways: no workspace with a cluster or one part, and partials
    of different sizes otherwise."""
    lib = kpa()
    cfg = lib.make_config(SPLITS[name], "bf16")
    size = {}
    for how, p in DECODES.items():
        pages = lib.make_pages(48, 4000, -(-p["max_len"] // 48), "bf16")
        size[how] = lib.kpa_paged_decode_workspace_size(cfg, pages, p["batch"], p["max_len"], p["window"], p["sinks"])
    assert size["cluster"] == size["one part"] == 0
    row = SPLITS[name].h * (SPLITS[name].dh + 2) * 4
    assert size["parts"] >= 20 * row                              # one sequence in twenty parts or more
    assert size["sized"] >= 48 * row                              # three parts a sequence or more


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(SPLITS))
@pytest.mark.parametrize("rows,past,window,sinks", [(17, 4001, 0, 0), (300, 3790, 0, 0), (130, 3001, 1100, 300)],
                         ids=["short", "long", "window"])
def test_prefill_meets_every_group(rows, past, window, sinks, name, fmt):
    lib = kpa()
    s, page, n = SPLITS[name], 48, rows + past
    c, k, v, table, (K, V, VA) = _cache(name, fmt, page, n, 5, 1, -(-n // page))
    cfg, pages, scale = lib.make_config(s, "bf16"), c.descriptor(lib), 1.0 / np.sqrt(s.dh)
    see = pu.visible(past, past + 1, window, sinks)               # what the first row sees, and the last
    t = pm.groups(past + 1, see & pu.visible(n - 1, n, window, sinks)[:past + 1])
    t = np.resize(t, (-(-len(t) // rows) * rows, 2))
    q = pm.select(K, t, scale)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, start = torch.tensor([0, rows], **i32), torch.tensor([past], **i32)
    ws = torch.full((max(256, lib.kpa_paged_prefill_workspace_size(cfg, pages, 1, rows, n, window, sinks)),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full((len(t), s.h, s.dh), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i in range(0, len(t), rows):
        lib.kpa_paged_prefill(cfg, pages, 1, rows, q[i:i + rows].contiguous(), cu, start, table, k, v, n, window, sinks, scale,
                              out[i:i + rows], ws)
    torch.cuda.synchronize()
    assert lib.kpa_read_device_error() == 0
    pos = np.resize(past + np.arange(rows), len(t))
    _check(out, q, pos, K, V, VA, window, sinks, scale, t)
