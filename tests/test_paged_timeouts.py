"""A copy of the paged decode that never arrives: its bounded wait runs out, the block lets its other
copies land and returns, the error word says so, and the next call is right (no GPU fault)."""
import numpy as np
import pytest
import torch

from gpu_util import kpa
from workloads import Shape

pytestmark = pytest.mark.gpu

SPLITS = {"kpa_4x8_8x16_r2": Shape(h1=4, h2=8, d1=8, d2=16, r_k=2, r_v=2),
          "tpa_16_64_r2": Shape(h1=16, h2=1, d1=1, d2=64, r_k=2, r_v=2)}
# one sequence in parts, a cluster per sequence, parts that the blocks size; a tile of the first ring
# and one behind it
CALLS = {"parts": (1, 200000, (0, 1, 2, 3)), "cluster": (8, 8200, (0, 1, 2)), "sized": (16, 40000, (0, 1, 2, 5))}


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", sorted(SPLITS))
@pytest.mark.parametrize("how", sorted(CALLS))
def test_paged_decode_wait_that_runs_out(how, name, fmt):
    lib = kpa()
    s = SPLITS[name]
    batch, n, tiles = CALLS[how]
    page, n_pages = 64, 9                                         # pages that all sequences share
    stride = -(-n // page)
    cfg, pages = lib.make_config(s, "bf16"), lib.make_pages(page, n_pages, stride, fmt)
    g = torch.Generator().manual_seed(1)
    rows = n_pages * page
    kf, vf = (torch.randn(rows, e, generator=g).to(torch.bfloat16).cuda() for e in (s.e_k, s.e_v))
    k, v = (torch.zeros(n_pages * b, dtype=torch.uint8, device="cuda") for b in lib.kpa_paged_page_bytes(cfg, pages))
    i32 = dict(dtype=torch.int32, device="cuda")
    lib.kpa_paged_append_factors(cfg, lib.make_pages(page, n_pages, n_pages, fmt), 1, rows, kf, vf, torch.tensor([0, rows], **i32),
                                 torch.zeros(1, **i32), torch.arange(n_pages, **i32)[None], k, v)
    table = torch.randint(0, n_pages, (batch, stride), generator=g).to(**i32)
    q = torch.randn(batch, s.h, s.dh, generator=g).to(torch.bfloat16).cuda()
    lens = torch.full((batch,), n, **i32)
    ws = torch.empty(max(256, lib.kpa_paged_decode_workspace_size(cfg, pages, batch, n)), dtype=torch.uint8, device="cuda")

    def run():
        out = torch.full((batch, s.h, s.dh), float("nan"), dtype=torch.bfloat16, device="cuda")
        lib.kpa_paged_decode(cfg, pages, batch, q, lens, table, k, v, n, 0, 0, 1.0 / np.sqrt(s.dh), out, ws)
        torch.cuda.synchronize()
        return out, lib.kpa_read_device_error()

    good, error = run()
    assert error == 0 and good.isfinite().all()
    for tile in tiles:
        lib.kpa_test_set_decode_hooks(tile, 0, 20_000_000)        # that tile of split 0 of sequence 0
        try:
            out, error = run()
            assert error == lib.KPA_ERR_TIMEOUT, tile
            assert torch.equal(out[1:], good[1:])                 # the other sequences
        finally:
            lib.kpa_test_set_decode_hooks(-1, -1, 1_000_000_000)
        out, error = run()
        assert error == 0 and torch.equal(out, good), tile
