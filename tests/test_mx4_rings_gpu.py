"""The 4-bit products' pipelines past their first turn, on the GPU: several work
items to a CTA of more K steps than the rings have stages, in every tile from 96
token rows on; K ranges in parts with 16- and 32-row tiles; pairs of CTAs whose second
one works past the last weight tile.  (test_block_fake_cpu.py shows on the CPU
that these sizes take these tiles.)"""
import numpy as np
import pytest
import torch

import block_ref as ref
from expert_routed_ffn_gemm_gb300 import binding
from test_mx4_gpu import check_product, dev, offsets_of, random_codes

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

K_LONG = 1312  # six K steps, the last of 32 columns
# token tile: rows of each group, weight rows (50 tiles of 128, gated of 64 features)
WRAPS = {96: [97, 30, 96, 80, 64, 90, 70, 1, 100, 88, 0, 75, 60],
         128: [129, 60, 128, 100, 90, 127, 110, 97, 140, 0, 105, 88, 131],
         240: [241, 240, 5, 190, 300, 481, 200, 239, 0, 350]}
WRAP_N = 6400
PARTS = ([20] * 7, 2048, 4096)  # groups, weight rows, columns
PARTS_16 = [([1] * 9, 2560, 4096), ([2, 0, 1], 640, 6400), ([1, 1, 0, 2], 1280, 12288)]  # 16-row tiles
# odd numbers of weight tiles; gated also with F no multiple of 16
ODD_TILES = [([300, 299, 310], 51 * 128, False), ([300, 299, 310], 2 * 51 * 64, True),
             ([300, 299, 310], 2 * (51 * 64 - 8), True)]
ODD_K = 800


def sample(counts, tile, rng):
    """Rows at the edges of every tile, and a few of each group between."""
    at = []
    for a, n in zip(offsets_of(counts)[:-1], counts):
        edges = [r for t in range(0, n, tile) for r in (t, t + 15, t + 16, min(n, t + tile) - 1)]
        at.append(sorted({int(a + r) for r in edges + rng.integers(0, max(n, 1), 4).tolist() if r < n}))
    return at


@pytest.mark.parametrize("tile", sorted(WRAPS))
@pytest.mark.parametrize("gated,dtype", [(False, torch.float32), (True, torch.float32), (True, torch.bfloat16),
                                         (False, torch.float16)])
def test_rings_that_wrap(tile, gated, dtype):
    counts = WRAPS[tile]
    G, R, F = len(counts), sum(counts), WRAP_N // 2 if gated else WRAP_N
    rng = np.random.default_rng(tile)
    wc, ws = random_codes((G, WRAP_N), K_LONG, tile + 1)
    ws[...] = np.where(ws > 0, ws - 6, 0)
    xc, xs = random_codes((R,), K_LONG, tile + 2)
    experts = binding.Mx4Experts(dev(wc), dev(ws), K_LONG, gated=gated)
    kw, out_rows, n_out = {}, np.arange(R, dtype=np.int32), R
    factor = np.ones(R, np.float32)
    if not gated:
        n_out = R + 9
        out_rows = rng.permutation(n_out)[:R].astype(np.int32)
        factor = rng.normal(size=n_out).astype(np.float32)
        kw = {"out_rows": dev(out_rows), "n_out": n_out, "row_scale": dev(factor)}
    out = torch.full((n_out, F), 7.0, dtype=dtype, device=DEV)
    args = (dev(xc), dev(xs), dev(offsets_of(counts)))
    experts.matmul(*args, out=out, **kw)
    again = torch.full_like(out, 7.0)
    experts.matmul(*args, out=again, **kw)
    assert experts.check() == binding.MOE_OK and torch.equal(out, again)
    written = np.zeros(n_out, bool)
    written[out_rows] = True
    assert bool((out[torch.from_numpy(~written).to(DEV)] == 7).all())
    got = out.cpu().double().numpy()
    for g, rows in enumerate(sample(counts, tile, rng)):
        if not rows:
            continue
        z, err = ref.grouped(ref.values_of(xc[rows], xs[rows], K_LONG), ref.values_of(wc[g], ws[g], K_LONG)[None],
                             [0, len(rows)], gated)
        f = factor[out_rows[rows]].astype(np.float64)[:, None]
        want, tol = z * f, err * np.abs(f) + np.abs(z * f) * ref.U * 4
        tol = tol + ref.half_step(dtype) * (np.abs(want) + tol) + torch.finfo(dtype).tiny
        bad = ~(np.abs(got[out_rows[rows]] - want) <= tol)
        assert not bad.any(), (g, int(bad.sum()), np.argwhere(bad)[:5].tolist())


@pytest.mark.parametrize("gated,dtype", [(False, torch.float32), (True, torch.float32), (True, torch.bfloat16)])
def test_parts_of_32_row_tiles(gated, dtype):
    counts, N, K = PARTS
    check_product(counts, N, K, gated, dtype, seed=51, scatter=not gated, scale=not gated)
    check_product([32, 17, 0, 31, 16, 20, 24], N, K, gated, dtype, seed=52)


@pytest.mark.parametrize("counts,N,K", PARTS_16)
@pytest.mark.parametrize("gated", [False, True])
def test_parts_of_16_row_tiles(counts, N, K, gated):
    check_product(counts, N, K, gated, torch.float32, seed=53, scatter=True, scale=True)


@pytest.mark.parametrize("counts,N,gated", ODD_TILES)
def test_pairs_past_the_last_weight_tile(counts, N, gated):
    for dtype in (torch.float32, torch.bfloat16):
        check_product(counts, N, ODD_K, gated, dtype, seed=N, scatter=not gated, scale=not gated)
