"""The operators that train the tile predictor at the edges of what their documentation allows."""
import math

import pytest
import torch

from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B

import train_util as T
from train_util import DEV, Geometry, randn

pytestmark = pytest.mark.gpu

REFS = dict(spans=[((2, 16, 16), (2, 8, 8)), ((1, 9, 21), (1, 8, 16)), ((6, 16, 24), (8, 4, 4))], text=150, gap=3)
LINE1500 = dict(spans=[((1500, 1, 1), (1, 1, 128))])


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    L.veda_device_check()
    yield
    assert L.veda_sync_status() == L.VEDA_OK


# --------------------------------------------------------------------------------------------- distillation


@pytest.mark.parametrize("geometry", [REFS, LINE1500], ids=["warp_per_row", "cta_per_row"])
@pytest.mark.parametrize("by_column", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_distill_rows_left_out_have_no_gradient_whatever_their_scores_are(geometry, by_column, weighted):
    geo = Geometry(**geometry)
    n, H = geo.n, 2
    scores = randn(1, H, n, n)
    teacher = randn(2, H, n, n)
    idx, val, cnt = T.top_lists(geo, teacher, 6)
    glob = geo.layout.n_tiles - n
    cnt[0, 0] = 0                                # an empty list
    if glob:
        idx[0, 1, :glob] = torch.arange(n, n + glob, device=DEV).int()
        cnt[0, 1] = glob                         # global tiles only
    else:
        cnt[0, 1] = 0
    val[0, 2] = -math.inf                        # listed, but no mass
    teacher[0, 2] = -math.inf
    for r, value in ((0, math.nan), (1, math.inf), (2, math.nan)):
        scores[0, r, r + 3] = value
        scores[0, r, n - 1 - r] = value
    scores[0, 0, 1] = -math.inf
    scores[1, 0] = math.nan
    cnt[1, 0] = 0
    scores[1, 1] = math.inf
    cnt[1, 1] = 0
    loss, d = torch.full((H, n), 7.0, device=DEV), torch.full((H, n, n), 7.0, device=DEV)
    weight = 0.5 + torch.rand(H, n, device=DEV) if weighted else None
    L.veda_distill(geo.layout, scores, idx, teacher if by_column else val, cnt, 1.0, loss, d_scores=d, row_weight=weight,
                   by_column=by_column)
    assert L.veda_sync_status() == L.VEDA_OK
    out = torch.zeros(H, n, dtype=torch.bool, device=DEV)
    out[0, :3] = out[1, :2] = True
    assert bool((loss[out] == 0).all()) and bool((d[out] == 0).all())
    assert bool(torch.isfinite(loss[~out]).all()) and bool(torch.isfinite(d[~out]).all()) and bool((d[~out] != 0).any(dim=1).all())
