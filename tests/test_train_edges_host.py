"""CPU checks of what the entry points that train the tile predictor refuse at the edges of their documentation."""
import pytest

from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


@pytest.mark.parametrize("by_column", [0, 1])
def test_distill_refuses_outputs_over_its_inputs(by_column):
    lay = L.veda_plan([(0, (8, 16, 16), (2, 8, 8))], 2048, (0.3, None), (1.0, None))
    n, heads, width = lay.n_video, 3, 8
    square, row = 4 * heads * n * n, 4 * heads * n
    value = square if by_column else 4 * heads * n * width
    names = ["scores", "t_idx", "t_val", "t_cnt", "row_weight", "loss", "d_scores"]
    size = dict(scores=square, t_idx=4 * heads * n * width, t_val=value, t_cnt=row, row_weight=row, loss=row, d_scores=square)
    apart = {name: (i + 1) << 30 for i, name in enumerate(names)}  # addresses that no call may follow

    def call(**at):
        p = {**apart, **at}
        return L.lib().veda_distill(lay.handle, p["scores"], heads, p["t_idx"], p["t_val"], p["t_cnt"], width, by_column, 1.0,
                                    p["row_weight"], p["loss"], p["d_scores"], None)

    for out in ("loss", "d_scores"):
        for other in names:
            if other == out:
                continue
            base = apart[other]
            # the same buffer, one that ends inside the other, one that begins at its last 16 bytes
            for at in (base, base - size[out] + 16, base + size[other] - 16):
                assert call(**{out: at}) == L.VEDA_ERR_INVALID, (out, other, at - base)
                assert "overlap" in L.veda_last_error()
