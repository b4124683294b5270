"""CPU checks of the entry points that train the tile predictor: the buckets of the relative position bias against a
plain restatement, and what the calls refuse before they touch a device."""
import numpy as np
import pytest
import torch

from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def axis_class(a, reach, far):
    """Distance class in whole numbers: exact distances first, then geometric steps."""
    exact = (reach + 1) // 2
    wide = reach - exact
    if a < exact:
        return a
    return min(reach - 1, exact + sum(a ** wide >= exact ** (wide - m) * far ** m for m in range(1, wide + 1)))


def plain_index(spans, reach, far):
    """Buckets of every pair from the definition: spans [(grid, box)], tiles of a span visited h, w, t."""
    places = []
    for s, (grid, box) in enumerate(spans):
        nt, nh, nw = (-(-g // b) for g, b in zip(grid, box))
        places += [(s, t, h, w) for h in range(nh) for w in range(nw) for t in range(nt)]
    pairs = int(np.prod([2 * r - 1 for r in reach]))
    out = np.empty((len(places), len(places)), np.int32)
    for i, q in enumerate(places):
        for j, k in enumerate(places):
            if k[0] != q[0]:
                out[i, j] = pairs + (k[0] > q[0])
                continue
            b = 0
            for a in range(3):
                r = k[a + 1] - q[a + 1]
                c = axis_class(abs(r), reach[a], far[a])
                b = b * (2 * reach[a] - 1) + (c if r <= 0 else reach[a] - 1 + c)
            out[i, j] = b
    return out


@pytest.mark.parametrize("spans,reach,far", [
    ([((8, 16, 16), (2, 8, 8))], (3, 3, 3), (8, 8, 8)),
    ([((2, 16, 16), (2, 8, 8)), ((6, 16, 24), (2, 8, 8))], (4, 2, 1), (16, 5, 3)),
    ([((1, 1, 1), (1, 8, 16))], (1, 1, 1), (2, 2, 2)),
    ([((40, 9, 30), (1, 8, 16)), ((3, 8, 16), (1, 8, 16)), ((5, 20, 20), (2, 8, 8))], (8, 5, 6), (32, 11, 60)),
    ([((70, 2, 2), (1, 1, 128))], (16, 2, 3), (64, 2, 4)),
])
def test_bias_index_matches_the_definition(spans, reach, far):
    at, plan = 5, []
    for grid, box in spans:
        plan.append((at, grid, box))
        at += int(np.prod(grid)) + 3
    lay = L.veda_plan(plan, at, (0.3, None), (0.5, None))
    want = plain_index(spans, reach, far)
    assert np.array_equal(L.veda_bias_index(lay, reach, far), want)
    buckets = L.veda_bias_buckets(reach, far)
    assert buckets == int(np.prod([2 * r - 1 for r in reach])) + 2 and want.max() < buckets


def test_class_borders_are_whole_numbers():
    # far a power of the first wide class: the border distance itself starts the class (a rounded logarithm may miss it)
    lay = L.veda_plan([(0, (300, 1, 1), (1, 1, 128))], 300, (0.3, None), (1.0, None))
    for reach, far in ((6, 24), (5, 48), (16, 2048), (8, 64), (9, 3125)):
        got = L.veda_bias_index(lay, (reach, 1, 1), (far, 2, 2))[:, 0]  # key 0: r = -distance
        assert got.tolist() == [axis_class(a, reach, far) for a in range(300)]


@pytest.mark.parametrize("reach,far,code", [
    ((0, 1, 1), (8, 8, 8), L.VEDA_ERR_INVALID), ((17, 1, 1), (99, 8, 8), L.VEDA_ERR_INVALID),
    ((4, 1, 1), (2, 8, 8), L.VEDA_ERR_INVALID), ((4, 1, 1), (32768, 8, 8), L.VEDA_ERR_INVALID),
    ((1, 1, 1), (1, 8, 8), L.VEDA_ERR_INVALID), ((16, 16, 16), (99, 99, 99), L.VEDA_ERR_UNSUPPORTED),
])
def test_bias_spec_refusals(reach, far, code):
    with pytest.raises(L.VedaError) as e:
        L.veda_bias_buckets(reach, far)
    assert e.value.code == code


def test_workspace_sizes():
    lay = L.veda_plan([(0, (8, 16, 16), (2, 8, 8))], 2048, (0.3, None), (1.0, None))
    # 4 x 2 x 2 tiles: 7 * 3 * 3 offsets and two buckets of other spans per head
    assert L.veda_score_bias_workspace_bytes(lay, 2, 64, (3, 3, 3)) >= 2 * (63 + 2) * 4
    assert L.veda_bias_backward_workspace_bytes(lay, 2, (3, 3, 3)) >= 2 * (125 + 2) * 4
    assert L.veda_score_backward_workspace_bytes(lay, 2, 64) >= 2 * 2 * 16 * 64 * 4
    assert L.lib().veda_score_bias_workspace_bytes(lay.handle, 0, 64) == 0
    assert L.lib().veda_score_backward_workspace_bytes(None, 2, 64) == 0


def test_c_entries_refuse_bad_arguments_before_any_device():
    lib, ok = L.lib(), 256  # a 16-byte aligned address that no call may follow
    lay = L.veda_plan([(0, (8, 16, 16), (2, 8, 8))], 2048, (0.3, None), (1.0, None))
    h = lay.handle
    big = 1 << 40
    spec = L.BiasSpec((3, 3, 3), (8, 8, 8))
    bad = L.BiasSpec((0, 3, 3), (8, 8, 8))
    import ctypes as C
    sp, bd = C.byref(spec), C.byref(bad)
    d = ok + (1 << 30)
    calls = [
        lib.veda_teacher(h, None, ok, 2, 64, None, ok, None), lib.veda_teacher(None, ok, ok, 2, 64, None, ok, None),
        lib.veda_teacher(h, ok, ok, 2, 96, None, ok, None), lib.veda_teacher(h, ok, ok, 0, 64, None, ok, None),
        lib.veda_teacher(h, ok + 8, ok, 2, 64, None, ok, None), lib.veda_teacher(h, ok, ok, 2, 64, ok + 4, ok, None),
        lib.veda_score_bias(h, ok, ok, 2, 64, ok, ok, sp, None, ok, ok, big, ok, None),
        lib.veda_score_bias(h, ok, ok, 2, 64, ok, ok, None, ok, ok, ok, big, ok, None),
        lib.veda_score_bias(h, ok, ok, 2, 64, ok, ok, bd, ok, ok, ok, big, ok, None),
        lib.veda_score_bias(h, ok, ok, 2, 64, ok, ok, sp, ok, ok, ok, 16, ok, None),
        lib.veda_score_bias(h, ok, ok, 2, 64, ok, ok, sp, ok, ok + 4, ok, big, ok, None),
        lib.veda_score_bias(h, ok, ok, 2, 32, ok, ok, sp, ok, ok, ok, big, ok, None),
        lib.veda_bias_backward(h, ok, 2, None, ok, big, ok, None), lib.veda_bias_backward(h, ok, 2, bd, ok, big, ok, None),
        lib.veda_bias_backward(h, ok, 2, sp, ok, 4, ok, None), lib.veda_bias_backward(h, None, 2, sp, ok, big, ok, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 0, 0, 1.0, None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, 0.0, None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, -1.0, None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, float("nan"), None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, float("inf"), None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, 1e-40, None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, 2e30, None, ok, d, None),
        lib.veda_distill(h, ok, 2, ok, ok, ok, 8, 0, 1.0, None, ok, ok + 16, None),  # overlaps scores
        lib.veda_distill(h, ok, 2, ok, ok, None, 8, 0, 1.0, None, ok, d, None),
        lib.veda_score_backward(h, ok, ok, 2, 64, ok, ok, ok, ok, ok, 4, None),
        lib.veda_score_backward(h, ok, ok, 2, 64, None, ok, ok, ok, ok, big, None),
        lib.veda_score_backward(h, ok, ok, -1, 64, ok, ok, ok, ok, ok, big, None),
    ]
    assert [i for i, rc in enumerate(calls) if rc != L.VEDA_ERR_INVALID] == []
    wide = L.veda_plan([(0, (16385, 1, 1), (1, 1, 128))], 16385, (None, 3), (1.0, None))
    assert wide.n_video == 16385
    assert lib.veda_teacher(wide.handle, ok, ok, 1, 64, None, ok, None) == L.VEDA_ERR_UNSUPPORTED
    assert lib.veda_distill(wide.handle, ok, 1, ok, ok, ok, 8, 0, 1.0, None, ok, None, None) == L.VEDA_ERR_UNSUPPORTED
    assert lib.veda_teacher(h, ok, ok, 65536, 64, None, ok, None) == L.VEDA_ERR_UNSUPPORTED


def test_binding_refuses_tensors_a_kernel_would_misread(monkeypatch):
    # host tensors, wrong types, shapes and strides are refused before the library sees their pointers
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    lay = L.veda_plan([(0, (8, 16, 16), (2, 8, 8))], 2048, (0.3, None), (1.0, None))
    n, f = lay.n_video, torch.zeros
    good = dict(scores=f(2, n, n), t_idx=f(2, n, 4, dtype=torch.int32), t_val=f(2, n, 4), t_cnt=f(2, n, dtype=torch.int32),
                tau=1.0, loss=f(2, n))
    bad = [dict(scores=f(2, n, n).double()), dict(scores=f(2, n, n + 1)), dict(scores=f(2, n, n).transpose(1, 2)),
           dict(t_idx=f(2, n, 4, dtype=torch.int64)), dict(t_val=f(2, n, 5)), dict(t_cnt=f(2, n)), dict(loss=f(n, 2)),
           dict(by_column=True), dict()]  # the last: all on the host
    for change in bad:
        with pytest.raises(L.VedaError) as e:
            L.veda_distill(lay, **{**good, **change})
        assert e.value.code == L.VEDA_ERR_INVALID
    with pytest.raises(L.VedaError):
        L.veda_teacher(lay, f(2, lay.n_slots, 64), f(2, lay.n_slots, 64), f(2, n, n))
    with pytest.raises(L.VedaError):
        L.veda_score_backward(lay, f(2, n, 192), f(2, n, 192), f(2, 2, n, 64), f(2, n, n), f(9), f(2, 192, 64), f(2, 64, 192))
    with pytest.raises(L.VedaError):
        L.veda_bias_backward(lay, f(2, n, n), (3, 3, 3), (8, 8, 8), f(9), f(2, 5))
    with pytest.raises(L.VedaError):
        L.veda_score_bias(lay, f(2, n, 192), f(2, n, 192), f(2, 192, 64), f(2, 192, 64), None, None, None, f(2, 2, n, 64),
                          f(9), f(2, n, n))
