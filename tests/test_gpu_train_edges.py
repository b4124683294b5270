"""The operators that train the tile predictor at the edges of what their documentation allows."""
import ctypes as C
import math
import threading

import pytest
import torch

from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B

import train_util as T
from train_util import DEV, EPS, SPLIT, Geometry, randn

pytestmark = pytest.mark.gpu

REFS = dict(spans=[((2, 16, 16), (2, 8, 8)), ((1, 9, 21), (1, 8, 16)), ((6, 16, 24), (8, 4, 4))], text=150, gap=3)
LINE1500 = dict(spans=[((1500, 1, 1), (1, 1, 128))])
SMEM = 227 * 1024  # a CTA's shared memory


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    L.veda_device_check()
    yield
    assert L.veda_sync_status() == L.VEDA_OK


def bytes_(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)


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


# ------------------------------------------------------------------------------------------- bias gradient


def bias_backward(geo, ds, reach, far):
    H = ds.shape[0]
    out = torch.full((H, L.veda_bias_buckets(reach, far)), 7.0, device=DEV)
    ws = bytes_(L.veda_bias_backward_workspace_bytes(geo.layout, H, reach))
    L.veda_bias_backward(geo.layout, ds, reach, far, ws, out)
    assert L.veda_sync_status() == L.VEDA_OK, L.veda_last_error()
    return out


def bucket_sums(geo, reach, far, x):
    """64-bit sums of each bucket, head by head."""
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long().reshape(-1)
    total = L.veda_bias_buckets(reach, far)
    return torch.stack([torch.zeros(total, dtype=torch.float64, device=DEV).index_add_(0, index, h.double().reshape(-1)) for h in x])


@pytest.mark.parametrize("spans,where", [
    ([((13, 48, 84), (1, 8, 16))], "first"), ([((61, 45, 80), (8, 1, 16))], "first"), ([((16, 128, 256), (1, 8, 16))], "first"),
    ([((5, 45, 80), (1, 8, 16)), ((2, 16, 16), (2, 8, 8))], "first"), ([((5, 45, 80), (1, 8, 16)), ((2, 16, 16), (2, 8, 8))], "cross")])
def test_bias_gradient_of_a_bucket_of_many_offsets(spans, where):
    # One value is so large that the others, added to it one by one in fp32, would all be lost. It is met first in its bucket:
    # the offset of the last query and the first key.
    geo, reach, far = Geometry(spans), (1, 1, 1), (2, 2, 2)
    n = geo.n
    ds = torch.ones(1, n, n, device=DEV)
    first = math.prod(-(-g // b) for g, b in zip(*spans[0]))  # tiles of the first span
    ds[0, first - 1 if where == "first" else n - 1, 0] = 2.0 ** 28
    got = bias_backward(geo, ds, reach, far).double()
    want = bucket_sums(geo, reach, far, ds)
    # additions that a value passes through: a chunk's rows (fewer than 64 up to 8,192 tiles), a run of offsets along each of
    # the three axes, the spans, the chunks (eight by eight, fewer than 64 times); across spans a thread's values (fewer
    # than 16 a row), the lanes and the warps in the place of the runs
    runs = sum(2 * -(-g // b) - 1 for g, b in zip(*spans[0]))
    adds = (64 + runs if where == "first" else 64 * 16 + 5 + 16) + len(spans) + 64
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV)
    big = int(index[first - 1 if where == "first" else n - 1, 0])
    # only the sum that holds the large value is that coarse: ones are exact
    assert float((got[0, big] - want[0, big]).abs()) <= adds * EPS * float(want[0, big])
    rest = torch.arange(got.shape[1], device=DEV) != big
    assert float(((got - want).abs() - EPS * want)[0, rest].max()) <= 0


def offsets_of(spans):
    """Entries of the table of every offset: (2 T - 1)(2 H - 1)(2 W - 1) of each span's array of tiles."""
    return sum(math.prod(2 * -(-g // b) - 1 for g, b in zip(grid, box)) for grid, box in spans)


@pytest.mark.parametrize("spans,heads,reach,far", [
    ([((20, 160, 320), (1, 8, 16))], 2, (4, 4, 6), (16, 16, 32)),                          # 20 x 20 x 20 tiles: too many offsets
    ([((20, 160, 320), (1, 8, 16)), ((4, 64, 64), (2, 8, 8))], 2, (3, 5, 2), (8, 11, 9)),  # and a second span
    ([((3, 24, 40), (1, 8, 16)), ((21, 160, 320), (1, 8, 16)), ((2, 16, 16), (2, 8, 8))], 1, (2, 3, 4), (9, 7, 12)),
    ([((90, 8, 1600), (1, 8, 16))], 2, (16, 1, 8), (64, 2, 32)),                           # more than 8,192 tiles, one along h
    ([((20, 160, 320), (1, 8, 16)), ((1, 8, 16), (1, 8, 16))], 1, (1, 1, 1), (2, 2, 2)),   # one bucket for all offsets
])
def test_bias_gradient_without_offset_sums(spans, heads, reach, far):
    geo = Geometry(spans)
    # this is what sends a layout to the kernel that sums boxes of each row
    assert 4 * offsets_of(spans) > SMEM or geo.n > 8192
    ds = randn(1, heads, geo.n, geo.n)
    got, want = bias_backward(geo, ds, reach, far), bucket_sums(geo, reach, far, ds)
    # a value passes through fewer than 2 n + 64 fp32 additions: its row's box, the chunk's rows, the chunks
    over = (got.double() - want).abs() - (2 * geo.n + 64) * EPS * bucket_sums(geo, reach, far, ds.abs())
    assert float(over.max()) <= 0
    assert torch.equal(bias_backward(geo, ds, reach, far), got)


def in_threads(jobs):
    """Runs every job (a C call, its arguments, how often, its stream) on a host thread of its own, all at once, and returns
    the sets of their status codes. The interpreter's lock is free during a call."""
    torch.cuda.synchronize()
    codes, start = [None] * len(jobs), threading.Barrier(len(jobs))

    def work(i, call, args, calls, stream):
        start.wait()
        codes[i] = {call(*args) for _ in range(calls)}
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i, *job)) for i, job in enumerate(jobs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return codes


def test_bias_gradient_of_wide_layouts_from_several_threads():
    # host threads whose layouts need different amounts of shared memory: neither's call is refused
    jobs, results, keep = [], [], []
    spec = L.BiasSpec((2, 1, 1), (9, 2, 2))
    for n, calls in ((16384, 400), (8200, 3000), (8200, 3000)):
        geo = Geometry([((n, 1, 1), (1, 1, 128))])
        ds = randn(n, 1, n, n)
        want = bias_backward(geo, ds, (2, 1, 1), (9, 2, 2))
        ws = bytes_(L.veda_bias_backward_workspace_bytes(geo.layout, 1, (2, 1, 1)))
        out, stream = torch.empty_like(want), torch.cuda.Stream()
        keep.append((geo, ds, ws))
        results.append((out, want))
        jobs.append((L.lib().veda_bias_backward, (geo.layout.handle, ds.data_ptr(), 1, C.byref(spec), ws.data_ptr(), ws.nbytes,
                                                  out.data_ptr(), C.c_void_p(stream.cuda_stream)), calls, stream))
    assert in_threads(jobs) == [{L.VEDA_OK}] * len(jobs)
    assert all(torch.equal(out, want) for out, want in results)


def test_selection_in_wide_layouts_from_several_threads():
    jobs, results, keep = [], [], []
    for n, calls in ((16384, 300), (12400, 1500), (12400, 1500)):  # both over the 48 KB that need no opt-in
        geo = Geometry([((n, 1, 1), (1, 1, 128))], ratio=0.001)
        scores = randn(n, 1, n, n)
        want, out = (torch.zeros(1, n, geo.layout.max_kept, dtype=torch.int32, device=DEV) for _ in range(2))
        cnt, stream = torch.zeros(1, n, dtype=torch.int32, device=DEV), torch.cuda.Stream()
        L.veda_select(geo.layout, scores, want, cnt)
        keep.append((geo, scores, cnt))
        results.append((out, want))
        jobs.append((L.lib().veda_select, (geo.layout.handle, scores.data_ptr(), 1, out.data_ptr(), cnt.data_ptr(),
                                           C.c_void_p(stream.cuda_stream)), calls, stream))
    assert in_threads(jobs) == [{L.VEDA_OK}] * len(jobs)
    assert all(torch.equal(out, want) for out, want in results)


# ------------------------------------------------------------------- values that are not finite, and the largest


def feats(seed, heads, n, dim):
    return torch.cat([0.3 * randn(seed, heads, n, dim), 2.4 + 0.4 * randn(seed + 1, heads, n, dim),
                      -2.4 + 0.4 * randn(seed + 2, heads, n, dim)], dim=2).contiguous()


def projections(seed, heads, dim):
    return randn(seed, heads, 3 * dim, dim) / math.sqrt(3 * dim)


LARGEST = torch.finfo(torch.float32).max


def magnitude(a, b):
    """Sums of the finite values' products, without signs."""
    return torch.nan_to_num(a, nan=0.0, posinf=0.0, neginf=0.0).abs() @ torch.nan_to_num(b, nan=0.0, posinf=0.0, neginf=0.0).abs()


def agrees(got, want, size, tol):
    """``got`` holds the 64-bit ``want`` within tol, NaN and infinities where want has them; returns how many those are.
    Passed over: sums whose finite terms alone can pass the type's range (size), which an fp32 sum may leave and not come
    back to."""
    seen = size < LARGEST / 2
    got, want = torch.where(seen, got.double(), 0.0), torch.where(seen, want, 0.0)
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)])
    assert float((torch.where(odd, 0.0, (got - want).abs()) - torch.where(seen, tol, 0.0)).max()) <= 0
    return int(odd.sum())


@pytest.mark.parametrize("dim,heads", [(64, 2), (128, 1), (128, 40)])  # whole tiles; cut along K; whole tiles of 128
def test_scores_of_values_that_are_not_finite(dim, heads):
    geo, reach, far = Geometry(**REFS), (3, 3, 3), (8, 8, 8)
    n = geo.n
    fq, fk = feats(1, heads, n, dim), feats(4, heads, n, dim)
    pq, pk = projections(7, heads, dim), projections(8, heads, dim)
    fq[0, 1, 5] = math.inf
    fq[0, 2, 3 * dim - 1] = -math.inf
    fq[0, 4, 7] = LARGEST           # finite, and so are its products with entries below one
    fk[0, 3, dim + 1] = math.nan
    fk[0, 5, 2] = -LARGEST
    fk[0, 6, 9], fk[0, 6, 10] = math.inf, -math.inf
    pk[heads - 1, dim + 3, 11] = math.inf
    pk[heads - 1, 2, 12] = LARGEST
    hats = torch.full((2, heads, n, dim), 7.0, device=DEV)
    scores = torch.full((heads, n, n), 7.0, device=DEV)
    bias = randn(9, heads, L.veda_bias_buckets(reach, far))
    bias[:, 0] = -math.inf
    ws = bytes_(L.veda_score_bias_workspace_bytes(geo.layout, heads, dim))
    L.veda_score_bias(geo.layout, fq, fk, pq, pk, reach, far, bias, hats, ws, scores)
    assert L.veda_sync_status() == L.VEDA_OK
    eye = torch.eye(3 * dim, dim, dtype=torch.float64, device=DEV)
    found = 0
    for got, f, p in ((hats[0], fq, pq), (hats[1], fk, pk)):
        f, p = f.double(), p.double() + eye
        size = magnitude(f, p.abs() + eye)
        found += agrees(got, f @ p, size, (SPLIT + (3 * dim + 9) * 2 * EPS) * size)
    assert found > 2 * dim
    huge = hats[0, 0, 4].abs() > 1e36  # (the finite one's row)
    assert int((huge & torch.isfinite(hats[0, 0, 4])).sum()) > dim // 2
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long()
    b = bias.double()[:, index]
    q, k = hats.double()
    size = magnitude(q, k.transpose(1, 2))
    # (rows that hold values of 2^11 or more on one side and infinities on the other give infinities or NaN)
    far_apart = (torch.isinf(q).any(2)[:, :, None] & (k.abs() >= 2048).any(2)[:, None]) | \
        ((q.abs() >= 2048).any(2)[:, :, None] & torch.isinf(k).any(2)[:, None])
    want = q @ k.transpose(1, 2) / math.sqrt(dim) + b
    assert not bool(torch.isfinite(scores[far_apart]).any())
    tol = (SPLIT + (dim + 12) * 2 * EPS) * size + 4 * EPS * torch.nan_to_num(b, neginf=0.0).abs()
    found = agrees(torch.where(far_apart, 0.0, scores), torch.where(far_apart, 0.0, want), size, tol)
    assert found > n and bool(torch.isnan(want).any()) and bool((want == -math.inf).any())
    # the rows and columns of the first head without such a value: scores as always
    rows = torch.tensor([0] + list(range(7, n)), device=DEV)
    if heads > 1:
        assert bool((torch.isfinite(scores[0, rows][:, rows]) | (b[0, rows][:, rows] == -math.inf)).all())


@pytest.mark.parametrize("spans,dim,heads", [(REFS["spans"], 64, 2), (REFS["spans"], 128, 1), ([((15, 24, 42), (1, 8, 16))], 128, 1),
                                             ([((5, 45, 80), (1, 8, 16))], 64, 3), ([((13, 48, 84), (1, 8, 16))], 128, 1)])
def test_projection_gradients_of_values_that_are_not_finite(spans, dim, heads):
    geo = Geometry(spans)
    n = geo.n
    fq, fk, hats = feats(1, heads, n, dim), feats(4, heads, n, dim), randn(7, 2, heads, n, dim)
    ds = torch.softmax(2 * randn(9, heads, n, n), 2) - torch.softmax(4 * randn(10, heads, n, n), 2)
    for case in range(4):
        f, h, g = fq.clone(), hats.clone(), ds.clone()
        if case == 0:
            g[0, 3, n - 2] = math.inf       # one infinite gradient: infinities of the signs that its features give
        elif case == 1:
            g[heads - 1, n - 1, 0] = LARGEST
            h[1, heads - 1, 0] *= 1e-3      # (its products stay in range)
            h[0, heads - 1, n - 1] *= 1e-3
        elif case == 2:
            f[0, 1, 5], f[0, 2, 6] = -math.inf, math.nan
        else:
            h[1, 0, 4, 7] = math.inf
        out = [torch.full((heads, 3 * dim, dim), 7.0, device=DEV) for _ in range(2)]
        ws = bytes_(L.veda_score_backward_workspace_bytes(geo.layout, heads, dim))
        L.veda_score_backward(geo.layout, f, fk, h, g, ws, *out)
        assert L.veda_sync_status() == L.VEDA_OK
        q, k = h.double()
        c = 1 / math.sqrt(dim)
        found = 0
        for got, x, m, y in ((out[0], f, g.double(), k), (out[1], fk, g.double().transpose(1, 2), q)):
            dx, ft = c * (m @ y), x.double().transpose(1, 2)
            bound = c * (SPLIT + (n + 12) * 2 * EPS) * magnitude(m, y)
            size = magnitude(ft, dx.abs() + bound)
            found += agrees(got, ft @ dx, size, magnitude(ft, bound) + (SPLIT + (n + 8) * 2 * EPS) * size)
        assert (found > 0) == (case != 1)
