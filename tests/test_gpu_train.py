"""The operators that train the tile predictor against plain 64-bit restatements: pooled teacher, scores with the
relative position bias, distillation, and the gradients of projections and bias."""
import math

import pytest
import torch

from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B

import train_util as T
from train_util import DEV, EPS, SPLIT, Geometry, randn

pytestmark = pytest.mark.gpu

GEOMETRIES = {
    "one": dict(spans=[((1, 1, 1), (1, 8, 16))]),                                   # a single tile with one real row
    "tiny": dict(spans=[((8, 16, 16), (2, 8, 8))]),                                 # whole tiles, 16
    "ragged": dict(spans=[((3, 10, 12), (2, 8, 8))], text=200),                     # partial tiles, global tiles
    "refs": dict(spans=[((2, 16, 16), (2, 8, 8)), ((1, 9, 21), (1, 8, 16)), ((6, 16, 24), (8, 4, 4))], text=150, gap=3),
    "wide": dict(spans=[((5, 45, 50), (1, 8, 16))], text=1),                        # 120 tiles of odd fill
    "odd135": dict(spans=[((15, 24, 42), (1, 8, 16))]),                             # just over one MMA tile, an odd number
    "even150": dict(spans=[((5, 45, 80), (1, 8, 16))]),                             # 150 = 2 modulo 4
    "odd259": dict(spans=[((37, 8, 112), (1, 8, 16))], text=40),                    # three MMA tiles, 3 modulo 4
    "quad260": dict(spans=[((65, 8, 60), (1, 8, 16))]),                             # rows of whole 16-byte pieces
    "line": dict(spans=[((259, 1, 3), (128, 1, 1))]),                               # boxes longer than the grid is
}


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    L.veda_device_check()
    yield
    assert L.veda_sync_status() == L.VEDA_OK


@pytest.fixture(params=sorted(GEOMETRIES))
def geo(request):
    return Geometry(**GEOMETRIES[request.param])


def bytes_(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)


def within(got, want, tol):
    """Every entry within its tolerance; infinities and NaN where the other has them."""
    got, want = got.double(), want.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)])
    err = torch.where(odd, 0.0, (got - want).abs())
    over = err - tol
    assert float(over.max()) <= 0, (float(err.max()), float(over.max()))


# ------------------------------------------------------------------------------------------------ teacher


def teacher(geo, q, k, lse=None, **kw):
    out = torch.full((q.shape[0], geo.n, geo.n), 7.0, device=DEV)
    L.veda_teacher(geo.layout, q, k, out, row_lse=lse, **kw)
    assert L.veda_sync_status() == L.VEDA_OK, L.veda_last_error()
    return out


def teacher_tol(q, k, lse):
    # products of bf16 are exact in fp32; each of the D additions loses at most 2^-23 of the sum of magnitudes, which is
    # at most |q| |k| (Cauchy-Schwarz); scaling and the difference with lse round the result three times
    D = q.shape[2]
    big = float(q.double().norm(dim=2).max() * k.double().norm(dim=2).max()) / math.sqrt(D)
    off = 0.0 if lse is None else float(lse[torch.isfinite(lse)].abs().max())
    return (D + 4) * 2 * EPS * big + 4 * EPS * (big + off)


@pytest.mark.parametrize("dim,heads", [(64, 1), (128, 3)])
@pytest.mark.parametrize("with_lse", [False, True])
def test_teacher(geo, dim, heads, with_lse):
    q, k = T.tile_rows(geo, 1, heads, dim), T.tile_rows(geo, 3, heads, dim)
    lse = 5 + 2 * randn(5, heads, geo.seq) if with_lse else None
    within(teacher(geo, q, k, lse), T.plain_teacher(geo, q, k, lse), teacher_tol(q, k, lse))


def test_teacher_negative_logits_are_not_beaten_by_padding():
    # every real logit is negative: a padding slot (zeros, logit 0) must not become the maximum
    geo = Geometry(**GEOMETRIES["ragged"])
    q = T.tile_rows(geo, 1, 2, 64).abs()
    k = -T.tile_rows(geo, 3, 2, 64).abs()
    out = teacher(geo, q, k)
    assert float(out.max()) < 0
    within(out, T.plain_teacher(geo, q, k), teacher_tol(q, k, None))


def test_teacher_passes_over_rows_without_a_softmax_sum_and_nan():
    geo = Geometry(**GEOMETRIES["refs"])
    q, k = T.tile_rows(geo, 1, 2, 128), T.tile_rows(geo, 3, 2, 128)
    lse = 5 + randn(5, 2, geo.seq)
    rows = geo.perm[:geo.n]
    lse[0, rows[2][rows[2] >= 0]] = -math.inf      # a tile whose rows see no key: nothing is left
    lse[1, rows[3][0]] = math.inf
    lse[1, rows[4][5]] = math.nan
    q[0, 128 * 5] = math.nan                       # one row of NaN logits
    k[1, 128 * 7 + 1] = math.nan
    out = teacher(geo, q, k, lse)
    want = T.plain_teacher(geo, q, k, lse)
    assert bool((out[0, 2] == -math.inf).all()) and bool(torch.isfinite(out[1]).all())
    clean = lambda x: torch.nan_to_num(x.float(), nan=0.0).to(torch.bfloat16)  # noqa: E731
    within(out, want, teacher_tol(clean(q), clean(k), lse))


# ------------------------------------------------------------------------------------- scores with a bias


def feats(seed, heads, n, dim):
    return torch.cat([0.3 * randn(seed, heads, n, dim), 2.4 + 0.4 * randn(seed + 1, heads, n, dim),
                      -2.4 + 0.4 * randn(seed + 2, heads, n, dim)], dim=2).contiguous()


def projections(seed, heads, dim):
    return randn(seed, heads, 3 * dim, dim) / math.sqrt(3 * dim)


def score_bias(geo, fq, fk, pq, pk, reach=None, far=None, bias=None, **kw):
    H, _, D = pq.shape
    hats = torch.full((2, H, geo.n, D), 7.0, device=DEV)
    out = torch.full((H, geo.n, geo.n), 7.0, device=DEV)
    ws = bytes_(L.veda_score_bias_workspace_bytes(geo.layout, H, D, reach))
    L.veda_score_bias(geo.layout, fq, fk, pq, pk, reach, far, bias, hats, ws, out, **kw)
    assert L.veda_sync_status() == L.VEDA_OK, L.veda_last_error()
    return out, hats


def product_tol(a, b, terms):
    """Bound of a split-tf32 product with fp32 sums of ``terms`` terms: what the split leaves out, and at most 2^-23 of the
    magnitudes' sum for each addition."""
    return (SPLIT + (terms + 8) * 2 * EPS) * (a.abs() @ b.abs())


@pytest.mark.parametrize("dim,heads,reach,far", [(64, 2, (3, 3, 3), (8, 8, 8)), (128, 1, (6, 1, 4), (20, 5, 9)),
                                                 (128, 2, None, None)])
def test_score_bias(geo, dim, heads, reach, far):
    n = geo.n
    fq, fk = feats(1, heads, n, dim), feats(4, heads, n, dim)
    pq, pk = projections(7, heads, dim), projections(8, heads, dim)
    bias = None if reach is None else randn(9, heads, L.veda_bias_buckets(reach, far))
    out, hats = score_bias(geo, fq, fk, pq, pk, reach, far, bias)
    q, k = T.plain_hats(fq, fk, pq, pk)
    eye = torch.eye(3 * dim, dim, dtype=torch.float64, device=DEV)
    tq, tk = (product_tol(f.double(), p.double().abs() + eye, 3 * dim + 1) for f, p in ((fq, pq), (fk, pk)))
    within(hats[0], q, tq)
    within(hats[1], k, tk)
    want = q @ k.transpose(1, 2) / math.sqrt(dim)
    tol = (tq @ k.abs().transpose(1, 2) + (q.abs() + tq) @ tk.transpose(1, 2) +
           product_tol(q.abs() + tq, (k.abs() + tk).transpose(1, 2), dim)) / math.sqrt(dim)
    if bias is not None:
        index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long()
        want = want + bias.double()[:, index]
        tol = tol + 2 * EPS * bias.abs().max()
    within(out, want, tol + 4 * EPS * want.abs())


@pytest.mark.parametrize("dim", [64, 128])
def test_score_bias_masks(dim):
    # -inf and the type's lowest value in buckets: the first leaves -inf, the second a finite score below all others
    geo, reach, far = Geometry(**GEOMETRIES["refs"]), (3, 3, 3), (8, 8, 8)
    n, low = geo.n, torch.finfo(torch.float32).min
    total = L.veda_bias_buckets(reach, far)
    bias = torch.zeros(1, total, device=DEV)
    bias[0, ::3], bias[0, 1::3], bias[0, -1] = -math.inf, low, 3e38
    fq, fk, pq, pk = feats(1, 1, n, dim), feats(4, 1, n, dim), projections(7, 1, dim), projections(8, 1, dim)
    out, _ = score_bias(geo, fq, fk, pq, pk, reach, far, bias)
    plain, _ = score_bias(geo, fq, fk, pq, pk)
    kind = bias[0][torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long()][None]
    assert bool((out[kind == -math.inf] == -math.inf).all())
    for value, sign in ((low, -1.0), (3e38, 1.0)):
        got = out[kind == value].double()
        assert bool(((got - sign * 2.0 ** 120).abs() <= 4 * EPS * 2.0 ** 120).all())
    assert float((out - plain)[kind == 0].abs().max()) <= 8 * EPS * float(plain.abs().max())


# ------------------------------------------------------------------------------------------- bias gradient


def bias_backward(geo, ds, reach, far, **kw):
    H = ds.shape[0]
    out = torch.full((H, L.veda_bias_buckets(reach, far)), 7.0, device=DEV)
    ws = bytes_(L.veda_bias_backward_workspace_bytes(geo.layout, H, reach))
    L.veda_bias_backward(geo.layout, ds, reach, far, ws, out, **kw)
    assert L.veda_sync_status() == L.VEDA_OK, L.veda_last_error()
    return out


@pytest.mark.parametrize("heads,reach,far", [(1, (3, 3, 3), (8, 8, 8)), (3, (8, 8, 8), (32, 11, 60)), (2, (1, 1, 1), (2, 2, 2)),
                                             (2, (16, 2, 1), (90, 3, 2))])
def test_bias_backward(geo, heads, reach, far):
    ds = randn(1, heads, geo.n, geo.n)
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long().reshape(-1)
    total = L.veda_bias_buckets(reach, far)

    def sums(x):
        return torch.zeros(heads, total, dtype=torch.float64, device=DEV).index_add_(1, index, x.reshape(heads, -1))

    # a bucket's value passes through fewer than 3 n + 64 additions (its row, its rows, the partial sums)
    within(bias_backward(geo, ds, reach, far), sums(ds.double()), (3 * geo.n + 64) * EPS * sums(ds.double().abs()))


@pytest.mark.parametrize("spans,heads", [([((13, 48, 84), (1, 8, 16))], 2), ([((61, 45, 80), (8, 1, 16))], 1),
                                         ([((4000, 1, 1), (1, 1, 128))], 1), ([((29, 90, 160), (1, 8, 16)), ((7, 64, 64), (2, 8, 8))], 1),
                                         ([((7300, 1, 1), (1, 1, 128))], 1), ([((72, 80, 170), (1, 8, 16))], 1)])
def test_bias_backward_wide_layouts(spans, heads):
    # every width of the kernel: 468, 1800, 4000, 3686 + 224, 7300 tiles, and 7920 tiles whose offsets fit no shared memory
    geo, reach, far = Geometry(spans), (4, 4, 6), (16, 16, 32)
    ds = randn(1, heads, geo.n, geo.n)
    total = L.veda_bias_buckets(reach, far)
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long().reshape(-1)

    def sums(x):
        return torch.zeros(heads, total, dtype=torch.float64, device=DEV).index_add_(1, index, x.reshape(heads, -1))

    got = bias_backward(geo, ds, reach, far)
    within(got, sums(ds.double()), (3 * geo.n + 64) * EPS * sums(ds.double().abs()))
    assert torch.equal(bias_backward(geo, ds, reach, far), got)


# --------------------------------------------------------------------------------------------- distillation


def distill(geo, scores, idx, val, cnt, tau, weight=None, grad=True, by_column=False, status=L.VEDA_OK, **kw):
    loss = torch.full(cnt.shape, 7.0, device=DEV)
    d = torch.full(scores.shape, 7.0, device=DEV) if grad else None
    L.veda_distill(geo.layout, scores, idx, val, cnt, tau, loss, d_scores=d, row_weight=weight, by_column=by_column, **kw)
    assert L.veda_sync_status() == status, L.veda_last_error()
    return loss, d


def check_distill(geo, scores, idx, val, cnt, tau, weight, loss, d):
    n = geo.n
    want, grad, p, q = T.plain_distill(scores, idx, val, cnt, tau, weight, n)
    # arguments of exp are off by 2^-22 of their size (the inverse of tau and the product round), exp by 2^-22 relative,
    # a sum of m terms by m 2^-24 relative
    top = float(scores[torch.isfinite(scores)].abs().max()) / tau
    topt = float(val[torch.isfinite(val)].abs().max()) / tau
    r = 4 * EPS * (2 * top + 1) + n * EPS
    rt = 4 * EPS * (2 * topt + 1) + idx.shape[2] * EPS
    w = torch.ones_like(want) if weight is None else weight.double()
    within(d, grad, (w / tau)[..., None] * (2 * (r + EPS * 4) * q + 2 * (rt + EPS * 4) * p) + 4 * EPS * grad.abs())
    gap = 2 * (top + topt) + math.log(max(n, 2))
    within(loss, want, w * (4 * r + 4 * rt) * (1 + gap))


@pytest.mark.parametrize("k,tau,heads", [(1, 1.0, 2), (5, 0.5, 1), (40, 3.7, 3), (1000, 1.0, 1)])
def test_distill(geo, k, tau, heads):
    scores = 2 * randn(1, heads, geo.n, geo.n)
    idx, val, cnt = T.top_lists(geo, scores + 2 * randn(2, heads, geo.n, geo.n), k)
    weight = (0.5 + torch.rand(heads, geo.n, device=DEV)) / geo.n
    loss, d = distill(geo, scores, idx, val, cnt, tau, weight)
    check_distill(geo, scores, idx, val, cnt, tau, weight, loss, d)
    assert torch.equal(distill(geo, scores, idx, val, cnt, tau, weight, grad=False)[0], loss)
    # the dense form of the same teacher gives the same bits
    dense = torch.full_like(scores, math.nan)
    inside = idx < geo.n
    dense.scatter_(2, torch.where(inside, idx, idx[..., :1]).long(), torch.where(inside, val, val[..., :1]))
    loss2, d2 = distill(geo, scores, idx, dense, cnt, tau, weight, by_column=True)
    assert torch.equal(loss2, loss) and torch.equal(d2, d)


@pytest.mark.parametrize("n_side,heads", [(((259, 1, 40), (2, 1, 64)), 2), (((1500, 1, 1), (1, 1, 128)), 1),
                                          (((2100, 2, 1), (1, 2, 64)), 1), (((5000, 1, 1), (1, 1, 128)), 1),
                                          (((16384, 1, 1), (1, 1, 128)), 1)])
def test_distill_long_rows(n_side, heads):
    geo = Geometry([n_side])
    scores = 2 * randn(1, heads, geo.n, geo.n)
    idx, val, cnt = T.top_lists(geo, 3 * randn(2, heads, geo.n, geo.n), 70)
    cnt -= (torch.arange(geo.n, device=DEV) % 3).int()
    loss, d = distill(geo, scores, idx, val, cnt, 2.0)
    rows = slice(0, geo.n) if geo.n < 6000 else slice(3, geo.n, 1021)  # the widest: some rows

    class Some:
        n = geo.n

    want = [x[:, rows] for x in (scores, idx, val, cnt, loss, d)]
    t = torch.full((heads, want[0].shape[1], geo.n), -math.inf, dtype=torch.float64, device=DEV)
    on = torch.arange(idx.shape[2], device=DEV) < want[3][..., None]
    s = want[0].double() / 2.0
    for h in range(heads):
        for r in range(t.shape[1]):
            t[h, r, want[1][h, r][on[h, r]].long()] = want[2][h, r][on[h, r]].double() / 2.0
    p, q = torch.softmax(t, 2), torch.softmax(s, 2)
    e = 4 * EPS * (2 * float(s.abs().max()) + 20) + geo.n * EPS
    within(want[5], (q - p) / 2, e * (q + p) + 8 * EPS * (q - p).abs())
    ref = torch.where(p > 0, p * (torch.log_softmax(t, 2) - torch.log_softmax(s, 2)), 0.0).sum(2)
    within(want[4], ref, 8 * e * (1 + ref.abs() + float(s.abs().max())))


def test_distill_rows_left_out_and_infinities():
    geo = Geometry(**GEOMETRIES["refs"])
    n, H = geo.n, 2
    scores = randn(1, H, n, n)
    idx, val, cnt = T.top_lists(geo, randn(2, H, n, n), 6)
    glob = geo.layout.n_tiles - n
    cnt[0, 0] = 0                                # an empty list
    idx[0, 1, :glob] = torch.arange(n, n + glob, device=DEV).int()
    cnt[0, 1] = glob                             # global tiles only
    val[0, 2] = -math.inf                        # listed, but no mass
    val[0, 3, 1:4] = -math.inf                   # mass on some
    scores[0, 4] = -math.inf                     # no student column
    scores[0, 5, int(idx[0, 5, 0])] = -math.inf  # the teacher has mass where the student has none
    scores[0, 6, 2] = torch.finfo(torch.float32).min  # a mask of the type's lowest value
    scores[0, 7, :] = torch.finfo(torch.float32).min
    val[0, 8, :2] = torch.finfo(torch.float32).min
    loss, d = distill(geo, scores, idx, val, cnt, 1.0)
    for r in (0, 1, 2, 4):
        assert float(loss[0, r]) == 0 and not bool(d[0, r].any())
    assert float(loss[0, 5]) == math.inf and bool(torch.isfinite(d[0, 5]).all())
    fine = torch.ones(H, n, dtype=torch.bool, device=DEV)
    fine[0, 4] = fine[0, 7] = False
    want, grad, p, q = T.plain_distill(scores, idx, val, cnt, 1.0, None, n)
    # sizes below 2^5 after the shift by the maxima
    tol = 64 * EPS * 32 + n * EPS
    within(torch.where(fine, loss, 0.0), torch.where(fine, want, 0.0), 16 * tol)
    within(d[fine], grad[fine], tol)
    # an even row of lowest values: q is uniform, whatever the level
    assert float((d[0, 7] + p[0, 7].float()).sub(1 / n).abs().max()) <= 8 * EPS
    scores[1, 0, 3] = math.nan
    scores[1, 1, 4] = math.inf
    val[1, 2, 0] = math.nan
    loss, d = distill(geo, scores, idx, val, cnt, 1.0)
    assert bool(torch.isnan(loss[1, :3]).all()) and bool(torch.isfinite(loss[1, 3:]).all())
    assert bool(torch.isnan(d[1, :2]).all()) and bool(torch.isfinite(d[1, 3:]).all())


def test_distill_malformed_lists_are_cut_and_reported():
    geo = Geometry(**GEOMETRIES["refs"])
    n, H = geo.n, 1
    scores = randn(1, H, n, n)
    idx, val, cnt = T.top_lists(geo, randn(2, H, n, n), 6)
    good_idx, good_cnt = idx.clone(), cnt.clone()
    changes = {0: (3, -1), 1: (2, geo.layout.n_tiles), 2: (4, int(idx[0, 2, 3])), 3: (0, -5), 4: (1, 1 << 30)}
    for r, (e, v) in changes.items():
        idx[0, r, e] = v
        good_cnt[0, r] = e
    cnt[0, 5] = idx.shape[2] + 7   # longer than its row: what is there counts
    cnt[0, 6] = -3
    good_cnt[0, 6] = 0
    got = distill(geo, scores, idx, val, cnt, 1.0, status=L.VEDA_ERR_BAD_LIST)
    want = distill(geo, scores, good_idx, val, good_cnt, 1.0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ----------------------------------------------------------------------------------- projections' gradients


def score_backward(geo, fq, fk, hats, ds, **kw):
    H, D = hats.shape[1], hats.shape[3]
    out = [torch.full((H, 3 * D, D), 7.0, device=DEV) for _ in range(2)]
    ws = bytes_(L.veda_score_backward_workspace_bytes(geo.layout, H, D))
    L.veda_score_backward(geo.layout, fq, fk, hats, ds, ws, *out, **kw)
    assert L.veda_sync_status() == L.VEDA_OK, L.veda_last_error()
    return out


@pytest.mark.parametrize("spans,dim,heads", [([((13, 48, 84), (1, 8, 16))], 128, 1), ([((13, 48, 84), (1, 8, 16))], 64, 5),
                                             ([((26, 48, 84), (2, 16, 4))], 128, 2)])
def test_score_backward_cut_along_k(spans, dim, heads):
    # 468 and 819 tiles of few heads: the products' K is cut over the CTAs and joined
    check_score_backward(Geometry(spans), dim, heads)


@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 1), (128, 2)])
def test_score_backward(geo, dim, heads):
    check_score_backward(geo, dim, heads)


def check_score_backward(geo, dim, heads):
    n = geo.n
    fq, fk, hats = feats(1, heads, n, dim), feats(4, heads, n, dim), randn(7, 2, heads, n, dim)
    ds = torch.softmax(2 * randn(9, heads, n, n), 2) - torch.softmax(4 * randn(10, heads, n, n), 2)
    got = score_backward(geo, fq, fk, hats, ds)
    q, k = hats.double()
    for out, f, m, x in ((got[0], fq, ds.double(), k), (got[1], fk, ds.double().transpose(1, 2), q)):
        c = 1 / math.sqrt(dim)
        dx, tx = c * (m @ x), c * product_tol(m, x, n + 4)
        ft = f.double().transpose(1, 2)
        within(out, ft @ dx, ft.abs() @ tx + product_tol(ft, dx.abs() + tx, n))


# ---------------------------------------------------------------------------------------- limits of the sizes


def test_many_heads():
    # more heads than SMs, and than the bias gradient has chunks for
    geo, H, D, reach, far = Geometry([((2, 16, 24), (2, 8, 8))], text=130), 301, 64, (3, 2, 3), (8, 8, 8)
    n = geo.n
    q, k = T.tile_rows(geo, 1, H, D), T.tile_rows(geo, 3, H, D)
    within(teacher(geo, q, k), T.plain_teacher(geo, q, k), teacher_tol(q, k, None))
    fq, fk, pq, pk = feats(1, H, n, D), feats(4, H, n, D), projections(7, H, D), projections(8, H, D)
    bias = randn(9, H, L.veda_bias_buckets(reach, far))
    out, hats = score_bias(geo, fq, fk, pq, pk, reach, far, bias)
    qh, kh = T.plain_hats(fq, fk, pq, pk)
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long()
    want = qh @ kh.transpose(1, 2) / math.sqrt(D) + bias.double()[:, index]
    # 3 D and D additions, each at most 2^-23 of sums of magnitudes below 2^9
    within(out, want, torch.full_like(want, 4 * D * 2 * EPS * 2.0 ** 9))
    scores = randn(11, H, n, n)
    idx, val, cnt = T.top_lists(geo, randn(12, H, n, n), 3)
    loss, d = distill(geo, scores, idx, val, cnt, 2.0)
    check_distill(geo, scores, idx, val, cnt, 2.0, None, loss, d)
    sums = torch.zeros(H, bias.shape[1], dtype=torch.float64, device=DEV)
    sums.index_add_(1, index.reshape(-1), d.double().reshape(H, -1))
    within(bias_backward(geo, d, reach, far), sums, torch.full_like(sums, (3 * n + 64) * EPS * n * n))
    got = score_backward(geo, fq, fk, hats, d)
    again = score_backward(geo, fq, fk, hats, d)
    assert all(torch.equal(a, b) and bool(torch.isfinite(a).all()) for a, b in zip(got, again))


def test_largest_layout():
    # 16,384 tiles of one row each: every operator at the limit, compared on some rows
    geo, D, reach, far = Geometry([((16384, 1, 1), (1, 1, 128))]), 64, (8, 1, 1), (4000, 2, 2)
    n, some = geo.n, torch.tensor([0, 1, 127, 128, 8191, 12345, 16383], device=DEV)
    q, k = T.tile_rows(geo, 1, 1, D), T.tile_rows(geo, 3, 1, D)
    rows, keys = (x[0].reshape(n, 128, D)[:, 0].double() for x in (q, k))
    out = teacher(geo, q, k)
    within(out[0, some], rows[some] @ keys.T / 8, teacher_tol(q, k, None))
    del out
    fq, fk, pq, pk = feats(1, 1, n, D), feats(4, 1, n, D), projections(7, 1, D), projections(8, 1, D)
    bias = randn(9, 1, L.veda_bias_buckets(reach, far))
    scores, hats = score_bias(geo, fq, fk, pq, pk, reach, far, bias)
    qh, kh = T.plain_hats(fq, fk, pq, pk)
    r = torch.arange(n, device=DEV)[None] - some[:, None]
    classes = torch.as_tensor(L.veda_bias_index(Geometry([((300, 1, 1), (1, 1, 128))]).layout, (8, 1, 1), (4000, 2, 2))[0], device=DEV)
    near = (r.abs() < 300)
    index = torch.where(r > 0, classes[r.clamp(0, 299)].long(), torch.zeros_like(r))
    want = qh[0, some] @ kh[0].T / 8
    got = scores[0, some].double() - want
    # offsets of 0 to 299 keys behind have the buckets of a short line; differences stay within the scores' error
    ahead = near & (r >= 0)
    tol = 4 * D * 2 * EPS * 2.0 ** 9
    assert float((got - bias[0].double()[index])[ahead].abs().max()) <= tol
    del scores
    ds = randn(11, 1, n, n)
    dq, dk = score_backward(geo, fq, fk, hats, ds)
    dx = ds[0].double() @ hats[1, 0].double() / 8
    want = fq[0].double().T @ dx
    bound = fq[0].abs().double().T @ product_tol(ds[0].double(), hats[1, 0].double() / 8, n)
    within(dq[0], want, bound + product_tol(fq[0].double().T, dx, n))
    total = bias_backward(geo, ds, reach, far)
    assert abs(float(total.double().sum()) - float(ds.double().sum())) <= (3 * n + 64) * EPS * float(ds.abs().double().sum())
    zero = float(torch.diagonal(ds[0]).double().sum())  # distance 0 is a bucket of its own
    at = int(L.veda_bias_index(Geometry([((1, 1, 1), (1, 1, 128))]).layout, reach, far)[0, 0])
    assert abs(float(total[0, at]) - zero) <= (3 * n + 64) * EPS * float(torch.diagonal(ds[0]).abs().double().sum())


# ------------------------------------------------------------------------------------------------ together


def step(geo, fq, fk, pq, pk, reach, far, bias, idx, val, cnt, tau, weight):
    """One training step through the entry points: summed loss, gradients of both projections and the bias."""
    scores, hats = score_bias(geo, fq, fk, pq, pk, reach, far, bias)
    loss, ds = distill(geo, scores, idx, val, cnt, tau, weight)
    dq, dk = score_backward(geo, fq, fk, hats, ds)
    return loss, dq, dk, bias_backward(geo, ds, reach, far)


def plain_loss(geo, fq, fk, pq, pk, index, bias, idx, val, cnt, tau, weight):
    D = pq.shape[2]
    q, k = (f.double() @ p + f.double()[..., :D] for f, p in ((fq, pq), (fk, pk)))
    s = q @ k.transpose(1, 2) / math.sqrt(D) + bias[:, index]
    on = (torch.arange(idx.shape[2], device=DEV) < cnt[..., None]) & (idx < geo.n)
    t = torch.where(on, val.double() / tau, -math.inf)
    p, logp = torch.softmax(t, 2), torch.log_softmax(t, 2)
    logq = torch.log_softmax(s / tau, 2).gather(2, torch.where(on, idx, 0).long())
    return (weight.double() * torch.where(on, p * (logp - logq), 0.0).sum(2)).sum()


def test_gradients_of_a_step_match_differences():
    geo = Geometry(**GEOMETRIES["refs"])
    H, D, tau, reach, far = 2, 64, 2.0, (3, 2, 4), (8, 8, 8)
    fq, fk, pq, pk = feats(1, H, geo.n, D), feats(4, H, geo.n, D), projections(7, H, D), projections(8, H, D)
    bias = randn(9, H, L.veda_bias_buckets(reach, far))
    index = torch.as_tensor(L.veda_bias_index(geo.layout, reach, far), device=DEV).long()
    idx, val, cnt = T.top_lists(geo, 2 * randn(10, H, geo.n, geo.n), 7)
    weight = torch.full((H, geo.n), 1.0 / (H * geo.n), device=DEV)
    loss, dq, dk, db = step(geo, fq, fk, pq, pk, reach, far, bias, idx, val, cnt, tau, weight)
    f = lambda a, b, c: float(plain_loss(geo, fq, fk, a, b, index, c, idx, val, cnt, tau, weight))  # noqa: E731
    base = [x.double() for x in (pq, pk, bias)]
    assert abs(float(loss.double().sum()) - f(*base)) <= 1e-5 * abs(f(*base))
    for which, grad in enumerate((dq, dk, db)):
        for seed in range(3):
            dirn = torch.sign(randn(20 + seed, *base[which].shape)).double()
            h = 1e-5  # central difference in 64 bits: truncation of order h^2, rounding of order 1e-16 / h
            ends = []
            for sign in (1, -1):
                moved = list(base)
                moved[which] = base[which] + sign * h * dirn
                ends.append(f(*moved))
            slope, got = (ends[0] - ends[1]) / (2 * h), float((grad.double() * dirn).sum())
            # the kernels' own error: well under 2^-15 of the gradient's 1-norm
            assert abs(slope - got) <= 2.0 ** -15 * float(grad.double().abs().sum()) + 1e-8, (which, slope, got)


def test_step_is_deterministic_on_streams_and_in_a_graph():
    geo = Geometry(**GEOMETRIES["wide"])
    H, D, tau, reach, far = 2, 128, 1.0, (4, 4, 4), (8, 8, 8)
    n, buckets = geo.n, L.veda_bias_buckets((4, 4, 4), (8, 8, 8))
    lay = geo.layout
    weight = torch.full((H, n), 1.0 / n, device=DEV)

    def inputs(seed):
        x = dict(q=T.tile_rows(geo, seed, H, D), k=T.tile_rows(geo, seed + 2, H, D), fq=feats(seed, H, n, D),
                 fk=feats(seed + 4, H, n, D), pq=projections(seed + 7, H, D), pk=projections(seed + 8, H, D),
                 bias=randn(seed + 9, H, buckets))
        return x

    def buffers():
        f = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
        return dict(teacher=f(H, n, n), hats=f(2, H, n, D), scores=f(H, n, n), loss=f(H, n), ds=f(H, n, n),
                    dq=f(H, 3 * D, D), dk=f(H, 3 * D, D), db=f(H, buckets),
                    idx=torch.zeros(H, n, lay.max_kept, dtype=torch.int32, device=DEV),
                    cnt=torch.zeros(H, n, dtype=torch.int32, device=DEV),
                    ws=[bytes_(L.veda_score_bias_workspace_bytes(lay, H, D, reach)),
                        bytes_(L.veda_score_backward_workspace_bytes(lay, H, D)),
                        bytes_(L.veda_bias_backward_workspace_bytes(lay, H, reach))])

    def all_steps(x, b, stream=None):
        L.veda_teacher(lay, x["q"], x["k"], b["teacher"], stream=stream)
        L.veda_select(lay, b["teacher"], b["idx"], b["cnt"], stream)
        L.veda_score_bias(lay, x["fq"], x["fk"], x["pq"], x["pk"], reach, far, x["bias"], b["hats"], b["ws"][0],
                          b["scores"], stream)
        L.veda_distill(lay, b["scores"], b["idx"], b["teacher"], b["cnt"], tau, b["loss"], b["ds"], weight, True, stream)
        L.veda_score_backward(lay, x["fq"], x["fk"], b["hats"], b["ds"], b["ws"][1], b["dq"], b["dk"], stream)
        L.veda_bias_backward(lay, b["ds"], reach, far, b["ws"][2], b["db"], stream)

    outs = ("teacher", "hats", "scores", "loss", "ds", "dq", "dk", "db", "cnt")
    xs = [inputs(100), inputs(200)]
    want = []
    for x in xs:
        b = buffers()
        all_steps(x, b)
        torch.cuda.synchronize()
        want.append({o: b[o].clone() for o in outs})
        assert not any(bool(torch.isnan(b[o].float()).any()) for o in outs)
    # two at once on streams of their own, again and again
    streams, bufs = [torch.cuda.Stream() for _ in xs], [buffers() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, b, s in zip(xs, bufs, streams):
            all_steps(x, b, s)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert all(torch.equal(b[o], w[o]) for o in outs)
    # captured, and replayed on new inputs in the same buffers
    x, b = {k: v.clone() for k, v in xs[0].items()}, buffers()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        all_steps(x, b)
    for new, w in zip(xs[::-1], want[::-1]):
        for k, v in new.items():
            x[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[o], w[o]) for o in outs)
    assert L.veda_sync_status() == L.VEDA_OK


def test_binding_refuses_host_tensors():
    geo = Geometry(**GEOMETRIES["tiny"])
    n = geo.n
    with pytest.raises(L.VedaError) as e:
        L.veda_bias_backward(geo.layout, torch.zeros(1, n, n), (3, 3, 3), (8, 8, 8), bytes_(1 << 20),
                             torch.zeros(1, 127, device=DEV))
    assert e.value.code == L.VEDA_ERR_INVALID and "cpu" in str(e.value)
