"""Plain 64-bit restatements of the operators that train the tile predictor, for their GPU tests."""
import math

import torch

import oracle as O
from learned_block_sparse_tile_b200 import _lib as L

DEV = "cuda"
EPS = 2.0 ** -24   # half a step of fp32
SPLIT = 1.25 * 2.0 ** -20  # what a split-tf32 product leaves out, relative to |a b|


class Geometry:
    """Spans [(grid, box)] behind ``text`` global rows: the library's layout and the oracle's."""

    def __init__(self, spans, text=0, gap=0, ratio=0.3):
        at, plan = text, []
        for grid, box in spans:
            plan.append((at, grid, box))
            at += math.prod(grid) + gap
        self.seq = at
        self.layout = L.veda_plan(plan, at, (ratio, None), (0.5, None))
        self.oracle = O.build_layout(plan, at)
        self.n = self.layout.n_video
        self.valid = torch.as_tensor(self.oracle.valid_count[:self.n].copy(), device=DEV)
        self.perm = torch.as_tensor(self.oracle.perm.reshape(-1, 128).copy(), device=DEV).long()


def randn(seed, *shape):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV)


def tile_rows(geo, seed, heads, dim):
    """bf16 [heads, N, D] in tile order, zeros in the padding slots, rows of a tile alike."""
    x = randn(seed, heads, len(geo.perm), 128, dim) + randn(seed + 1, heads, len(geo.perm), 1, dim)
    return (x * (geo.perm >= 0)[..., None]).reshape(heads, -1, dim).to(torch.bfloat16)


def plain_teacher(geo, q_t, k_t, lse=None):
    H, _, D = q_t.shape
    n = geo.n
    q, k = (x.double().reshape(H, -1, 128, D)[:, :n] for x in (q_t, k_t))
    x = torch.einsum("hird,hjsd->hijrs", q, k) / math.sqrt(D)
    real = geo.perm[:n] >= 0
    off = torch.zeros(H, n, 128, dtype=torch.float64, device=DEV)
    if lse is not None:
        off = lse.double()[:, geo.perm[:n].clamp_min(0)]
    rows = real & torch.isfinite(off)
    x = x - torch.where(rows, off, 0.0)[:, :, None, :, None]
    keep = rows[:, :, None, :, None] & real[None, None, :, None, :] & ~x.isnan()
    return torch.where(keep, x, -math.inf).amax(dim=(3, 4))


def plain_hats(fq, fk, pq, pk):
    D = pq.shape[2]
    return tuple(f.double() @ p.double() + f.double()[..., :D] for f, p in ((fq, pq), (fk, pk)))


def plain_distill(scores, idx, val, cnt, tau, weight, n):
    """(loss, d_scores, p, q) of rows whose lists are well formed."""
    H, _, W = idx.shape
    on = (torch.arange(W, device=DEV) < cnt[..., None]) & (idx < n)
    t = torch.full((H, n, n + 1), -math.inf, dtype=torch.float64, device=DEV)
    t.scatter_(2, torch.where(on, idx.long(), n), torch.where(on, val.double(), -math.inf))
    t = t[..., :n] / tau
    s = scores.double() / tau
    has = (t.amax(dim=2, keepdim=True) > -math.inf) & (s.amax(dim=2, keepdim=True) > -math.inf)
    p = torch.where(has, torch.softmax(t, dim=2), 0.0)
    q = torch.where(has, torch.softmax(s, dim=2), 0.0)
    logp, logq = torch.log_softmax(t, dim=2), torch.log_softmax(s, dim=2)
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(dim=2)
    w = torch.ones(H, n, dtype=torch.float64, device=DEV) if weight is None else weight.double()
    return w * loss, (w / tau)[..., None] * (q - p), p, q


def top_lists(geo, teacher, k):
    """The k best columns of each row in ascending order, then the layout's global tiles; values beside them."""
    n, H = geo.n, teacher.shape[0]
    idx = teacher.topk(min(k, n), dim=2).indices.sort(dim=2).values
    extra = torch.arange(n, geo.layout.n_tiles, device=DEV).expand(H, n, -1)
    val = torch.cat([teacher.gather(2, idx), torch.zeros(extra.shape, device=DEV)], dim=2)
    idx = torch.cat([idx, extra], dim=2).int().contiguous()
    return idx, val.float().contiguous(), torch.full((H, n), idx.shape[2], dtype=torch.int32, device=DEV)
