"""Cases of the operators that train the tile predictor: the pooled teacher, the scores with a learned relative position
bias, the distillation loss and the gradients.

``own`` False computes each operator from elementary torch operations in 32 bits; ``own`` True calls the library.
"""
import functools
import math

import torch

own = False

TILE = 128
DEV = "cuda"

# Geometries: a target grid in (t, h, w) rows cut into boxes of 128 rows, reference grids before it, text rows first.
# They are the workloads the repository's benchmark and tests run: the 104,832-row layer (26, 48, 84), the 219,600-row
# layer (61, 45, 80), a ragged quarter of its length, the 2,048-row layer and a text + reference + target sequence.
_TINY = {"text": 0, "refs": "", "ref_box": "", "grid": "8,16,16", "box": "2,8,8"}
_MIXED = {"text": 150, "refs": "2,16,16", "ref_box": "2,8,8", "grid": "6,16,24", "box": "2,8,8"}
_RAGGED = {"text": 300, "refs": "", "ref_box": "", "grid": "7,45,80", "box": "1,8,16"}
_L104K = {"text": 0, "refs": "", "ref_box": "", "grid": "26,48,84", "box": "2,16,4"}
_LONG = {"text": 0, "refs": "", "ref_box": "", "grid": "61,45,80", "box": "8,1,16"}


def listed():
    return [
        # pooled teacher: a short clip (latency), a ragged sequence weighted by the softmax sums, a quarter of the heads
        # of a full layer (the tensor-core bound)
        dict(_TINY, name="teacher 2k", op="teacher", heads=2, dim=64, lse=False),
        dict(_RAGGED, name="teacher 25k ragged", op="teacher", heads=24, dim=128, lse=True),
        dict(_L104K, name="teacher 104k", op="teacher", heads=4, dim=128, lse=False),
        # scores with the bias: a head group of a small mixed sequence, all heads of the full layer
        dict(_MIXED, name="score_bias mixed", op="score_bias", heads=3, dim=64, reach="3,3,3", far="8,8,8"),
        dict(_L104K, name="score_bias 104k", op="score_bias", heads=24, dim=128, reach="4,4,6", far="16,16,32"),
        # gradient of the bias table from the gradient of the scores
        dict(_MIXED, name="bias_grad mixed", op="bias_grad", heads=3, dim=64, reach="3,3,3", far="8,8,8"),
        dict(_L104K, name="bias_grad 104k", op="bias_grad", heads=24, dim=128, reach="4,4,6", far="16,16,32"),
        # loss and its gradient: the small sequence, the full layer at ratio 0.10, the long layer at ratio 0.05
        dict(_MIXED, name="distill mixed", op="distill", heads=3, dim=64, ratio=0.30, tau=2.0),
        dict(_L104K, name="distill 104k", op="distill", heads=24, dim=128, ratio=0.10, tau=1.0),
        dict(_LONG, name="distill 220k", op="distill", heads=24, dim=128, ratio=0.05, tau=1.0),
        # gradients of the two projections: the small sequence, the full layer
        dict(_MIXED, name="score_grad mixed", op="score_grad", heads=3, dim=64),
        dict(_L104K, name="score_grad 104k", op="score_grad", heads=24, dim=128),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["teacher", "score_bias", "bias_grad", "distill", "score_grad"])
    exps = rng.choice([(a, b, 7 - a - b) for a in range(5) for b in range(8 - a)])
    box = [1 << e for e in exps]
    grid = [_logint(rng, 1, 61), _logint(rng, 3, 48), _logint(rng, 4, 84)]
    heads, dim = _logint(rng, 1, 24), rng.choice([64, 128])
    while math.prod(-(-g // b) for g, b in zip(grid, box)) > 1700 or (
            op == "teacher" and math.prod(math.ceil(g / b) * b for g, b in zip(grid, box)) ** 2 * heads > 4.2e10):
        if heads > 4 and op == "teacher":
            heads //= 2
        else:
            a = grid.index(max(grid))
            grid[a] = max(1, int(grid[a] * 0.8))
    case = {"op": op, "text": rng.choice([0, 1, rng.randint(2, 600)]), "refs": "", "ref_box": "",
            "grid": ",".join(map(str, grid)), "box": ",".join(map(str, box)), "heads": heads, "dim": dim}
    if rng.random() < 0.4:
        case.update(refs="%d,%d,%d" % (rng.randint(1, 2), rng.randint(2, 20), rng.randint(3, 24)), ref_box="1,8,16")
    if op == "teacher":
        case["lse"] = rng.random() < 0.5
    if op in ("score_bias", "bias_grad"):
        reach = [rng.randint(1, 8) for _ in range(3)]
        case.update(reach=",".join(map(str, reach)), far=",".join(str(rng.choice([8, 11, 16, 32, 60])) for _ in range(3)))
    if op == "distill":
        case.update(ratio=round(rng.uniform(0.03, 0.5), 3), tau=rng.choice([0.5, 1.0, 2.0, 3.7]))
    return case


# ------------------------------------------------------------------------------------------------------- geometry


def _ints(text):
    return tuple(int(x) for x in text.split(",")) if text else ()


def _spans(case):
    """[(first row, grid, box)] in packed order (text rows, references, target) and the number of rows."""
    at, out = int(case["text"]), []
    for grid, box in ((_ints(case["refs"]), _ints(case["ref_box"])), (_ints(case["grid"]), _ints(case["box"]))):
        if grid:
            out.append((at, grid, box))
            at += math.prod(grid)
    return out, at


@functools.lru_cache(maxsize=None)
def _geometry(text, refs, ref_box, grid, box):
    """perm [n_tiles, 128] (packed row of each tile slot, real rows first, -1 behind them) and coord [n_video, 4]
    (span, t, h, w in tiles); video tiles in box order (h, w, t), then the text rows in runs of 128."""
    spans, seq = _spans({"text": text, "refs": refs, "ref_box": ref_box, "grid": grid, "box": box})
    perms, coords = [], []
    for number, (start, g, b) in enumerate(spans):
        nt, nh, nw = (-(-x // y) for x, y in zip(g, b))
        bh, bw, bt = (x.reshape(-1, 1) for x in torch.meshgrid(torch.arange(nh), torch.arange(nw), torch.arange(nt), indexing="ij"))
        it, ih, iw = (x.reshape(1, -1) for x in torch.meshgrid(*(torch.arange(x) for x in b), indexing="ij"))
        t, h, w = bt * b[0] + it, bh * b[1] + ih, bw * b[2] + iw
        real = (t < g[0]) & (h < g[1]) & (w < g[2])
        rows = torch.where(real, start + (t * g[1] + h) * g[2] + w, -1)
        perms.append(rows.gather(1, (~real).int().argsort(dim=1, stable=True)))
        coords.append(torch.cat([torch.full_like(bt, number), bt, bh, bw], dim=1))
    coord = torch.cat(coords)
    rest = torch.full((-(-text // TILE) * TILE,), -1)
    rest[:text] = torch.arange(text)
    perm = torch.cat(perms + [rest.reshape(-1, TILE)])
    return perm.to(DEV), coord.to(DEV), seq


def _of(case):
    return _geometry(case["text"], case["refs"], case["ref_box"], case["grid"], case["box"])


@functools.lru_cache(maxsize=None)
def _layout(text, refs, ref_box, grid, box):
    import learned_block_sparse_tile_b200 as B
    spans, seq = _spans({"text": text, "refs": refs, "ref_box": ref_box, "grid": grid, "box": box})
    return B.veda_plan(spans, seq, (0.10, None), (0.50, None))


def _classes(reach, far, top):
    """Distance class of 0..top tiles: `reach` classes, the first half one distance each, the others widening
    geometrically up to `far` tiles. Compared in whole numbers: no rounding at a border."""
    exact = (reach + 1) // 2
    wide = reach - exact
    out = []
    for a in range(top + 1):
        c = a if a < exact else exact + sum(a ** wide >= exact ** (wide - m) * far ** m for m in range(1, wide + 1))
        out.append(min(c, reach - 1))
    return out


def _buckets(case, coord):
    """Bucket of every (query tile, key tile) pair, and how many there are."""
    reach, far = _ints(case["reach"]), _ints(case["far"])
    index = torch.zeros(len(coord), len(coord), dtype=torch.int64, device=DEV)
    for axis in range(3):
        r = coord[None, :, axis + 1] - coord[:, None, axis + 1]
        table = torch.tensor(_classes(reach[axis], far[axis], int(r.abs().max())), device=DEV)
        c = table[r.abs()]
        index = index * (2 * reach[axis] - 1) + torch.where(r > 0, reach[axis] - 1 + c, c)
    pairs = math.prod(2 * x - 1 for x in reach)
    span = coord[None, :, 0] - coord[:, None, 0]
    return torch.where(span < 0, pairs, torch.where(span > 0, pairs + 1, index)), pairs + 2


# --------------------------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    perm, coord, seq = _of(case)
    H, D, n = case["heads"], case["dim"], len(coord)
    f = functools.partial(torch.randn, generator=g, device=DEV)
    s = dict(case=case, n=n, perm=perm, coord=coord)
    if own:
        s["layout"] = _layout(case["text"], case["refs"], case["ref_box"], case["grid"], case["box"])
    if case["op"] == "teacher":
        # rows of a tile share a direction, as neighbouring patches do; bf16 in tile order, zeros behind real rows
        flat = perm.reshape(-1)
        for name in ("q", "k"):
            x = f(H, len(perm), TILE, D) + f(H, len(perm), 1, D)
            s[name] = (x.reshape(H, -1, D) * (flat >= 0)[:, None]).to(torch.bfloat16)
            del x
        s["lse"] = 8 + 2 * f(H, seq) if case["lse"] else None
        s["out"] = torch.empty(H, n, n, device=DEV)
    # per tile and channel: mean, maximum and minimum over the rows, as pooling N(0, 1) rows leaves them
    feats = lambda: torch.cat([0.3 * f(H, n, D), 2.4 + 0.4 * f(H, n, D), -2.4 + 0.4 * f(H, n, D)], dim=2)  # noqa: E731
    if case["op"] in ("score_bias", "score_grad"):
        s["fq"], s["fk"] = feats(), feats()
    if case["op"] == "score_bias":
        s["pq"], s["pk"] = (f(H, 3 * D, D) / math.sqrt(3 * D) for _ in range(2))
    if case["op"] in ("score_bias", "bias_grad"):
        s["index"], s["buckets"] = _buckets(case, coord)
        s["reach"], s["far"] = _ints(case["reach"]), _ints(case["far"])
    if case["op"] == "score_bias":
        s["bias"] = 0.5 * f(H, s["buckets"])
        s["hats"], s["out"] = torch.empty(2, H, n, D, device=DEV), torch.empty(H, n, n, device=DEV)
    if case["op"] in ("bias_grad", "score_grad"):
        # a softmax less a few teacher entries, over the rows that the mean is taken of
        q = torch.softmax(2 * f(H, n, n), dim=2)
        s["ds"] = (q - torch.softmax(4 * f(H, n, n), dim=2)) / (H * n)
    if case["op"] == "score_grad":
        s["hats"] = f(2, H, n, D)
        s["out"] = [torch.empty(H, 3 * D, D, device=DEV) for _ in range(2)]
    if case["op"] == "bias_grad":
        s["out"] = torch.empty(H, s["buckets"], device=DEV)
    if case["op"] == "distill":
        # the teacher's list of a row: its best columns in ascending order, then the global tiles (no column of the
        # scores); every other row holds one fewer, a few rows hold none
        near = (coord[None, :, 1:] - coord[:, None, 1:]).abs().sum(dim=2).float()
        s["scores"] = 2 * f(H, n, n) - 0.2 * near
        teacher = 0.6 * s["scores"] + 2 * f(H, n, n)
        k = max(1, round(case["ratio"] * n))
        idx = teacher.topk(k, dim=2).indices.sort(dim=2).values
        extra = torch.arange(n, len(perm), device=DEV).expand(H, n, -1)
        s["idx"] = torch.cat([idx, extra], dim=2).int().contiguous()
        s["val"] = torch.cat([teacher.gather(2, idx), torch.zeros_like(extra, dtype=torch.float32)], dim=2).contiguous()
        less = (torch.arange(n, device=DEV) % 2).expand(H, n) if not len(extra[0, 0]) and k > 1 else 0
        s["cnt"] = torch.where(torch.rand(H, n, generator=g, device=DEV) < 0.01, 0, s["idx"].shape[2] - less).int()
        s["weight"] = (0.5 + torch.rand(H, n, generator=g, device=DEV)) / (H * n)
        s["out"] = [torch.empty(H, n, device=DEV), torch.empty(H, n, n, device=DEV)]
    if own and case["op"] in ("score_bias", "bias_grad", "score_grad"):
        import learned_block_sparse_tile_b200 as B
        size = {"score_bias": lambda: B.veda_score_bias_workspace_bytes(s["layout"], H, D, s["reach"]),
                "bias_grad": lambda: B.veda_bias_backward_workspace_bytes(s["layout"], H, s["reach"]),
                "score_grad": lambda: B.veda_score_backward_workspace_bytes(s["layout"], H, D)}[case["op"]]()
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------------ operators


def _teacher(s):
    q, k, n = s["q"].float(), s["k"].float(), s["n"]
    H, _, D = q.shape
    real = (s["perm"][:n] >= 0).reshape(-1)
    off = torch.zeros(H, n * TILE, device=DEV)
    if s["lse"] is not None:
        off = s["lse"][:, s["perm"][:n].reshape(-1).clamp_min(0)]
    off = torch.where(real, off, math.inf)
    out = torch.empty(H, n, n, device=DEV)
    step = max(1, (1 << 33) // (n * TILE * TILE))  # 34 GB of logits at a time
    for h in range(H):
        for lo in range(0, n, step):
            r = slice(lo * TILE, min(n, lo + step) * TILE)
            x = q[h, r] @ k[h, :n * TILE].T
            x *= D ** -0.5
            x -= off[h, r, None]
            x.masked_fill_(~real, -math.inf)
            out[h, lo:lo + step] = x.reshape(-1, TILE, n, TILE).amax(dim=(1, 3))
    return out


def _score_bias(s):
    D = s["pq"].shape[2]
    q = s["fq"] @ s["pq"] + s["fq"][..., :D]
    k = s["fk"] @ s["pk"] + s["fk"][..., :D]
    return {"scores": q @ k.transpose(1, 2) * D ** -0.5 + s["bias"][:, s["index"]], "hats": torch.stack([q, k])}


def _bias_grad(s):
    H = len(s["ds"])
    out = torch.zeros(H, s["buckets"], dtype=torch.float64, device=DEV)
    return out.index_add_(1, s["index"].reshape(-1), s["ds"].reshape(H, -1).double()).float()


def _distill(s):
    tau, n = s["case"]["tau"], s["n"]
    idx = s["idx"].long()
    on = (torch.arange(idx.shape[2], device=DEV) < s["cnt"][..., None]) & (idx < n)
    idx = torch.where(on, idx, 0)
    x = s["scores"] / tau
    x = x - x.amax(dim=2, keepdim=True)
    e = x.exp()
    total = e.sum(dim=2, keepdim=True)
    t = torch.where(on, s["val"] / tau, -math.inf)
    t = t - torch.where(on.any(dim=2, keepdim=True), t.amax(dim=2, keepdim=True), 0.0)
    p = t.exp()
    mass = p.sum(dim=2, keepdim=True)
    has = mass > 0
    p = torch.where(has, p / mass, 0.0)
    gap = torch.where(on, t - x.gather(2, idx), 0.0)
    loss = torch.where(has, (p * gap).sum(dim=2, keepdim=True) - mass.log() + total.log(), 0.0)[..., 0]
    scale = s["weight"][..., None] / tau * has
    return {"loss": loss * s["weight"], "d_scores": (scale * e / total).scatter_add_(2, idx, -scale * p)}


def _score_grad(s):
    q, k = s["hats"]
    c = q.shape[2] ** -0.5
    dq = s["ds"] @ k * c
    dk = s["ds"].transpose(1, 2) @ q * c
    return {"d_proj_q": s["fq"].transpose(1, 2) @ dq, "d_proj_k": s["fk"].transpose(1, 2) @ dk}


def run(s):
    op = s["case"]["op"]
    if own:
        import learned_block_sparse_tile_b200 as B
        lay, out = s["layout"], s["out"]
        if op == "teacher":
            B.veda_teacher(lay, s["q"], s["k"], out, row_lse=s["lse"])
            return out
        if op == "score_bias":
            B.veda_score_bias(lay, s["fq"], s["fk"], s["pq"], s["pk"], s["reach"], s["far"], s["bias"], s["hats"],
                              s["workspace"], out)
            return {"scores": out, "hats": s["hats"]}
        if op == "bias_grad":
            B.veda_bias_backward(lay, s["ds"], s["reach"], s["far"], s["workspace"], out)
            return out
        if op == "distill":
            B.veda_distill(lay, s["scores"], s["idx"], s["val"], s["cnt"], s["case"]["tau"], out[0], d_scores=out[1],
                           row_weight=s["weight"])
            return {"loss": out[0], "d_scores": out[1]}
        B.veda_score_backward(lay, s["fq"], s["fk"], s["hats"], s["ds"], s["workspace"], out[0], out[1])
        return {"d_proj_q": out[0], "d_proj_k": out[1]}
    return {"teacher": _teacher, "score_bias": _score_bias, "bias_grad": _bias_grad, "distill": _distill,
            "score_grad": _score_grad}[op](s)


def work(case):
    spans, _ = _spans(case)
    n = sum(math.prod(-(-a // b) for a, b in zip(g, box)) for _, g, box in spans)
    rows = sum(math.prod(g) for _, g, _ in spans)
    H, D, op = case["heads"], case["dim"], case["op"]
    square, feats, proj, hats = H * n * n, 2 * H * n * 3 * D, 2 * H * 3 * D * D, 2 * H * n * D
    if op == "teacher":
        return {"bytes": 4 * H * rows * D + 4 * square, "flops": 2 * H * rows * rows * D}
    if op == "score_bias":
        return {"bytes": 4 * (feats + proj + hats + square), "flops": 4 * H * n * 3 * D * D + 2 * square * D}
    if op == "bias_grad":
        return {"bytes": 4 * square, "flops": square}
    if op == "distill":
        return {"bytes": 8 * square + 8 * H * n * max(1, round(case["ratio"] * n)), "flops": 8 * square}
    return {"bytes": 4 * (square + feats + hats + proj), "flops": 4 * square * D + 4 * H * n * 3 * D * D}


# ---------------------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    s = prepare(case, seed)
    n, op = s["n"], case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "teacher":
        H, D = case["heads"], case["dim"]
        counts = (s["perm"][:n] >= 0).sum(dim=1).tolist()
        full = min(counts) == TILE
        out = torch.empty(H, n, n, dtype=torch.float64, device=DEV)
        keys = d["k"].reshape(H, -1, TILE, D)[:, :n]
        rows = d["q"].reshape(H, -1, TILE, D)[:, :n]
        slot_real = s["perm"][:n] >= 0
        for i, c in enumerate(counts):
            logits = torch.einsum("hrd,hjsd->hrjs", rows[:, i, :c], keys) / math.sqrt(D)
            if not full:
                logits = torch.where(slot_real, logits, -math.inf)
            best = logits.amax(dim=3)
            if "lse" in d:
                best = best - d["lse"][:, s["perm"][i, :c]][..., None]
            out[:, i] = best.amax(dim=1)
        return out
    if op == "score_bias":
        D = case["dim"]
        eye = torch.eye(3 * D, D, dtype=torch.float64, device=DEV)
        q, k = (torch.einsum("hnf,hfd->hnd", d[a], d[b] + eye) for a, b in (("fq", "pq"), ("fk", "pk")))
        bias = torch.gather(d["bias"], 1, s["index"].reshape(1, -1).expand(case["heads"], -1)).reshape(-1, n, n)
        return {"scores": torch.einsum("hid,hjd->hij", q, k) / math.sqrt(D) + bias, "hats": torch.stack([q, k])}
    if op == "bias_grad":
        index = s["index"].reshape(-1).cpu()
        rows = d["ds"].reshape(case["heads"], -1).cpu()
        return torch.stack([torch.bincount(index, weights=row, minlength=s["buckets"]) for row in rows])
    if op == "distill":
        tau = case["tau"]
        width = s["idx"].shape[2]
        on = (torch.arange(width, device=DEV) < s["cnt"][..., None]) & (s["idx"] < n)
        at = torch.where(on, s["idx"].long(), n)  # a column behind the last takes what is not listed
        t = torch.full((case["heads"], n, n + 1), -math.inf, dtype=torch.float64, device=DEV)
        t.scatter_(2, at, torch.where(on, d["val"], -math.inf))
        t = t[..., :n] / tau
        has = on.any(dim=2)
        logp = torch.where(has[..., None], torch.log_softmax(t, dim=2), -math.inf)
        p = logp.exp()
        logq = torch.log_softmax(d["scores"] / tau, dim=2)
        loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(dim=2)
        grad = d["weight"][..., None] * (logq.exp() - p) / tau * has[..., None]
        return {"loss": d["weight"] * loss, "d_scores": grad}
    q, k = d["hats"]
    c = 1 / math.sqrt(case["dim"])
    return {"d_proj_q": c * torch.einsum("hif,hij,hjd->hfd", d["fq"], d["ds"], k),
            "d_proj_k": c * torch.einsum("hjf,hij,hid->hfd", d["fk"], d["ds"], q)}
