"""Training the tile predictor of a VedaLayer: the teacher, the distillation loss and the gradients.

The pages summarise the method ("max-pooled full attention gives the tile-level distribution", which the predictor's
scores learn) and print no training code. Here the teacher pools full attention's logits, or its probabilities when the
rows' softmax sums are given; its top tiles under the layer's own budgets are the target, and the predictor's scores
(with the layer's relative position bias, if it has one) are trained on them. Q and K are a frozen model's.

    trainer = PredictorTrainer(layer)          # a VedaLayer with set_projections, and set_bias or not
    trainer.teach(q, k)                        # once per batch
    loss, grads = trainer.step()               # mean loss; gradients of proj_q, proj_k and bias
    ...                                        # the caller's optimizer, then layer.set_projections / set_bias

The operators run in libveda's kernels; PyTorch allocates the buffers, supplies the stream, puts the groups' gradients into
the layer's head order and sums the loss.
"""
from __future__ import annotations

import torch

from . import _lib as L


class PredictorTrainer:
    """Teacher lists and gradient buffers for one layer. ``tau``: the temperature of both distributions."""

    def __init__(self, layer, tau=1.0):
        self.layer, self.tau = layer, float(tau)
        self.state = None

    def _buffers(self, g):
        n, lay, dim = len(g["heads_list"]), g["layout"], self.layer.dim
        f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=self.layer.device)  # noqa: E731
        i = lambda *shape: torch.empty(shape, dtype=torch.int32, device=self.layer.device)  # noqa: E731
        b = lambda size: torch.empty(max(size, 256), dtype=torch.uint8, device=self.layer.device)  # noqa: E731
        nv = lay.n_video
        return dict(feats_q=f(n, nv, 3 * dim), feats_k=f(n, nv, 3 * dim), teacher=f(n, nv, nv), idx=i(n, nv, lay.max_kept),
                    cnt=i(n, nv), hats=f(2, n, nv, dim), scores=f(n, nv, nv), d_scores=f(n, nv, nv), loss=f(n, nv),
                    d_q=f(n, 3 * dim, dim), d_k=f(n, 3 * dim, dim), weight=f(n, nv),
                    score_ws=b(L.veda_score_bias_workspace_bytes(lay, n, dim)),
                    back_ws=b(L.veda_score_backward_workspace_bytes(lay, n, dim)))

    def teach(self, q, k, row_lse=None, stream=None):
        """Pools the features of q and k (bf16 [S, H, D] cuda, any strides veda_gather takes) and makes the teacher's
        lists. ``row_lse``: fp32 [H, S], the logarithm of each row's softmax sum under full attention (the teacher then
        pools probabilities), or None (it pools logits)."""
        layer = self.layer
        st = stream if stream is not None else torch.cuda.current_stream(layer.device)
        if tuple(q.shape) != (layer.seq_len, layer.heads, layer.dim) or q.shape != k.shape:
            raise ValueError("PredictorTrainer.teach: q and k must be [S, H, D] of the layer")
        if row_lse is not None and tuple(row_lse.shape) != (layer.heads, layer.seq_len):
            raise ValueError("PredictorTrainer.teach: row_lse must be [H, S]")
        if q.dtype is not torch.bfloat16 or k.dtype is not torch.bfloat16:
            raise ValueError("PredictorTrainer.teach: q and k must be bf16")
        with torch.cuda.stream(st):
            if self.state is None:
                self.state = [self._buffers(g) for g in layer.groups]
                rows = sum(s["loss"].numel() for s in self.state)
                for s in self.state:
                    s["weight"].fill_(1.0 / rows)
            for g, s in zip(layer.groups, self.state):
                lay, n = g["layout"], len(g["heads_list"])
                # the tile-order copies live for this call only
                q_t = torch.empty(n, lay.n_slots, layer.dim, dtype=torch.bfloat16, device=layer.device)
                k_t = torch.empty_like(q_t)
                L.veda_gather(lay, q, g["heads"], q_t, s["feats_q"], st)
                L.veda_gather(lay, k, g["heads"], k_t, s["feats_k"], st)
                lse = None if row_lse is None else row_lse.index_select(0, g["heads"].long())
                L.veda_teacher(lay, q_t, k_t, s["teacher"], row_lse=lse, stream=st)
                L.veda_select(lay, s["teacher"], s["idx"], s["cnt"], st)

    def step(self, stream=None):
        """(loss, gradients) of the layer's present projections and bias on the batch of the last teach: the mean loss
        over heads and query tiles (a 0-d fp32 cuda tensor) and a dict of fp32 cuda tensors in the layer's head order,
        proj_q and proj_k [H, 3D, D] and, with a bias, bias [H, buckets]. teach and step share buffers: whoever makes
        them on several streams orders them, as with every tensor that torch hands out on a stream."""
        layer = self.layer
        if self.state is None:
            raise ValueError("PredictorTrainer.step: call teach first")
        st = stream if stream is not None else torch.cuda.current_stream(layer.device)
        spec = layer.bias_spec
        with torch.cuda.stream(st):
            f = lambda *shape: torch.zeros(shape, dtype=torch.float32, device=layer.device)  # noqa: E731
            grads = {"proj_q": f(layer.heads, 3 * layer.dim, layer.dim), "proj_k": f(layer.heads, 3 * layer.dim, layer.dim)}
            if spec is not None:
                grads["bias"] = f(layer.heads, L.veda_bias_buckets(*spec))
            losses = []
            for g, s in zip(layer.groups, self.state):
                lay, heads = g["layout"], g["heads"].long()
                reading = layer._before_read(st)
                L.veda_score_bias(lay, s["feats_q"], s["feats_k"], g["proj_q"], g["proj_k"], *(spec or (None, None)),
                                  g["bias"] if spec else None, s["hats"], s["score_ws"], s["scores"], st)
                layer._after_read(reading)
                L.veda_distill(lay, s["scores"], s["idx"], s["teacher"], s["cnt"], self.tau, s["loss"],
                               d_scores=s["d_scores"], row_weight=s["weight"], by_column=True, stream=st)
                L.veda_score_backward(lay, s["feats_q"], s["feats_k"], s["hats"], s["d_scores"], s["back_ws"], s["d_q"],
                                      s["d_k"], st)
                grads["proj_q"][heads] = s["d_q"]
                grads["proj_k"][heads] = s["d_k"]
                if spec is not None:
                    n = len(g["heads_list"])
                    ws = torch.empty(max(L.veda_bias_backward_workspace_bytes(lay, n, spec[0]), 256), dtype=torch.uint8,
                                     device=layer.device)
                    d_bias = torch.empty_like(g["bias"])
                    L.veda_bias_backward(lay, s["d_scores"], *spec, ws, d_bias, st)
                    grads["bias"][heads] = d_bias
                losses.append(s["loss"].sum())
            return torch.stack(losses).sum(), grads
