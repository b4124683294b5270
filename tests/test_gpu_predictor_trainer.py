"""A layer's predictor training end to end: the teacher's lists, the loss and the gradients against 64-bit autograd, the
layer with a relative position bias."""
import math

import pytest
import torch

import oracle as O
import veda_synth as V
from learned_block_sparse_tile_b200 import PredictorTrainer, VedaLayer
from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B

pytestmark = pytest.mark.gpu
REACH, FAR = (3, 4, 3), (8, 12, 8)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    L.veda_device_check()


def make(name, bias=True):
    wl = V.workload(name)
    q, k, v = (x.cuda() for x in V.make_qkv(wl))
    layer = VedaLayer(wl.seq_len, wl.ref_spans, wl.target, wl.head_shapes, (wl.generated, wl.reference), wl.heads, wl.dim)
    pq, pk = V.make_projections(wl)
    layer.set_projections(pq, pk)
    table = None
    if bias:
        g = torch.Generator("cpu").manual_seed(5)
        table = 0.3 * torch.randn(wl.heads, L.veda_bias_buckets(REACH, FAR), generator=g)
        layer.set_bias(REACH, FAR, table)
    return wl, layer, q, k, v, pq, pk, table


def plain_teacher(wl, lay_o, q, k, h, lse):
    rows = torch.as_tensor(lay_o.perm.reshape(-1, 128)[:lay_o.n_video].copy()).cuda().long()
    real = rows >= 0
    n, D = len(rows), q.shape[2]
    x = torch.einsum("ird,jsd->ijrs", q[rows.clamp_min(0), h].double(), k[rows.clamp_min(0), h].double()) / math.sqrt(D)
    if lse is not None:
        x = x - lse[h][rows.clamp_min(0)].double()[:, None, :, None]
    return torch.where(real[:, None, :, None] & real[None, :, None, :], x, -math.inf).amax(dim=(2, 3))


@pytest.mark.parametrize("name,bias,with_lse", [("small_mixed", True, False), ("padded_tiny", False, True), ("tiny", True, True)])
def test_step_matches_autograd(name, bias, with_lse):
    wl, layer, q, k, v, pq, pk, table = make(name, bias)
    lse = None
    if with_lse:  # full attention's own softmax sums
        lse = torch.logsumexp(torch.einsum("shd,thd->hst", q.double(), k.double()) / math.sqrt(wl.dim), dim=2).float()
    trainer = PredictorTrainer(layer, tau=1.5)
    trainer.teach(q, k, row_lse=lse)
    loss, grads = trainer.step()
    assert L.veda_sync_status() == L.VEDA_OK
    leaves = [x.double().cuda().requires_grad_() for x in (pq, pk)] + ([table.double().cuda().requires_grad_()] if bias else [])
    total, rows = 0.0, sum(len(g["heads_list"]) * g["layout"].n_video for g in layer.groups)
    for g, s in zip(layer.groups, trainer.state):
        lay = g["layout"]
        spans = O.layer_spans(wl.ref_spans, (wl.target[0], wl.target[1], g["box"]), not O.keeps_all(wl.reference))
        lay_o = O.build_layout(spans, wl.seq_len)
        for at, h in enumerate(g["heads_list"]):
            t = plain_teacher(wl, lay_o, q, k, h, lse)
            # bf16 products summed in fp32: D + 8 roundings of at most 2^-23 of |q| |k| / sqrt(D), and lse's own
            big = float(q[:, h].float().norm(dim=1).max() * k[:, h].float().norm(dim=1).max()) / math.sqrt(wl.dim)
            assert float((s["teacher"][at].double() - t).abs().max()) <= (wl.dim + 8) * 2.0 ** -23 * (big + 40)
            on = torch.zeros(lay.n_video, lay.n_tiles, dtype=torch.bool, device="cuda")
            for r in range(lay.n_video):
                on[r, s["idx"][at, r, :int(s["cnt"][at, r])].long()] = True
            on = on[:, :lay.n_video]
            assert bool(on.any(dim=1).all())
            D = wl.dim
            qh = s["feats_q"][at].double() @ leaves[0][h] + s["feats_q"][at, :, :D].double()
            kh = s["feats_k"][at].double() @ leaves[1][h] + s["feats_k"][at, :, :D].double()
            x = qh @ kh.T / math.sqrt(D)
            if bias:
                x = x + leaves[2][h][torch.as_tensor(L.veda_bias_index(lay, REACH, FAR), device="cuda").long()]
            p = torch.softmax(torch.where(on, s["teacher"][at].double() / 1.5, -math.inf), dim=1)
            logq = torch.log_softmax(x / 1.5, dim=1)
            total = total + torch.where(on, p * (p.clamp_min(1e-300).log() - logq), 0.0).sum() / rows
    want, total = torch.autograd.grad(total, leaves), total.detach()
    # the scores are right to about 1e-6 of their size (below 2^6), which moves q, loss and gradients by 2^-13 at most
    assert abs(float(loss) - float(total)) <= 2.0 ** -13 * abs(float(total))
    for key, w in zip(("proj_q", "proj_k", "bias"), want):
        got = grads[key].double()
        assert got.shape == w.shape
        assert float((got - w).norm()) <= 2.0 ** -13 * float(w.norm()), key
    assert set(grads) == {"proj_q", "proj_k"} | ({"bias"} if bias else set())


def test_layer_with_a_bias_selects_by_score_plus_bias():
    wl, layer, q, k, v, pq, pk, table = make("small_mixed")
    out, plain = (torch.zeros(wl.seq_len, wl.heads, wl.dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    launches = layer.launches
    layer.forward(q, k, v, out)
    assert L.veda_sync_status() == L.VEDA_OK
    biased = [(g["scores"].clone(), g["kept_idx"].clone(), g["kept_cnt"].clone()) for g in layer.groups]
    layer.set_bias()
    assert layer.launches == launches + len(layer.groups)
    layer.forward(q, k, v, plain)
    for g, (s, idx, cnt) in zip(layer.groups, biased):
        lay = g["layout"]
        index = torch.as_tensor(L.veda_bias_index(lay, REACH, FAR), device="cuda").long()
        want = g["scores"].double() + table.double().cuda()[g["heads"].long()][:, index]
        tol = 1e-5 * float(want.abs().max())  # the score tolerance of both paths
        assert float((s.double() - want).abs().max()) <= 2 * tol
        again_idx, again_cnt = torch.full_like(idx, -1), torch.empty_like(cnt)
        L.veda_select(lay, s, again_idx, again_cnt)
        assert torch.equal(again_cnt, cnt)
        on = torch.arange(idx.shape[2], device="cuda") < cnt[..., None]
        assert torch.equal(torch.where(on, again_idx, 0), torch.where(on, idx, 0))
    assert not torch.equal(out, plain)
    # a zero bias gives veda_score's scores, and no bias restores the layer's results bit for bit
    layer.set_bias(REACH, FAR, torch.zeros_like(table))
    layer.forward(q, k, v, out)
    layer.set_bias()
    again = torch.zeros_like(plain)
    layer.forward(q, k, v, again)
    assert torch.equal(again, plain)
    assert L.veda_sync_status() == L.VEDA_OK


@pytest.mark.parametrize("direct", [True, False])
def test_bias_on_both_attend_paths(direct):
    wl = V.workload("padded_tiny")
    q, k, v = (x.cuda() for x in V.make_qkv(wl))
    layer = VedaLayer(wl.seq_len, wl.ref_spans, wl.target, wl.head_shapes, (wl.generated, wl.reference), wl.heads, wl.dim,
                      direct=direct)
    layer.set_projections(*V.make_projections(wl))
    layer.set_bias(REACH, FAR, torch.randn(wl.heads, L.veda_bias_buckets(REACH, FAR)))
    out = torch.zeros(wl.seq_len, wl.heads, wl.dim, dtype=torch.bfloat16, device="cuda")
    layer.forward(q, k, v, out)
    assert L.veda_sync_status() == L.VEDA_OK and bool(torch.isfinite(out.float()).all())


def test_steps_follow_the_parameters():
    wl, layer, q, k, v, pq, pk, table = make("tiny")
    trainer = PredictorTrainer(layer)
    with pytest.raises(ValueError):
        trainer.step()
    trainer.teach(q, k)
    loss, grads = trainer.step()
    again, same = trainer.step()
    assert torch.equal(loss, again) and all(torch.equal(grads[x], same[x]) for x in grads)
    layer.set_projections(pq - 0.1 * grads["proj_q"].cpu(), pk - 0.1 * grads["proj_k"].cpu())
    layer.set_bias(REACH, FAR, table - 0.1 * grads["bias"].cpu())
    after, moved = trainer.step()
    assert bool(torch.isfinite(after)) and not torch.equal(after, loss)
    assert all(bool(torch.isfinite(moved[x]).all()) and not torch.equal(moved[x], grads[x]) for x in grads)
    layer.set_bias()
    plain, without = trainer.step()
    assert bool(torch.isfinite(plain)) and set(without) == {"proj_q", "proj_k"}


def test_refusals():
    wl, layer, q, k, v, pq, pk, table = make("tiny")
    trainer = PredictorTrainer(layer)
    for args in ((q[:-1], k[:-1]), (q.float(), k.float()), (q, k, torch.zeros(wl.heads, 3, device="cuda"))):
        with pytest.raises(ValueError):
            trainer.teach(*args)
    with pytest.raises(ValueError):
        layer.set_bias(REACH, FAR, table[:, :-1])
    with pytest.raises(ValueError):
        layer.set_bias(REACH, FAR)
