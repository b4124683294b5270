"""A layer's parameters set while work that reads them is queued on other streams, and behind a captured forward."""
import pytest
import torch

import veda_synth as V
from learned_block_sparse_tile_b200 import PredictorTrainer, VedaLayer
from learned_block_sparse_tile_b200 import _lib as L
from learned_block_sparse_tile_b200 import build as B

pytestmark = pytest.mark.gpu
REACH, FAR = (3, 4, 3), (8, 12, 8)
BUSY = 100_000_000  # clocks that a stream is kept busy for, some 50 ms


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    L.veda_device_check()
    yield
    assert L.veda_sync_status() == L.VEDA_OK


class Made:
    """A layer, its inputs and two sets of parameters (of one shape) with the output of each."""

    def __init__(self, name="small_mixed", direct=None):
        wl = V.workload(name)
        self.q, self.k, self.v = (x.cuda() for x in V.make_qkv(wl))
        self.layer = VedaLayer(wl.seq_len, wl.ref_spans, wl.target, wl.head_shapes, (wl.generated, wl.reference), wl.heads, wl.dim,
                               direct=direct)
        pq, pk = V.make_projections(wl)
        g = torch.Generator("cpu").manual_seed(5)
        table = 2 * torch.randn(wl.heads, L.veda_bias_buckets(REACH, FAR), generator=g)
        self.sets = [(pq, pk, table), (pk, pq, -table)]
        self.outs = []
        for s in self.sets:
            self.set(s)
            self.outs.append(self.forward())
        assert not torch.equal(*self.outs)

    def set(self, s):
        self.layer.set_projections(s[0], s[1])
        self.layer.set_bias(REACH, FAR, s[2])

    def forward(self, stream=None):
        out = torch.zeros_like(self.q)
        torch.cuda.current_stream().synchronize()  # (out is zeroed before another stream writes it)
        return self.layer.forward(self.q, self.k, self.v, out, stream=stream)


def churn():
    """Blocks of many sizes taken and overwritten on the current stream, as a program that goes on would."""
    for size in [1 << e for e in range(9, 25)] * 2:
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("direct", [True, False])
def test_a_queued_forward_keeps_the_parameters_it_was_called_with(direct):
    m, side = Made(direct=direct), torch.cuda.Stream()
    for change in (lambda: m.set(m.sets[1]), lambda: m.layer.set_bias(),
                   lambda: m.layer.set_bias((2, 2, 2), FAR, torch.ones(m.layer.heads, 29))):
        m.set(m.sets[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        out = m.forward(side)
        change()
        churn()
        torch.cuda.synchronize()
        assert torch.equal(out, m.outs[0])


def test_a_forward_elsewhere_waits_for_the_parameters():
    m, side = Made(), torch.cuda.Stream()
    table = m.sets[1][2].cuda()
    m.layer.set_projections(*m.sets[1][:2])
    m.layer.set_bias(REACH, FAR, m.sets[0][2])
    torch.cuda.synchronize()
    out = torch.zeros_like(m.q)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)                       # the current stream is behind, and with it the new bias
    m.layer.set_bias(REACH, FAR, table)
    m.layer.forward(m.q, m.k, m.v, out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, m.outs[1])


def test_a_queued_step_keeps_the_parameters_it_was_called_with():
    m, side = Made(), torch.cuda.Stream()
    trainer = PredictorTrainer(m.layer)
    trainer.teach(m.q, m.k)
    m.set(m.sets[0])
    want, grads = trainer.step()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    loss, got = trainer.step(stream=side)
    m.set(m.sets[1])
    churn()
    torch.cuda.synchronize()
    assert torch.equal(loss, want) and all(torch.equal(got[x], grads[x]) for x in grads)
    other, _ = trainer.step()
    assert not torch.equal(other, want)


def test_a_captured_forward_replays_with_new_parameters():
    m = Made()
    out = torch.zeros_like(m.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.layer.forward(m.q, m.k, m.v, out)
    for i in (0, 1, 0):
        m.set(m.sets[i])
        churn()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, m.outs[i])
    assert L.veda_sync_status() == L.VEDA_OK


def test_parameters_from_the_device():
    # as an optimizer leaves them: on the GPU, leaves that require a gradient
    m = Made()
    for i in (0, 1):
        pq, pk, table = (x.cuda().requires_grad_() for x in m.sets[i])
        m.layer.set_projections(pq, pk)
        m.layer.set_bias(REACH, FAR, table)
        out = m.forward()
        torch.cuda.synchronize()
        assert torch.equal(out, m.outs[i]) and not out.requires_grad
        assert not any(g[key].requires_grad for g in m.layer.groups for key in ("proj_q", "proj_k", "bias"))
