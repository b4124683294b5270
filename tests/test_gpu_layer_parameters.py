"""A layer's parameters set while work that reads them is queued on other streams, and behind a captured forward; the
launches it counts."""
import ctypes as C
import math

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


def test_streams_by_handle_and_streams_that_are_gone():
    # a stream as its handle, made and destroyed by its owner between two changes of the parameters
    m = Made(direct=True)
    rt = C.CDLL("libcudart.so.12")
    for i in (0, 1):
        m.set(m.sets[i])
        handle = C.c_void_p()
        assert rt.cudaStreamCreate(C.byref(handle)) == 0
        out = m.forward(handle.value)
        assert rt.cudaStreamSynchronize(handle) == 0
        assert torch.equal(out, m.outs[i])
        assert rt.cudaStreamDestroy(handle) == 0
    m.layer.set_bias()
    m.layer.set_bias((2, 2, 2), FAR, torch.ones(m.layer.heads, 29))
    m.forward()
    torch.cuda.synchronize()


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


def kernel_nodes(call):
    """Kernels that ``call`` launches, counted in a captured graph."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    rt = C.CDLL("libcudart.so.12")
    raw, count = C.c_void_p(graph.raw_cuda_graph()), C.c_size_t()
    assert rt.cudaGraphGetNodes(raw, None, C.byref(count)) == 0
    nodes = (C.c_void_p * count.value)()
    assert rt.cudaGraphGetNodes(raw, nodes, C.byref(count)) == 0
    kernels = 0
    for node in nodes:
        kind = C.c_int()
        assert rt.cudaGraphNodeGetType(C.c_void_p(node), C.byref(kind)) == 0
        kernels += kind.value == 0
    return kernels


@pytest.mark.parametrize("dim,heads,grid", [(64, 2, (8, 16, 16)), (128, 2, (8, 16, 16)), (128, 40, (8, 16, 16)), (128, 3, (8, 48, 48))])
def test_a_layer_counts_the_launches_it_makes(dim, heads, grid):
    seq = math.prod(grid)
    layer = VedaLayer(seq, (), (0, grid), ((2, 8, 8),) * heads, ((0.3, None), (1.0, None)), heads, dim)
    layer.set_projections(*(torch.randn(heads, 3 * dim, dim) / math.sqrt(3 * dim) for _ in range(2)))
    q, k, v = (torch.randn(seq, heads, dim, device="cuda").to(torch.bfloat16) for _ in range(3))
    out = torch.empty_like(q)
    plain = kernel_nodes(lambda: layer.forward(q, k, v, out))
    assert layer.launches == plain
    table = torch.zeros(heads, L.veda_bias_buckets((3, 3, 3), (8, 8, 8)))
    for _ in range(2):
        layer.set_bias((3, 3, 3), (8, 8, 8), table)
        assert layer.launches == kernel_nodes(lambda: layer.forward(q, k, v, out))
    layer.set_bias()
    assert layer.launches == plain == kernel_nodes(lambda: layer.forward(q, k, v, out))


def test_a_captured_step_follows_the_parameters_and_the_teacher():
    m = Made()
    trainer = PredictorTrainer(m.layer)
    inputs = [(m.q, m.k), (m.k, m.q)]
    want = {}
    for i in (0, 1):
        for j in (0, 1):
            m.set(m.sets[i])
            trainer.teach(*inputs[j])
            loss, grads = trainer.step()
            want[i, j] = loss.clone(), {x: grads[x].clone() for x in grads}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads = trainer.step()
    for i, j in ((0, 0), (1, 0), (1, 1), (0, 1)):
        m.set(m.sets[i])
        trainer.teach(*inputs[j])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[i, j][0]) and all(torch.equal(grads[x], want[i, j][1][x]) for x in grads)


@pytest.mark.parametrize("fp8,int8", [(True, False), (False, True)])
def test_a_bias_on_layers_of_8_bit_codes(fp8, int8):
    wl = V.workload("small_d128")
    q, k, v = (x.cuda() for x in V.make_qkv(wl))
    layer = VedaLayer(wl.seq_len, wl.ref_spans, wl.target, wl.head_shapes, (wl.generated, wl.reference), wl.heads, wl.dim,
                      fp8_qk=fp8, int8_qk=int8)
    layer.set_projections(*V.make_projections(wl))
    outs, kept = [], []
    for bias in (None, torch.zeros(wl.heads, L.veda_bias_buckets(REACH, FAR)), 4 * torch.randn(wl.heads, L.veda_bias_buckets(REACH, FAR))):
        layer.set_bias(*((None, None, None) if bias is None else (REACH, FAR, bias)))
        out = torch.zeros(wl.seq_len, wl.heads, wl.dim, dtype=torch.bfloat16, device="cuda")
        layer.forward(q, k, v, out)
        torch.cuda.synchronize()
        outs.append(out)
        kept.append([g["kept_cnt"].clone() for g in layer.groups])
        assert bool(torch.isfinite(out.float()).all())
    # the budgets stay, what is kept under them changes with a bias that is not zero
    assert all(torch.equal(a, b) for other in kept[1:] for a, b in zip(kept[0], other))
    assert not torch.equal(outs[0], outs[2])
