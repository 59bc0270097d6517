"""GPU checks of registered calls that take their own workspaces: launched on a
stream behind other work and dropped at once, launched on two streams at the
same time, and captured into a graph that outlives them."""
import gc

import numpy as np
import pytest

from tests import training_reference as ref
from tests.test_gpu_checkpoint import close, grad_inputs
from tests.test_gpu_vocab_loss import Run, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


class Loss:
    """A registered loss with gradients, and what its results have to be."""

    def __init__(self, tide, seed, tokens=600, size=72, vocab=3001):
        import torch

        self.sizes = tokens, size, vocab
        self.h, self.w = (torch.empty(n, size, dtype=torch.bfloat16, device="cuda") for n in (tokens, vocab))
        self.t = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.g, self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(3))
        self.dh, self.dw = torch.empty_like(self.h), torch.empty_like(self.w)
        self.call = tide.vocab_loss_grad_call(self.h, self.w, self.t, self.g, self.loss, self.lse, self.dh, self.dw)
        self.bytes = tide.vocab_loss_workspace(self.h, self.w, self.dw)
        self.fill(seed)

    def fill(self, seed):
        import torch

        h, w, t, g = make(np.random.default_rng(seed), *self.sizes, 0.2)
        self.want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
        for to, x in ((self.h, h), (self.w, w), (self.t, torch.from_numpy(t)), (self.g, torch.from_numpy(g))):
            to.copy_(x)
        for out in (self.loss, self.lse, self.dh, self.dw):
            out.fill_(float("nan"))
        torch.cuda.synchronize()

    def check(self):
        r = Run.__new__(Run)
        r.loss, r.lse, r.dh, r.dw = self.loss, self.lse, self.dh, self.dw
        r.check(self.want)


def busy(stream):
    """A few milliseconds of work on `stream`."""
    import torch

    with torch.cuda.stream(stream):
        a = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
        for _ in range(4):
            a = a @ a


def scribble(nbytes):
    """Takes and overwrites blocks of the current stream's memory."""
    import torch

    return [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]


def test_dropped_behind_other_work(tide):
    import torch

    side = torch.cuda.Stream()
    busy(side)
    torch.cuda.synchronize()
    for seed in range(3):
        job = Loss(tide, seed)
        torch.cuda.synchronize()
        busy(side)
        job.call(side)
        job.call = None
        gc.collect()
        blocks = scribble(job.bytes)
        torch.cuda.synchronize()
        job.check()
        assert all(bool((b == 255).all()) for b in blocks)


def test_weight_gradient_dropped_behind_other_work(tide):
    import torch

    side = torch.cuda.Stream()
    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(1), 5000, 65, 90, "e4m3")
    need = tide.checkpoint_weight_grad_workspace(dy, 90)
    assert need > 0
    dw = torch.full((65, 90), float("nan"), device="cuda")
    torch.cuda.synchronize()
    busy(side)
    tide.checkpoint_weight_grad_call(dy, codes, scales, dw)(side)
    blocks = scribble(need)
    torch.cuda.synchronize()
    close(dw, *ref.weight_grad(y, x), "f32")
    assert all(bool((b == 255).all()) for b in blocks)


def test_two_streams_at_once(tide):
    """One registered call on two streams at the same time: the same results
    from two workspaces."""
    import torch

    job = Loss(tide, 5)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            job.call(s)
    torch.cuda.synchronize()
    job.check()


def test_a_graph_outlives_its_calls(tide):
    import torch

    job = Loss(tide, 7)
    side = torch.cuda.Stream()
    job.call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        job.call()
    job.call = None
    gc.collect()
    for seed in range(8, 12):
        job.fill(seed)
        blocks = scribble(job.bytes)
        graph.replay()
        torch.cuda.synchronize()
        job.check()
        assert all(bool((b == 255).all()) for b in blocks)
