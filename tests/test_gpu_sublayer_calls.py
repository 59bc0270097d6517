"""GPU checks of registered calls of layer norm's gradients, the gated block and
the orthogonalized updates that take their own workspaces: launched on a stream
behind other work and dropped at once, on two streams at the same time, and
captured into graphs that outlive them."""
import gc

import pytest

from tests.test_gpu_training_calls import busy, scribble

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


class Job:
    """A registered call with a workspace, its inputs and its outputs."""

    def __init__(self, tide, kind, seed):
        import torch

        gen = torch.Generator("cuda").manual_seed(seed)
        b = torch.bfloat16

        def rand(*shape, unit=1.0, dtype=b):
            return (torch.randn(*shape, generator=gen, device="cuda") * unit).to(dtype)

        if kind == "norm":
            rows, n = 3000, 1100
            x, dy, w = rand(rows, n), rand(rows, n), rand(n, dtype=torch.float32)
            mean, rstd = (rand(rows, dtype=torch.float32) for _ in range(2))
            self.inputs = [dy, x, w, mean, rstd]
            self.outputs = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
            self.call = tide.layer_norm_grad_call(*self.inputs, *self.outputs)
            self.bytes = tide.layer_norm_grad_workspace(x, dy)
        elif kind == "block":
            tokens, n, f = 700, 333, 1041
            x, wg, wu, dh = rand(tokens, n), rand(f, n, unit=0.05), rand(f, n, unit=0.05), rand(tokens, f)
            self.inputs = [dh, x, wg, wu]
            self.outputs = [torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)]
            self.call = tide.gated_block_grad_call(*self.inputs, *self.outputs)
            self.bytes = tide.gated_block_workspace(x, wg, wu, gradients=True)
        else:
            self.inputs = [rand(500, 900, dtype=torch.float32) for _ in range(5)]
            self.outputs = [torch.empty(500, 900, dtype=b, device="cuda") for _ in range(5)]
            self.call = tide.orthogonalize_call(self.inputs, self.outputs)
            self.bytes = tide.orthogonalize_workspace(self.inputs)
        assert self.bytes > 0
        self.call()
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.outputs]
        assert all(bool(t.isfinite().all()) for t in self.want)
        self.clear()

    def clear(self):
        import torch

        for t in self.outputs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()

    def check(self):
        import torch

        assert all(torch.equal(t, w) for t, w in zip(self.outputs, self.want))


KINDS = ["norm", "block", "updates"]


@pytest.mark.parametrize("kind", KINDS)
def test_dropped_behind_other_work(tide, kind):
    import torch

    side = torch.cuda.Stream()
    busy(side)
    torch.cuda.synchronize()
    for seed in range(2):
        job = Job(tide, kind, seed)
        busy(side)
        job.call(side)
        job.call = None
        gc.collect()
        blocks = scribble(job.bytes)
        torch.cuda.synchronize()
        job.check()
        assert all(bool((b == 255).all()) for b in blocks)


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(tide, kind):
    """Two registered calls of the same kind on two streams, several times: each
    launch has queues and partial sums of its own."""
    import torch

    jobs = [Job(tide, kind, seed) for seed in range(2)]
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        for job in jobs:
            job.clear()
        for _ in range(4):
            for job, s in zip(jobs, streams):
                job.call(s)
        torch.cuda.synchronize()
        for job in jobs:
            job.check()


@pytest.mark.parametrize("kind", KINDS)
def test_graphs_outlive_their_calls(tide, kind):
    """Two captured graphs replayed one beside the other, with eager work between
    the replays."""
    import torch

    jobs = [Job(tide, kind, seed) for seed in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in jobs]
    for job in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            job.call()
        job.call = None
    gc.collect()
    for _ in range(3):
        blocks = scribble(jobs[0].bytes)
        for job in jobs:
            job.clear()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for job in jobs:
            job.check()
        assert all(bool((b == 255).all()) for b in blocks)
