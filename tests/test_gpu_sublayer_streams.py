"""GPU checks that every call of the sublayer's operators runs on the stream it is
given, behind that stream's work: its inputs are only filled there, and outputs hold
NaN until it has run.  Registered, called once with a stream, and on the current
one; two streams at once, each with outputs of its own."""
import pytest

from tests.test_gpu_training_calls import busy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


# (function, sizes): a few rows and many, rows read by loops; tokens that are streamed past, small tiles, larger ones with
# copies; from kept gates and without; a small matrix and a list
KINDS = {
    "norm": ("layer_norm", (3000, 1100)), "norm_few": ("layer_norm", (5, 200)), "norm_wide": ("layer_norm", (40, 17000)),
    "norm_grad": ("layer_norm_grad", (3000, 1100)), "norm_grad_wide": ("layer_norm_grad", (40, 17000)),
    "block_few": ("gated_block", (9, 333, 1041)), "block_small": ("gated_block", (60, 320, 640)),
    "block": ("gated_block", (700, 333, 1041)), "block_grad_few": ("gated_block_grad", (9, 333, 1041)),
    "block_grad": ("gated_block_grad", (700, 333, 1041)), "block_grad_kept": ("gated_block_grad", (700, 320, 640, True)),
    "update": ("orthogonalize", (1, 100, 260)), "updates": ("orthogonalize", (5, 500, 900)),
}


class Job:
    """Inputs that hold NaN until fill(), outputs that do until a call has run, and what
    they have to be then."""

    def __init__(self, tide, kind, seed):
        import torch

        self.function, sizes = KINDS[kind]
        gen = torch.Generator("cuda").manual_seed(seed)
        b, f = torch.bfloat16, torch.float32

        def rand(*shape, unit=1.0, dtype=b):
            return (torch.randn(*shape, generator=gen, device="cuda") * unit).to(dtype)

        def blank(*shape, dtype=b):
            return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

        if self.function == "layer_norm":
            rows, n = sizes
            ins = [rand(rows, n, dtype=f), rand(n), rand(n)]
            self.outs = [blank(rows, n), blank(rows, dtype=f), blank(rows, dtype=f)]
            self.arguments = lambda i: (*i, *self.outs)
        elif self.function == "layer_norm_grad":
            rows, n = sizes
            ins = [rand(rows, n), rand(rows, n), rand(n, dtype=f), rand(rows, dtype=f), rand(rows, dtype=f).abs()]
            self.outs = [blank(rows, n), blank(n, dtype=f), blank(n, dtype=f)]
            self.arguments = lambda i: (*i, *self.outs)
        elif self.function == "gated_block":
            t, n, k = sizes
            ins = [rand(t, n), rand(k, n, unit=0.05), rand(k, n, unit=0.05)]
            self.outs = [blank(t, k), blank(t, 2 * k)]
            self.arguments = lambda i: (*i, *self.outs)
        elif self.function == "gated_block_grad":
            t, n, k, *kept = sizes
            ins = [rand(t, k), rand(t, n), rand(k, n, unit=0.05), rand(k, n, unit=0.05)] + ([rand(t, 2 * k)] if kept else [])
            self.outs = [blank(t, n), blank(k, n), blank(k, n)]
            self.arguments = lambda i: (*i[:4], *self.outs, *i[4:])
        else:
            count, r, c = sizes
            ins = [rand(r, c, dtype=f) for _ in range(count)]
            self.outs = [blank(r, c) for _ in ins]
            self.arguments = lambda i: (list(i), self.outs)
        self.values, self.ins = ins, [torch.full_like(t, float("nan")) for t in ins]
        getattr(tide, self.function)(*self.arguments(ins))
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.outs]
        assert all(bool(t.isfinite().all()) for t in self.want)
        self.clear()

    def clear(self):
        import torch

        for t in (*self.outs, *self.ins):
            t.fill_(float("nan"))
        torch.cuda.synchronize()

    def fill(self):
        for t, v in zip(self.ins, self.values):
            t.copy_(v)

    def check(self):
        import torch

        assert all(torch.equal(t, w) for t, w in zip(self.outs, self.want))


def launch(tide, job, how, stream):
    import torch

    function, args = getattr(tide, job.function), job.arguments(job.ins)
    if how == "registered":
        getattr(tide, job.function + "_call")(*args)(stream)
    elif how == "once":
        function(*args, stream=stream)
    else:
        with torch.cuda.stream(stream):
            function(*args)


@pytest.mark.parametrize("how", ["registered", "once", "current"])
@pytest.mark.parametrize("kind", KINDS)
def test_on_its_stream(tide, kind, how):
    import torch

    jobs = [Job(tide, kind, seed) for seed in range(2)]
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(2):
        for job in jobs:
            job.clear()
        for job, s in zip(jobs, streams):
            busy(s)
            with torch.cuda.stream(s):
                job.fill()
            launch(tide, job, how, s)
        torch.cuda.synchronize()
        for job in jobs:
            job.check()
