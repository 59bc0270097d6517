"""A training step of a feed-forward sublayer on two simulated ranks, of the
library's operators alone: layer norm, the gated block, its output packed for the
backward pass, all the gradients, their reduce-scatter into shards, the mean
gathered back, and the matrices' mean orthogonalized.  Each operator's results are
checked against 64-bit references of what it was given; the whole step also as a
captured graph."""
import numpy as np
import pytest

from tests import sublayer_reference as ref, training_reference
from tests.test_gpu_checkpoint import close as close_packed, device
from tests.test_gpu_gated_block import check_grads
from tests.test_gpu_layer_norm import close, held, nan
from tests.test_gpu_orthogonalize import check as check_update

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def f64(t):
    return t.double().cpu().numpy()


class Step:
    """The buffers and registered calls of a step."""

    def __init__(self, tide, tokens, hidden, ffn, act, keep, world=2):
        import torch

        self.tide, self.act, self.world = tide, act, world
        self.shapes = [(ffn, hidden), (ffn, hidden), (hidden, ffn), (hidden,), (hidden,)]
        self.plan = plan = tide.Plan(world, self.shapes)
        self.params = [nan(s, "bf16") for s in self.shapes]
        wg, wu, wd, nw, nb = self.params
        c, s = tide.checkpoint_layout(ffn)
        self.ranks, self.calls = [], []
        for _ in range(world):
            r = dict(x=nan((tokens, hidden), "f32"), y=nan((tokens, hidden), "bf16"), mean=nan((tokens,), "f32"),
                     rstd=nan((tokens,), "f32"), h=nan((tokens, ffn), "bf16"),
                     gates=nan((tokens, 2 * ffn), "bf16") if keep else None, dout=nan((tokens, hidden), "bf16"),
                     dh=nan((tokens, ffn), "bf16"), dy=nan((tokens, hidden), "bf16"), dx=nan((tokens, hidden), "f32"),
                     codes=torch.zeros(tokens, c, dtype=torch.int8, device="cuda"),
                     scales=torch.zeros(tokens, s, dtype=torch.uint8, device="cuda"),
                     grads=[nan(s, "bf16") for s in self.shapes])
            dwg, dwu, dwd, dnw, dnb = r["grads"]
            self.ranks.append(r)
            self.calls += [
                tide.layer_norm_call(r["x"], nw, nb, r["y"], r["mean"], r["rstd"], eps=EPS),
                tide.gated_block_call(r["y"], wg, wu, r["h"], r["gates"], activation=act),
                tide.checkpoint_pack_call(r["h"], r["codes"], r["scales"]),
                tide.checkpoint_weight_grad_call(r["dout"], r["codes"], r["scales"], dwd),
                tide.gated_block_grad_call(r["dh"], r["y"], wg, wu, r["dy"], dwg, dwu, gates=r["gates"], activation=act),
                tide.layer_norm_grad_call(r["dy"], r["x"], nw, r["mean"], r["rstd"], r["dx"], dnw, dnb),
            ]
        self.shards = [nan((plan.shard_elems,), "f32") for _ in range(world)]
        self.flat = nan((world * plan.shard_elems,), "bf16")
        self.means = [nan(s, "bf16") for s in self.shapes]
        self.updates = [nan(s, "bf16") for s in self.shapes[:3]]
        self.calls += [
            tide.reduce_scatter_call(plan, [r["grads"] for r in self.ranks], self.shards, alpha=1.0 / world),
            tide.allgather_copyin_call(plan, [[t[o:o + n] for o, n in zip(plan.shard_offset, real)]
                                              for t, real in zip(self.shards, plan.n_real)], self.flat),
            tide.allgather_copyout_call(plan, self.flat, self.means),
            tide.orthogonalize_call(self.means[:2], self.updates[:2]),
            tide.orthogonalize_call(self.means[2:3], self.updates[2:]),
        ]

    def fill(self, seed):
        rng = np.random.default_rng(seed)
        for p, unit in zip(self.params, (0.05, 0.05, 0.05, 0.3, 1.0)):
            p.copy_(device(held(rng.standard_normal(tuple(p.shape)) * unit + (unit == 0.3), "bf16"), "bf16"))
        for r in self.ranks:
            for k, t, unit in (("x", "f32", 2.0), ("dout", "bf16", 0.01), ("dh", "bf16", 0.01)):
                r[k].copy_(device(held(rng.standard_normal(tuple(r[k].shape)) * unit, t), t))

    def outputs(self):
        own = [r[k] for r in self.ranks for k in ("y", "mean", "rstd", "h", "gates", "dy", "dx") if r[k] is not None]
        return own + [g for r in self.ranks for g in r["grads"]] + self.shards + self.means + self.updates

    def clear(self):
        for t in self.outputs():
            t.fill_(float("nan"))

    def run(self):
        for c in self.calls:
            c()

    def check(self):
        import torch

        wg, wu, _, nw, nb = (f64(p) for p in self.params)
        for r in self.ranks:
            want = ref.layer_norm(f64(r["x"]), nw, nb, EPS)
            for k, name, t in (("y", "out", "bf16"), ("mean", "mean", "f32"), ("rstd", "rstd", "f32")):
                close(r[k], want[name], t, k)
            want = ref.gated_block(f64(r["y"]), wg, wu, self.act)
            close(r["h"], want["out"], "bf16", "h")
            gates = None
            if r["gates"] is not None:
                close(r["gates"], want["gates"], "bf16", "gates")
                gates = f64(r["gates"])
            dwg, dwu, dwd, dnw, dnb = r["grads"]
            packed = training_reference.unpack(r["codes"].cpu().numpy(), r["scales"].cpu().numpy(), "int8", wg.shape[0])
            close_packed(dwd, *training_reference.weight_grad(f64(r["dout"]), packed), "bf16")
            check_grads((r["dy"], dwg, dwu), ref.gated_block_grad(f64(r["dh"]), f64(r["y"]), wg, wu, self.act, gates), "bf16")
            want = ref.layer_norm_grad(f64(r["dy"]), f64(r["x"]), nw, f64(r["mean"]), f64(r["rstd"]))
            close(r["dx"], want["dx"], "f32", "dx")
            close(dnw, want["dweight"], "bf16", "dweight")
            close(dnb, want["dbias"], "bf16", "dbias")
        for i, mean in enumerate(self.means):  # two addends have one order
            total = sum(r["grads"][i].float() for r in self.ranks) / self.world
            assert torch.equal(mean, total.bfloat16())
        for mean, update in zip(self.means, self.updates):
            check_update(update, f64(mean), dtype="bf16")


@pytest.mark.parametrize("tokens,hidden,ffn,act,keep", [(1, 64, 96, "silu", True), (16, 256, 520, "gelu", False),
                                                        (301, 200, 333, "silu", False), (600, 512, 768, "gelu", True)])
def test_a_step(tide, tokens, hidden, ffn, act, keep):
    import torch

    step = Step(tide, tokens, hidden, ffn, act, keep)
    step.fill(tokens)
    step.run()
    torch.cuda.synchronize()
    step.check()


def test_a_captured_step(tide):
    """After one eager step with the same buffers; with new inputs before each
    replay."""
    import torch

    step = Step(tide, 301, 200, 333, "silu", True)
    step.fill(0)
    step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for seed in range(1, 4):
        step.fill(seed)
        step.clear()
        graph.replay()
        torch.cuda.synchronize()
        step.check()
        got = [t.clone() for t in step.outputs()]
        step.clear()
        step.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step.outputs()))
