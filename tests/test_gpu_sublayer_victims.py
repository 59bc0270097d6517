"""Layer norm's and the gated block's gradients and the orthogonalized update as
victims of the interference study: they run on the study's stream beside the
reduce-scatter and leave its shards alone, and their own results are those of a
run by themselves."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def study():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import interference

    return interference, interference.Study("llama3.1-8b-layer")


def tensors(call):
    import torch

    flat = []
    for t in call._tensors:
        flat += t if isinstance(t, (list, tuple)) else [t]
    return [t for t in flat if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("kind", ["NORM_GRADS", "GATED_GRADS", "UPDATES"])
def test_victim_beside_the_reduce_scatter(study, kind):
    import torch

    interference, st = study
    call = st.victim(next(iter(getattr(interference, kind))))
    vs = st.stream_v.torch
    call(vs)
    torch.cuda.synchronize()
    alone = [t.clone() for t in tensors(call)]
    assert all(bool(t.isfinite().all()) for t in alone)
    agg, stream, _ = st.aggressor("tide", budget=64)
    agg(stream.torch)
    torch.cuda.synchronize()
    shards = [s.clone() for s in st.outs]
    for _ in range(3):
        agg(stream.torch)
        call(vs)
    torch.cuda.synchronize()
    for got, want in zip(tensors(call) + st.outs, alone + shards):
        assert torch.equal(got, want)
    ms = st.time_alone(call, vs, reps=3)
    assert len(ms) == 3 and all(m > 0 for m in ms)
    stream.destroy()
