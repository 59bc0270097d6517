"""The training-step operators as victims of the interference study: they run
on the study's stream beside the reduce-scatter and leave its shards alone, and
their own results are those of a run by themselves."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def study():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import interference

    return interference, interference.Study("llama3.1-8b-layer")


@pytest.mark.parametrize("kind", ["WEIGHT_GRADS", "VOCAB_LOSSES"])
def test_victim_beside_the_reduce_scatter(study, kind):
    import torch

    interference, st = study
    call = st.victim(next(iter(getattr(interference, kind))))
    outputs = [t for t in call._tensors if isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16]
    vs = st.stream_v.torch
    call(vs)
    torch.cuda.synchronize()
    alone = [t.clone() for t in outputs]
    agg, stream, _ = st.aggressor("tide", budget=64)
    agg(stream.torch)
    torch.cuda.synchronize()
    shards = [s.clone() for s in st.outs]
    for _ in range(3):
        agg(stream.torch)
        call(vs)
    torch.cuda.synchronize()
    for got, want in zip(outputs + st.outs, alone + shards):
        assert torch.equal(got, want)
    ms = st.time_alone(call, vs, reps=3)
    assert len(ms) == 3 and all(m > 0 for m in ms)
    stream.destroy()
