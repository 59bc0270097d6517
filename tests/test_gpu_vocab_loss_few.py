"""GPU checks of the vocabulary loss of few tokens, whose kernel keeps two blocks
of 256 k in turn: every fragment count (16, 32, 48 and 64 tokens) with all its
rows in use and with the last ones missing, and hidden sizes of three blocks and
more, where both halves of the pipelined loop run."""
import numpy as np
import pytest

from tests import training_reference as ref
from tests.test_gpu_vocab_loss import Run, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


@pytest.mark.parametrize("tokens", [16, 17, 25, 32, 41, 48, 57, 64])
@pytest.mark.parametrize("size", [768, 1024, 1288, 2048])
def test_blocks(tide, tokens, size):
    h, w, t, g = make(np.random.default_rng(size + tokens), tokens, size, 2005)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    Run(tide, h, w, t, None).check(want)
    Run(tide, h, w, t, g).check(want)


@pytest.mark.parametrize("tokens", [17, 32, 64])
def test_runs_repeat_bit_for_bit(tide, tokens):
    import torch

    h, w, t, g = make(np.random.default_rng(tokens), tokens, 2048, 16000)
    h, w = h.cuda(), w.cuda()
    runs = [Run(tide, h, w, t, None) for _ in range(8)]
    for r in runs[1:]:
        assert torch.equal(r.loss, runs[0].loss) and torch.equal(r.lse, runs[0].lse)
