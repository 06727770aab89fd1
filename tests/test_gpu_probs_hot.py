"""idx_logit_probs at temperatures without bound: what is left has the same chance, what is masked none."""

import pytest
import torch
from test_gpu_probs import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [5, 1000, 30_001, 200_003])
def test_infinite_temperature(lib, dtype, vocab):
    for more in (dict(penalties=False), dict(biases=5, grammar=True), dict(seen=0.7, grammar=True)):
        c = Case([0, 2, 3], vocab, dtype, pad=1, gap=3, **more)
        c.args["temperature"][:] = torch.tensor([float("inf"), 3.4e38], device="cuda")
        c.logits[0, 2] = float("-inf")
        c.check(lib)
        assert torch.isfinite(c.probs).all() and c.probs[0, 2] == 0
