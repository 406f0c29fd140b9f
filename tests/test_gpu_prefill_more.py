"""GPU tests of the prompt attention's rarer paths, with the definition in 64
bits, the cases and the tolerances of test_gpu_prefill."""
import numpy as np
import pytest
import torch

from test_gpu_prefill import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [np.bool_(True), np.bool_(False), np.int64(1), 0])
def test_causal_as_any_truth_value(cuda_dev, causal):
    c = Case([70], [200], 2, seed=21)
    o, lse = c.run(causal)
    want = c.run(bool(causal))
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for bad in (None, "yes", 0.5):
        with pytest.raises(TypeError):
            c.run(bad)
