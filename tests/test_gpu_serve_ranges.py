"""The norm and the packed layer's product at the ends of what
include/pwq_serve.h allows, each against its own definition.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_19_amd as P
from test_gpu_serve import DT, hidden

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,n", [(3, 5), (40, 256), (3, 4096), (700, 4096), (2, 40960)])
@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
def test_norm_codes_are_the_rounded_quotient(tokens, n, x_kind):
    """q = rint(value / step), in float32, of the values that the float32
    output has: equal, ties and all."""
    rng = np.random.default_rng([tokens, n])
    x, res = (hidden(rng, tokens, n).to(DT[x_kind]).cuda() for _ in range(2))
    # weights of few bits: many values at a tie of the step
    w = torch.from_numpy(rng.integers(1, 9, n).astype(np.float32) / 4).cuda()
    x[0], res[0] = 1, 0
    y = P.rms_norm(x, w, res, out_dtype=torch.float32)[0].cpu().numpy()
    q, step, _ = P.rms_norm(x, w, res, out_dtype=torch.int8)
    want = np.abs(y).max(axis=1) / np.float32(127)
    assert np.array_equal(step.cpu().numpy(), want)
    assert np.array_equal(q.cpu().numpy(), np.rint(y / want[:, None]).astype(np.int8))
