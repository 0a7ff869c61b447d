"""Calls of the key-value cache that its documentation allows and few make.  Bounds as in
test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import oracle.cache_oracle as C
import post_weight_quantization_19_amd as P
from test_gpu_cache import DT, batch_of, check_attention, f64, filled, keys_values, queries, up

pytestmark = pytest.mark.gpu


def test_outputs_between_the_heads_of_inputs():
    """q and the output, or k and v, of one projection [tokens, heads, parts, head_dim]."""
    rng = np.random.default_rng(40)
    b = batch_of(rng, [50, 9], [20, 9], 32)
    cache, records = filled(rng, b[3], 2, 64, 8, 32)
    args = up(*b[:3])
    qkv = torch.from_numpy(rng.standard_normal((29, 4, 3, 64)).astype(np.float32)).cuda()
    keep = qkv.clone()
    y = P.cached_attention(qkv[:, :, 0], cache, *args, out=qkv[:, :, 2])
    check_attention(y, qkv[:, :, 0], records, b[:3], 64, 8, 32)
    assert torch.equal(qkv[:, :, :2], keep[:, :, :2])
    k, v = P.cache_read(cache, *args, 29, dtype=torch.float32)
    for shape, pick in (((29, 2, 2, 64), lambda t, i: t[:, :, i]),
                        ((2, 2, 29, 64), lambda t, i: t[:, i].transpose(0, 1)),
                        ((2, 29, 2, 64), lambda t, i: t[:, :, i].transpose(0, 1))):
        kv = torch.full(shape, 7.0, device="cuda")
        P.cache_read(cache, *args, 29, out=(pick(kv, 0), pick(kv, 1)))
        assert torch.equal(pick(kv, 0), k) and torch.equal(pick(kv, 1), v)
