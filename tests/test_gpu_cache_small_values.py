"""Attention over values near the ends of float32.  Bounds as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import post_weight_quantization_19_amd as P
from test_gpu_cache import batch_of, check_attention, keys_values, queries, up

pytestmark = pytest.mark.gpu

WIDE = 40000      # pages of a table whose entries are none: room for many tokens, so tiles of rows


@pytest.mark.parametrize("power", [-100, -110, -118])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 8)])
@pytest.mark.parametrize("new,extra", [(2, 0), (2, WIDE), (90, WIDE)])
def test_values_near_the_smallest(dim, bits, dtype, power, new, extra):
    """Values around 2^power, whose steps are 2^-3 to 2^-7 of them."""
    rng = np.random.default_rng(dim - power)
    n, page = 150, 32
    b = batch_of(rng, [n], [new], page, extra=extra)
    cache = P.new_cache(b[3], 1, dim, bits, page)
    k, v = keys_values(rng, (n, 1, dim), torch.float32)
    P.cache_write(k, v * 2.0 ** power, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
    records = cache["records"].cpu().numpy()
    q = queries(rng, new, 4, dim, dtype)
    y = P.cached_attention(q, cache, *up(*b[:3]))
    check_attention(y, q, records, b[:3], dim, bits, page)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,extra", [(2, 0), (2, WIDE), (90, WIDE)])
def test_values_that_step_up_to_the_largest(new, extra, dtype):
    """Values of 2^-110 first, then of 2^60: small ones count where no others are seen."""
    rng = np.random.default_rng(new)
    n, page, dim = 160, 32, 64
    b = batch_of(rng, [n], [new], page, extra=extra)
    cache = P.new_cache(b[3], 1, dim, 8, page)
    k, v = keys_values(rng, (n, 1, dim), torch.float32)
    v[:128] *= 2.0 ** -110
    v[128:] *= 2.0 ** 60
    P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
    records = cache["records"].cpu().numpy()
    q = queries(rng, new, 4, dim, dtype)
    y = P.cached_attention(q, cache, *up(*b[:3]))
    check_attention(y, q, records, b[:3], dim, 8, page)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,extra", [(2, 0), (2, WIDE), (90, 2), (90, WIDE)])
def test_values_near_the_largest(new, extra, dtype):
    """Steps just below 2^84, equal weights: sums of 160 or 3000 tokens stay in float32."""
    rng = np.random.default_rng(new)
    page, dim = 32, 64
    for n in (160, 3000):
        b = batch_of(rng, [n], [new], page, extra=extra)
        cache = P.new_cache(b[3], 1, dim, 8, page)
        k, v = keys_values(rng, (n, 1, dim), torch.float32)
        v = v.clamp(-8, 8) * (2.0 ** 84 * 255 / 16.2)
        P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
        records = cache["records"].cpu().numpy()
        for size in (0.0, 1.5):
            q = queries(rng, new, 4, dim, dtype, size)
            y = P.cached_attention(q, cache, *up(*b[:3]))
            check_attention(y, q, records, b[:3], dim, 8, page)
