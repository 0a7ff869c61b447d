"""Attention whose scores are far from zero.  Bounds as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import post_weight_quantization_19_amd as P
from test_gpu_cache import batch_of, check_attention, f64, keys_values, queries, up

pytestmark = pytest.mark.gpu

WIDE = 40000      # pages of a table whose entries are none: room for many tokens, so tiles of rows


@pytest.mark.parametrize("power", [20, 28, 31, 50, 100])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,extra", [(1, 0), (1, WIDE), (100, WIDE)])
def test_scores_far_from_zero(new, extra, dtype, sign, power):
    """All keys alike: whatever the scores, every token that a row sees weighs the same,
    and a single one gives its value.  (Scores are some 2^power; the sums of equal weights
    are exact, so what is left is the values' part of the bound.)"""
    rng = np.random.default_rng(power)
    dim = 128
    for n in (new, new + 50):
        b = batch_of(rng, [n], [new], 32, extra=extra)
        cache = P.new_cache(b[3], 1, dim, 8, 32)
        _, v = keys_values(rng, (n, 1, dim), torch.float32)
        key = torch.from_numpy(np.abs(rng.standard_normal(dim)).astype(np.float32)).cuda()
        P.cache_write(key.expand(n, 1, dim), v, cache, up(np.array([0, n], np.int32))[0],
                      *up(*b[1:3]))
        records = cache["records"].cpu().numpy()
        q = queries(rng, new, 4, dim, dtype).abs() * (sign * 2.0 ** power)
        y = P.cached_attention(q, cache, *up(*b[:3]))
        check_attention(y, q * 0, records, b[:3], dim, 8, 32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,extra", [(2, 0), (2, WIDE), (90, WIDE)])
def test_one_token_far_above_the_others(new, extra, dtype):
    """A key whose score is 2^30 or more above all others takes all of the weight."""
    rng = np.random.default_rng(new)
    n, at, dim = 300, 40, 64
    b = batch_of(rng, [n], [new], 32, extra=extra)
    cache = P.new_cache(b[3], 1, dim, 8, 32)
    k, v = keys_values(rng, (n, 1, dim), torch.float32)
    k = -k.abs()
    k[at] *= -1
    P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
    _, held = P.cache_read(cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]), n,
                           dtype=torch.float32)
    for power in (30, 60):
        q = queries(rng, new, 3, dim, dtype).abs() * 2.0 ** power
        y = P.cached_attention(q, cache, *up(*b[:3]))
        want = f64(held[at])[None]
        err = np.abs(f64(y) - want)
        step = f64(held).max() * 2 / 255
        # (float16 has 11 significant bits: one rounding is off by 2^-11 at most)
        tol = (3 * 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) * np.abs(want)
        tol = tol + 2.0 ** -25 * step * 255 + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want)
        assert np.all(err <= tol * 1.01)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [0, WIDE])
def test_far_scores_behind_a_prefix(extra, dtype):
    """The prefix's keys like the sequences' own: its tokens and theirs weigh the same."""
    rng = np.random.default_rng(50)
    n, own, before, dim, page = 40, 20, 70, 64, 32
    starts, lengths, table, pages = batch_of(rng, [own] * n, [1] * n, page, spare=4)
    free = np.array([p for p in range(pages) if p not in set(table.ravel())][:3], np.int32)
    cache = P.new_cache(pages, 1, dim, 8, page)
    key = torch.from_numpy(np.abs(rng.standard_normal(dim)).astype(np.float32)).cuda()
    for tab, count in ((table, [own] * n), (free[None], [before])):
        _, v = keys_values(rng, (sum(count), 1, dim), torch.float32)
        P.cache_write(key.expand(sum(count), 1, dim), v, cache,
                      *up(np.concatenate([[0], np.cumsum(count)]).astype(np.int32),
                          np.array(count, np.int32), tab))
    records = cache["records"].cpu().numpy()
    wide = np.concatenate([free, np.full(extra, -1, np.int32)])
    for power in (24, 27, 30, 33, 80):
        q = queries(rng, n, 8, dim, dtype).abs() * 2.0 ** power
        y = P.cached_attention(q, cache, *up(starts, lengths, table),
                               prefix=tuple(up(wide, np.array([before], np.int32))))
        check_attention(y, q * 0, records, (starts, lengths, table), dim, 8, page,
                        prefix=(free, before))


@pytest.mark.parametrize("heads,dim,dtype", [(256, 64, "f32"), (256, 128, "bf16")])
def test_far_scores_over_many_records(heads, dim, dtype):
    """So many key heads, and rows of each, that a tile of rows takes all of its tokens."""
    rng = np.random.default_rng(dim)
    n, new = 450, 250
    b = batch_of(rng, [n], [new], 32)
    cache = P.new_cache(b[3], heads, dim, 8, 32)
    _, v = keys_values(rng, (n, heads, dim), torch.float32)
    key = torch.from_numpy(np.abs(rng.standard_normal(dim)).astype(np.float32)).cuda()
    P.cache_write(key.expand(n, heads, dim), v, cache, up(np.array([0, n], np.int32))[0],
                  *up(*b[1:3]))
    records = cache["records"][:, -2:].cpu().numpy()
    for power in (24, 27, 31, 90):
        q = queries(rng, new, heads, dim, dtype).abs() * 2.0 ** power
        y = P.cached_attention(q, cache, *up(*b[:3]))[:, -2:]
        check_attention(y, q[:, -2:] * 0, records, b[:3], dim, 8, 32)
