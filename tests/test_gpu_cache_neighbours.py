"""What a row of attention must not depend on: the other rows that a kernel takes with it,
and the values of tokens that it does not see.  Bounds as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import oracle.cache_oracle as C
import post_weight_quantization_19_amd as P
from test_gpu_cache import DT, batch_of, check_attention, f64, filled, keys_values, queries, up

pytestmark = pytest.mark.gpu

WIDE = 40000      # pages of a table whose entries are none: room for many tokens, so tiles of rows


@pytest.mark.parametrize("power", [40, 110])
@pytest.mark.parametrize("heads,kv_heads,dim,bits,dtype", [
    (4, 1, 128, 8, "bf16"), (14, 2, 64, 4, "f32"), (6, 2, 256, 8, "bf16"), (3, 3, 128, 4, "f32")])
def test_a_query_far_above_its_neighbours(heads, kv_heads, dim, bits, dtype, power):
    """One head of one token 2^power above the others, 16 rows taken together."""
    rng = np.random.default_rng(dim + power)
    lens, new, page = [90, 700], [5, 3], 32
    b = batch_of(rng, lens, new, page)
    cache, records = filled(rng, b[3], kv_heads, dim, bits, page)
    q = queries(rng, 8, heads, dim, dtype)
    q[2, heads - 1] *= 2.0 ** power
    q[6, 0] *= 2.0 ** power
    y = P.cached_attention(q, cache, *up(*b[:3]))
    check_attention(y, q, records, b[:3], dim, bits, page)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_query_far_above_those_of_other_sequences(dtype):
    """Rows of a prefix belong to different sequences."""
    rng = np.random.default_rng(31)
    n, page, before, dim = 12, 32, 100, 64
    starts, lengths, table, pages = batch_of(rng, [9] * n, [1] * n, page, spare=5)
    free = np.array([p for p in range(pages) if p not in set(table.ravel())][:4], np.int32)
    cache, records = filled(rng, pages, 2, dim, 8, page)
    q = queries(rng, n, 6, dim, dtype)
    q[7] *= 2.0 ** 40
    y = P.cached_attention(q, cache, *up(starts, lengths, table),
                           prefix=tuple(up(free, np.array([before], np.int32))))
    check_attention(y, q, records, (starts, lengths, table), dim, 8, page, prefix=(free, before))


@pytest.mark.parametrize("power", [7, 9, 40, 110])
@pytest.mark.parametrize("heads,kv_heads,dim,bits,dtype", [
    (4, 1, 128, 8, "bf16"), (14, 2, 64, 4, "f32"), (6, 2, 256, 8, "bf16"), (3, 1, 128, 4, "f32"),
    (2, 1, 64, 8, "bf16")])
def test_a_query_far_above_those_of_its_tile(heads, kv_heads, dim, bits, dtype, power):
    """The same in tiles of many rows, with rows of zeros and a NaN among them."""
    rng = np.random.default_rng(dim + power)
    lens, new, page = [300, 140], [150, 100], 32
    b = batch_of(rng, lens, new, page, extra=WIDE)
    cache, records = filled(rng, b[3], kv_heads, dim, bits, page)
    q = queries(rng, 250, heads, dim, dtype)
    q[2, heads - 1] *= 2.0 ** power
    q[200, 0] *= 2.0 ** power
    q[5] = 0
    args = up(*b[:3])
    y = P.cached_attention(q, cache, *args)
    check_attention(y, q, records, b[:3], dim, bits, page)
    q[9, 0, 3] = float("nan")
    z = P.cached_attention(q, cache, *args)
    assert torch.isnan(z[9, 0]).all()
    z[9, 0] = y[9, 0]
    assert torch.equal(y, z)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 64)])
def test_a_query_far_above_others_behind_a_prefix_in_tiles(dtype, dim):
    rng = np.random.default_rng(32)
    n, page, before = 40, 32, 200
    starts, lengths, table, pages = batch_of(rng, [9] * n, [1] * n, page, spare=9)
    free = np.array([p for p in range(pages) if p not in set(table.ravel())][:7], np.int32)
    wide = np.concatenate([free, np.full(WIDE, -1, np.int32)])
    cache, records = filled(rng, pages, 1, dim, 8, page)
    q = queries(rng, n, 8, dim, dtype)
    q[30] *= 2.0 ** 50
    y = P.cached_attention(q, cache, *up(starts, lengths, table),
                           prefix=tuple(up(wide, np.array([before], np.int32))))
    check_attention(y, q, records, (starts, lengths, table), dim, 8, page, prefix=(free, before))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_of_all_sizes_in_a_tile(dtype):
    """Rows from 2^-100 to 2^44 and from 2^-60 to 2^120, with keys for which some of the
    scores are of ordinary size."""
    rng = np.random.default_rng(33)
    n, page, dim = 130, 32, 64
    b = batch_of(rng, [n], [n], page, extra=WIDE)
    for lo, hi, size in ((-100, 44, 2.0 ** 70), (-60, 120, 2.0 ** -100)):
        cache = P.new_cache(b[3], 1, dim, 8, page)
        k, v = keys_values(rng, (n, 1, dim), torch.float32)
        P.cache_write(k * size, v, cache, *up(*b[:3]))
        records = cache["records"].cpu().numpy()
        q = queries(rng, n, 2, dim, "f32")
        q *= torch.from_numpy(np.exp2(np.linspace(lo, hi, n))).float().cuda()[:, None, None]
        q = q.to(DT[dtype])
        y = P.cached_attention(q, cache, *up(*b[:3]))
        check_attention(y, q, records, b[:3], dim, 8, page)


def check_by_what_is_seen(y, q, records, b, dim, bits, page):
    """check_attention of one sequence, where a row's bound counts the steps of the values
    that it sees (a step of 2^-33 of the largest so far, times a code of at most 255).  A
    rounding to float16, of 11 significant bits, is off by 2^-11 at most."""
    starts, lens, table = b
    new, group, bf16 = starts[1], q.shape[1] // records.shape[1], q.dtype == torch.bfloat16
    k, v, there = C.stored(records, table[0], lens[0], dim, bits, page)
    n, qn, got = lens[0], f64(q), f64(y)
    seen = there & (np.arange(n) <= (n - new + np.arange(new))[:, None])
    for h in range(q.shape[1]):
        vh = v[h // group]
        want, size, score = C.attention(qn[:new, h], k[h // group], vh, dim ** -0.5, seen)
        steps = (vh.max(-1).clip(0) - vh.min(-1).clip(max=0)) / (2 ** bits - 1) * 1.02
        step = np.where(seen, steps, 0).max(1)[:, None]
        off = score * ((dim + 4 + 1.45) * 2.0 ** -24 + (0 if bf16 else 2.0 ** -22))
        rel = 2 * off + 2.0 ** -21 + (3 * 2.0 ** -11 if bf16 else 2.0 ** -22)
        rel = rel + (n / 16 + 64) * 2.0 ** -24
        tol = rel[:, None] * (size + np.abs(want)) + (n + 9) * 2.0 ** -33 * step * 255
        tol = tol * 1.01 + (2.0 ** -8 * 1.01 if bf16 else 2.0 ** -23) * np.abs(want)
        err = np.abs(got[:new, h] - want)
        assert np.all(err <= tol), (h, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("power", [20, 34, 60])
@pytest.mark.parametrize("heads,kv_heads,dim,bits,dtype", [
    (4, 1, 128, 8, "bf16"), (2, 2, 64, 4, "f32"), (3, 1, 256, 8, "f32"), (8, 8, 64, 8, "bf16")])
def test_values_of_tokens_that_a_row_does_not_see(heads, kv_heads, dim, bits, dtype, power):
    """The last two of eight new tokens have values 2^power above the others': the rows
    before them are as exact as without."""
    rng = np.random.default_rng(dim + power)
    for n in (20, 90, 1500):
        b = batch_of(rng, [n], [8], 32)
        cache = P.new_cache(b[3], kv_heads, dim, bits, 32)
        k, v = keys_values(rng, (n, kv_heads, dim), torch.float32)
        v[-2:] *= 2.0 ** power
        P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
        records = cache["records"].cpu().numpy()
        q = queries(rng, 8, heads, dim, dtype)
        y = P.cached_attention(q, cache, *up(*b[:3]))
        check_by_what_is_seen(y, q, records, b[:3], dim, bits, 32)


# So many key heads, and rows of each, that a tile of rows takes all of its tokens.
MANY = [(256, 64, 8, "bf16"), (256, 64, 4, "f32"), (256, 128, 8, "bf16"), (300, 128, 4, "f32")]


@pytest.mark.parametrize("power", [34, 90, 170])
@pytest.mark.parametrize("heads,dim,bits,dtype", MANY)
def test_values_behind_a_row_in_tiles(heads, dim, bits, dtype, power):
    """Tokens from a multiple of 32 on have values 2^power above the others': rows of the
    same tile that end before are as exact as without."""
    rng = np.random.default_rng(dim + power)
    n, new = 450, 250
    b = batch_of(rng, [n], [new], 32)
    cache = P.new_cache(b[3], heads, dim, bits, 32)
    k, v = keys_values(rng, (n, heads, dim), torch.float32)
    v[:352] *= 2.0 ** -min(power, 100)
    v[352:] *= 2.0 ** (power - min(power, 100))
    P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
    q = queries(rng, new, heads, dim, dtype)
    y = P.cached_attention(q, cache, *up(*b[:3]))
    rows = 352 - (n - new)                     # those that end before
    cut = (np.array([0, rows], np.int32), [352], b[2])
    for some in (slice(0, 3), slice(heads - 2, heads)):
        records = cache["records"][:, some].cpu().numpy()
        check_by_what_is_seen(y[:rows, some], q[:rows, some], records, cut, dim, bits, 32)
        check_attention(y[:, some], q[:, some], records, b[:3], dim, bits, 32)


@pytest.mark.parametrize("power", [9, 40, 110])
@pytest.mark.parametrize("heads,dim,bits,dtype", MANY)
def test_queries_far_above_others_over_many_records(heads, dim, bits, dtype, power):
    rng = np.random.default_rng(dim + power)
    n, new = 450, 250
    b = batch_of(rng, [n], [new], 32)
    cache = P.new_cache(b[3], heads, dim, bits, 32)
    k, v = keys_values(rng, (n, heads, dim), torch.float32)
    P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
    q = queries(rng, new, heads, dim, dtype)
    q[[7, 130]] *= 2.0 ** power
    q[200] = 0
    y = P.cached_attention(q, cache, *up(*b[:3]))
    for some in (slice(0, 2), slice(heads - 1, heads)):
        records = cache["records"][:, some].cpu().numpy()
        check_attention(y[:, some], q[:, some], records, b[:3], dim, bits, 32)


@pytest.mark.parametrize("power", [9, 20, 34, 90])
@pytest.mark.parametrize("heads,dim,bits,dtype", MANY + [(4, 64, 8, "bf16"), (2, 128, 4, "f32"),
                                                         (3, 256, 8, "bf16"), (3, 256, 4, "f32")])
def test_values_in_the_record_of_a_row_in_tiles(heads, dim, bits, dtype, power):
    """Tokens here and there with values 2^power above the others', in the 32 tokens that rows
    end in: a row is as exact as what it sees lets it be.  Some read as NaN."""
    rng = np.random.default_rng(dim + power)
    n, new = 450, 250
    b = batch_of(rng, [n], [new], 32, extra=0 if heads > 200 else WIDE)
    cache = P.new_cache(b[3], heads, dim, bits, 32)
    k, v = keys_values(rng, (n, heads, dim), torch.float32)
    for t in (203, 230, 231, 290, 300, 310, 395, 448):
        v[t] *= 2.0 ** power
    v[[350, 351]] = 0
    v[430, :, 5] = float("nan")
    k[440, :, 7] = float("inf")
    P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
    q = queries(rng, new, heads, dim, dtype)
    y = P.cached_attention(q, cache, *up(*b[:3]))
    rows = 430 - (n - new)
    assert torch.isnan(y[rows:]).all() and not torch.isnan(y[:rows]).any()
    cut = (np.array([0, rows], np.int32), [430], b[2])
    for some in (slice(0, 2), slice(heads - 1, heads)):
        records = cache["records"][:, some].cpu().numpy()
        check_by_what_is_seen(y[:rows, some], q[:rows, some], records, cut, dim, bits, 32)


@pytest.mark.parametrize("heads,dim,bits,dtype", MANY + [(4, 64, 8, "bf16"), (2, 128, 4, "f32"),
                                                         (3, 256, 8, "bf16"), (3, 256, 4, "f32")])
@pytest.mark.parametrize("new", [8, 250])
def test_the_largest_values_and_keys_behind_a_row(new, heads, dim, bits, dtype):
    """Tokens behind a row with values and keys near float32's largest: the row is as without,
    whether they share its record, or some of it, or none."""
    rng = np.random.default_rng(dim)
    n = 450
    b = batch_of(rng, [n], [new], 32, extra=0 if heads > 200 or new == 8 else WIDE)
    for first in (447, 446, 420, 416):
        if first < n - new + 1:
            continue
        cache = P.new_cache(b[3], heads, dim, bits, 32)
        k, v = keys_values(rng, (n, heads, dim), torch.float32)
        k[first:], v[first:] = 1.6e38 * torch.sign(k[first:]), 1.6e38 * torch.sign(v[first:])
        P.cache_write(k, v, cache, up(np.array([0, n], np.int32))[0], *up(*b[1:3]))
        q = queries(rng, new, heads, dim, dtype)
        y = P.cached_attention(q, cache, *up(*b[:3]))
        rows = first - (n - new)
        cut = (np.array([0, rows], np.int32), [first], b[2])
        for some in (slice(0, 2), slice(heads - 1, heads)):
            records = cache["records"][:, some].cpu().numpy()
            check_by_what_is_seen(y[:rows, some], q[:rows, some], records, cut, dim, bits, 32)
