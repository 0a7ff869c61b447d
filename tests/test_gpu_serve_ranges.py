"""The norm and the packed layer's product at the ends of what
include/pwq_serve.h allows, each against its own definition.

Linear tolerances, from the arithmetic: a matrix instruction adds the products
of 32 columns (64 in 8 bits, exact) to a float32 with at most four roundings,
three times over for float32 x in its three bf16 parts; steps, waves, splits
and scales add fewer than n / 32 + 64 more.  A rounding is at most 2^-24 of the
sum of the terms' absolute values.  A bf16 output adds half a unit in its last
place, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle.serve_oracle as S
import post_weight_quantization_19_amd as P
from test_gpu_serve import (DT, HALF_BF16, U, activations, f64, hidden, layer,
                            packed_layer)

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


@pytest.mark.parametrize("n", [6, 300, 4096, 40960])
def test_norm_codes_of_the_smallest_values(n):
    """A step of one or two units of the smallest float32 is far from 1 / 127
    of the maximum: codes stay within -127 .. 127."""
    tiny = 2.0 ** -149
    for units in (1, 63, 64, 100, 190, 200, 300):
        x = torch.ones((2, n), device="cuda")
        x[1] = -1
        w = torch.full((n,), units * tiny, device="cuda", dtype=torch.float32)
        w[n // 2:] = 0
        q, step, _ = P.rms_norm(x, w, eps=0.0, out_dtype=torch.int8)
        s = np.float32(units * tiny) / np.float32(127)
        s = np.float32(1) if s == 0 else s
        want = min(127, int(np.rint(np.float32(units * tiny) / s)))
        assert step.tolist() == [float(s)] * 2
        print(f"[ranges] tiny {n} {units} {want}", flush=True)
        assert torch.all(q[0, :n // 2] == want) and torch.all(q[1, :n // 2] == -want)
        assert torch.all(q[:, n // 2:] == 0)


@pytest.mark.parametrize("n", [6, 300, 4096, 40960])
def test_norm_codes_beside_an_infinity(n):
    """A value beyond float32's range: an infinite step and codes 0, in its
    token alone."""
    x = torch.ones((3, n), device="cuda")
    x[1, 2], x[2, 2] = 0, -2
    w = torch.ones(n, device="cuda")
    w[2] = 3.4e38
    x[0, 2] = 2
    q, step, _ = P.rms_norm(x, w, eps=0.0, out_dtype=torch.int8)
    print(f"[ranges] infinity {n}", flush=True)
    assert torch.isinf(step[[0, 2]]).all() and torch.isfinite(step[1])
    assert torch.all(q[[0, 2]] == 0) and torch.all(q[1, 3:] == 127) and q[1, 2] == 0


def wide_layer(rng, m, n, group, density):
    """ASYM codes with zero points 16 .. 127 and steps to +-127."""
    ng = n // (group or n)
    zeros = rng.integers(16, 128, (m, ng)).astype(np.int32)
    zeros[rng.random((m, ng)) < 0.3] = 127
    z = np.repeat(zeros, n // ng, axis=1)
    codes = rng.integers(0, 16, (m, n))
    far = rng.random((m, n)) < density
    far[0, n // 2] = True
    codes = np.where(far, z + rng.integers(-127, 128, (m, n)), codes)
    codes = np.where(far & (rng.random((m, n)) < 0.3), z + 127, codes)
    codes[0, n // 2] = z[0, n // 2] + 127
    scales = (0.003 * np.exp(0.3 * rng.standard_normal((m, ng)))).astype(np.float32)
    return codes.astype(np.int32), scales, zeros


def product(x, xs, codes, scales, zeros):
    """(y, sum of the terms' absolute values), float64, by the definition."""
    step = codes.astype(np.float64)
    ng = scales.shape[1]
    if zeros is not None:
        step = step - np.repeat(zeros.astype(np.float64), codes.shape[1] // ng, axis=1)
    w = step * np.repeat(scales.astype(np.float64), codes.shape[1] // ng, axis=1)
    x = f64(x) * (1 if xs is None else f64(xs)[:, None])
    return x @ w.T, np.abs(x) @ np.abs(w).T


def check(y, x, xs, codes, scales, zeros):
    n = codes.shape[1]
    want, size = product(x, xs, codes, scales, zeros)
    parts = 3 if x.dtype == torch.float32 else 1
    tol = (parts * n / 8 + n / 32 + 64) * U * size
    if y.dtype == torch.bfloat16:
        tol = tol + HALF_BF16 * np.abs(want)
    worst = (np.abs(f64(y) - want) / np.maximum(tol, 1e-300)).max()
    assert worst <= 1, float(worst)


@pytest.mark.parametrize("x_kind", ["int8", "f32", "bf16"])
@pytest.mark.parametrize("n,group", [(1024, 128), (640, 64), (1152, 192), (416, 32), (1000, 0),
                                     (200, 20)])
def test_overflow_entries_above_127(n, group, x_kind):
    """With zero points above 15 an overflow entry, code - 15, goes to 239."""
    m = 50
    for density in (0.002, 0.05, 1.0):
        rng = np.random.default_rng([n, group, int(1000 * density)])
        codes, scales, zeros = wide_layer(rng, m, n, group, density)
        pk = packed_layer(codes, scales, zeros, group)
        assert int((pk["outliers"] >> 16).max()) > 127
        for tokens in (1, 2, 8, 9, 16, 17, 40, 140):
            print(f"[ranges] above 127 {n} {group} {x_kind} {density} {tokens}", flush=True)
            x, xs = activations(rng, tokens, n, x_kind)
            y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                                out_dtype=torch.float32)
            check(y, x, xs, codes, scales, zeros)


def test_overflow_entries_above_127_past_whole_tiles():
    """The same layer for a prompt whose last tokens go to the kernels for few."""
    rng = np.random.default_rng(127)
    codes, scales, zeros = wide_layer(rng, 4096, 4096, 128, 0.001)
    pk = packed_layer(codes, scales, zeros, 128)
    x, xs = activations(rng, 1030, 4096, "int8")
    y = P.packed_linear(x.cuda(), pk, x_scales=xs.cuda(), out_dtype=torch.float32)
    check(y[-16:], x[-16:], xs[-16:], codes, scales, zeros)
    check(y[:16], x[:16], xs[:16], codes, scales, zeros)


@pytest.mark.parametrize("multiplier", [0.0625, 0.3])
def test_layer_of_small_steps(multiplier):
    """Steps made small by the grid's multiplier: zero points near 120, codes
    to 240, quantized, packed and multiplied."""
    rng = np.random.default_rng(16)
    m, n = 48, 512
    W = torch.from_numpy(rng.uniform(-1, 1, (m, n)).astype(np.float32)).cuda()
    grid = P.Grid("asym", 4, 128, kappa=multiplier)
    scales, zeros = P.grid_steps(W, grid)
    s = f64(scales).repeat(128, axis=1)
    z = zeros.cpu().numpy().astype(np.int64).repeat(128, axis=1)
    codes = np.clip(np.rint(f64(W) / s), -127, 127).astype(np.int64) + z
    pk = P.pack_weights(torch.from_numpy(codes.astype(np.int32)).cuda(), scales, grid, zeros)
    for x_kind in ("int8", "bf16"):
        for tokens in (1, 16, 17):
            x, xs = activations(rng, tokens, n, x_kind)
            y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                                out_dtype=torch.float32)
            check(y, x, xs, codes, scales.cpu().numpy(), zeros.cpu().numpy())


@pytest.mark.parametrize("x_kind", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("tokens", [1, 7, 16, 17, 140])
def test_rows_of_zero_steps_give_zero(tokens, x_kind):
    """Every code at its zero point: the product is 0, not its rounding."""
    rng = np.random.default_rng(tokens)
    m, n = 40, 1000
    for kind in ("sym", "asym"):
        zeros = rng.integers(0, 16, (m, 1)).astype(np.int32) if kind == "asym" else None
        codes = np.zeros((m, n), np.int32) if zeros is None else zeros.repeat(n, axis=1)
        pk = packed_layer(codes.astype(np.int32), np.ones((m, 1), np.float32), zeros, 0)
        x, xs = activations(rng, tokens, n, x_kind)
        y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                            out_dtype=torch.float32)
        assert torch.all(y == 0), (kind, float(y.abs().max()))


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 5, 16, 17, 140])
def test_large_finite_tokens(tokens, x_kind):
    """x of 2^125 and steps of 1 and -1: finite, and exact."""
    m, n = 33, 256
    for kind in ("sym", "asym"):
        codes = np.zeros((m, n), np.int32)
        codes[:, 3], codes[:, 200] = 1, -1
        zeros = None
        if kind == "asym":
            codes += 9
            zeros = np.full((m, 2), 9, np.int32)
        pk = packed_layer(codes, np.full((m, 2), 0.5, np.float32), zeros, 128)
        x = torch.zeros((tokens, n), dtype=DT[x_kind])
        x[:, 3], x[:, 200] = 2.0 ** 125, 2.0 ** 124
        y = P.packed_linear(x.cuda(), pk, out_dtype=torch.float32)
        assert torch.all(y == 2.0 ** 123), (kind, y.flatten()[:4].tolist())


@pytest.mark.parametrize("x_kind", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("tokens", [1, 16, 33, 140])
def test_small_steps_next_to_large_x(tokens, x_kind):
    """Steps of a few units: the error follows |step| |x|, whatever the stored
    code and zero point are."""
    rng = np.random.default_rng([tokens, 5])
    m, n, group = 64, 4096, 128
    for kind in ("sym", "asym"):
        step = rng.integers(-1, 2, (m, n)) * (rng.random((m, n)) < 0.05)
        zeros = rng.integers(1, 15, (m, n // group)).astype(np.int32) if kind == "asym" else None
        codes = step if zeros is None else step + zeros.repeat(group, axis=1)
        scales = np.full((m, n // group), 0.25, np.float32)
        codes = codes.astype(np.int32)
        pk = packed_layer(codes, scales, zeros, group)
        x, xs = activations(rng, tokens, n, x_kind)
        y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                            out_dtype=torch.float32)
        check(y, x, xs, codes, scales, zeros)


def test_norm_of_sixteen_million_tokens():
    """More workgroups than a launch takes, of the kernel for short rows."""
    tokens, n = 2 ** 24 + 5, 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((tokens, n), generator=gen, device="cuda")
    w = torch.tensor([0.5, 1.0, 2.0, -1.0], device="cuda")
    print("[ranges] 2^24 tokens", flush=True)
    y, _, _ = P.rms_norm(x, w)
    q, step, _ = P.rms_norm(x, w, out_dtype=torch.int8)
    rel = 16 * U                                       # a sum of 4 squares, root, 3 roundings
    for part in (slice(0, 1000), slice(2 ** 24 - 500, None)):
        want, s, _, _ = S.rms_norm(f64(x[part]), f64(w), None, 1e-6, True)
        assert np.all(np.abs(f64(y[part]) - want) <= rel * np.abs(want))
        assert np.all(np.abs(f64(step[part]) - s) <= rel * s)
        assert np.all(np.abs(f64(q[part]) - want / s[:, None]) <= 0.5 + 254 * rel)
    assert torch.isfinite(y).all() and int((step <= 0).sum()) == 0


def test_product_of_sixty_million_rows():
    """More workgroups than a launch takes, of the kernel for groups that are
    no multiple of 32 columns."""
    m, n, group = 2 ** 26 + 9, 6, 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(0, 256, (m, 16), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand((m, 2), generator=gen, device="cuda")
    x = torch.randn((2, n), generator=gen, device="cuda")
    print("[ranges] 2^26 rows", flush=True)
    y = P.packed_linear(x, {"qweight": q, "scales": scales, "zeros": None, "n": n, "group": group,
                            "outlier_off": None, "outliers": None})
    for part in (slice(0, 1000), slice(2 ** 26 - 500, None)):
        codes = S.unpack(q[part].cpu().numpy(), n, False)
        check(y[:, part], x, None, codes, f64(scales[part]), None)
    assert torch.isfinite(y).all()


# ------------------------------------------------------------------ kernels by their sizes

NORM_WALKS = [(1700, 4097), (1600, 8200), (900, 14336), (6200, 2047), (6200, 300), (600, 20001)]


def norm_tolerance(n):
    """Of a value: the sum of squares (halved by the root) and 8 roundings."""
    return (0.5 * (n / 64 + 32) + 8) * U


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,n", NORM_WALKS)
def test_norm_walks_over_tokens(tokens, n, x_kind):
    """More tokens than workgroups: each kernel for many tokens, every token
    against 64 bits, in every output type, with a residual and without."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((tokens, n), generator=gen, device="cuda").to(DT[x_kind])
    res = (2 * torch.randn((tokens, n), generator=gen, device="cuda")).to(DT[x_kind])
    w = 1 + 0.1 * torch.randn(n, generator=gen, device="cuda")
    rel = norm_tolerance(n)
    for residual in (None, res):
        h = x.double() if residual is None else x.double() + residual.double()
        want = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
        for out in ("int8", "bf16", "f32"):
            print(f"[ranges] walk {tokens} {n} {x_kind} {residual is not None} {out}", flush=True)
            y, step, total = P.rms_norm(x, w, residual, out_dtype=DT[out])
            if residual is not None:
                tol = h.abs() * (2 * U + (HALF_BF16 if x_kind == "bf16" else 0))
                assert bool(((total.double() - h).abs() <= tol).all())
            if out == "int8":
                s = want.abs().amax(1) / 127
                assert bool(((step.double() - s).abs() <= (rel + 2 * U) * s).all())
                off = (y.double() - want / s[:, None]).abs()
                assert float(off.max()) <= 0.5 + 127 * (2 * rel + 8 * U)
            else:
                tol = want.abs() * (rel + (HALF_BF16 if out == "bf16" else 0))
                assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("tokens,n", NORM_WALKS)
def test_norm_walks_in_place(tokens, n):
    """The sum on x's or the residual's memory, in rows of a wider tensor, and
    tokens of NaN and infinity: the other tokens as without any of it."""
    gen = torch.Generator(device="cuda").manual_seed(n + 1)
    x = torch.randn((tokens, n), generator=gen, device="cuda").bfloat16()
    res = torch.randn((tokens, n), generator=gen, device="cuda").bfloat16()
    w = torch.rand(n, generator=gen, device="cuda")
    y0, s0, t0 = P.rms_norm(x, w, res, out_dtype=torch.int8)
    for shift, pad in ((0, 8), (3, 5)):
        for place in ("x", "residual"):
            print(f"[ranges] in place {tokens} {n} {shift} {place}", flush=True)
            wide = torch.full((tokens, n + pad), 7.0, device="cuda", dtype=torch.bfloat16)
            view = wide[:, shift:shift + n]
            view.copy_(x if place == "x" else res)
            args = (view, w, res) if place == "x" else (x, w, view)
            y, s, t = P.rms_norm(*args, out_dtype=torch.int8, sum_out=view)
            assert torch.equal(y, y0) and torch.equal(s, s0) and torch.equal(view, t0)
            assert bool((wide[:, :shift] == 7).all()) and bool((wide[:, shift + n:] == 7).all())
    bad = torch.tensor([0, tokens // 3, tokens // 2, tokens - 1], device="cuda")
    x[bad, n - 1] = torch.tensor([float("nan"), float("inf"), float("-inf"), float("nan")],
                                 device="cuda").bfloat16()
    y, s, _ = P.rms_norm(x, w, res, out_dtype=torch.int8)
    good = torch.ones(tokens, dtype=torch.bool, device="cuda")
    good[bad] = False
    assert torch.equal(y[good], y0[good]) and torch.equal(s[good], s0[good])
    assert bool(torch.isnan(s[bad]).all()) and bool((y[bad] == 0).all())


@pytest.mark.parametrize("x_kind", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("n,group", [(34560, 128), (34560, 192), (33792, 64), (10240, 32),
                                     (34560, 0), (34470, 0)])
def test_long_rows_for_few_tokens(n, group, x_kind):
    """More tiles of columns to a wave than it stages the steps of at a time:
    steps, zero points and overflow entries are staged again, in mid-group too."""
    m = 33
    for kind, density in (("sym", 0.02), ("asym", 0.02), ("sym", 0.6), ("asym", 0.0)):
        rng = np.random.default_rng([n, group])
        codes, scales, zeros = layer(rng, m, n, group, kind, density)
        pk = packed_layer(codes, scales, zeros, group)
        for tokens in (1, 6, 16):
            print(f"[ranges] long rows {n} {group} {x_kind} {kind} {density} {tokens}", flush=True)
            x, xs = activations(rng, tokens, n, x_kind)
            y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                                out_dtype=torch.float32)
            check(y, x, xs, codes, scales, zeros)


def test_many_rows_and_long_rows_for_few_tokens():
    """A layer of 8200 rows of 14336: several chunks of a wave in every strip."""
    m, n, group = 8200, 14336, 64
    rng = np.random.default_rng(14336)
    codes, scales, zeros = layer(rng, m, n, group, "asym", 0.01)
    pk = packed_layer(codes, scales, zeros, group)
    rows = np.r_[0:40, 4000:4040, m - 40:m]
    for x_kind in ("bf16", "int8", "f32"):
        for tokens in (1, 16):
            x, xs = activations(rng, tokens, n, x_kind)
            y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                                out_dtype=torch.float32)
            check(y[:, torch.from_numpy(rows).cuda()], x, xs, codes[rows], scales[rows],
                  zeros[rows])


@pytest.mark.parametrize("tokens", [1, 20, 200])
@pytest.mark.parametrize("n,group", [(256, 128), (320, 64), (140032, 0)])
def test_largest_integers_are_exact(n, group, tokens):
    """8-bit x of -128 against steps of -127: partial sums are multiples of 128 x
    127, and added by twos or more, at most 70016 of them, exact in 24 bits."""
    m = 17
    zeros = np.full((m, n // (group or n)), 127, np.int32)
    pk = packed_layer(np.zeros((m, n), np.int32), np.full(zeros.shape, 0.5, np.float32), zeros,
                      group)
    x = torch.full((tokens, n), -128, dtype=torch.int8, device="cuda")
    y = P.packed_linear(x, pk, x_scales=torch.ones(tokens, device="cuda"),
                        out_dtype=torch.float32)
    assert bool((y == 0.5 * 128 * 127 * n).all())


@pytest.mark.parametrize("x_kind", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("tokens,m,n,group", [(1, 70, 4096, 128), (12, 70, 4096, 32),
                                              (50, 200, 1408, 128), (200, 300, 2048, 64),
                                              (700, 300, 2048, 0), (650, 700, 1152, 192),
                                              (90, 40, 600, 20)])
def test_error_follows_the_steps(tokens, m, n, group, x_kind):
    """Every kernel within its roundings of |step| |x|."""
    for kind, density in (("sym", 0.0), ("asym", 0.01)):
        rng = np.random.default_rng([tokens, m, n])
        codes, scales, zeros = layer(rng, m, n, group, kind, density)
        pk = packed_layer(codes, scales, zeros, group)
        x, xs = activations(rng, tokens, n, x_kind)
        for out in ("f32", "bf16"):
            y = P.packed_linear(x.cuda(), pk, x_scales=None if xs is None else xs.cuda(),
                                out_dtype=DT[out])
            check(y, x, xs, codes, scales, zeros)
