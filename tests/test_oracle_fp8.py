"""Pins of the oracle's FP8 projection against torch's casts and closed forms."""
import numpy as np
import torch

from oracle import csa_oracle as O


def test_block_exponent_is_the_least_that_holds_the_block():
    for e in range(-127, 128):
        top = np.ldexp(448.0, e)
        assert O.fp8_block_exponent(top) == e
        if e < 127:
            assert O.fp8_block_exponent(np.nextafter(top, np.inf)) == e + 1
    assert O.fp8_block_exponent(0.0) == 0
    assert O.fp8_block_exponent(2.0 ** -149) == -127
    assert O.fp8_block_exponent(3.0e38) == 120


def test_codes_agree_with_torch_and_scales_cover_rows_and_columns():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2 * 200)) * np.exp(3 * rng.standard_normal((5, 400)))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    codes, scales = O.fp8_quantize_blocks(x, groups=2)
    assert scales.shape == (5, 4)
    for g in range(2):
        for b, (c0, c1) in enumerate(((0, 128), (128, 200))):
            at = (slice(None), slice(200 * g + c0, 200 * g + c1))
            e = scales[:, 2 * g + b].astype(int) - 127
            want = torch.from_numpy(np.ldexp(x[at], -e[:, None])).float().to(torch.float8_e4m3fn)
            assert np.array_equal(codes[at], want.view(torch.uint8).numpy())
            top = np.abs(x[at]).max(1)
            assert np.all(top <= np.ldexp(448.0, e)) and np.all(top > np.ldexp(224.0, e))
    back = O.fp8_dequantize_blocks(codes, scales, groups=2)
    # E4M3 keeps 4 significant bits (half a step 2^-4 of a normal value; below
    # 2^-6 of the scale a step is 2^-9 of it)
    step = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), [128, 72, 128, 72], axis=1)
    assert np.all(np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10))


def test_a_block_that_is_not_finite_becomes_nan_and_no_other():
    x = np.ones((3, 300))
    x[1, 130] = np.inf
    x[2, 299] = np.nan
    w = np.ones((130, 300))
    wc, ws = O.fp8_quantize_blocks(w, rows=128)
    y = O.fp8_linear(x, wc, ws)
    assert np.all(y[0] == 300) and np.isnan(y[1]).all() and np.isnan(y[2]).all()


def test_grouped_product_is_block_diagonal():
    rng = np.random.default_rng(4)
    x, w = rng.integers(-8, 9, (4, 48)).astype(float), rng.integers(-8, 9, (256, 24)).astype(float)
    wc, ws = O.fp8_quantize_blocks(w, rows=128)
    y = O.fp8_linear(x, wc, ws, groups=2)          # small integers are exact in E4M3
    assert np.array_equal(y[:, :128], x[:, :24] @ w[:128].T)
    assert np.array_equal(y[:, 128:], x[:, 24:] @ w[128:].T)
