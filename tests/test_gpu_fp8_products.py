"""The 8-bit quantiser's code bytes, and the products where a CTA works on many tiles and blocks."""

import numpy as np
import pytest
import torch

from tests.test_gpu_fp8 import (BF16, E4M3, F32, check_product, dequantized, make_layer, np32,
                                quantize_ref, weight_values)

pytestmark = pytest.mark.gpu


def code_bytes(values):
    """Bytes of e4m3 values, the sign of zero included."""
    return (np.searchsorted(E4M3, np.abs(values)) | (np.signbit(values) << 7)).astype(np.uint8)


@pytest.mark.parametrize("form", ["rows", "columns", "blocks"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_bytes(lib, cuda_device, form, dtype):
    """The codes are those of the division's quotient, byte for byte: zeros of either sign and
    numbers that round to them keep their sign, at ordinary scales, extreme ones and in groups
    that hold nothing else."""
    rng = np.random.default_rng(41)
    x = rng.standard_normal((520, 400)) * np.exp2(rng.integers(-14, 1, (520, 400)))
    x[rng.random(x.shape) < 0.2] = -0.0
    x[rng.random(x.shape) < 0.2] = 0.0
    x[:128] *= 2.0 ** -100              # scales below 2^-80, where the division itself is taken
    x[128:256] *= 2.0 ** 110            # and above 2^100
    x[256:384, :128] = np.where(rng.random((128, 128)) < 0.5, -0.0, 0.0)
    xt = torch.from_numpy(x.astype(np.float32)).to(dtype)
    codes, scales = lib.gptq_fp8_quantize(xt.to(cuda_device), form)
    ref, sref = quantize_ref(np32(xt), form)
    assert np.array_equal(scales.cpu().numpy(), sref)
    want = code_bytes(ref)
    assert (want == 0x80).sum() > 10000
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want)


def test_linear_gradients_are_exact_differences(lib, cuda_device):
    """On inputs that the quantisers represent exactly, an entry of x moves one token's outputs
    and an entry of W one column of them, and the gradients are those differences, weighted by dy.
    Both sides are within check_product's bound, 128 2^-23 + 3 blocks 2^-24 of the terms'
    magnitudes, which at the entries taken is under 5 % of the gradient."""
    rng = np.random.default_rng(11)
    t, n, k = 6, 130, 260
    grid = E4M3[(E4M3 >= 1) & (E4M3 <= 448)]
    def exact_grid(r, c):
        m = rng.choice(grid, (r, c)) * rng.choice([-1.0, 1.0], (r, c))
        # every group (1 x 128 either way, 128 x 128) reaches 448, so that its scale is 1
        m[np.arange(r) % 128 == 0, :] = 448
        m[:, np.arange(c) % 128 == 0] = 448
        return m
    x, w, dy = exact_grid(t, k), exact_grid(n, k), exact_grid(t, n)
    points = [(1, 1), (5, 259), (3, 130), (2, 77), (4, 200)]
    for i, j in points:
        x[i, j] = w[i, j] = 448 if (i + j) % 2 else -416
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).to(cuda_device)
    gamma = lambda m: 128 * 2.0 ** -23 + 3 * -(-m // 128) * 2.0 ** -24
    def outputs():
        y = lib.gptq_fp8_linear(dev(x), *lib.gptq_fp8_quantize(dev(w)), dtype=F32)
        return y.double().cpu().numpy(), gamma(k) * (np.abs(x) @ np.abs(w).T)
    codes, scales = lib.gptq_fp8_quantize(dev(w))
    dx, dw = lib.gptq_fp8_linear_backward(dev(dy), dev(x), codes, scales)
    base, tol = outputs()
    bx, bw = gamma(n) * (np.abs(dy) @ np.abs(w)), gamma(t) * (np.abs(dy).T @ np.abs(x))
    for i, j in points:
        for m, grad, own, part in ((x, dx, bx, np.s_[i, :]), (w, dw, bw, np.s_[:, i])):
            old = m[i, j]
            m[i, j] = -old
            moved = outputs()[0]
            m[i, j] = old
            diff = ((moved - base)[part] * dy[part]).sum() / (-2 * old)
            bound = 2 * (tol[part] * np.abs(dy[part])).sum() / (2 * abs(old)) + own[i, j]
            got = float(grad[i, j])
            assert bound <= 0.05 * abs(diff), (bound, diff)
            assert abs(diff - got) <= bound, (diff, got, bound)


def varied(rng, r, c, dtype, dev):
    """Values whose groups of 128, along either axis, differ in size by powers of two."""
    x = rng.standard_normal((r, c))
    x *= np.exp2(rng.integers(-6, 7, (r, -(-c // 128))).repeat(128, 1)[:, :c])
    x *= np.exp2(rng.integers(-6, 7, (-(-r // 128), c)).repeat(128, 0)[:r])
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(dev)


@pytest.mark.parametrize("t,n,k", [(2500, 2600, 2300),    # 99 tiles, 20 token blocks
                                   (300, 4200, 2400),     # 170 tiles, 3 blocks
                                   (4300, 300, 200)])     # 2 tiles, 34 blocks
@pytest.mark.parametrize("wdt", [F32, BF16])
def test_weight_gradient_of_many_tiles(lib, cuda_device, t, n, k, wdt):
    """More tiles than pairs of SMs and more token blocks than scale slots, with scales that
    differ from block to block and from column to column."""
    rng = np.random.default_rng(t + n + k)
    x, dy = varied(rng, t, k, BF16, cuda_device), varied(rng, t, n, BF16, cuda_device)
    g = torch.Generator().manual_seed(43)
    codes, scales = make_layer(lib, g, n, k, cuda_device)
    _, dw = lib.gptq_fp8_linear_backward(dy, x, codes, scales, need_dx=False, dw_dtype=wdt)
    check_product(dw, dequantized(np32(dy), "columns").T, dequantized(np32(x), "columns"))
    for _ in range(5):                                # the same bits every time
        assert torch.equal(lib.gptq_fp8_linear_backward(dy, x, codes, scales, need_dx=False,
                                                        dw_dtype=wdt)[1], dw)
    lib.gptq_async_status()


# many tiles; 9 x 9 tiles with a shared last wave; shared contractions; few tokens with more
# blocks a CTA than scale slots; tokens that the product quantises itself
@pytest.mark.parametrize("t,n,k", [(2600, 4400, 2300), (2300, 2200, 4200), (700, 1100, 5003),
                                   (12, 300, 40000), (50, 300, 40000), (100, 300, 40000),
                                   (3, 300, 40000), (8, 1000, 16000)])
def test_products_with_scales_of_every_size(lib, cuda_device, t, n, k):
    """Output and input gradient with a scale for each token and block that differs from its
    neighbours' by powers of two, repeated."""
    rng = np.random.default_rng(t + n + k)
    w = varied(rng, n, k, F32, cuda_device) * 2.0 ** -5
    codes, scales = lib.gptq_fp8_quantize(w)
    x = varied(rng, t, k, BF16, cuda_device)
    y = lib.gptq_fp8_linear(x, codes, scales, dtype=F32)
    check_product(y, dequantized(np32(x), "rows"), weight_values(codes, scales).T)
    tcodes, tscales = lib.gptq_fp8_quantize(w.t().contiguous())
    back = lambda: lib.gptq_fp8_linear_backward(x, None, tcodes, tscales, need_dw=False)[0]
    dx = back()
    check_product(dx, dequantized(np32(x), "rows"), weight_values(tcodes, tscales))
    for _ in range(5):
        assert torch.equal(lib.gptq_fp8_linear(x, codes, scales, dtype=F32), y)
        assert torch.equal(back(), dx)
    lib.gptq_async_status()


def test_gradients_of_a_long_vocabulary(lib, cuda_device):
    """An output head: the input gradient contracts over 131072 entries, the weight gradient has as
    many rows."""
    t, n, k = 300, 131072, 256
    g = torch.Generator().manual_seed(47)
    codes, scales = make_layer(lib, g, n, k, cuda_device)
    rng = np.random.default_rng(47)
    x, dy = varied(rng, t, k, BF16, cuda_device), varied(rng, t, n, BF16, cuda_device)
    dx, dw = lib.gptq_fp8_linear_backward(dy.float(), x, codes, scales)
    check_product(dx, dequantized(np32(dy), "rows"), weight_values(codes, scales))
    check_product(dw, dequantized(np32(dy), "columns").T, dequantized(np32(x), "columns"))
    lib.gptq_async_status()
