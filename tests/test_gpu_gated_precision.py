"""The gated product's activations in fp32 outputs, where the factors are exact:
one nonzero code a row and channel and scales that are powers of two, so that
what is off is the activation's own."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _gated(scale, act, rows, out=torch.float32):
    """(g, act(g)) for g = a c scale, all codes a of the rows and c of the channels."""
    a, c = np.resize(np.arange(-127, 128), rows), np.arange(-127, 128)
    x, wg, wu = (np.zeros((n, 16), np.int8) for n in (rows, len(c), len(c)))
    x[:, 0], x[:, 1], wg[:, 0], wu[:, 1] = a, 1, c, 1
    one = torch.ones(max(rows, len(c)), device="cuda")
    got = vq.gated_w8a8(torch.from_numpy(wg).cuda(), scale * one[:len(c)], torch.from_numpy(wu).cuda(), one[:len(c)],
                        torch.from_numpy(x).cuda(), one[:rows], torch.empty(rows, len(c), device="cuda", dtype=out),
                        activation=act)
    return (a[:, None] * c).astype(np.float64) * scale, got.double().cpu().numpy()


def _exact(g, act):
    t = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return np.where(t > 0, g / (1 + np.exp(-np.abs(t))), g * np.exp(-np.abs(t)) / (1 + np.exp(-np.abs(t))))


SCALES = [2.0 ** -16, 2.0 ** -13, 2.0 ** -11, 2.0 ** -9, 2.0 ** -7]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("rows", [5, 255, 600])
def test_silu_to_fp32(scale, rows):
    """In half units U of fp32: the power 2, its correction 1 and 0.1 (what is
    left of the argument's roundings), the sum 1, the reciprocal 2, the product
    1: 7.1.  Results below 2^-126 |g| may be 0."""
    g, got = _gated(scale, "silu", rows)
    want = _exact(g, "silu")
    off = np.abs(got - want) / (8 * U * np.abs(want) + (np.abs(g) + 1) * 2.0 ** -126)
    assert off.max() <= 1.0, (off.max(), g.flat[off.argmax()])


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("rows", [5, 255, 600])
def test_tanh_gelu_to_fp32(scale, rows):
    """The power 2, the sum 1, the reciprocal 2, the product 1; and the exponent,
    whose roundings are 2 |z| times as large relative to the result: 5 of the
    cubic term's constant, 3 where the two terms are put together.  Results
    below 2^-126 |g| may be 0."""
    g, got = _gated(scale, "gelu_tanh", rows)
    want, z = _exact(g, "gelu_tanh"), np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    off = np.abs(got - want) / ((7 + 16 * np.abs(z)) * U * np.abs(want) + (np.abs(g) + 1) * 2.0 ** -126)
    assert off.max() <= 1.0, (off.max(), g.flat[off.argmax()])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_16_bit_outputs(act, out):
    """The output's rounding, the exponent's (2^-15 of the result) and the rest
    (7 U); results below 2^-126 |g| may be 0."""
    for scale in (2.0 ** -13, 2.0 ** -9, 2.0 ** -7):
        g, got = _gated(scale, act, 300, out)
        want = _exact(g, act)
        fi = torch.finfo(out)
        bound = (fi.eps / 2 + 1.01 * 2.0 ** -15 + 7 * U) * np.abs(want) + fi.smallest_normal * fi.eps / 2 + \
            2.0 ** -126 * (np.abs(g) + 1)
        assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_large_arguments(act, out):
    """Far from zero the activations are g and 0 (below 2^-126 |g|), infinity
    and NaN pass."""
    scales = torch.tensor([1.0, 300.0, 1e4, 1e9, 1e20, 1e36, float("inf"), float("nan")], device="cuda")
    w = torch.zeros(2 * len(scales), 16, dtype=torch.int8, device="cuda")
    w[:len(scales), 0], w[len(scales):, 1] = 100, 1
    x = torch.zeros(2, 16, dtype=torch.int8, device="cuda")
    x[0, 0], x[1, 0], x[:, 1] = 1, -1, 1
    one, f = torch.ones(len(scales), device="cuda"), len(scales)
    got = vq.gated_w8a8(w[:f], scales, w[f:], one, x, one[:2], torch.empty(2, f, device="cuda", dtype=out),
                        activation=act).double().cpu()
    g = 100.0 * scales.double().cpu()
    assert ((got[0, :6] - g[:6]).abs() <= torch.finfo(out).eps / 2 * g[:6]).all() and got[0, 6] == float("inf")
    assert (got[1, :6].abs() <= 2.0 ** -126 * g[:6]).all(), got[1]
    assert torch.isnan(got[:, 7]).all()
