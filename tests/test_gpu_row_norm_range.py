"""The norm of rows whose squares leave the range of fp32, against the 64-bit
definition."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R

pytestmark = pytest.mark.gpu
POWERS = [-130, -100, -64, -50, -46, -45, -44, 0, 50, 57, 60, 64, 100, 120]
TINY = [p for p in POWERS if p < 0]


def _np(t):
    return t.double().cpu().numpy()


def _rows(c, dtype, seed):
    """A row of about 2^p for each p, the last one with both ends in it."""
    x = torch.randn(len(POWERS) + 1, c, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    for i, p in enumerate(POWERS):
        x[i] *= 2.0 ** p
    x[-1, ::2] *= 2.0 ** 100
    x[-1, 1::2] *= 2.0 ** -100
    return x.to(dtype).cuda()


def _within(got, want, bound, out):
    worst = np.abs(_np(got) - want) / R.rounded(want, bound, out)
    assert worst.max() <= 1.0, (worst.max(1))


@pytest.mark.parametrize("c", [16, 5120, 16400, 32768])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 3e38])
def test_norm_of_any_magnitude(c, dtype, eps):
    x = _rows(c, dtype, c)
    w = (1 + 0.2 * torch.randn(c, generator=torch.Generator().manual_seed(1))).cuda()
    out = vq.residual_norm(x, weight=w, eps=eps, out=torch.empty(x.shape, dtype=torch.bfloat16, device="cuda"))
    _, _, h, eh = R.norm(_np(x), None, _np(w), None, None, 1.0, float(np.float32(eps)))
    _within(out, h, eh, "bf16")
    q, s = vq.residual_norm(x, weight=w, eps=eps, out=torch.empty(x.shape, dtype=torch.int8, device="cuda"),
                            scales_out=torch.empty(len(x), device="cuda"))
    # the largest element's error, and two roundings of the scale; scales below the normal numbers to 2^-150
    assert (np.abs(_np(s) * 127 - np.abs(h).max(1)) <= eh.max(1) + 2 * R.U * np.abs(h).max(1) + 127 * 2.0 ** -149).all()


@pytest.mark.parametrize("c", [64, 8208])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_behind_a_block_of_any_magnitude(c, eps):
    """The norm of y (bf16, so that its squares leave the range too), in the
    sum with a residual of about 1."""
    y = _rows(c, torch.bfloat16, 7 * c)
    r = torch.randn(y.shape, generator=torch.Generator().manual_seed(2)).cuda()
    pw = (1 + 0.2 * torch.randn(c, generator=torch.Generator().manual_seed(3))).cuda()
    ro, out = torch.empty_like(r), torch.empty_like(y)
    vq.residual_norm(r, y, post_weight=pw, alpha=0.35, eps=eps, out=out, residual_out=ro)
    x, ex, h, eh = R.norm(_np(r), _np(y), None, _np(pw), None, float(np.float32(0.35)), float(np.float32(eps)))
    _within(ro, x, ex, "f32")
    _within(out, h, eh, "bf16")


def test_infinities_and_nan_mark_their_row_alone():
    x = torch.randn(4, 80, device="cuda")
    x[0, 3], x[1, 5] = float("inf"), float("nan")
    x[2] *= 1e30
    out = vq.residual_norm(x, out=torch.empty(4, 80, dtype=torch.bfloat16, device="cuda"))
    finite = torch.ones(80, dtype=torch.bool, device="cuda")
    finite[3] = False
    assert (out[0][finite] == 0).all() and torch.isnan(out[0, 3]) and torch.isnan(out[1]).all()
    assert torch.isfinite(out[2:]).all()
