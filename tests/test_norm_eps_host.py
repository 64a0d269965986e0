"""The norm's eps on the host: every finite one is taken, nothing else."""
import math

import pytest
import torch

import block_quantized_gemm_amd as vq
from test_layer_host import _norm


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would run")
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-6, 3.1e38, 3.4028234e38])
def test_finite_eps(eps):
    assert _norm(eps=eps) == vq.VQ_ERR_DEVICE  # past the checks of the arguments


@pytest.mark.parametrize("eps", [-2.0 ** -149, -1.0, math.inf, -math.inf, math.nan])
def test_other_eps(eps):
    assert _norm(eps=eps) == vq.VQ_ERR_BAD_CONFIG
