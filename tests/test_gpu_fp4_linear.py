"""The dense linear with MXFP4 weights is the one-expert grouped product: output
and both gradients, with and without each of them."""

import numpy as np
import pytest

from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(32, 128, 128), (416, 1152, 640)])
@pytest.mark.parametrize("wants", [(True, True), (True, False), (False, True)])
def test_linear_and_its_gradients(M, N, K, wants):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"fp4 linear {M}x{N}x{K} {wants}")
    x = to_dev_bf16(inp.random_bf16((M, K), seed=31, outliers=True)).requires_grad_(wants[0])
    W = to_dev_bf16(inp.random_bf16((N, K), seed=32, std=0.02)).requires_grad_(wants[1])
    grad = to_dev_bf16(inp.random_bf16((M, N), seed=33, std=0.1))
    leaves = [t for t in (x, W) if t.requires_grad]
    out = mx.mx_linear(x, W, weight_format="mxfp4")
    want = mx.mx_grouped_mm(x, W.unsqueeze(0), to_dev_i32(np.array([M])), weight_format="mxfp4")
    assert out.shape == (M, N) and torch.equal(out, want) and out.any()
    got, ref = torch.autograd.grad(out, leaves, grad), torch.autograd.grad(want, leaves, grad)
    assert [g.shape for g in got] == [t.shape for t in leaves]
    assert all(torch.equal(g, r) and g.any() for g, r in zip(got, ref))
    with torch.no_grad():
        assert torch.equal(mx.mx_linear(x, W, weight_format="mxfp4"), out)
