"""Few-token layers of different sizes called from several host threads at once:
every call launches, and gives the bits of a call on its own."""

import threading

import numpy as np
import pytest

from mxfp8_block_scaled_06_amd import inputs as inp
from gpu_util import require_gpu, to_dev_bf16, to_dev_i32, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_layers_from_two_threads(fmt):
    torch = require_gpu()
    import mxfp8_block_scaled_06_amd as mx
    log(f"moe from threads {fmt}")
    quantize = mx.mx_quantize_weights_fp4 if fmt == "mxfp4" else mx.mx_quantize_weights

    def layer(T, k, E, K, N, seed):
        rng = np.random.default_rng(seed)
        w13 = quantize(to_dev_bf16(inp.random_bf16((E, 2 * N, K), seed=seed, std=0.05)))[:2]
        w2 = quantize(to_dev_bf16(inp.random_bf16((E, K, N), seed=seed + 1, std=0.05)))[:2]
        return (to_dev_bf16(inp.random_bf16((T, K), seed=seed + 2)),
                to_dev_i32(rng.integers(0, E, size=(T, k)).astype(np.int32)),
                torch.from_numpy(rng.random((T, k), dtype=np.float32)).to("cuda:0"), w13, w2)

    # the same kernels, with the least and with much LDS
    cases = [layer(2, 1, 4, 128, 128, 1), layer(15, 4, 16, 2048, 256, 5)]
    want = [mx.mx_moe_few_tokens(*c, weight_format=fmt) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [mx.mx_moe_few_tokens(*cases[i], weight_format=fmt, check=False) for _ in range(200)]
            stream.synchronize()
            assert all(torch.equal(g, want[i]) for g in got)
        except Exception as e:      # reported in the test's own thread
            failed.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
