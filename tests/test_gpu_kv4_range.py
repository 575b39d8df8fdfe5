"""The 4-bit cache's attention where scores, value steps and pages are far from ordinary: scores far below zero, references
that are outgrown inside a tile, value steps of very different sizes, pages that are not there, contexts never written; and
kernels that follow one another while the one before still runs.

The tolerance is that of test_gpu_kv4 (its docstring derives it); where a test needs another, it stands there."""
import numpy as np
import pytest

from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import weight_only_int4_act_b200 as awq  # noqa: E402
from test_gpu_kv4 import DT, _check, _f64, _fill, _rand, _read  # noqa: E402


# ---------------------------------------------------------------- kernels behind one another
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_then_the_8_bit_layer(dim):
    """A prompt's attention, the row quantiser and the few-token product, each launched while the one before still runs."""
    heads, share, n, batch = 8, 8, 16, 8
    cfg, cache, table, lens, slots = _fill([200 + 40 * i for i in range(batch)], heads, dim, dim, 32, "bf16", 200)
    W = _rand((256, heads * share * dim), "bf16", 201, 0.05)
    wq, w_step = awq.quantize_int8(W)
    start = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n

    def step(q, wait):
        out = awq.kv4_attention(q, cache, table, lens, cfg, q_start=start, max_q=n)
        wait()
        xq, x_step = awq.quantize_int8(out.view(n * batch, -1))
        wait()
        return awq.w8a8_gemm(xq, x_step, wq, w_step)
    for i in range(10):
        q = _rand((n * batch, heads * share, dim), "bf16", 210 + i)
        want = step(q, torch.cuda.synchronize)
        torch.cuda.synchronize()
        got = [step(q, lambda: None) for _ in range(5)]
        assert all(torch.equal(want, g) for g in got) and want.any()
