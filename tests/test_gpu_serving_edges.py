"""Serving operators at the edges of their contracts, against the plain 64-bit forms (tests/serving_helpers.py):
query rows that are not finite, offsets that decrease next to sound ones, float32 sums over very long rows.
Tolerances: tests/test_gpu_serving.py, unless a test derives its own."""
import numpy as np
import pytest
import torch

import serving_helpers as R
from gpu_helpers import BF, lib
from test_gpu_serving import F32, U32, UBF, Prompt, check_out, check_weight, host, i32, score_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("n_q,n_kv,row", [(400, 400, 264), (400, 400, 265), (400, 400, 266), (400, 400, 3), (450, 480, 384),
                                          (5, 2500, 0), (5, 2500, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prompt_nonfinite_query_row(cuda, kernel, dtype, d, n_q, n_kv, row, value):
    """One query row of one head is not finite: its output and the weights of every key that it sees are NaN,
    wherever the row lies in a tile; all else is as without it."""
    p = Prompt(lib(), dtype, d, 2, 2, [n_q], [n_kv], seed=row + d, kernel=kernel)
    q = host(p.q)
    q[row, 0] = 0
    p.q[row, 0, :3] = value
    p.run()
    k, v = host(p.k), host(p.v)
    ref, w = R.prompt_attention(q, k, v, p.cu_q, p.cu_kv, p.n_w)
    spread, _ = R.prompt_attention(q, k, np.abs(v), p.cu_q, p.cu_kv, p.n_w)
    e, seen = score_step(q, k, n_kv), row + n_kv - n_q + 1
    o, got = host(p.o), host(p.w)
    assert np.isnan(o[row, 0]).all() and np.isnan(got[0, 0, :seen]).all()
    o[row, 0], ref[row, 0] = 0, 0
    check_out(o, ref, spread, e, dtype, UBF if dtype == BF and kernel == 0 else 0.0)
    check_weight(got[0, 0, seen:], host(p.w0)[0, 0, seen:], w[0, 0, seen:], e)
    check_weight(got[0, 1], host(p.w0)[0, 1], w[0, 1], e)
