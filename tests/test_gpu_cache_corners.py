"""Corners of the paged 8-bit cache: inputs at the ends of their ranges, rows whose sum is
empty, tokens taken back, tensors that change under the cache."""

import numpy as np
import pytest
import torch

import cache_reference as ref
from test_gpu_cache import DEV, Case, host, i32, mask_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from dynamic_causal_attention_gb300 import api as _api
    return _api


KERNELS = [(3, "cache_attn"), (70, "cache_chunk")]


@pytest.mark.parametrize("n_q,kernel", KERNELS)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("e_q,e_k", [(-80, -64), (-30, -126), (-110, -10)])
def test_small_queries_against_small_scales(api, d, e_q, e_k, n_q, kernel):
    # the factor of a logit underflows: the weights are equal, keys behind a row weigh nothing
    c = Case(api, mask_of(4, (1,)), 2, d, 16, [200, n_q + 13], n_q, seed=d, kernel=kernel)
    c.k_scales = np.where(np.isfinite(c.k_scales), 2.0 ** e_k, c.k_scales).astype(np.float32)
    c.q = (c.q.float() * 2.0 ** e_q).to(torch.bfloat16)
    c.put()
    c.check(*c.run())


@pytest.mark.parametrize("page,tail", [(64, 1), (16, 3), (32, 1)])
def test_nan_in_a_table_that_ends_inside_a_tile(api, page, tail):
    # seq_len lies far behind the table, whose keys are no multiple of 128: every row sees all
    # of them, the NaN among them too
    cols = 2 ** 18 // page + tail
    length = cols * page + 1000
    holes = [(0, j) for j in range(2, cols - 3)]
    c = Case(api, mask_of(4, (1,)), 1, 32, page, [length], 80, holes=holes, cols=cols, seed=page)
    c.kernel = "cache_chunk"
    c.v_codes[c.table[0, cols - 1], 0, page - 5, 3] = 0x7F
    c.v_codes[c.table[0, cols - 1], 0, 0, 30] = 0xFF
    c.put()
    out, lse = c.run()
    assert bool(torch.isnan(out[0, :, :, [3, 30]].float()).all())
    c.check(out, lse)
