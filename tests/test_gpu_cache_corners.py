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
