"""GPU tests of which keys the paged attention leaves out, in every variant.

Tolerances are those derived in test_gpu_paged.py.
"""

import math

import pytest
import torch

from tests.test_gpu_paged import Setup
from tests.test_gpu_serving import VARIANTS

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")


@pytest.fixture(autouse=True)
def _no_device_errors():
    tg.tg_device_error(clear=True)
    yield
    assert tg.tg_device_error() == 0


@pytest.fixture(params=list(VARIANTS))
def variant(request):
    lens, hq, hkv, dh, page, dt = VARIANTS[request.param]
    return Setup(lens, hq, hkv, dh, page, dt, seed=60).fill()


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_without_gains_the_biases_are_not_read(variant, junk):
    """gain=None is a call without a bias, whatever the cache holds there."""
    st = variant
    q = st.queries()
    bare = tg.PagedKV(st.k, st.v, st.table)
    want = tg.tg_paged_attn(bare, q, st.cu, st.kv_len)
    st.bias.fill_(junk)
    assert torch.equal(tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len), want)
