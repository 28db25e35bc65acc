"""GPU tests of which keys the paged attention leaves out, in every variant.

Tolerances are those derived in test_gpu_paged.py.
"""

import math

import pytest
import torch

from tests.test_gpu_paged import Setup, U
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


@pytest.mark.parametrize("gain", [None, 0.0, 1.0])
def test_products_alone_remove_no_key(variant, gain):
    """Logits of about -1e33 from the products, all alike: the outputs are the
    means of the values. Tolerance: the weights are equal, so that the sums'
    roundings (keys x 2^-24) and one rounding of the weights and of the output
    remain, of at most the largest value."""
    st = variant
    for b, (n, p) in enumerate(st.lens):
        pg, r = st.where(b, 0, n + p)
        st.k[pg, r] = -1e16
    st.bias.fill_(0.0)
    q = torch.full((st.rows, st.hq, st.dh), 1e16, device="cuda").to(st.dtype)
    lse = torch.full((st.hq, st.rows), 7.0, device="cuda")
    g = None if gain is None else torch.full((st.hq,), gain, device="cuda")
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=g, lse=lse)
    want = float(q[0, 0, 0]) * float(st.k[st.table[0, 0], 0, 0, 0]) * math.sqrt(st.dh)
    assert ((lse / want - 1).abs() <= 2.0 ** -20).all()
    u = U[st.dtype]
    for b, (n, p) in enumerate(st.lens):
        pg, r = st.where(b, 0, n + p)
        vb = st.v[pg, r].double()
        mean = (vb.cumsum(0) / torch.arange(1, n + p + 1, device="cuda")[:, None, None])[p:]
        mean = mean.repeat_interleave(st.hq // st.hkv, 1)
        got = out[st.cu_host[b]:st.cu_host[b + 1]].double()
        tol = u * mean.abs() + (2 * u + (n + p) * 2.0 ** -24) * vb.abs().amax()
        assert ((got - mean).abs() <= tol).all(), float(((got - mean).abs() - tol).max())
