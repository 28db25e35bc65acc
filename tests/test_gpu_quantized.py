"""GPU parity of the 8-bit projections against their definitions in 64 bits.

tg_quantize_rows: the integers are those of the exact quotient (64 bits
decide every value: 127 x is exact there and the quotient of at most 31-bit
integers is rounded far below its distance from a half-integer); the scale
is one rounded fp32 quotient, 2^-24.
tg_linear_quantized: the integer sum is exact; its conversion, two products
and the residual's sum are one fp32 rounding each (4 x 2^-24 of the terms'
sizes), then one rounding to the output type (bf16 2^-8, fp32 2^-24).
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _no_device_errors():
    tg.tg_device_error(clear=True)
    yield
    assert tg.tg_device_error() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check_quantize(x, got):
    xq, scale = got
    w = x.double()
    amax = w.abs().amax(1)
    safe = torch.where(amax > 0, amax, 1.0)
    assert torch.equal(xq, torch.round(127.0 * w / safe[:, None]).to(torch.int8))
    assert ((scale.double() - amax / 127).abs() <= 2.0 ** -24 * amax / 127 + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 2048), (3, 48), (17, 4096), (130, 6144),
                                       (2, 12288), (5, 40000), (1000, 128), (4, 131056)])
def test_quantize(dtype, rows, cols):
    x = torch.randn(rows, cols, generator=gen(rows + cols), device="cuda")
    x *= torch.exp(4 * torch.randn(rows, 1, generator=gen(1), device="cuda"))
    x = x.to(dtype)
    check_quantize(x, tg.tg_quantize_rows(x))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_borders_and_extremes(dtype):
    """Quotients on and next to half-integers, rows of zeros, of one value, of
    the smallest and largest numbers."""
    fi = torch.finfo(dtype)
    k = torch.arange(-128, 128, device="cuda", dtype=torch.float64)
    rows = [k / 2, k / 2 + 0.25, (k + 0.5) * 127 / 128, torch.zeros_like(k), torch.full_like(k, -3.0),
            k * fi.smallest_normal / 16, k * (fi.max / 128), k * fi.tiny * 40,
            torch.where(k == 5, 127.0, k / 2)]
    for step in range(1, 8):  # one unit of the type's mantissa around the borders
        rows.append(torch.where(k == 0, 127.0, (k + 0.5) * (1 + (step - 4) * fi.eps)).clamp(-127, 127))
    x = torch.stack(rows).to(dtype)
    check_quantize(x, tg.tg_quantize_rows(x))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_rows_that_are_not_finite(dtype):
    x = torch.randn(6, 256, generator=gen(3), device="cuda").to(dtype)
    x[1, 7], x[3, 200], x[4, 0] = float("inf"), float("nan"), -float("inf")
    xq, scale = tg.tg_quantize_rows(x)
    bad = torch.tensor([False, True, False, True, True, False], device="cuda")
    assert torch.equal(torch.isnan(scale), bad) and (xq[bad] == 0).all()
    check_quantize(x[~bad], (xq[~bad], scale[~bad]))


def test_quantize_strided_rows():
    big = torch.randn(40, 3, 128, generator=gen(4), device="cuda").to(BF)
    x = big[:, 1]
    check_quantize(x, tg.tg_quantize_rows(x))
    assert tg.tg_quantize_rows(x[:0])[0].shape == (0, 128)


def check_linear(m, n, k, dtype, residual, seed=0, lo=-127, in_place=False):
    g = gen(seed)
    xq = torch.randint(lo, 128, (m, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    wq = torch.randint(lo, 128, (n, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    xs = torch.rand(m, generator=g, device="cuda") * 1e-2
    ws = torch.rand(n, generator=g, device="cuda") * 1e-2
    res = torch.randn(m, n, generator=g, device="cuda").to(dtype) if residual else None
    want = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    tol = 4 * 2.0 ** -24 * want.abs()
    if residual:
        tol += 2.0 ** -24 * (want + res.double()).abs()
        want = want + res.double()
    tol += U[dtype] * want.abs()
    y = None
    if in_place:
        y = res
    got = tg.tg_linear_quantized(xq, xs, wq, ws, residual=res, y=y, dtype=dtype)
    assert got.dtype == dtype and got.shape == (m, n)
    diff = (got.double() - want).abs()
    assert (diff <= tol * 1.001).all(), (float((diff - tol).max()), float(diff.max()))


@pytest.mark.parametrize("dtype,residual", [(BF, False), (BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("m,n,k", [
    (1, 32, 16), (1, 4096, 2048), (2, 64, 48), (3, 2048, 6144), (5, 12288, 2048), (8, 96, 1040),
    (9, 2048, 2048), (16, 4096, 2048), (17, 160, 272), (31, 2048, 6144), (33, 480, 2048),
    (64, 4096, 2048), (100, 2048, 6144), (127, 256, 128), (128, 256, 128), (129, 288, 144),
    (255, 4096, 2048), (257, 544, 1008), (700, 2048, 528), (1025, 1024, 2064), (2500, 4096, 2048)])
def test_linear(m, n, k, dtype, residual):
    check_linear(m, n, k, dtype, residual, seed=m + n)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_linear_extreme_values_and_long_rows(m):
    """-128 everywhere and the longest rows: the largest integer sums."""
    k, n = 131056, 64
    xq = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    wq[1::2] = 127
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    y = tg.tg_linear_quantized(xq, one_m, wq, one_n, dtype=F32)
    want = torch.tensor([128.0 * 128 * k, -128.0 * 127 * k], dtype=torch.float64)
    got = y[:, :2].double().cpu()
    assert ((got - want).abs() <= 2.0 ** -24 * want.abs()).all()
    assert (y == y[:1, :2].repeat(1, n // 2)).all()
    check_linear(m, 96, 4096, BF, False, seed=9, lo=-128)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_linear_in_place_residual_and_nan_scale(m):
    check_linear(m, 256, 512, BF, True, seed=5, in_place=True)
    xq = torch.ones(m, 64, dtype=torch.int8, device="cuda")
    wq = torch.ones(32, 64, dtype=torch.int8, device="cuda")
    xs, ws = torch.ones(m, device="cuda"), torch.ones(32, device="cuda")
    xs[m // 2] = float("nan")
    y = tg.tg_linear_quantized(xq, xs, wq, ws)
    bad = torch.isnan(y.float())
    assert bad[m // 2].all() and int(bad.sum()) == 32
    assert tg.tg_linear_quantized(xq[:0], xs[:0], wq, ws).shape == (0, 32)


@pytest.mark.parametrize("m", [1, 50, 400])
def test_linear_is_deterministic_and_replays(m):
    g = gen(6)
    x = torch.randn(m, 2048, generator=g, device="cuda").to(BF)
    w = torch.randn(1024, 2048, generator=g, device="cuda").to(BF)
    wq, ws = tg.tg_quantize_rows(w)
    y = torch.empty(m, 1024, dtype=BF, device="cuda")

    def step():
        xq, xs = tg.tg_quantize_rows(x)
        return tg.tg_linear_quantized(xq, xs, wq, ws, y=y)

    ref = step().clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            xq, xs = tg.tg_quantize_rows(x)
            outs.append(tg.tg_linear_quantized(xq, xs, wq, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -ref)


def test_quantized_projection_is_near_the_bf16_one():
    """What a user sees: the 8-bit projection of a row against tg_linear. Each
    integer is off by at most half a step: |dy| <= sum_k (|x| ws/2 + |w| xs/2 +
    xs ws/4), far above what is met; held here in full."""
    g = gen(7)
    x = torch.randn(70, 2048, generator=g, device="cuda").to(BF)
    w = (0.02 * torch.randn(4096, 2048, generator=g, device="cuda")).to(BF)
    xq, xs = tg.tg_quantize_rows(x)
    wq, ws = tg.tg_quantize_rows(w)
    y = tg.tg_linear_quantized(xq, xs, wq, ws).double()
    ref = x.double() @ w.double().t()
    bound = (x.double().abs().sum(1, keepdim=True) * ws.double() / 2
             + w.double().abs().sum(1) * xs.double()[:, None] / 2
             + 2048 * xs.double()[:, None] * ws.double() / 4 + 2.0 ** -8 * y.abs())
    assert ((y - ref).abs() <= bound * 1.001).all()
