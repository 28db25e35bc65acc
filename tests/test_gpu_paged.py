"""GPU parity of the paged cache: tg_paged_append and tg_paged_attn against the
definitions in 64 bits.

Tolerances, from the arithmetic (u = eps / 2 of a type: bf16 2^-8, fp32 2^-24):

append   q, k: one rounding to the type, u |y|; in fp32 before it the norm
         (a sum of dh squares, a square root, two products: (dh + 8) 2^-24)
         and the rotation (cos and sin within 2^-22, two products and a sum),
         all relative to |x| |w| (|c| + |s|) <= 2 max |pair|. v exact.
         bias: logsigmoid in fp32, 2^-21 relative plus 2^-24 absolute.
attn     the logit's error e (log units): (dh + 8) 2^-24 sum |q k| scale, the
         bias product 2^-22 |gain bias|, and 2^-22 |logit| for the scaling and
         the exponential's argument. An output is a weighted mean of v, so it
         moves by at most 2 max(e) A with A = sum_j P_ij |v_j|, and by
         (keys + 8) 2^-24 A in the fp32 sums. bf16 also rounds the weights P
         (u each: u A) and the exponential may be a polynomial within 7.5e-5
         (twice, in numerator and sum: 1.5e-4 A). Then one rounding of the
         output, u |o|.
         lse: max(e) + (keys + 8) 2^-24 + 1.5e-4 (bf16) + 2^-22 |lse|.
"""

import math

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


class Setup:
    """A batch of requests [(new rows, cached rows before them)] with pages
    dealt at random; stale rows are NaN."""

    def __init__(self, lens, hq, hkv, dh, page, dtype, bias=True, seed=0, stale=float("nan"),
                 layers=1, spare=2):
        g = gen(seed)
        self.g, self.lens, self.hq, self.hkv, self.dh, self.page = g, lens, hq, hkv, dh, page
        self.dtype = dtype
        need = [-(-max(n + p, 0) // page) for n, p in lens]
        pool = sum(need) + spare
        shape = (pool, layers, page, hkv, dh)
        self.pool_k = torch.full(shape, stale, dtype=dtype, device="cuda")
        self.pool_v = torch.full(shape, stale, dtype=dtype, device="cuda")
        self.k, self.v = self.pool_k[:, layers - 1], self.pool_v[:, layers - 1]
        self.bias = torch.full((pool, page), stale, device="cuda") if bias else None
        perm = torch.randperm(pool, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = perm[at:at + c]
            at += c
        self.cache = tg.PagedKV(self.k, self.v, self.table, self.bias)
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        self.cu_host, self.rows = cu, cu[-1]
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([n + p for n, p in lens], dtype=torch.int32, device="cuda")

    def where(self, b, lo, hi):
        j = torch.arange(lo, hi, device="cuda")
        return self.table[b, j // self.page].long(), j % self.page

    def fill(self):
        """Random rows for every request; gate biases of random scores."""
        for b, (n, p) in enumerate(self.lens):
            t = n + p
            if t <= 0:
                continue
            pg, r = self.where(b, 0, t)
            for dst in (self.k, self.v):
                dst[pg, r] = torch.randn(t, self.hkv, self.dh, generator=self.g,
                                         device="cuda").to(self.dtype)
            if self.bias is not None:
                s = 2 * torch.randn(t, generator=self.g, device="cuda")
                self.bias[pg, r] = torch.nn.functional.logsigmoid(s)
        return self

    def queries(self, extra=0):
        q = torch.randn(self.rows + extra, self.hq, self.dh, generator=self.g, device="cuda")
        return q.to(self.dtype)

    def gates(self):
        return (2 * torch.rand(self.hq, generator=self.g, device="cuda"),
                0.5 + torch.rand(self.hq, generator=self.g, device="cuda"))


def attn_reference(st, q, gain, tau):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
    grp, dh = st.hq // st.hkv, st.dh
    out = torch.zeros(st.rows, st.hq, dh, dtype=torch.float64, device="cuda")
    lse = torch.full((st.hq, st.rows), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    u = U[st.dtype]
    for b, (n, p) in enumerate(st.lens):
        if n == 0 or n + p <= 0:
            continue
        t0, total = st.cu_host[b], n + p
        pg, r = st.where(b, 0, total)
        kb, vb = st.k[pg, r].double(), st.v[pg, r].double()
        bb = st.bias[pg, r].double() if st.bias is not None else None
        see = (torch.arange(total, device="cuda")[None]
               < torch.arange(p + 1, p + n + 1, device="cuda")[:, None])
        for h in range(st.hq):
            scale = 1.0 / (math.sqrt(dh) * (float(tau[h]) if tau is not None else 1.0))
            qh, kh, vh = q[t0:t0 + n, h].double(), kb[:, h // grp], vb[:, h // grp]
            lg = qh @ kh.t() * scale
            err = (dh + 8) * 2.0 ** -24 * (qh.abs() @ kh.abs().t()) * scale + 2.0 ** -22 * lg.abs()
            if bb is not None and gain is not None and float(gain[h]) != 0.0:
                add = float(gain[h]) * bb
                lg = lg + add
                err = err + 2.0 ** -22 * torch.where(add > -1e30, add.abs(), 0.0)
            lg = torch.where(see & (lg > -1e29), lg, -math.inf)
            e = torch.where(lg > -math.inf, err, 0.0).amax(1, keepdim=True)
            ls = torch.logsumexp(lg, 1, keepdim=True)
            w = torch.where(lg > -math.inf, torch.exp(lg - torch.where(ls > -math.inf, ls, 0.0)), 0.0)
            # values that a row does not see never reach it
            clean = torch.where(torch.isfinite(vh), vh, 0.0)
            o, a = w @ clean, w @ clean.abs()
            bad = w @ (~torch.isfinite(vh)).double() > 0
            extra = (u + 1.5e-4) if st.dtype == BF else 0.0
            out[t0:t0 + n, h] = torch.where(bad, float("nan"), o)
            tol[t0:t0 + n, h] = a * (2 * e + (total + 8) * 2.0 ** -24 + extra) * 1.01 + u * o.abs()
            lse[h, t0:t0 + n] = ls[:, 0]
            tol_l[h, t0:t0 + n] = (e[:, 0] + (total + 8) * 2.0 ** -24
                                   + (1.5e-4 if st.dtype == BF else 0.0) + 2.0 ** -22 * ls[:, 0].abs()
                                   + 2.0 ** -23)
    return out, lse, tol, tol_l


def check_attn(st, q, gain, tau, max_kv=None):
    out = torch.full_like(q, 7.0)
    lse = torch.full((st.hq, q.shape[0]), 7.0, device="cuda")
    tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, max_kv=max_kv, out=out,
                     lse=lse)
    want, wlse, tol, tol_l = attn_reference(st, q, gain, tau)
    got, glse = out[:st.rows].double(), lse[:, :st.rows].double()
    assert (out[st.rows:] == 7).all() and (lse[:, st.rows:] == 7).all()
    bad = torch.isnan(want)
    assert torch.equal(~torch.isfinite(got), bad)
    diff = torch.where(bad, 0.0, (got - torch.where(bad, 0.0, want)).abs())
    worst = (diff - torch.where(bad, 0.0, tol)).max()
    assert worst <= 0, (float(worst), float(diff.max()))
    none = torch.isneginf(wlse)
    assert torch.equal(torch.isneginf(glse), none)
    dl = torch.where(none, 0.0, glse - wlse).abs()
    assert (dl <= torch.where(none, 0.0, tol_l)).all(), float((dl - tol_l)[~none].max())
    return out


SHAPES = [  # hq, hkv, dh, page, dtype
    (16, 8, 128, 64, BF), (4, 2, 64, 16, BF), (8, 1, 128, 128, BF), (6, 2, 64, 256, BF),
    (5, 5, 128, 32, BF), (10, 2, 128, 16, BF), (4, 2, 64, 32, F32), (6, 2, 128, 16, F32),
]
LENS = {
    "decode": [(1, 0), (1, 1), (1, 126), (1, 127), (1, 128), (1, 700), (1, 31), (1, 2049)],
    "ragged": [(0, 5), (7, 0), (65, 200), (0, 0), (129, 1), (1, 511), (128, 128), (33, 1000)],
    "chunk": [(300, 517)],
    "empty_past": [(257, 0), (64, 0)],
}


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[1]}x{s[2]}-p{s[3]}-{str(s[4])[6:]}")
def test_attn_parity(shape, lens, bias):
    st = Setup(LENS[lens], *shape, bias=bias, seed=len(lens)).fill()
    gain, tau = st.gates()
    check_attn(st, st.queries(extra=3), gain if bias else None, tau if bias else None)


def test_attn_long_context():
    """Contexts of thousands of keys of very different lengths, one to a few
    new rows: the split of one row's keys over many thread blocks."""
    st = Setup([(1, 20000), (3, 50), (2, 9000), (1, 0), (5, 4096)], 16, 8, 128, 64, BF, seed=3).fill()
    check_attn(st, st.queries(), *st.gates(), max_kv=20001)


def test_attn_many_short_requests():
    """More requests than a warp or a thread block counts at once."""
    lens = [(i % 4, (i * 37) % 190) for i in range(700)]
    st = Setup(lens, 4, 2, 64, 16, BF, seed=4).fill()
    check_attn(st, st.queries(), *st.gates())


def test_attn_wide_group():
    """More query heads to a KV head than a tile has rows for one token."""
    st = Setup([(3, 100), (1, 300)], 160, 1, 64, 32, BF, seed=5).fill()
    check_attn(st, st.queries(), *st.gates())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_masked_keys(dtype):
    """Biases of -inf and of the lowest value remove keys, for every row or
    some; a head of gain 0 sees them; rows without a key are zero."""
    st = Setup([(40, 90), (2, 0), (1, 130)], 4, 2, 64, 32, dtype, seed=6).fill()
    gain = torch.tensor([1.0, 0.0, 0.5, 2.0], device="cuda")
    tau = torch.ones(4, device="cuda")
    pg, r = st.where(0, 0, 100)
    st.bias[pg, r] = -math.inf            # rows 0 .. 9 of the chunk have no key left
    st.bias[pg[50:60], r[50:60]] = torch.finfo(F32).min
    pg, r = st.where(1, 0, 2)
    st.bias[pg, r] = -math.inf            # nothing left at all
    pg, r = st.where(2, 0, 131)
    st.bias[pg[::2], r[::2]] = -math.inf  # every other key
    out = check_attn(st, st.queries(), gain, tau)
    assert (out[40:42, 0] == 0).all() and (out[40:42, 1] != 0).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[(150, 70)], [(9, 3), (4, 250)], [(300, 0)]])
def test_attn_values_behind_a_row_never_reach_it(dtype, lens):
    """Infinite and NaN values of later rows of the chunk: rows before them
    are finite, rows that see them are not."""
    st = Setup(lens, 8, 4, 64, 16, dtype, seed=7).fill()
    for b, (n, p) in enumerate(lens):
        pg, r = st.where(b, p + n // 2, p + n // 2 + 2)
        st.v[pg[0], r[0], 0, 3] = float("nan")
        st.v[pg[1], r[1], 2, 63] = math.inf
    check_attn(st, st.queries(), *st.gates())


def test_attn_more_new_rows_than_cached_ones():
    """kv_len below the chunk's rows: the first ones see nothing."""
    st = Setup([(5, 10), (6, -4), (3, -3)], 4, 2, 64, 16, BF, seed=8).fill()
    out = check_attn(st, st.queries(), *st.gates())
    assert (out[5:9] == 0).all() and (out[11:] == 0).all() and (out[9:11] != 0).any()


def test_attn_strided_queries_and_layered_pool():
    """q as a slice of a fused projection, one layer of a pool of three."""
    st = Setup([(17, 60), (1, 33)], 8, 2, 128, 32, BF, seed=9, layers=3).fill()
    fused = torch.randn(st.rows, 12, 128, generator=st.g, device="cuda").to(BF)
    gain, tau = st.gates()
    got = tg.tg_paged_attn(st.cache, fused[:, :8], st.cu, st.kv_len, gain=gain, tau=tau)
    want = check_attn(st, fused[:, :8].contiguous(), gain, tau)
    assert torch.equal(got, want)
    assert torch.isnan(st.pool_k[:, :2].float()).all()


def test_attn_matches_the_contiguous_kernel():
    """The whole chunk in an empty cache is tg_gated_attn_prefill."""
    n, hq, hkv, dh = 700, 16, 8, 128
    st = Setup([(n, 0)], hq, hkv, dh, 64, BF, seed=10, stale=0.0)
    q = torch.randn(n, hq, dh, generator=st.g, device="cuda").to(BF)
    k = torch.randn(n, hkv, dh, generator=st.g, device="cuda").to(BF)
    v = torch.randn(n, hkv, dh, generator=st.g, device="cuda").to(BF)
    s = torch.randn(n, generator=st.g, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 3
    gain, tau = st.gates()
    qr = tg.tg_paged_append(st.cache, k, v, st.cu, st.kv_len, q=q, pos=pos, s=s)
    out = tg.tg_paged_attn(st.cache, qr, st.cu, st.kv_len, gain=gain, tau=tau)
    want = tg.tg_gated_attn_prefill(q, k, v, pos, s=s, gain=gain, tau=tau)
    _, _, tol, _ = attn_reference(st, qr, gain, tau)
    # both are within the tolerance of the 64-bit result of the same rotated
    # rows; the two rotations round alike up to one bf16 step of q and k
    # (2^-7 of a logit's |q||k| sum: measured against 2e-2, the bf16 bound)
    assert ((out.double() - want.double()).abs() <= 2 * tol + 2e-2).all()


def test_attn_reports_pages_out_of_range():
    st = Setup([(1, 40), (1, 40)], 4, 2, 64, 16, BF, seed=11).fill()
    q, (gain, tau) = st.queries(), st.gates()
    good = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    st.table[0, 1] = 10 ** 6
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    assert tg.tg_device_error(clear=True) == 2
    assert torch.isfinite(out.float()).all() and torch.equal(out[1], good[1])
    st.table[0, 1] = -1
    tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    assert tg.tg_device_error(clear=True) == 2
    # a length above max_kv is cut there
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, max_kv=16)
    assert tg.tg_device_error(clear=True) == 2 and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_is_deterministic_and_replays(dtype):
    """The same bits twice, on another stream, beside another call, and from a
    captured graph whose lengths have grown since."""
    st = Setup([(1, 3000), (2, 100), (1, 17)], 8, 4, 128 if dtype == BF else 64, 16, dtype,
               seed=12).fill()
    st2 = Setup([(64, 700)], 8, 4, st.dh, 16, dtype, seed=13).fill()
    q, (gain, tau) = st.queries(), st.gates()
    q2 = st2.queries()
    ref = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    ref2 = tg.tg_paged_attn(st2.cache, q2, st2.cu, st2.kv_len, gain=gain, tau=tau)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(8):
        with torch.cuda.stream(sa):
            outs.append((ref, tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)))
        with torch.cuda.stream(sb):
            outs.append((ref2, tg.tg_paged_attn(st2.cache, q2, st2.cu, st2.kv_len, gain=gain,
                                                tau=tau)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(graph):
        tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    st.kv_len[1] -= 60  # other lengths, the same graph
    want = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not torch.equal(want, ref)


def test_pool_beyond_32_bits():
    """Pages whose element offsets pass 2^31."""
    hkv, dh, page, pool = 8, 128, 256, 8400
    k = torch.empty(pool, page, hkv, dh, dtype=BF, device="cuda")
    v = torch.empty(pool, page, hkv, dh, dtype=BF, device="cuda")
    assert (pool - 2) * page * hkv * dh > 2 ** 31
    g = gen(14)
    table = torch.tensor([[pool - 1, 3, pool - 2]], dtype=torch.int32, device="cuda")
    cache = tg.PagedKV(k, v, table)
    n = 600
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = torch.randn(n, 32, dh, generator=g, device="cuda").to(BF)
    q = tg.tg_paged_append(cache, x[:, 16:24], x[:, 24:], cu, ln, q=x[:, :16], rope_base=0.0)
    assert torch.equal(q, x[:, :16])
    assert torch.equal(k[pool - 1], x[:256, 16:24]) and torch.equal(v[pool - 2, :88], x[512:, 24:])
    st = Setup([(n, 0)], 16, hkv, dh, page, BF, bias=False)
    st.k, st.v, st.table, st.cache = k, v, table, cache
    check_attn(st, q.contiguous(), None, None)


# ------------------------------------------------------------------ append


def append_reference(x, w, pos, base, eps=1e-6):
    """(y, tolerance without the final rounding) in 64 bits; x [rows, heads, dh]."""
    dh = x.shape[-1]
    x = x.double()
    rel = 0.0
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
        rel = (dh + 8) * 2.0 ** -24
    if not base:
        return x, rel * x.abs()
    i = torch.arange(dh // 2, device="cuda", dtype=torch.float64)
    ang = pos.double()[:, None, None] * base ** (-2.0 * i / dh)
    lo, hi = x[..., :dh // 2], x[..., dh // 2:]
    y = torch.cat([lo * ang.cos() - hi * ang.sin(), hi * ang.cos() + lo * ang.sin()], -1)
    size = (lo.abs() + hi.abs()).repeat(1, 1, 2)
    return y, size * (rel + 2.0 ** -21)


@pytest.mark.parametrize("mode", ["norm", "plain", "knorm", "copy"])
@pytest.mark.parametrize("shape", [(16, 8, 128, 64, BF), (4, 2, 64, 16, BF), (3, 3, 128, 32, F32),
                                   (10, 2, 64, 256, F32), (7, 1, 128, 128, BF)],
                         ids=lambda s: f"{s[0]}-{s[1]}x{s[2]}-p{s[3]}-{str(s[4])[6:]}")
def test_append_parity(shape, mode):
    hq, hkv, dh, page, dt = shape
    lens = [(1, 0), (5, 130), (0, 9), (1, 63), (200, 0), (33, 250), (1, 64)]
    st = Setup(lens, hq, hkv, dh, page, dt, seed=20, stale=5.0)
    g, rows = st.g, st.rows
    fused = torch.randn(rows + 4, hq + 2 * hkv, dh, generator=g, device="cuda").to(dt)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    pos = torch.randint(0, 200000, (rows + 4,), generator=g, device="cuda").int()
    s = 3 * torch.randn(rows + 4, generator=g, device="cuda")
    s[0], s[1], s[2] = math.inf, -math.inf, -200.0
    w = 1 + 0.1 * torch.randn(2, dh, generator=g, device="cuda")
    kw = dict(norm=dict(q_norm=w[0], k_norm=w[1]), plain={}, knorm=dict(k_norm=w[1]),
              copy=dict(rope_base=0.0))[mode]
    base = kw.get("rope_base", 1e6)
    q_out = torch.full((rows + 4, hq, dh), 5.0, dtype=dt, device="cuda")
    tg.tg_paged_append(st.cache, k, v, st.cu, st.kv_len, q=q, pos=pos, s=s, q_out=q_out, **kw)
    u = U[dt]
    touched = torch.zeros(st.k.shape[:2], dtype=torch.bool, device="cuda")
    yq, tq = append_reference(q[:rows], kw.get("q_norm"), pos[:rows], base)
    yk, tk = append_reference(k[:rows], kw.get("k_norm"), pos[:rows], base)
    assert ((q_out[:rows].double() - yq).abs() <= u * yq.abs() + tq * 1.01).all()
    assert (q_out[rows:] == 5).all()
    for b, (n, p) in enumerate(lens):
        if n == 0:
            continue
        pg, r = st.where(b, p, p + n)
        touched[pg, r] = True
        sl = slice(st.cu_host[b], st.cu_host[b] + n)
        assert ((st.k[pg, r].double() - yk[sl]).abs() <= u * yk[sl].abs() + tk[sl] * 1.01).all()
        assert torch.equal(st.v[pg, r], v[sl])
        want = torch.where(torch.isneginf(s[sl]), -math.inf,
                           -torch.logaddexp(torch.zeros_like(s[sl].double()), -s[sl].double()))
        got = st.bias[pg, r].double()
        near = (got - want).abs() <= 2.0 ** -21 * want.abs() + 2.0 ** -24
        assert (near | (got == want)).all()
    for t in (st.k, st.v, st.bias):
        assert (t[~touched] == 5).all()  # nothing else is written


def test_append_default_positions_in_place_and_without_queries():
    st = Setup([(3, 70), (2, 0)], 4, 2, 64, 16, BF, seed=21, stale=5.0)
    x = torch.randn(5, 8, 64, generator=st.g, device="cuda").to(BF)
    q = x[:, :4].contiguous()
    pos = torch.tensor([70, 71, 72, 0, 1], dtype=torch.int32, device="cuda")
    want = tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len, q=q, pos=pos)
    k1 = st.k.clone()
    assert (st.bias[st.table[0, 4], 6:9] == 0).all()  # no scores: generated rows, bias 0
    got = tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len, q=q, q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(st.k, k1)
    st.k.fill_(5.0)
    assert tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len) is None
    assert torch.equal(st.k, k1)


def test_append_skips_and_reports_rows_out_of_range():
    st = Setup([(2, 14), (2, -1), (1, 3)], 4, 2, 64, 16, BF, seed=22, stale=5.0)
    x = torch.randn(5, 8, 64, generator=st.g, device="cuda").to(BF)
    a = (x[:, 4:6], x[:, 6:], st.cu, st.kv_len)
    tg.tg_paged_append(st.cache, *a, rope_base=0.0)  # request 1: row -1, skipped
    assert tg.tg_device_error(clear=True) == 2
    assert torch.equal(st.k[st.table[1, 0].long(), 0], x[3, 4:6])
    before = st.k.clone()
    st.table[0, 0] = 99
    st.kv_len[2] = 10 ** 6  # behind the table
    tg.tg_paged_append(st.cache, *a, rope_base=0.0)
    assert tg.tg_device_error(clear=True) == 2 and torch.equal(st.k, before)


def test_append_graph_replay():
    st = Setup([(1, 20), (1, 5)], 4, 2, 64, 16, BF, seed=23, stale=5.0)
    x = torch.randn(2, 8, 64, generator=st.g, device="cuda").to(BF)
    q_out = torch.empty(2, 4, 64, dtype=BF, device="cuda")
    call = lambda: tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len, q=x[:, :4],  # noqa: E731
                                      q_out=q_out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    st.kv_len += 1
    graph.replay()
    got_k, got_q = st.k.clone(), q_out.clone()
    call()
    assert torch.equal(st.k, got_k) and torch.equal(q_out, got_q)
    assert torch.equal(st.v[st.table[0, 1].long(), 5], x[0, 6:])


def test_no_rows_and_no_requests():
    st = Setup([(0, 5), (0, 0)], 4, 2, 64, 16, BF, seed=24, stale=5.0)
    x = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    assert tg.tg_paged_attn(st.cache, x, st.cu, st.kv_len).shape == (0, 4, 64)
    assert tg.tg_paged_append(st.cache, x[:, :2], x[:, :2], st.cu, st.kv_len, q=x).shape == (0, 4, 64)
    # rows that belong to no request
    y = torch.full((3, 4, 64), 5.0, dtype=BF, device="cuda")
    out = torch.full_like(y, 9.0)
    tg.tg_paged_attn(st.cache, y, st.cu, st.kv_len, out=out)
    tg.tg_paged_append(st.cache, y[:, :2], y[:, 2:], st.cu, st.kv_len, q=y, q_out=out)
    assert (out == 9).all() and (st.k == 5).all()
