"""GPU tests of the serving calls together, and of the paged attention's
variants at the calls that its parity tests do not make: other streams, shared
pages, values and logits that are not finite, growing maxima.

Tolerances are those derived in test_gpu_paged.py and test_gpu_quantized.py.
"""

import math

import pytest
import torch

from tests.test_gpu_paged import BF, F32, Setup, attn_reference, check_attn, gen
from tests.test_gpu_quantized import check_linear

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")


@pytest.fixture(autouse=True)
def _no_device_errors():
    tg.tg_device_error(clear=True)
    yield
    assert tg.tg_device_error() == 0


# one of each variant: single rows over a short cache (a cluster merges) and a
# long one (a second kernel merges), drafts (both softmax groups on the same
# rows), chunks (256-row tiles), fp32
VARIANTS = {
    "cluster": ([(1, 300), (1, 900)], 8, 4, 128, 32, BF),
    "split": ([(1, 5000), (2, 2500), (1, 10)], 8, 4, 64, 64, BF),
    "draft": ([(6, 1500), (9, 40), (1, 700)], 16, 2, 64, 16, BF),
    "draft128": ([(5, 900), (12, 3000)], 16, 2, 128, 128, BF),
    "chunk": ([(200, 500), (150, 0)], 8, 2, 128, 64, BF),
    "fp32": ([(20, 300), (1, 90)], 4, 2, 64, 32, F32),
}


@pytest.fixture(params=list(VARIANTS))
def variant(request):
    lens, hq, hkv, dh, page, dt = VARIANTS[request.param]
    return Setup(lens, hq, hkv, dh, page, dt, seed=40).fill()


def test_variants(variant):
    st = variant
    check_attn(st, st.queries(extra=2), *st.gates())
    check_attn(st, st.queries(), None, None)


def test_values_of_removed_keys_never_reach_a_row(variant):
    """NaN values under biases of -inf: heads with a gain are finite, the head
    of gain 0 sees the key and is not."""
    st = variant
    gain, tau = st.gates()
    gain[1] = 0.0
    for b, (n, p) in enumerate(st.lens):
        pg, r = st.where(b, 0, n + p)
        for j in range(0, n + p, 7):
            st.bias[pg[j], r[j]] = -math.inf
            st.v[pg[j], r[j], :, j % st.dh] = math.nan if j % 2 else math.inf
    out = check_attn(st, st.queries(), gain, tau)
    grp = st.hq // st.hkv
    assert torch.isfinite(out[:, [h for h in range(st.hq) if h != 1]].float()).all()
    assert grp >= 1 and not torch.isfinite(out[-1, 1].float()).all()


def test_logits_that_are_not_finite_show(variant):
    """A NaN in a query or in a key that a row sees makes its outputs NaN (or
    infinite), and no other row's."""
    st = variant
    q, (gain, tau) = st.queries(), st.gates()
    good = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    q2 = q.clone()
    q2[0, 2, 5] = math.nan
    out = tg.tg_paged_attn(st.cache, q2, st.cu, st.kv_len, gain=gain, tau=tau)
    hit = torch.zeros(st.rows, st.hq, dtype=torch.bool, device="cuda")
    hit[0, 2] = True
    assert torch.equal(~torch.isfinite(out.float()).all(-1), hit)
    assert torch.equal(out[~hit], good[~hit])
    for j in (0, 3, 14):  # a key of the second request: every row of its group there
        st.k[st.table[1, 0].long(), j, 0, 1] = math.nan
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    bad = ~torch.isfinite(out.float()).all(-1)
    lo, hi = st.cu_host[1], st.cu_host[2]
    grp = st.hq // st.hkv
    sees = bad[lo:hi, :grp]
    assert sees[-1].all() and not bad[:lo].any() and not bad[hi:].any() and not bad[:, grp:].any()


def test_growing_maxima(variant):
    """Keys that grow along the cache: the running maximum moves again and
    again, within a tile and from tile to tile."""
    st = variant
    for b, (n, p) in enumerate(st.lens):
        pg, r = st.where(b, 0, n + p)
        ramp = torch.linspace(0.01, 6.0, n + p, device="cuda")[:, None, None]
        st.k[pg, r] = (st.k[pg, r].float().abs() * ramp).to(st.dtype)
    q = st.queries().abs()
    check_attn(st, q, None, None)
    check_attn(st, q, *st.gates())


def test_shared_prefix_pages():
    """Two requests whose tables begin with the same pages."""
    st = Setup([(1, 127), (3, 200), (70, 128)], 8, 2, 64, 64, BF, seed=41).fill()
    st.table[1, :2] = st.table[0, :2]
    st.table[2, :2] = st.table[0, :2]
    check_attn(st, st.queries(), *st.gates())


def test_pages_out_of_range_count_as_zero_keys():
    """Chunks, too: the keys and values of a page that does not exist are
    zeros, with bias 0."""
    for lens, dt in (([(90, 200)], BF), ([(1, 290)], BF), ([(30, 200)], F32)):
        st = Setup(lens, 8, 2, 64, 16, dt, seed=42).fill()
        q, (gain, tau) = st.queries(), st.gates()
        real = int(st.table[0, 4])
        st.k[real], st.v[real], st.bias[real] = 0, 0, 0
        want = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
        st.table[0, 4] = 1 << 30
        got = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
        assert tg.tg_device_error(clear=True) == 2
        assert torch.equal(got, want)


def test_calls_on_a_given_stream():
    """`stream=` with results and workspace allocated by the call: the memory is
    not handed out again while the other stream works."""
    st = Setup([(1, 4000), (1, 2000)], 16, 8, 128, 64, BF, seed=43).fill()
    q, (gain, tau) = st.queries(), st.gates()
    want = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
    x = torch.randn(64, 2048, generator=st.g, device="cuda").to(BF)
    wq, ws = tg.tg_quantize_rows(torch.randn(512, 2048, generator=st.g, device="cuda"))
    xq0, xs0 = tg.tg_quantize_rows(x)
    y0 = tg.tg_linear_quantized(xq0, xs0, wq, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(20):
        out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, stream=side)
        xq, xs = tg.tg_quantize_rows(x, stream=side)
        y = tg.tg_linear_quantized(xq, xs, wq, ws, stream=side)
        outs.append((out, xq, y))
        torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda")  # on the current stream
    torch.cuda.synchronize()
    for out, xq, y in outs:
        assert torch.equal(out, want) and torch.equal(xq, xq0) and torch.equal(y, y0)


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn."""
    a = Setup([(1, 3000)], 16, 8, 128, 64, BF, seed=44).fill()
    b = Setup([(70, 600)], 16, 8, 128, 64, BF, seed=45).fill()
    qa, qb = a.queries(), b.queries()
    need = max(tg.tg_workspace_size(tg.TG_OP_PAGED_ATTN, n=1, k=s.rows, n_heads_q=16, n_heads_kv=8,
                                    head_dim=128) for s in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    wa = tg.tg_paged_attn(a.cache, qa, a.cu, a.kv_len)
    wb = tg.tg_paged_attn(b.cache, qb, b.cu, b.kv_len)
    oa, ob = torch.empty_like(qa), torch.empty_like(qb)
    graphs = []
    for s, q, o in ((a, qa, oa), (b, qb, ob)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tg.tg_paged_attn(s.cache, q, s.cu, s.kv_len, out=o, ws=ws)
        graphs.append(g)
    for _ in range(3):
        ws.fill_(255)  # nothing is carried from call to call
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


@pytest.mark.parametrize("dtype,residual", [(BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("m,n,k", [(5000, 1056, 1008), (4097, 1312, 144), (130, 12288, 272),
                                   (60, 2080, 6144), (6, 32, 131056)])
def test_linear_tails(m, n, k, dtype, residual):
    """Rows, columns and k that end inside a tile, in each of the kernels."""
    check_linear(m, n, k, dtype, residual, seed=m + n, lo=-128)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(100, 160, 512), (300, 1024, 400), (70, 256, 1040), (520, 2048, 3600),
                                   (700, 2048, 64), (6622, 928, 48), (4096, 96, 640)])
def test_linear_plans(m, n, k, dtype):
    """Each number of parts of k, wide tiles below and above a wave, with the
    residual that the product overwrites."""
    check_linear(m, n, k, dtype, True, seed=m, lo=-128)
    g = gen(m)
    xq, xs = tg.tg_quantize_rows(torch.randn(m, k, generator=g, device="cuda"))
    wq, ws = tg.tg_quantize_rows(torch.randn(n, k, generator=g, device="cuda"))
    r = torch.randn(m, n, generator=g, device="cuda").to(dtype)
    want = tg.tg_linear_quantized(xq, xs, wq, ws, residual=r, dtype=dtype)
    y = r.clone()
    tg.tg_linear_quantized(xq, xs, wq, ws, residual=y, y=y, dtype=dtype)
    assert torch.equal(y, want)


def test_linear_on_the_first_rows_of_a_buffer():
    """y is a part of a larger buffer: nothing behind it is written."""
    g = gen(46)
    for m, n in ((3, 96), (50, 352), (3000, 1312)):
        xq, xs = tg.tg_quantize_rows(torch.randn(m, 256, generator=g, device="cuda"))
        wq, ws = tg.tg_quantize_rows(torch.randn(n, 256, generator=g, device="cuda"))
        buf = torch.full((m + 2, n), 5.0, dtype=BF, device="cuda")
        tg.tg_linear_quantized(xq, xs, wq, ws, y=buf[1:m + 1])
        assert (buf[0] == 5).all() and (buf[m + 1] == 5).all()
        assert torch.equal(buf[1:m + 1], tg.tg_linear_quantized(xq, xs, wq, ws))


def test_unaligned_scales_are_refused_or_read():
    g = gen(47)
    xq, xs = tg.tg_quantize_rows(torch.randn(40, 256, generator=g, device="cuda"))
    wq, ws = tg.tg_quantize_rows(torch.randn(64, 256, generator=g, device="cuda"))
    want = tg.tg_linear_quantized(xq, xs, wq, ws)
    off = torch.empty(65, device="cuda")[1:]
    off.copy_(ws)
    with pytest.raises(tg.TokenGateError):
        tg.tg_linear_quantized(xq, xs, wq, off)
    xoff = torch.empty(41, device="cuda")[1:]
    xoff.copy_(xs)
    assert torch.equal(tg.tg_linear_quantized(xq, xoff, wq, ws), want)
    # norm weights, gains and temperatures may sit anywhere
    st = Setup([(3, 20)], 4, 2, 64, 16, BF, seed=48, stale=1.0)
    x = torch.randn(3, 8, 64, generator=st.g, device="cuda").to(BF)
    w = 1 + 0.1 * torch.randn(65, generator=st.g, device="cuda")
    a = tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len, q=x[:, :4],
                           q_norm=w[1:], k_norm=w[1:])
    b = tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len, q=x[:, :4],
                           q_norm=w[1:].clone(), k_norm=w[1:].clone())
    assert torch.equal(a, b)


@pytest.mark.parametrize("most,dtype", [(1, BF), (6, BF), (40, BF), (1, F32), (40, F32)])
def test_thousands_of_requests(most, dtype):
    """Requests found among thousands, empty ones between them, by the append
    and by each of the attention's row tiles."""
    r = torch.Generator().manual_seed(most)
    n = torch.randint(0, most + 1, (2500,), generator=r)
    p = torch.randint(0, 40, (2500,), generator=r)
    n[100:170], n[-1] = 0, most
    st = Setup(list(zip(n.tolist(), p.tolist())), 4, 2, 64, 16, dtype, seed=53, stale=5.0)
    x = torch.randn(st.rows, 8, 64, generator=st.g, device="cuda").to(dtype)
    st.fill()
    before = st.k.clone()
    q = tg.tg_paged_append(st.cache, x[:, 4:6], x[:, 6:], st.cu, st.kv_len, q=x[:, :4], rope_base=0.0)
    owner = torch.repeat_interleave(torch.arange(2500), n).cuda()
    row = torch.arange(st.rows, device="cuda") - st.cu[owner].long() + p.cuda()[owner]
    pg, at = st.table[owner, row // 16].long(), row % 16
    assert torch.equal(st.k[pg, at], x[:, 4:6]) and torch.equal(st.v[pg, at], x[:, 6:])
    untouched = torch.ones(st.k.shape[:2], dtype=torch.bool, device="cuda")
    untouched[pg, at] = False
    assert torch.equal(st.k[untouched], before[untouched])
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len)
    # the same requests a few at a time
    for b0 in (0, 90, 1203, 2490):
        sub = tg.PagedKV(st.k, st.v, st.table[b0:b0 + 10].contiguous(), st.bias)
        lo, hi = st.cu_host[b0], st.cu_host[b0 + 10]
        cu = (st.cu[b0:b0 + 11] - lo).contiguous()
        part = tg.tg_paged_attn(sub, q[lo:hi], cu, st.kv_len[b0:b0 + 10].contiguous())
        # The weights and the output are rounded once in either call, each by at
        # most 2^-8 of the largest value; in fp32 the logits' sums of 64 products are
        # what differs, and each moves a weight and the sum that divides it.
        logit = 64 * float(q.abs().max()) * float(st.k.abs().max()) / 8
        unit = 2.0 ** -8 if dtype == BF else 64 * 2.0 ** -24 * logit
        tol = 4 * unit * float(st.v.abs().max())
        assert ((part.float() - out[lo:hi].float()).abs() <= tol).all()


def test_append_many_requests_and_heads():
    """More requests than a warp counts at once, more heads than a pass holds,
    more tokens than the blocks' first groups."""
    lens = [(i % 5, 3 * i % 70) for i in range(400)]
    st = Setup(lens, 40, 8, 128, 16, BF, seed=49, stale=5.0)
    x = torch.randn(st.rows, 56, 128, generator=st.g, device="cuda").to(BF)
    s = torch.randn(st.rows, generator=st.g, device="cuda")
    q = tg.tg_paged_append(st.cache, x[:, 40:48], x[:, 48:], st.cu, st.kv_len, q=x[:, :40], s=s,
                           rope_base=0.0)
    assert torch.equal(q, x[:, :40])
    touched = torch.zeros(st.k.shape[:2], dtype=torch.bool, device="cuda")
    for b, (n, p) in enumerate(lens):
        if n == 0:
            continue
        pg, r = st.where(b, p, p + n)
        touched[pg, r] = True
        sl = slice(st.cu_host[b], st.cu_host[b] + n)
        assert torch.equal(st.k[pg, r], x[sl, 40:48]) and torch.equal(st.v[pg, r], x[sl, 48:])
        assert torch.allclose(st.bias[pg, r], torch.nn.functional.logsigmoid(s[sl]), atol=1e-6)
    assert (st.k[~touched] == 5).all() and (st.v[~touched] == 5).all()


def test_serving_a_layer():
    """A layer's serving loop as a program runs it: 8-bit QKV projection, append,
    attention, 8-bit output projection onto the residual stream; three requests
    prefilled in chunks of different sizes, then decoded together (the decoding
    step from a captured graph). The cache is that of one call over the whole
    sequences, bit for bit, and every attention output is within its tolerance
    of the 64-bit result over that cache."""
    d, hq, hkv, dh, page = 512, 8, 4, 64, 16
    g = gen(50)
    total = [150, 93, 40]  # rows of each request in the end
    plan = [[(70, 31, 5), (60, 60, 20), (18, 0, 13)], [(1, 1, 1)] * 2]
    width = (hq + 2 * hkv) * dh
    wqkv, sqkv = tg.tg_quantize_rows(torch.randn(width, d, generator=g, device="cuda") * 0.05)
    wo, so = tg.tg_quantize_rows(torch.randn(d, hq * dh, generator=g, device="cuda") * 0.05)
    xs = [torch.randn(t, d, generator=g, device="cuda").to(BF) for t in total]
    scores = [torch.randn(t, generator=g, device="cuda") for t in total]
    norm = 1 + 0.1 * torch.randn(2, dh, generator=g, device="cuda")
    gain = torch.rand(hq, generator=g, device="cuda")
    tau = 0.5 + torch.rand(hq, generator=g, device="cuda")

    def project(x):
        xq, sc = tg.tg_quantize_rows(x)
        return tg.tg_linear_quantized(xq, sc, wqkv, sqkv).view(-1, hq + 2 * hkv, dh)

    def step(st, x, s):
        h = project(x)
        q = tg.tg_paged_append(st.cache, h[:, hq:hq + hkv], h[:, hq + hkv:], st.cu, st.kv_len,
                               q=h[:, :hq], s=s, q_norm=norm[0], k_norm=norm[1])
        o = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau)
        oq, sc = tg.tg_quantize_rows(o.view(-1, hq * dh))
        return q, o, tg.tg_linear_quantized(oq, sc, wo, so, residual=x)

    # the whole sequences at once
    ref = Setup([(t, 0) for t in total], hq, hkv, dh, page, BF, seed=51)
    q_all, o_all, _ = step(ref, torch.cat(xs), torch.cat(scores))
    want, _, tol, _ = attn_reference(ref, q_all, gain, tau)
    assert ((o_all.double() - want).abs() <= tol).all()

    live = Setup([(t, 0) for t in total], hq, hkv, dh, page, BF, seed=52)
    done = [0, 0, 0]

    def spans(ns):
        live.lens = list(zip(ns, done))
        cu = [0]
        for n in ns:
            cu.append(cu[-1] + n)
        live.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        live.kv_len.copy_(torch.tensor([n + p for n, p in live.lens], dtype=torch.int32))
        return (torch.cat([xs[b][done[b]:done[b] + n] for b, n in enumerate(ns)]),
                torch.cat([scores[b][done[b]:done[b] + n] for b, n in enumerate(ns)]))

    def x_of(ns):  # (after `done` has moved)
        return torch.cat([xs[b][done[b] - n:done[b]] for b, n in enumerate(ns)])

    def compare(ns, q, o, y):
        at = 0
        for b, n in enumerate(ns):
            sl = slice(ref.cu_host[b] + done[b], ref.cu_host[b] + done[b] + n)
            assert torch.equal(q[at:at + n], q_all[sl])
            assert ((o[at:at + n].double() - want[sl]).abs() <= tol[sl]).all()
            at += n
            done[b] += n
        # the block's output is what its two calls give for these rows
        oq, sc = tg.tg_quantize_rows(o.view(-1, hq * dh))
        assert torch.equal(y, tg.tg_linear_quantized(oq, sc, wo, so, residual=x_of(ns)))

    for ns in plan[0]:
        x, s = spans(ns)
        compare(ns, *step(live, x, s))
    x, s = spans(plan[1][0])
    xb, sb = x.clone(), s.clone()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step(live, xb, sb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(live, xb, sb)
    for ns in plan[1]:
        x, s = spans(ns)
        xb.copy_(x)
        sb.copy_(s)
        graph.replay()
        compare(ns, *res)
    assert done == [150, 93, 40]
    for b, t in enumerate(total):
        pr, rr = ref.where(b, 0, t)
        pl, rl = live.where(b, 0, t)
        assert torch.equal(ref.k[pr, rr], live.k[pl, rl])
        assert torch.equal(ref.v[pr, rr], live.v[pl, rl])
        assert torch.equal(ref.bias[pr, rr], live.bias[pl, rl])
