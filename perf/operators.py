"""Cases, plain forms and exact values of the operators that serve a pruned,
paged key/value cache:

    append    tg_paged_append        per-head norm of q and k, position rotation,
                                     keys / values / gate biases into pages
    attn      tg_paged_attn          token-gated attention of chunks of new tokens
                                     over the paged cache
    quant     tg_quantize_rows       8-bit integers with one scale per row
    linear    tg_linear_quantized    the projection product on 8-bit integers

With `own` false, `run` computes an operator from elementary torch operations;
with `own` true it makes the library's call. Sizes are those of this
repository's workloads: 16 query and 8 KV heads of 128 (the 28-layer prefill),
4 and 2 heads of 64 (the fp32 block), widths 2048 / 4096 / 6144 / 12288,
prompts of up to 32768 tokens of which 2048 to 8192 are kept.
"""

import math
import random

import torch

own = False

ROPE_BASE = 1e6
EPS = 1e-6


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one new token for each of 64 running requests, ragged histories:
        # the append of every layer of every decoding step (latency)
        dict(name="append_decode_64", op="append", dtype="bf16", batch=64, n_lo=1, n_hi=1,
             past_lo=100, past_hi=8192, hq=16, hkv=8, dh=128, page=64, norm=True, bias=True,
             lens=1),
        # one whole prompt going into an empty cache, keys and queries normed
        # and rotated on the way (bandwidth)
        dict(name="append_prompt_32k", op="append", dtype="bf16", batch=1, n_lo=32768, n_hi=32768,
             past_lo=0, past_hi=0, hq=16, hkv=8, dh=128, page=128, norm=True, bias=True, lens=2),
        # one generated token over the 4096 kept tokens of a pruned prompt,
        # gate bias on: the decoding step of a layer above the gate (latency)
        dict(name="attn_decode_1", op="attn", dtype="bf16", batch=1, n_lo=1, n_hi=1, past_lo=4096,
             past_hi=4096, hq=16, hkv=8, dh=128, page=64, bias=True, lens=3),
        # a batch of 64 decoding requests with full caches of very different
        # lengths: the layers below the gate (cache bandwidth)
        dict(name="attn_decode_64", op="attn", dtype="bf16", batch=64, n_lo=1, n_hi=1,
             past_lo=500, past_hi=32767, hq=16, hkv=8, dh=128, page=64, bias=False, lens=4),
        # drafted continuations of 2 to 9 tokens of 8 requests, heads of 64,
        # small pages, eight query heads to a KV head
        dict(name="attn_draft_8", op="attn", dtype="bf16", batch=8, n_lo=2, n_hi=9, past_lo=1000,
             past_hi=9000, hq=16, hkv=2, dh=64, page=16, bias=True, lens=5),
        # the last 2048 tokens of a prompt prefilled in chunks, after 30720
        # tokens that are in the cache (tensor-core rate)
        dict(name="attn_chunk_2k", op="attn", dtype="bf16", batch=1, n_lo=2048, n_hi=2048,
             past_lo=30720, past_hi=30720, hq=16, hkv=8, dh=128, page=128, bias=True, lens=6),
        # the fp32 block: ragged chunks over short caches, full precision
        dict(name="attn_fp32", op="attn", dtype="fp32", batch=3, n_lo=17, n_hi=130, past_lo=0,
             past_hi=400, hq=4, hkv=2, dh=64, page=32, bias=True, lens=7),
        # the activation row of one decoded token (latency)
        dict(name="quant_1", op="quant", dtype="bf16", rows=1, cols=2048),
        # the SwiGLU activations of a whole prompt (bandwidth)
        dict(name="quant_32k", op="quant", dtype="bf16", rows=32768, cols=6144),
        # the fused QKV projection of one decoded token (weight bandwidth)
        dict(name="linear_1", op="linear", dtype="bf16", m=1, n=4096, k=2048, residual=False),
        # the down projection of a decoding batch, onto the residual stream
        dict(name="linear_100", op="linear", dtype="bf16", m=100, n=2048, k=6144, residual=True),
        # the gate/up projection of a chunk of 8192 rows (tensor-core rate)
        dict(name="linear_8k", op="linear", dtype="bf16", m=8192, n=12288, k=2048,
             residual=False),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def _heads(rng, dtype):
    dh = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8] if dtype == "bf16" else [1, 2, 3])
    return min(hkv * group, 40) // hkv * hkv, hkv, dh


def _draw_once(rng):
    op = rng.choice(["append", "attn", "attn", "quant", "linear", "linear"])
    if op == "quant":
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), rows=_log_int(rng, 1, 32768),
                    cols=16 * _log_int(rng, 4, 768))
    if op == "linear":
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), m=_log_int(rng, 1, 32768),
                    n=32 * _log_int(rng, 2, 384), k=16 * _log_int(rng, 4, 384),
                    residual=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    hq, hkv, dh = _heads(rng, dtype)
    batch = _log_int(rng, 1, 64)
    if dtype == "fp32":  # the full-precision block is a small one
        n_hi, past_hi, batch = _log_int(rng, 1, 256), _log_int(rng, 1, 1024), min(batch, 8)
    else:
        n_hi = _log_int(rng, 1, 8192 if op == "append" else 2048)
        past_hi = _log_int(rng, 1, 32768)
    n_lo = n_hi if rng.random() < 0.3 else _log_int(rng, 1, n_hi)
    past_lo = 0 if rng.random() < 0.2 else _log_int(rng, 1, past_hi)
    c = dict(op=op, dtype=dtype, batch=batch, n_lo=n_lo, n_hi=n_hi, past_lo=past_lo,
             past_hi=past_hi, hq=hq, hkv=hkv, dh=dh, page=rng.choice([16, 32, 64, 128, 256]),
             bias=rng.random() < 0.6, lens=rng.randrange(1 << 30))
    if op == "append":
        c["norm"] = rng.random() < 0.7
    return c


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        t = tops.setdefault(c["op"], [0, 0])
        tops[c["op"]] = [max(t[0], w["bytes"]), max(t[1], w["flops"])]
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= tops[c["op"]][0] and w["flops"] <= tops[c["op"]][1]:
            return c


def _lens(case):
    """(new rows, cached rows before them) of each request of the case."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["batch"]):
        n = r.randint(case["n_lo"], case["n_hi"])
        past = r.randint(case["past_lo"], case["past_hi"])
        out.append((n, past))
    return out


def _elem(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e = _elem(case)
    if case["op"] == "quant":  # a maximum, a product and a rounding per element
        return dict(bytes=case["rows"] * (case["cols"] * (e + 1) + 4),
                    flops=3 * case["rows"] * case["cols"])
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(bytes=m * k + n * k + 4 * (m + n) + m * n * e * (2 if case["residual"] else 1),
                    flops=2 * m * n * k)
    hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
    lens = _lens(case)
    rows = sum(n for n, _ in lens)
    if case["op"] == "append":  # rows in, rows out; about ten operations an element
        b = rows * ((hq + 2 * hkv) * dh * 2 * e + 4 + (8 if case["bias"] else 0))
        return dict(bytes=b, flops=10 * rows * (hq + hkv) * dh)
    keys = sum(n + p for n, p in lens)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in lens)
    b = 2 * rows * hq * dh * e + keys * (2 * hkv * dh * e + (4 if case["bias"] else 0))
    return dict(bytes=b, flops=4 * pairs * hq * dh)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62) + 17)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _paged_inputs(case, seed):
    """A page pool whose pages are dealt to the requests in random order, with
    the cached rows filled in and what earlier requests left (for the attention
    NaN: memory that nothing wrote) behind them; the chunk's projections; the
    gate scores."""
    g = _gen(seed)
    dt, dev = _dtype(case), "cuda"
    hq, hkv, dh, page = case["hq"], case["hkv"], case["dh"], case["page"]
    lens = _lens(case)
    n_of = [(n + p + page - 1) // page for n, p in lens]
    used = sum(n_of)
    pool = used + 3
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(n_of)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(n_of):
        table[b, :c] = perm[at:at + c]
        at += c
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    rows = cu[-1]
    kv_len = torch.tensor([n + p for n, p in lens], dtype=torch.int32, device=dev)
    left = float("nan") if case["op"] == "attn" else 7.0
    k_pages = torch.full((pool, page, hkv, dh), left, dtype=dt, device=dev)
    v_pages = torch.full((pool, page, hkv, dh), left, dtype=dt, device=dev)
    bias = torch.full((pool, page), left, device=dev) if case["bias"] else None
    fill = [p + (n if case["op"] == "attn" else 0) for n, p in lens]
    for b, t in enumerate(fill):
        if t == 0:
            continue
        at_page, at_row = _slots(table, b, 0, t, page)
        k_pages[at_page, at_row] = torch.randn(t, hkv, dh, generator=g, device=dev).to(dt)
        v_pages[at_page, at_row] = torch.randn(t, hkv, dh, generator=g, device=dev).to(dt)
        if bias is not None:  # kept tokens' scores; the last eighth was generated: no bias
            lsig = _logsigmoid(2.0 * torch.randn(t, generator=g, device=dev) + 1.0)
            lsig[t - t // 8:] = 0.0
            bias[at_page, at_row] = lsig
    st = dict(case=case, lens=lens, table=table, kv_len=kv_len, k_pages=k_pages, v_pages=v_pages,
              bias=bias, cu=torch.tensor(cu, dtype=torch.int32, device=dev), cu_host=cu,
              max_kv=max(n + p for n, p in lens))
    if case["op"] == "append":
        # the fused projection's rows, [q | k | v], 1% of the tokens four times as large
        qkv = torch.randn(rows, (hq + 2 * hkv) * dh, generator=g, device=dev)
        qkv *= 1.0 + 3.0 * (torch.rand(rows, 1, generator=g, device=dev) < 0.01).float()
        st["qkv"] = qkv.to(dt)
        # original positions of kept tokens: ascending with gaps
        gaps = torch.randint(1, 9, (rows,), generator=g, device=dev)
        st["pos"] = torch.cat([torch.cumsum(gaps[cu[b]:cu[b + 1]], 0) - 1 + 8 * lens[b][1]
                               for b in range(len(lens))]).to(torch.int32)
        st["s"] = 2.0 * torch.randn(rows, generator=g, device=dev) if case["bias"] else None
        st["q_norm"] = st["k_norm"] = None
        if case["norm"]:
            st["q_norm"] = 1.0 + 0.1 * torch.randn(dh, generator=g, device=dev)
            st["k_norm"] = 1.0 + 0.1 * torch.randn(dh, generator=g, device=dev)
    else:
        st["q"] = torch.randn(rows, hq, dh, generator=g, device=dev).to(dt)
        st["gain"] = 2.0 * torch.rand(hq, generator=g, device=dev) if case["bias"] else None
        st["tau"] = 0.5 + torch.rand(hq, generator=g, device=dev)
    return st


def _quantized(x):
    """8-bit rows of x, for the product's inputs."""
    amax = x.abs().amax(dim=1, keepdim=True).clamp_min(1e-20)
    return torch.round(x * (127.0 / amax)).clamp(-127, 127).to(torch.int8), (amax / 127.0)[:, 0]


def prepare(case, seed):
    if case["op"] in ("append", "attn"):
        st = _paged_inputs(case, seed)
        if own:
            import learned_token_pruning_score_b200 as tg

            st["cache"] = tg.PagedKV(st["k_pages"], st["v_pages"], st["table"], st["bias"])
        return st
    g = _gen(seed)
    if case["op"] == "quant":
        x = torch.randn(case["rows"], case["cols"], generator=g, device="cuda")
        x *= 1.0 + 3.0 * (torch.rand(case["rows"], 1, generator=g, device="cuda") < 0.01).float()
        return dict(case=case, x=x.to(_dtype(case)))
    m, n, k = case["m"], case["n"], case["k"]
    xq, xs = _quantized(torch.randn(m, k, generator=g, device="cuda"))
    wq, ws = _quantized(0.02 * torch.randn(n, k, generator=g, device="cuda"))
    res = None
    if case["residual"]:
        res = torch.randn(m, n, generator=g, device="cuda").to(_dtype(case))
    return dict(case=case, xq=xq, xs=xs, wq=wq, ws=ws, residual=res)


# ------------------------------------------------------------------ plain forms


def _logsigmoid(s):
    return torch.minimum(s, torch.zeros_like(s)) - torch.log1p(torch.exp(-s.abs()))


def _slots(table, b, lo, hi, page):
    """(page, row in the page) of rows lo .. hi - 1 of request b."""
    r = torch.arange(lo, hi, device=table.device)
    return table[b, r // page].long(), r % page


def _norm_rotate(x, w, pos):
    """Per-head RMSNorm (when w is given) and rotate-half rotation of x
    [rows, heads, dh]; the angles in 64 bits."""
    dh = x.shape[-1]
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    i = torch.arange(dh // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None] * torch.exp(-(2.0 * i / dh) * math.log(ROPE_BASE))[None]
    cos, sin = torch.cos(ang).to(x.dtype)[:, None], torch.sin(ang).to(x.dtype)[:, None]
    lo, hi = x[..., :dh // 2], x[..., dh // 2:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def _append_plain(st):
    c = st["case"]
    hq, hkv, dh, page = c["hq"], c["hkv"], c["dh"], c["page"]
    dt = _dtype(c)
    rows = st["qkv"].shape[0]
    x = st["qkv"].float().view(rows, hq + 2 * hkv, dh)
    q = _norm_rotate(x[:, :hq], st["q_norm"], st["pos"]).to(dt)
    k = _norm_rotate(x[:, hq:hq + hkv], st["k_norm"], st["pos"]).to(dt)
    v = st["qkv"].view(rows, hq + 2 * hkv, dh)[:, hq + hkv:]
    lens, cu = st["lens"], st["cu_host"]
    at = [_slots(st["table"], b, p, p + n, page) for b, (n, p) in enumerate(lens)]
    at_page, at_row = torch.cat([a[0] for a in at]), torch.cat([a[1] for a in at])
    st["k_pages"][at_page, at_row] = k
    st["v_pages"][at_page, at_row] = v
    if st["bias"] is not None:
        st["bias"][at_page, at_row] = _logsigmoid(st["s"])
    return _append_outputs(st, q)


def _append_outputs(st, q):
    out = dict(q=q, k_pages=st["k_pages"], v_pages=st["v_pages"])
    if st["bias"] is not None:
        out["bias"] = st["bias"]
    return out


def _attend(st, wide, rows_at_once):
    """out [rows, hq, dh], by request, KV head and block of query rows, with
    the arithmetic in the type `wide`."""
    c = st["case"]
    hq, hkv, dh, page = c["hq"], c["hkv"], c["dh"], c["page"]
    grp = hq // hkv
    q = st["q"]
    out = torch.empty(q.shape, dtype=wide, device=q.device)
    for b, (n, past) in enumerate(st["lens"]):
        t0, total = st["cu_host"][b], n + past
        at_page, at_row = _slots(st["table"], b, 0, total, page)
        kb = st["k_pages"][at_page, at_row].to(wide)
        vb = st["v_pages"][at_page, at_row].to(wide)
        bb = st["bias"][at_page, at_row].to(wide) if st["bias"] is not None else None
        for h0 in range(hkv):
            hs = slice(h0 * grp, (h0 + 1) * grp)
            for i0 in range(0, n, rows_at_once):
                i1 = min(n, i0 + rows_at_once)
                qb = q[t0 + i0:t0 + i1, hs].to(wide).transpose(0, 1)      # [grp, r, dh]
                logits = torch.matmul(qb, kb[:, h0].t()) / (
                    math.sqrt(dh) * st["tau"][hs].to(wide)[:, None, None])
                if bb is not None:
                    logits = logits + st["gain"][hs].to(wide)[:, None, None] * bb
                seen = torch.arange(total, device=q.device)[None] <= torch.arange(
                    past + i0, past + i1, device=q.device)[:, None]
                logits = torch.where(seen[None], logits, torch.full_like(logits[:1, :1, :1],
                                                                         -math.inf))
                logits = torch.exp(logits - logits.amax(-1, keepdim=True))
                o = torch.matmul(logits, vb[:, h0]) / logits.sum(-1, keepdim=True)
                out[t0 + i0:t0 + i1, hs] = o.transpose(0, 1)
    return out


def _quant_plain(x):
    # In 64 bits, so that a value next to the border between two integers
    # goes to the side that the definition says.
    w = x.double()
    amax = w.abs().amax(dim=1)
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    return torch.round(w * 127.0 / safe[:, None]).to(torch.int8), (amax / 127.0).float()


def _linear_plain(st):
    acc = torch.matmul(st["xq"].float(), st["wq"].float().t())
    y = acc * st["xs"][:, None] * st["ws"][None]
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(_dtype(st["case"]))


def run(state):
    c = state["case"]
    if own:
        return _run_own(state)
    if c["op"] == "append":
        return _append_plain(state)
    if c["op"] == "attn":
        return _attend(state, torch.float32, 1024).to(_dtype(c))
    if c["op"] == "quant":
        xq, scale = _quant_plain(state["x"])
        return dict(xq=xq, scale=scale)
    return _linear_plain(state)


def _run_own(st):
    import learned_token_pruning_score_b200 as tg

    c = st["case"]
    if c["op"] == "append":
        hq, hkv, dh = c["hq"], c["hkv"], c["dh"]
        x = st["qkv"].view(-1, hq + 2 * hkv, dh)
        q = tg.tg_paged_append(st["cache"], x[:, hq:hq + hkv], x[:, hq + hkv:], st["cu"],
                               st["kv_len"], q=x[:, :hq], pos=st["pos"], s=st["s"],
                               q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS,
                               rope_base=ROPE_BASE)
        return _append_outputs(st, q)
    if c["op"] == "attn":
        return tg.tg_paged_attn(st["cache"], st["q"], st["cu"], st["kv_len"], gain=st["gain"],
                                tau=st["tau"], max_kv=st["max_kv"])
    if c["op"] == "quant":
        xq, scale = tg.tg_quantize_rows(st["x"])
        return dict(xq=xq, scale=scale)
    return tg.tg_linear_quantized(st["xq"], st["xs"], st["wq"], st["ws"],
                                  residual=st["residual"], dtype=_dtype(c))


# ------------------------------------------------------------------ exact values


def exact(case, seed):
    """The operators' definitions in 64 bits, written apart from the plain forms."""
    if case["op"] == "quant":
        x = prepare(case, seed)["x"].double()
        top = x.abs().max(dim=1).values
        step = top / 127.0
        ints = torch.round(127.0 * x / torch.where(top == 0, 1.0, top)[:, None])
        return dict(xq=ints.to(torch.int8), scale=step)
    if case["op"] == "linear":
        st = prepare(case, seed)
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        wt = st["wq"].double().t().contiguous()
        for i in range(0, case["m"], 4096):  # sums of products of 8-bit integers: exact
            y[i:i + 4096] = st["xq"][i:i + 4096].double() @ wt
        y *= st["xs"].double()[:, None]
        y *= st["ws"].double()[None, :]
        if st["residual"] is not None:
            y += st["residual"].double()
        return y
    st = _paged_inputs(case, seed)
    if case["op"] == "append":
        return _append_exact(case, st)
    return _attn_exact(case, st)


def _append_exact(case, st):
    hq, hkv, dh, page = case["hq"], case["hkv"], case["dh"], case["page"]
    x = st["qkv"].double().view(-1, hq + 2 * hkv, dh)
    half = dh // 2
    freq = ROPE_BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(len(x), half),
                       st["pos"].double()[:, None] * freq)

    def turned(y, w):
        if w is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * w.double()
        z = torch.complex(y[..., :half], y[..., half:]) * turn[:, None]
        return torch.cat([z.real, z.imag], -1)

    q = turned(x[:, :hq], st["q_norm"])
    k = turned(x[:, hq:hq + hkv], st["k_norm"])
    v = x[:, hq + hkv:]
    k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
    bias = None
    if st["bias"] is not None:
        bias = st["bias"].double()
        b_new = -torch.logaddexp(torch.zeros_like(st["s"].double()), -st["s"].double())
    at = 0
    for b, (n, past) in enumerate(st["lens"]):
        done = 0
        while done < n:  # page by page
            row = past + done
            p, r = int(st["table"][b, row // page]), row % page
            take = min(page - r, n - done)
            src = slice(at + done, at + done + take)
            k_pages[p, r:r + take], v_pages[p, r:r + take] = k[src], v[src]
            if bias is not None:
                bias[p, r:r + take] = b_new[src]
            done += take
        at += n
    out = dict(q=q, k_pages=k_pages, v_pages=v_pages)
    if bias is not None:
        out["bias"] = bias
    return out


def _attn_exact(case, st):
    hq, hkv, dh, page = case["hq"], case["hkv"], case["dh"], case["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, past) in enumerate(st["lens"]):
        total = n + past
        pages = st["table"][b, :(total + page - 1) // page].long()
        kb = st["k_pages"][pages].flatten(0, 1)[:total].double()
        vb = st["v_pages"][pages].flatten(0, 1)[:total].double()
        for h in range(hq):
            add = 0.0
            if st["bias"] is not None:
                add = st["gain"][h].double() * st["bias"][pages].flatten()[:total].double()
            for i in range(0, n, 512):
                j = min(n, i + 512)
                lg = st["q"][at + i:at + j, h].double() @ kb[:, h // (hq // hkv)].T
                lg = lg / (dh ** 0.5 * st["tau"][h].double()) + add
                late = torch.ones(j - i, total, dtype=torch.bool, device="cuda").triu(past + i + 1)
                lg[late] = -math.inf
                out[at + i:at + j, h] = torch.exp(
                    lg - torch.logsumexp(lg, -1, keepdim=True)) @ vb[:, h // (hq // hkv)]
        at += n
    return out
