"""Cases of the rotary paged appends and of the attention over block-scaled e4m3 pages.

Three operators, each in its plain form (elementary torch operations, 32-bit) and as the call a
user makes of the library:

  rope_append      rotate this step's queries and keys, write keys and values into bf16 pages
  rope_append_fp8  the same into e4m3 pages with one power-of-two scale per block of tokens and
                   KV head
  attention_fp8    decode / verify attention over such pages

A request's position t lives in row t % page_rows of page page_table[b][t // page_rows].
"""
import math

import torch

own = False

#: Largest e4m3 magnitude, and the range of the scales' exponents.
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -100, 100


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, op, batch, k, q_heads, kv_heads, head_dim, ctx_lo, ctx_hi, page_rows=128,
            block_rows=16, rotary_dim=None, interleaved=False, ragged=False, fused_qkv=False):
    return {"name": name, "op": op, "batch": batch, "k": k, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "page_rows": page_rows, "block_rows": block_rows,
            "rotary_dim": head_dim if rotary_dim is None else rotary_dim,
            "interleaved": interleaved, "ragged": ragged, "fused_qkv": fused_qkv}


def _attend(name, batch, k, q_heads, kv_heads, head_dim, key_lo, key_hi, page_rows=128,
            block_rows=16, window=0):
    return {"name": name, "op": "attention_fp8", "batch": batch, "k": k, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "key_lo": key_lo, "key_hi": key_hi,
            "page_rows": page_rows, "block_rows": block_rows, "window": window}


def listed():
    return [
        # one user's next token in a global layer: pure latency
        _append("rope decode 1", "rope_append", 1, 1, 16, 2, 512, 6004, 6004),
        # a verify step of a full batch, straight from the fused QKV projection's output
        _append("rope verify 64x4", "rope_append", 64, 4, 16, 2, 512, 512, 4096, fused_qkv=True),
        # prompts of several users after prefill, ragged, sliding-layer heads, partial rotation
        _append("rope prompts 8x2048", "rope_append", 8, 2048, 16, 8, 256, 0, 0, page_rows=256,
                rotary_dim=64, interleaved=True, ragged=True),
        # the same three situations with an 8-bit cache
        _append("rope fp8 decode 1", "rope_append_fp8", 1, 1, 16, 2, 512, 6004, 6004),
        _append("rope fp8 verify 64x4", "rope_append_fp8", 64, 4, 16, 2, 512, 512, 4096,
                block_rows=32, fused_qkv=True),
        _append("rope fp8 prompts 8x2048", "rope_append_fp8", 8, 2048, 16, 8, 256, 0, 0,
                page_rows=256, block_rows=64, rotary_dim=64, interleaved=True, ragged=True),
        # one long prompt's next chunk behind 1000 tokens that are already cached
        _append("rope fp8 chunk 8191", "rope_append_fp8", 1, 8191, 16, 2, 512, 1000, 1000,
                block_rows=128),
        # one request's decode, sliding-layer heads: a short chain of latencies
        _attend("attn fp8 1x1 1500", 1, 1, 16, 8, 256, 1500, 1500, window=1024),
        # one request's verify of 4 proposals in a global layer
        _attend("attn fp8 1x4 6005", 1, 4, 16, 2, 512, 6005, 6005, block_rows=32),
        # batched decode, sliding-layer heads
        _attend("attn fp8 56x1 sliding", 56, 1, 16, 8, 256, 1024, 4096, page_rows=256,
                block_rows=64, window=1024),
        # the longest contexts under a 15-proposal verify: 120 rows share each KV head
        _attend("attn fp8 8x15 32768", 8, 15, 16, 2, 512, 1024, 32768, block_rows=128),
        # a full batch's verify in a global layer: the bandwidth case
        _attend("attn fp8 64x4 32768", 64, 4, 16, 2, 512, 512, 32768, block_rows=16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_append", "rope_append_fp8", "attention_fp8", "attention_fp8"])
    head_dim = rng.choice([256, 512])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    q_heads = group * kv_heads
    page_rows = rng.choice([128, 256, 384])
    block_rows = rng.choice([16, 32, 64, 128])
    if op == "attention_fp8":
        k = rng.randint(1, 16)
        batch = _log_int(rng, 1, 64)
        # at most about 0.4 million cached tokens of 1024 bytes a row over the batch
        rows = 400000 * 1024 // (batch * kv_heads * head_dim)
        key_hi = _log_int(rng, 32, max(33, min(32768, rows)))
        key_lo = max(k, _log_int(rng, 16, key_hi))
        key_hi = max(key_hi, key_lo)
        window = rng.choice([0, 0, 1024, rng.randint(k, 2000)])
        case = _attend("", batch, k, q_heads, kv_heads, head_dim, key_lo, key_hi, page_rows,
                       block_rows, window)
    else:
        if rng.random() < 0.5:                  # a step
            batch, k = _log_int(rng, 1, 64), rng.randint(1, 16)
        else:                                   # prompts, at most 16384 tokens
            batch = _log_int(rng, 1, 16)
            k = _log_int(rng, 17, 16384 // batch)
        ctx_hi = rng.choice([0, _log_int(rng, 1, 4096)])
        case = _append("", op, batch, k, q_heads, kv_heads, head_dim, min(ctx_hi, rng.randint(0, 64)),
                       ctx_hi, page_rows, block_rows, rng.choice([head_dim, head_dim // 4, 64]),
                       rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(case, lo, hi, seed):
    """One length per request, spread over [lo, hi] by its logarithm (both ends met where the
    batch has two requests or more), in a seeded order.  Host integers."""
    n = case["batch"]
    a, b = math.log(lo + 1), math.log(hi + 1)
    v = [int(round(math.exp(a + (b - a) * (i / (n - 1) if n > 1 else 1.0)) - 1)) for i in range(n)]
    g = torch.Generator().manual_seed(seed * 2 + 1)
    return [min(hi, max(lo, v[i])) for i in torch.randperm(n, generator=g).tolist()]


def _contexts(case, seed):
    if case["op"] == "attention_fp8":
        return [n - case["k"] for n in _lengths(case, case["key_lo"], case["key_hi"], seed)]
    return _lengths(case, case["ctx_lo"], case["ctx_hi"], seed)


def _counts(case, seed):
    """New tokens of each request of an append (all k, or ragged: one request has none)."""
    n, k = case["batch"], case["k"]
    if not case["ragged"]:
        return [k] * n
    g = torch.Generator().manual_seed(seed * 2 + 2)
    c = [int(x) for x in torch.randint(max(1, k // 4), k + 1, (n,), generator=g)]
    c[0] = k
    if n > 2:
        c[-1] = 0
    return c


def _pages(case, ctx):
    most = max(c + case["k"] for c in ctx)
    return max(1, -(-most // case["page_rows"]))


def _normal(shape, gen, dtype=torch.bfloat16, mul=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, mul, generator=gen)


def _e4m3_pool(shape, gen):
    """Bytes of normal draws, as a block's quantisation leaves them (largest near 256)."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for page in out.split(max(1, (64 << 20) // max(1, out[0].numel()))):
        x = _normal(page.shape, gen, torch.float32, 64.0).clamp_(-E4M3_MAX, E4M3_MAX)
        page.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _pow2(e):
    """2^e in fp32, exactly (e in the normal range)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scales(shape, gen):
    """Power-of-two scales that give the pool's bytes a spread of about 1/2 to 2."""
    return _pow2(torch.randint(-7, -4, shape, device="cuda", generator=gen))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, k, H, D = case["batch"], case["k"], case["kv_heads"], case["head_dim"]
    Hq, rows = case["q_heads"], case["page_rows"]
    ctx = _contexts(case, seed)
    per = _pages(case, ctx)
    num_pages = B * per + 1
    perm = torch.randperm(num_pages, device="cuda", generator=gen)
    st = {"case": dict(case), "page_table": perm[:B * per].view(B, per).to(torch.int32).contiguous(),
          "context_lengths": torch.tensor(ctx, dtype=torch.int32, device="cuda")}
    pool = (num_pages, rows, H, D)
    if case["op"] == "rope_append":
        st["key_pages"], st["value_pages"] = _normal(pool, gen), _normal(pool, gen)
    else:
        st["key_pages"], st["value_pages"] = _e4m3_pool(pool, gen), _e4m3_pool(pool, gen)
        blocks = (num_pages, rows // case["block_rows"], H)
        st["k_scales"], st["v_scales"] = _scales(blocks, gen), _scales(blocks, gen)
    if case["op"] == "attention_fp8":
        st["queries"] = _normal((B, k, Hq, D), gen)
        st["scale"] = 1.0 / math.sqrt(D)
        st["most"] = max(ctx) + k
        st["out"] = torch.empty((B, k, Hq, D), dtype=torch.bfloat16, device="cuda")
        if own:                                 # the library's workspace: kept by its caller
            from sliding_window_gqa_ring_gb300 import carat
            st["workspace"] = carat.workspace_tensor(carat.paged_fp8_workspace_bytes(
                B, k, Hq, H, D, per * rows))
        return st
    if case["fused_qkv"]:
        qkv = _normal((B, k, (Hq + 2 * H) * D), gen)
        st["queries"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        st["k_new"] = qkv[..., Hq * D:(Hq + H) * D].unflatten(-1, (H, D))
        st["v_new"] = qkv[..., (Hq + H) * D:].unflatten(-1, (H, D))
    else:
        st["queries"] = _normal((B, k, Hq, D), gen)
        st["k_new"], st["v_new"] = _normal((B, k, H, D), gen), _normal((B, k, H, D), gen)
    st["queries_out"] = torch.zeros((B, k, Hq, D), dtype=torch.bfloat16, device="cuda")
    counts = _counts(case, seed)
    st["new_counts"] = (torch.tensor(counts, dtype=torch.int32, device="cuda")
                        if case["ragged"] else None)
    half = case["rotary_dim"] // 2
    pos = torch.arange(per * rows, dtype=torch.float64, device="cuda")
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = pos[:, None] * freq
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).contiguous()
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _rotate(x, cos_sin, positions, interleaved):
    """Rotary embedding of x [B][k][heads][D] (any type) in fp32."""
    x = x.float()
    r = cos_sin.shape[1]
    cs = cos_sin[positions][:, :, None, :]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _rows(st, t):
    """Pool rows of positions t [B][n]."""
    rows = st["case"]["page_rows"]
    return st["page_table"].long().gather(1, t // rows) * rows + t % rows


def _plain_append(st):
    c = st["case"]
    B, k = c["batch"], c["k"]
    ctx = st["context_lengths"].long()[:, None]
    n = st["new_counts"].long()[:, None] if st["new_counts"] is not None else torch.full_like(ctx, k)
    j = torch.arange(k, device="cuda")[None]
    pos = ctx + j
    live = (j < n)[..., None, None]
    q = _rotate(st["queries"], st["cos_sin"], pos, c["interleaved"]).bfloat16()
    q_out = torch.where(live, q, st["queries_out"])
    k_rot = _rotate(st["k_new"], st["cos_sin"], pos, c["interleaved"])
    if c["op"] == "rope_append":
        row = _rows(st, pos)
        for pages, new in ((st["key_pages"], k_rot), (st["value_pages"], st["v_new"])):
            flat = pages.view(-1, *pages.shape[2:])
            flat[row] = torch.where(live, new.to(flat.dtype), flat[row])
        return {"key_pages": st["key_pages"], "value_pages": st["value_pages"],
                "queries_out": q_out}
    # Every block that some request writes, as [B][blocks][R] positions.  Requests that touch
    # fewer blocks name their last one again (the same values are written twice).
    R = c["block_rows"]
    first, last = ctx // R, torch.maximum(ctx + n - 1, ctx) // R
    blocks = torch.minimum(first + torch.arange((k + R - 2) // R + 1, device="cuda")[None], last)
    nb = blocks.shape[1]
    t = (blocks[..., None] * R + torch.arange(R, device="cuda")).flatten(1)      # [B][nb*R]
    t = t.clamp(max=st["page_table"].shape[1] * c["page_rows"] - 1)
    row = _rows(st, t)
    is_new = ((t >= ctx) & (t < ctx + n)).view(B, nb, R, 1, 1)
    is_old = (t < ctx).view(B, nb, R, 1, 1)
    fresh = (blocks * R >= ctx)[..., None]                                       # [B][nb][1]
    touched = is_new.any(2).view(B, nb, 1)
    src = (t - ctx).clamp(0, k - 1)[..., None, None].expand(-1, -1, *k_rot.shape[2:])
    for pages, scales, new in ((st["key_pages"], st["k_scales"], k_rot),
                               (st["value_pages"], st["v_scales"], st["v_new"].float())):
        flat = pages.view(-1, *pages.shape[2:])
        sflat = scales.view(-1, scales.shape[2])
        x = new.gather(1, src).view(B, nb, R, *new.shape[2:])
        amax = torch.where(is_new & x.isfinite(), x.abs(), 0.0).amax((2, 4))     # [B][nb][H]
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), EXP_MIN).clamp(EXP_MIN, EXP_MAX)
        need = _pow2(e)
        brow = (row.view(B, nb, R)[:, :, 0]) // R
        old = sflat[brow]
        scale = torch.where(touched, torch.where(fresh, need, torch.maximum(need, old)), old)
        held = flat[row].view(torch.float8_e4m3fn).float().view_as(x)
        again = held * (old / scale)[:, :, None, :, None]
        y = torch.where(is_new, x / scale[:, :, None, :, None], torch.where(is_old, again, held))
        y = y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        flat[row] = y.flatten(1, 2)
        sflat[brow] = scale
    e4m3 = torch.float8_e4m3fn
    return {"key_pages": st["key_pages"].view(e4m3), "value_pages": st["value_pages"].view(e4m3),
            "k_scales": st["k_scales"], "v_scales": st["v_scales"], "queries_out": q_out}


def _plain_attention(st):
    c = st["case"]
    B, k, H, D, Hq, R = (c[x] for x in ("batch", "k", "kv_heads", "head_dim", "q_heads",
                                        "block_rows"))
    ctx = st["context_lengths"].long()[:, None]
    t = torch.arange(st["most"], device="cuda")[None].expand(B, -1)
    row = _rows(st, t)
    held = (t < ctx + k)[..., None, None]

    def cache(pages, scales):
        x = pages.view(-1, H, D)[row].view(torch.float8_e4m3fn).float()
        x = x * scales.view(-1, H)[row // R][..., None]
        return torch.where(held, x, 0.0).transpose(1, 2)                         # [B][H][S][D]

    q = st["queries"].float().view(B, k, H, Hq // H, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, cache(st["key_pages"], st["k_scales"]).transpose(2, 3)) * st["scale"]
    p = (ctx + torch.arange(k, device="cuda"))[..., None]                        # [B][k][1]
    seen = t[:, None] <= p
    if c["window"]:
        seen = seen & (t[:, None] > p - c["window"])
    seen = seen[:, None, :, None].expand(-1, H, -1, Hq // H, -1).flatten(2, 3)
    s = torch.where(seen, s, -math.inf)
    w = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(w, cache(st["value_pages"], st["v_scales"])) / w.sum(-1, keepdim=True)
    return o.view(B, H, k, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, k, Hq, D).bfloat16()


def _own(st):
    from sliding_window_gqa_ring_gb300 import carat
    c = st["case"]
    if c["op"] == "attention_fp8":
        carat.carat_paged_verify_attention_fp8(
            st["out"], st["queries"], st["key_pages"], st["value_pages"], st["k_scales"],
            st["v_scales"], st["page_table"], st["context_lengths"], scale=st["scale"],
            window=c["window"], workspace=st["workspace"])
        return st["out"]
    rope = {"cos_sin": st["cos_sin"], "interleaved": c["interleaved"], "queries": st["queries"],
            "queries_out": st["queries_out"], "new_counts": st["new_counts"]}
    if c["op"] == "rope_append":
        carat.carat_paged_rope_append(st["key_pages"], st["value_pages"], st["page_table"],
                                      st["k_new"], st["v_new"], st["context_lengths"], **rope)
        return {"key_pages": st["key_pages"], "value_pages": st["value_pages"],
                "queries_out": st["queries_out"]}
    carat.carat_paged_rope_append_fp8(st["key_pages"], st["value_pages"], st["k_scales"],
                                      st["v_scales"], st["page_table"], st["k_new"], st["v_new"],
                                      st["context_lengths"], **rope)
    e4m3 = torch.float8_e4m3fn
    return {"key_pages": st["key_pages"].view(e4m3), "value_pages": st["value_pages"].view(e4m3),
            "k_scales": st["k_scales"], "v_scales": st["v_scales"],
            "queries_out": st["queries_out"]}


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "attention_fp8":
        return _plain_attention(state)
    return _plain_append(state)


# ---------------------------------------------------------------------------
# Work and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations of one pass.  Ragged counts are taken at their expected sum."""
    B, k, H, D, Hq = (case[x] for x in ("batch", "k", "kv_heads", "head_dim", "q_heads"))
    ctx = _contexts(case, 0)
    if case["op"] == "attention_fp8":
        w, group, total, pairs = case["window"], Hq // H, 0, 0
        for n in ctx:
            total += n + k - (max(0, n - w + 1) if w else 0)
            pairs += sum(min(n + j + 1, w) if w else n + j + 1 for j in range(k))
        return {"bytes": total * H * (2 * D + 8 / case["block_rows"]) + 2 * B * k * Hq * D * 2,
                "flops": 4 * pairs * H * group * D}
    tokens = sum(_counts(case, 0))
    new = tokens * 2 * H * D
    table = tokens * case["rotary_dim"] * 4
    bytes_ = 2 * new + 2 * tokens * Hq * D * 2 + table
    if case["op"] == "rope_append":
        bytes_ += 2 * new
    else:
        bytes_ += new + 8 * H * tokens / case["block_rows"]
    return {"bytes": bytes_, "flops": 3 * tokens * (H + Hq) * case["rotary_dim"]}


def _e4m3_round(x):
    """Nearest e4m3 value of a double (ties to even, magnitudes past 448 to 448)."""
    a = x.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(a.clamp(min=2.0 ** -6))           # a in [2^(e-1), 2^e): steps of 2^(e-4)
    step = ((e.to(torch.int64) - 4 + 1023) << 52).view(torch.float64)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _turned(x, table, positions, interleaved):
    """Rotation of rows x [n][heads][D] as complex products, in 64 bits."""
    x = x.double()
    r = table.shape[1]
    cs = table[positions].double()
    turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None, :]
    part = x[..., :r].unflatten(-1, (r // 2, 2) if interleaved else (2, r // 2))
    dim = -1 if interleaved else -2
    z = torch.complex(*part.unbind(dim)) * turn
    return torch.cat([torch.stack([z.real, z.imag], dim).flatten(-2), x[..., r:]], -1)


def _exact_append(case, seed, st):
    rows, R = case["page_rows"], case["block_rows"]
    fp8 = case["op"] == "rope_append_fp8"
    ctx, counts = _contexts(case, seed), _counts(case, seed)
    powers = torch.tensor([2.0 ** e for e in range(EXP_MIN, EXP_MAX + 1)], dtype=torch.float64,
                          device="cuda")
    table = st["page_table"].tolist()
    q_out = st["queries_out"].double()
    if fp8:
        pages = [st[x].view(torch.float8_e4m3fn).double() for x in ("key_pages", "value_pages")]
        scales = [st[x].double() for x in ("k_scales", "v_scales")]
    else:
        pages = [st[x].double() for x in ("key_pages", "value_pages")]
    for b in range(case["batch"]):
        n = counts[b]
        if n == 0:
            continue
        pos = torch.arange(ctx[b], ctx[b] + n, device="cuda")
        q_out[b, :n] = _turned(st["queries"][b, :n], st["cos_sin"], pos, case["interleaved"])
        new = [_turned(st["k_new"][b, :n], st["cos_sin"], pos, case["interleaved"]),
               st["v_new"][b, :n].double()]
        step = R if fp8 else rows
        for t0 in range(ctx[b] // step * step, ctx[b] + n, step):
            lo, hi = max(t0, ctx[b]), min(t0 + step, ctx[b] + n)
            page, r0 = table[b][t0 // rows], t0 % rows
            for i in range(2):
                x = new[i][lo - ctx[b]:hi - ctx[b]]
                at = pages[i][page, r0 + lo - t0:r0 + hi - t0]
                if not fp8:
                    at.copy_(x)
                    continue
                s = scales[i][page, r0 // R]
                top = x.abs().amax((0, 2))
                need = powers[(top[:, None] > E4M3_MAX * powers[:-1]).sum(1)]
                if lo > t0:
                    need = torch.maximum(need, s)
                    before = pages[i][page, r0:r0 + lo - t0]
                    before.copy_(_e4m3_round(before * (s / need)[:, None]))
                at.copy_(_e4m3_round(x / need[:, None]))
                s.copy_(need)
    got = {"key_pages": pages[0], "value_pages": pages[1], "queries_out": q_out}
    if fp8:
        got["k_scales"], got["v_scales"] = scales
    return got


def _exact_attention(case, seed, st):
    k, H, D, Hq, R, w = (case[x] for x in ("k", "kv_heads", "head_dim", "q_heads", "block_rows",
                                           "window"))
    rows, group = case["page_rows"], Hq // H
    out = torch.zeros(st["queries"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_contexts(case, seed)):
        used = st["page_table"][b, :-(-(n + k) // rows)].long()
        for h in range(H):
            kk, vv = (st[p][used, :, h].view(torch.float8_e4m3fn).double()
                      * st[s][used, :, h].double().repeat_interleave(R, 1)[..., None]
                      for p, s in (("key_pages", "k_scales"), ("value_pages", "v_scales")))
            kk, vv = kk.flatten(0, 1)[:n + k], vv.flatten(0, 1)[:n + k]
            for j in range(k):
                lo = max(0, n + j + 1 - w) if w else 0
                q = st["queries"][b, j, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ kk[lo:n + j + 1].T / math.sqrt(D), -1)
                out[b, j, h * group:(h + 1) * group] = p @ vv[lo:n + j + 1]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attention_fp8":
        return _exact_attention(case, seed, st)
    return _exact_append(case, seed, st)
