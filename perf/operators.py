"""Latent-cache operators: what is measured, and their plain forms.

A latent cache keeps, for every token, one latent vector c (R elements) and
one rotary key r (Dr elements) that all heads share, in pages behind a page
table. Four operators work on it:

  append   new rows are written into the pages, as bf16 or as e4m3 codes with
           one power-of-two scale a row;
  gather   rows are read back from the pages as contiguous bf16;
  decode   attention of a few query rows a sequence over the pages, in the
           absorbed form: keys are [c | r], values are c;
  prefill  attention of many query rows, in the expanded form: every head has
           keys and values of its own, made from c by a product, and all of
           them share r.

`run` takes the plain form in 32 bits where `own` is false and the library's
entry points where it is true.
"""

import math

import torch

own = False

SCALE_MIN, SCALE_MAX = -30, 30  # exponents of a row's power-of-two scale
OFF, BOTTOM_RIGHT = -1, -2      # causal offsets


def listed():
    return [
        # one new token for each of a batch of running requests: launch latency
        dict(name="append_step_bf16", op="append", fp8=False, batch=96, lo=1, hi=1, context=4000,
             page=64, latent=512, rope=64),
        # a round of prompt chunks of uneven length into an FP8 cache
        dict(name="append_chunks_fp8", op="append", fp8=True, batch=23, lo=1, hi=4099, context=8000,
             page=64, latent=512, rope=64),
        # a cached prefix read back before its keys and values are expanded
        dict(name="gather_prefix_bf16", op="gather", fp8=False, batch=5, lo=130, hi=2500, context=900,
             page=16, latent=256, rope=32),
        # the same for a full batch of long FP8 prefixes
        dict(name="gather_prefixes_fp8", op="gather", fp8=True, batch=31, lo=0, hi=5000, context=3000,
             page=128, latent=512, rope=64),
        # one interactive request: latency counts
        dict(name="decode_single_bf16", op="decode", fp8=False, batch=1, q_len=1, heads=20, lo=777,
             hi=777, page=16, latent=512, rope=64, causal=OFF, window=0),
        # a batch of uneven requests, heads shared out over several GPUs
        dict(name="decode_uneven_bf16", op="decode", fp8=False, batch=48, q_len=1, heads=32, lo=100,
             hi=8192, page=64, latent=512, rope=64, causal=OFF, window=0),
        # every head of the layer on one GPU
        dict(name="decode_heads128_bf16", op="decode", fp8=False, batch=56, q_len=1, heads=128,
             lo=3500, hi=4500, page=64, latent=512, rope=64, causal=OFF, window=0),
        # two speculated tokens a request over an FP8 cache, an empty request among them
        dict(name="decode_verify_fp8", op="decode", fp8=True, batch=72, q_len=3, heads=16, lo=0,
             hi=6000, page=128, latent=512, rope=64, causal=BOTTOM_RIGHT, window=0),
        # two very long contexts: few rows, a long axis
        dict(name="decode_long_fp8", op="decode", fp8=True, batch=2, q_len=1, heads=64, lo=90001,
             hi=131072, page=64, latent=512, rope=64, causal=OFF, window=0),
        # short prompts of uneven length
        dict(name="prefill_short", op="prefill", batch=9, heads=16, lo=33, hi=700, context=0, dim=128,
             rope=64, causal=BOTTOM_RIGHT, window=0),
        # chunks of prompts behind contexts that are cached already
        dict(name="prefill_chunks", op="prefill", batch=4, heads=32, lo=300, hi=1100, context=4000,
             dim=128, rope=64, causal=BOTTOM_RIGHT, window=0),
        # one long prompt
        dict(name="prefill_long", op="prefill", batch=1, heads=16, lo=8192, hi=8192, context=0,
             dim=128, rope=64, causal=BOTTOM_RIGHT, window=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prefill"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    latent, rope = rng.choice([(512, 64), (512, 64), (256, 64), (256, 32), (512, 32)])
    fp8 = rng.random() < 0.5
    if op in ("append", "gather"):
        batch = _log_int(rng, 1, 96)
        hi = _log_int(rng, 1, max(1, min(5000, 48000 // batch)))
        return dict(op=op, fp8=fp8, batch=batch, lo=rng.choice([0, hi]) if hi > 1 else 1, hi=hi,
                    context=_log_int(rng, 1, 8000), page=page, latent=latent, rope=rope)
    if op == "decode":
        batch = _log_int(rng, 1, 96)
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        heads = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 128])
        rows = batch * q_len * heads
        hi = _log_int(rng, 1, max(2, min(100000, 300000 // batch, 2 ** 31 // (4 * rows))))
        causal = BOTTOM_RIGHT if q_len > 1 else OFF
        return dict(op=op, fp8=fp8, batch=batch, q_len=q_len, heads=heads, lo=rng.choice([0, hi // 2, hi]),
                    hi=hi, page=page, latent=latent, rope=rope, causal=causal,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, 4000)]))
    batch = _log_int(rng, 1, 12)
    heads = rng.choice([1, 3, 8, 16, 32])
    hi = _log_int(rng, 2, max(2, 6000 // batch))
    context = rng.choice([0, 0, _log_int(rng, 1, 4000)])
    while batch * heads * hi * (hi + context) > 1 << 30:
        heads, hi = max(1, heads // 2), max(2, hi * 3 // 4)
    return dict(op=op, batch=batch, heads=heads, lo=rng.choice([0, 1, hi]), hi=hi, context=context,
                dim=128, rope=rng.choice([32, 64]), causal=rng.choice([BOTTOM_RIGHT, BOTTOM_RIGHT, OFF]),
                window=rng.choice([0, 0, _log_int(rng, 1, 2000)]))


# ---------------------------------------------------------------------------
# inputs

def _lengths(case, g, more):
    """A length of [lo, hi] for every sequence (one is hi, another lo) and a
    number up to `more` beside it. The pairs are the case's, their order is the seed's."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    fixed = torch.Generator().manual_seed(n + hi)
    v = torch.randint(lo, hi + 1, (n,), generator=fixed)
    v[-1] = lo
    v[0] = hi
    beside = torch.randint(0, more + 1, (n,), generator=fixed)
    order = torch.randperm(n, generator=g)
    return v[order], beside[order]


def _pages(lens, page, g):
    """A page table of shuffled pages that holds `lens` tokens a sequence, -1 behind them."""
    need = (lens + page - 1) // page
    width = max(1, int(need.max()))
    total = max(1, int(need.sum()))
    ids = torch.randperm(total + 3, generator=g)[:total].to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[torch.arange(width)[None, :] < need[:, None]] = ids[: int(need.sum())]
    return table, total + 3


def _quantise(c):
    """Rows of c (fp32) as e4m3 codes (their float8 type) and scale exponents, int32."""
    f, k = torch.frexp(c.abs().amax(dim=-1))
    e = torch.where(f > 0.875, k - 8, k - 9)
    e = torch.where(f == 0, torch.full_like(e, SCALE_MIN), e).clamp(SCALE_MIN, SCALE_MAX)
    return torch.ldexp(c, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), e.to(torch.int32)


def _rows(shape, g, spread=True):
    """bf16 rows as a norm or a projection leaves them: unit variance, some rows larger or smaller."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if spread:
        x = x * torch.exp2(torch.randint(-1, 2, shape[:-1] + (1,), generator=g, device="cuda").float())
    return x.to(torch.bfloat16)


def _pools(case, num_pages, gd):
    """Pools full of rows: latent, rope and, FP8, the scale bytes."""
    shape = (num_pages, case["page"])
    c = _rows(shape + (case["latent"],), gd)
    rope = _rows(shape + (case["rope"],), gd, spread=False)
    if not case["fp8"]:
        return c, rope, None
    codes, e = _quantise(c.float())
    return codes.view(torch.uint8), rope, (e + 127).to(torch.uint8)


def _offsets(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    op, n = case["op"], case["batch"]
    if op in ("append", "gather"):
        lens, first = _lengths(case, g, case["context"])
        table, num_pages = _pages(first + lens, case["page"], g)
        st.update(page_table=table.cuda(), first=first.to(torch.int32).cuda(),
                  row_offsets=_offsets(lens).cuda(), total=int(lens.sum()))
        if op == "gather":
            st["latent_pages"], st["rope_pages"], st["scales"] = _pools(case, num_pages, gd)
        else:
            # one projection writes both parts of a row, so each is a view of it
            both = _rows((st["total"], case["latent"] + case["rope"]), gd)
            st["c"], st["r"] = both[:, : case["latent"]], both[:, case["latent"]:]
            shape = (num_pages, case["page"])
            st["latent_pages"] = torch.zeros(shape + (case["latent"],), device="cuda",
                                             dtype=torch.uint8 if case["fp8"] else torch.bfloat16)
            st["rope_pages"] = torch.zeros(shape + (case["rope"],), device="cuda", dtype=torch.bfloat16)
            st["scales"] = torch.zeros(shape, device="cuda", dtype=torch.uint8) if case["fp8"] else None
    elif op == "decode":
        lens, _ = _lengths(case, g, 0)
        table, num_pages = _pages(lens, case["page"], g)
        st["latent_pages"], st["rope_pages"], st["scales"] = _pools(case, num_pages, gd)
        st["q"] = _rows((n, case["q_len"], case["heads"], case["latent"] + case["rope"]), gd, spread=False)
        st.update(page_table=table.cuda(), kv_lens=lens.to(torch.int32).cuda(),
                  scale=(128 + case["rope"]) ** -0.5)
    else:
        d, h = case["dim"], case["heads"]
        q_lens, before = _lengths(case, g, case["context"])
        kv_lens = q_lens + before
        tq, tk = int(q_lens.sum()), int(kv_lens.sum())
        st["q"] = _rows((tq, h, d + case["rope"]), gd, spread=False)
        st["kv"] = _rows((tk, h, 2 * d), gd, spread=False)
        st["r"] = _rows((tk, case["rope"]), gd, spread=False)
        st.update(q_offsets=_offsets(q_lens).cuda(), kv_offsets=_offsets(kv_lens).cuda(),
                  max_q=int(q_lens.max()), max_kv=int(kv_lens.max()), scale=(d + case["rope"]) ** -0.5)
    return st


# ---------------------------------------------------------------------------
# the plain forms (T: the type they compute in)

def _slots(st, owner, position):
    """Row of the flattened pools that holds `position` of sequence `owner`."""
    page = st["page_table"][owner, position // st["page"]].long()
    return page * st["page"] + position % st["page"]


def _row_map(st):
    """The sequence and the position of every ragged row."""
    row = torch.arange(st["total"], device="cuda")
    off = st["row_offsets"].long()
    owner = torch.searchsorted(off, row, right=True) - 1
    return owner, st["first"].long()[owner] + row - off[owner]


def _values(st, slots, T):
    """Latent and rope rows of `slots` as values."""
    c = st["latent_pages"].flatten(0, 1)[slots]
    r = st["rope_pages"].flatten(0, 1)[slots].to(T)
    if not st["fp8"]:
        return c.to(T), r
    e = st["scales"].flatten()[slots].int() - 127
    return torch.ldexp(c.view(torch.float8_e4m3fn).to(T), e.unsqueeze(-1).to(T)), r


def _append_plain(st):
    owner, position = _row_map(st)
    slots = _slots(st, owner, position)
    c = st["c"]
    if st["fp8"]:
        codes, e = _quantise(c.float())
        c = codes.view(torch.uint8)
        st["scales"].view(-1)[slots] = (e + 127).to(torch.uint8)
    st["latent_pages"].flatten(0, 1)[slots] = c
    st["rope_pages"].flatten(0, 1)[slots] = st["r"]


def _append_out(st):
    if not st["fp8"]:
        return st["latent_pages"], st["rope_pages"]
    return st["latent_pages"].view(torch.float8_e4m3fn), st["rope_pages"], st["scales"]


def _gather_plain(st, T):
    owner, position = _row_map(st)
    return _values(st, _slots(st, owner, position), T)


def _softmax(s, seen):
    """exp(s - lse) and lse over the last axis of the keys that are seen; rows that see none: 0 and -inf."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    lse = m + torch.log(total)
    return p / torch.where(total == 0, torch.ones_like(total), total), lse.squeeze(-1)


def _seen(case, q_index, q_lens, kv_lens, key):
    """Which keys a query row sees. q_index [rows], lengths [B], key [L] -> [B, rows, L]."""
    causal, window = case["causal"], case["window"]
    kv = kv_lens[:, None, None]
    position = kv - q_lens[:, None, None] + q_index[None, :, None]
    if causal == OFF:
        position = kv - 1 + torch.zeros_like(position)
    seen = (key < kv) & (key <= position)
    if window > 0:
        seen = seen & (key > position - window)
    return seen & (q_index[None, :, None] < q_lens[:, None, None])


def _decode_plain(st, T):
    lens = st["kv_lens"].long()
    key = torch.arange(max(1, int(st["page_table"].shape[1]) * st["page"]), device="cuda")
    table = st["page_table"].clamp(min=0)
    slots = table.long().repeat_interleave(st["page"], dim=1) * st["page"] + key % st["page"]
    c, r = _values(st, slots, T)
    live = (key < lens[:, None]).unsqueeze(-1)
    c, r = c.masked_fill(~live, 0.0), r.masked_fill(~live, 0.0)
    q = st["q"].to(T)
    s = torch.einsum("bihd,bjd->bihj", q[..., : st["latent"]], c)
    s = (s + torch.einsum("bihd,bjd->bihj", q[..., st["latent"]:], r)) * st["scale"]
    q_lens = torch.full_like(lens, st["q_len"])
    seen = _seen(st, torch.arange(st["q_len"], device="cuda"), q_lens, lens, key)
    p, lse = _softmax(s, seen[:, :, None, :])
    return torch.einsum("bihj,bjd->bihd", p, c), lse


def _padded(x, offsets, width):
    """Ragged rows [T, ...] as [B, width, ...], zeros behind each sequence."""
    off = offsets.long()
    row = off[:-1, None] + torch.arange(width, device="cuda")
    live = row < off[1:, None]
    y = x[torch.where(live, row, torch.zeros_like(row))]
    return y.masked_fill(~live.view(live.shape + (1,) * (x.dim() - 1)), 0.0), live


def _prefill_plain(st, T):
    d = st["dim"]
    q, q_live = _padded(st["q"].to(T), st["q_offsets"], st["max_q"])
    kv, _ = _padded(st["kv"].to(T), st["kv_offsets"], st["max_kv"])
    r, _ = _padded(st["r"].to(T), st["kv_offsets"], st["max_kv"])
    s = torch.einsum("bihd,bjhd->bhij", q[..., :d], kv[..., :d])
    s = (s + torch.einsum("bihd,bjd->bhij", q[..., d:], r)) * st["scale"]
    q_lens, kv_lens = (st[k].long().diff() for k in ("q_offsets", "kv_offsets"))
    seen = _seen(st, torch.arange(st["max_q"], device="cuda"), q_lens, kv_lens,
                 torch.arange(st["max_kv"], device="cuda"))
    p, lse = _softmax(s, seen[:, None])
    o = torch.einsum("bhij,bjhd->bihd", p, kv[..., d:])
    return o[q_live], lse.transpose(1, 2)[q_live]


# ---------------------------------------------------------------------------
# one pass

def run(state):
    op = state["op"]
    if own:
        return _run_own(state)
    if op == "append":
        _append_plain(state)
        return _append_out(state)
    if op == "gather":
        c, r = _gather_plain(state, torch.float32)
        return c.to(torch.bfloat16), r.to(torch.bfloat16)
    o, lse = (_decode_plain if op == "decode" else _prefill_plain)(state, torch.float32)
    return o.to(torch.bfloat16), lse


def _run_own(state):
    from paged_kv_decode_30_b200 import binding as B
    op = state["op"]
    if op == "append":
        B.paged_latent_append(state["c"], state["r"], state["row_offsets"], state["page_table"],
                              state["first"], state["latent_pages"], state["rope_pages"],
                              latent_scales=state["scales"])
        return _append_out(state)
    if op == "gather":
        return B.paged_latent_gather(state["latent_pages"], state["rope_pages"], state["page_table"],
                                     state["row_offsets"], starts=state["first"],
                                     total_rows=state["total"], latent_scales=state["scales"])
    if op == "decode":
        return B.paged_latent_decode(state["q"], state["latent_pages"], state["rope_pages"],
                                     state["page_table"], state["kv_lens"], scale=state["scale"],
                                     causal_offset=state["causal"], window=state["window"],
                                     latent_scales=state["scales"])
    return B.latent_prefill_attn(state["q"], state["kv"], state["r"], state["q_offsets"],
                                 state["kv_offsets"], scale=state["scale"],
                                 causal_offset=state["causal"], window=state["window"],
                                 max_q_len=state["max_q"])


# ---------------------------------------------------------------------------
# what a pass cannot do without

def _mean(case):
    """Mean length that _lengths gives."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return hi if n == 1 else (lo + hi + (n - 2) * (lo + hi) / 2) / n


def work(case):
    n, op = case["batch"], case["op"]
    rows = n * _mean(case)
    if op == "prefill":
        h, d, rope = case["heads"], case["dim"], case["rope"]
        before = case["context"] / 2
        keys = rows + n * before
        if n > 1:  # mean of squares of the uniform lengths
            lo, hi = case["lo"], case["hi"]
            square = (lo * lo + hi * hi + (n - 2) * (lo * lo + lo * hi + hi * hi) / 3) / n
        else:
            square = case["hi"] ** 2
        share = 1.0 if case["causal"] == OFF else 0.5
        pairs = n * (square * share + _mean(case) * before)
        if case["window"] > 0:
            pairs = min(pairs, rows * case["window"])
        return {"bytes": 2 * h * (rows * (2 * d + rope) + keys * 2 * d) + 2 * keys * rope + 4 * rows * h,
                "flops": 2 * pairs * h * (2 * d + rope)}
    c, rope = case["latent"], case["rope"]
    wide, narrow = 2 * (c + rope), (c + 1 if case["fp8"] else 2 * c) + 2 * rope
    if op in ("append", "gather"):
        return {"bytes": rows * (wide + narrow), "flops": 0}
    seen = _mean(case)
    if case["window"] > 0:
        seen = min(seen, case["window"] + case["q_len"] - 1)
    heads = case["q_len"] * case["heads"]
    return {"bytes": n * seen * narrow + n * heads * (wide + 2 * c + 4),
            "flops": 2 * n * seen * heads * (2 * c + rope)}


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence

def exact(case, seed):
    def attend(q, k, v, scale, position, window):
        """q [Q, h, d], k [L, h or 1, d], v [L, h or 1, e], position [Q] -> out [Q, h, e], lse [Q, h]."""
        n = k.shape[0]
        out = torch.zeros(q.shape[0], q.shape[1], v.shape[-1], dtype=torch.float64, device=q.device)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
        j = torch.arange(n, device=q.device)
        for h in range(q.shape[1]):
            for i in range(0, q.shape[0], 2048):
                pos = position[i: i + 2048, None]
                hidden = (j > pos) | ((j <= pos - window) if window > 0 else (j < 0))
                if n == 0:
                    continue
                x = scale * (q[i: i + 2048, h] @ k[:, h % k.shape[1]].T)
                x[hidden] = -math.inf
                total = torch.logsumexp(x, dim=1)
                w = torch.exp(x - total[:, None].nan_to_num(neginf=0.0))
                out[i: i + 2048, h] = w @ v[:, h % v.shape[1]]
                lse[i: i + 2048, h] = total
        return out, lse

    st = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "append":
        _, position = _row_map(st)
        owner = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"),
                                        st["row_offsets"].long().diff())
        slot = st["page_table"].long()[owner, position // case["page"]] * case["page"] + position % case["page"]
        rope = st["rope_pages"].double()
        rope.view(-1, case["rope"])[slot] = st["r"].double()
        pool = torch.zeros(st["latent_pages"].shape, dtype=D, device="cuda")
        c = st["c"].double()
        if not case["fp8"]:
            pool.view(-1, case["latent"])[slot] = c
            return pool, rope
        # what the code stands for before it is rounded to 8 bits
        top = c.abs().amax(dim=1)
        e = torch.ceil(torch.log2(top / 448)).nan_to_num(neginf=SCALE_MIN).clamp(SCALE_MIN, SCALE_MAX)
        pool.view(-1, case["latent"])[slot] = c * torch.exp2(-e)[:, None]
        return pool, rope, None
    off = {k: st[k].tolist() for k in ("row_offsets", "q_offsets", "kv_offsets", "kv_lens", "first") if k in st}
    if op == "prefill":
        d, outs = case["dim"], []
        for b in range(case["batch"]):
            i0, i1, j0, j1 = off["q_offsets"][b], off["q_offsets"][b + 1], off["kv_offsets"][b], off["kv_offsets"][b + 1]
            q, kv, r = st["q"][i0:i1].double(), st["kv"][j0:j1].double(), st["r"][j0:j1].double()
            k = torch.cat([kv[..., :d], r[:, None, :].expand(-1, case["heads"], -1)], dim=-1)
            pos = torch.arange(i1 - i0, device="cuda") + (j1 - j0) - (i1 - i0)
            if case["causal"] == OFF:
                pos = torch.full_like(pos, j1 - j0 - 1)
            outs.append(attend(q, k, kv[..., d:], st["scale"], pos, case["window"]))
        return torch.cat([o for o, _ in outs]), torch.cat([l for _, l in outs])
    # every row of the pools as the value that it stands for
    c, r = st["latent_pages"], st["rope_pages"].double()
    if case["fp8"]:
        c = c.view(torch.float8_e4m3fn).double() * torch.exp2(st["scales"].double() - 127)[..., None]
    else:
        c = c.double()

    def tokens(pool, b, start, count):
        ids = st["page_table"][b].long().clamp(min=0)
        j = torch.arange(start, start + count, device="cuda")
        return pool[ids[j // case["page"]], j % case["page"]]

    if op == "gather":
        parts = [(b, off["first"][b], off["row_offsets"][b + 1] - off["row_offsets"][b]) for b in range(case["batch"])]
        return tuple(torch.cat([tokens(p, *part) for part in parts]) for p in (c, r))
    outs = []
    for b, n in enumerate(off["kv_lens"]):
        k = torch.cat([tokens(c, b, 0, n), tokens(r, b, 0, n)], dim=-1)[:, None, :]
        pos = torch.arange(case["q_len"], device="cuda") + n - case["q_len"]
        if case["causal"] == OFF:
            pos = torch.full_like(pos, n - 1)
        q = st["q"][b].double().flatten(0, 1)[:, None, :]  # the heads of a row share its keys
        o, l = attend(q, k, k[..., : case["latent"]], st["scale"],
                         pos.repeat_interleave(case["heads"]), case["window"])
        outs.append((o.view(case["q_len"], case["heads"], -1), l.view(case["q_len"], case["heads"])))
    return torch.stack([o for o, _ in outs]), torch.stack([l for _, l in outs])
