"""Seeded inputs and 64-bit definitions for the latent-cache tests."""

import numpy as np
import torch

OFF, BOTTOM_RIGHT = -1, -2

# Half a step of bf16 relative to the value, and of fp32.
U16 = 2.0 ** -8
U32 = 2.0 ** -24


def page_table(lens, page, g, extra=3, width=None):
    """Shuffled pages that hold lens[b] tokens each, -1 behind them."""
    need = [(int(n) + page - 1) // page for n in lens]
    total = sum(need) + extra
    ids = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(need), width or max(1, *need, 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, total


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def quantise(x):
    """Rows of x (fp32 [n, R]) -> (codes uint8, scale bytes uint8), by the definition."""
    x = x.double()
    a = torch.where(x.isnan(), torch.zeros_like(x), x.abs()).amax(dim=1)
    e = torch.full(a.shape, 30, dtype=torch.int64)
    for k in range(30, -31, -1):
        e[a <= 448.0 * 2.0 ** k] = k
    y = (x * torch.pow(2.0, -e.double())[:, None]).clamp(-448, 448)
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def values(codes, scales):
    """e4m3 codes [..., R] and scale bytes [...] -> fp64 values."""
    e = scales.to(torch.int64).clamp(97, 157) - 127
    return codes.view(torch.float8_e4m3fn).double() * torch.pow(2.0, e.double())[..., None]


def cache(lens, page, R, Dr, fp8, seed, spread=1.0, poison=True):
    """A paged latent cache of these lengths. Bytes that belong to no token are
    NaN (poison). Returns a dict of CPU tensors and the rows' fp64 values."""
    g = torch.Generator().manual_seed(seed)
    table, num_pages = page_table(lens, page, g)
    rows = num_pages * page
    c = torch.randn((rows, R), generator=g) * torch.exp2(
        torch.randint(-2, 3, (rows, 1), generator=g).float() * spread)
    r = torch.randn((rows, Dr), generator=g).to(torch.bfloat16)
    used = torch.zeros(rows, dtype=torch.bool)
    for b, n in enumerate(lens):
        j = torch.arange(int(n))
        used[table[b].long()[j // page] * page + j % page] = True
    out = dict(page_table=table, kv_lens=torch.tensor([int(n) for n in lens], dtype=torch.int32),
               page=page, scales=None)
    if poison:
        r[~used] = float("nan")
    if fp8:
        codes, scales = quantise(c)
        if poison:
            codes[~used] = 0x7F
            scales[~used] = 255
        val = values(codes, scales)
        out.update(latent=codes.view(num_pages, page, R), scales=scales.view(num_pages, page))
    else:
        c = c.to(torch.bfloat16)
        if poison:
            c[~used] = float("nan")
        val = c.double()
        out.update(latent=c.view(num_pages, page, R))
    out.update(rope=r.view(num_pages, page, Dr), values=val, rope_values=r.double())
    return out


def rows_of(ch, b, n=None):
    """fp64 latent and rope rows of sequence b's first n tokens."""
    n = int(ch["kv_lens"][b]) if n is None else n
    j = torch.arange(n)
    slot = ch["page_table"][b].long()[j // ch["page"]] * ch["page"] + j % ch["page"]
    return ch["values"][slot], ch["rope_values"][slot]


def attend(q, k, v, scale, pos, causal, window):
    """q [n, d], k [L, d], v [L, e] fp64, pos [n]. Returns out, lse, the weighted
    mean of |v| (same shape as out) and the largest scale * sum |q k|."""
    n, L = q.shape[0], k.shape[0]
    j = torch.arange(L)
    seen = torch.ones((n, L), dtype=torch.bool)
    if causal != OFF:
        seen &= j[None, :] <= pos[:, None]
    if window > 0:
        seen &= j[None, :] > pos[:, None] - window
    s = scale * (q @ k.T) if L else torch.zeros((n, 0), dtype=torch.float64)
    s = torch.where(seen, s, torch.full_like(s, -np.inf))
    lse = torch.logsumexp(s, dim=1) if L else torch.full((n,), -np.inf, dtype=torch.float64)
    p = torch.where(seen, torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None]),
                    torch.zeros_like(s))
    big = float((scale * (q.abs() @ k.abs().T)).max()) if L and n else 0.0
    return p @ v, lse, p @ v.abs(), big


def positions(n_q, n_kv, causal):
    i = torch.arange(n_q)
    if causal == OFF:
        return torch.full((n_q,), n_kv - 1)
    return i + (n_kv - n_q if causal == BOTTOM_RIGHT else causal)


def decode_reference(q, ch, scale, causal, window):
    """q bf16 [B, q_len, H, R + Dr]. out, lse, |v| means and score bound, stacked."""
    B, q_len, H, _ = q.shape
    outs = []
    for b in range(B):
        c, r = rows_of(ch, b)
        pos = positions(q_len, c.shape[0], causal).repeat_interleave(H)
        o, l, a, big = attend(q[b].double().reshape(q_len * H, -1), torch.cat([c, r], 1), c, scale,
                              pos, causal, window)
        outs.append((o.view(q_len, H, -1), l.view(q_len, H), a.view(q_len, H, -1), big))
    return (*(torch.stack([x[k] for x in outs]) for k in range(3)), max(x[3] for x in outs))


def prefill_reference(q, kv, k_rope, q_lens, kv_lens, scale, causal, window):
    H, D = q.shape[1], kv.shape[2] // 2
    outs, q0, k0 = [], 0, 0
    big = 0.0
    for nq, nk in zip(q_lens, kv_lens):
        pos = positions(nq, nk, causal)
        heads = []
        for h in range(H):
            k = torch.cat([kv[k0:k0 + nk, h, :D], k_rope[k0:k0 + nk]], 1).double()
            o = attend(q[q0:q0 + nq, h].double(), k, kv[k0:k0 + nk, h, D:].double(), scale, pos,
                       causal, window)
            heads.append(o[:3])
            big = max(big, o[3])
        outs.append([torch.stack([x[k] for x in heads], 1) for k in range(3)])
        q0, k0 = q0 + nq, k0 + nk
    return (*(torch.cat([x[k] for x in outs]) for k in range(3)), big)


def check(got_out, got_lse, ref, width, what="", fp8=None):
    """out: every weight is rounded to 8 significant bits (relative error U16) and so
    is the result; the normaliser adds up the rounded weights, so
      |d out| <= U16 * (sum p |v| + |out|) + U16 * |out|,
    and fp32 accumulation adds at most about width * U32 of the same sums. FP8 (fp8
    = (keys, max |v|)): the two-term weights also carry an absolute error of up to
    2^-18 of the row's largest weight; over n keys, with random signs, seven
    standard deviations of the sum are below 4 sqrt(n) 2^-18 max |v|.
    lse: a score is a sum of `width` products in fp32, off by at most width * U32 *
    scale * sum |q k|; exp2, log2 and the sum over keys add a few U32 of lse and
    2^-20; FP8 queries are split to within 2^-21 of their row's maximum."""
    out, lse, mean_abs, big = ref
    got_out, got_lse = got_out.double().cpu(), got_lse.double().cpu()
    assert torch.equal(got_lse.isneginf(), lse.isneginf()), f"{what}: rows without keys differ"
    assert not got_out.isnan().any() and not got_lse.isnan().any(), f"{what}: NaN"
    d_s = width * U32 * big + (2.0 ** -20 * big if fp8 else 0.0)
    tol = U16 * (mean_abs + 2 * out.abs()) + 2 * (d_s + width * U32) * (mean_abs + out.abs()) + 1e-30
    if fp8:
        tol = tol + 4 * fp8[0] ** 0.5 * 2.0 ** -18 * fp8[1] * (~lse.isneginf()[..., None])
    bad = (got_out - out).abs() / tol
    worst = float(bad.max()) if bad.numel() else 0.0
    assert worst <= 1.0, f"{what}: out {worst:.3f} of its bound"
    fin = ~lse.isneginf()
    if fin.any():
        d = float(((got_lse - lse)[fin].abs() / (d_s + 8 * U32 * lse[fin].abs() + 2.0 ** -20)).max())
        assert d <= 1.0, f"{what}: lse {d:.3f} of its bound"
