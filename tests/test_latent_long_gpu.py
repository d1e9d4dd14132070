"""Latent decode over long ranges: many tiles of one sequence a CTA, weights of very
different sizes, values with a mean, against the definition in 64 bits.

Every sequence of a batch is the same one (the page table's rows repeat), and there are
two to three sequences a team, so that CTAs walk whole sequences as well as pieces."""

import math

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from tests import latent_util as L

pytestmark = pytest.mark.gpu

PAGE = 64


def clear():
    torch.cuda.synchronize()
    err = B.last_device_error()
    assert err == 0, B.STATUS.get(err, err)


def batch_of(rows, fp8, most):
    """Two and a half sequences for each team of CTAs (a CTA an SM; 32 packed rows a CTA
    over FP8 caches, 64 over bf16 ones)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = max(1, math.ceil(rows / (32 if fp8 else 64)))
    return min(most, sms // tiles * 5 // 2)


def cache(n, R, Dr, fp8, seed, scores=None, uneven=False):
    """n tokens whose latents have a mean of 1 (uneven: times 2^-3 .. 2^3 by rows), in
    shuffled pages. scores: element 0 of the rotated parts, the others being 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = 1 + 0.5 * torch.randn((n, R), generator=g, device="cuda")
    if uneven:
        c *= torch.exp2(torch.randint(-3, 4, (n, 1), generator=g, device="cuda").float())
    if scores is None:
        r = torch.randn((n, Dr), generator=g, device="cuda")
    else:
        r = torch.zeros((n, Dr), device="cuda")
        r[:, 0] = scores.cuda()
    r = r.to(torch.bfloat16)
    pages = (n + PAGE - 1) // PAGE
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    lat = torch.zeros((pages, PAGE, R), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    rope = torch.zeros((pages, PAGE, Dr), dtype=torch.bfloat16, device="cuda")
    sc = torch.zeros((pages, PAGE), dtype=torch.uint8, device="cuda") if fp8 else None
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    B.paged_latent_append(c.to(torch.bfloat16), r, off, table[None], off[:1], lat, rope, latent_scales=sc)
    slot = table.long()[torch.arange(n, device="cuda") // PAGE] * PAGE + torch.arange(n, device="cuda") % PAGE
    rows = lat.view(-1, R)[slot]
    exps = None
    if fp8:
        exps = sc.view(-1)[slot].double() - 127
        val = rows.view(torch.float8_e4m3fn).double() * torch.exp2(exps)[:, None]
    else:
        val = rows.double()
    return dict(latent=lat, rope=rope, scales=sc, table=table, n=n, c=val, r=r.double(), exps=exps)


def definition(q, ch, scale, pos, window=0):
    """q bf16 [rows, R + Dr] at positions pos [rows]: out, lse, mean |v|, sum of p 2^e (FP8)
    and the largest scale * sum |q k|."""
    q = q.double()
    R = ch["c"].shape[1]
    s = scale * (q[:, :R] @ ch["c"].T + q[:, R:] @ ch["r"].T)
    j = torch.arange(ch["n"], device="cuda")
    hidden = j > pos[:, None]
    if window > 0:
        hidden |= j <= pos[:, None] - window
    s[hidden] = -math.inf
    lse = torch.logsumexp(s, dim=1)
    p = torch.exp(s - lse[:, None])
    big = 0.0
    for a in range(0, q.shape[0], 16):
        x = q[a:a + 16].abs()
        big = max(big, float((x[:, :R] @ ch["c"].abs().T + x[:, R:] @ ch["r"].abs().T).max()) * scale)
    weight = (p * torch.exp2(ch["exps"])).sum(1) if ch["exps"] is not None else None
    return p @ ch["c"], lse, p @ ch["c"].abs(), weight, big


def check(o, l, ref, n, width, what):
    """o [B, rows, R], l [B, rows] of equal sequences. bf16: weights and the result are
    rounded to bf16 and the normaliser adds the rounded weights, 2^-8 (mean |v| + 2 |out|).
    FP8: a weight p 2^e is held to 2^-8 of itself, and what is rounded off beyond that is
    at most 2^-9 of the row's sum of p 2^e, times codes of up to 448; the normaliser is
    unrounded. The scores are off by d_s (width products in fp32, FP8 queries to 2^-21 of
    their row's largest), and a chain of n / 16 products is added up in fp32, each sum
    off by at most 2 U32 of it; the normaliser, n / 128 sums, and a factor of 2^-22 = 4 U32
    wherever a row's reference moves, at most once a tile."""
    out, lse, mean_abs, weight, big = ref
    o, l = o.double(), l.double()
    assert not o.isnan().any() and not l.isnan().any(), what
    d_s = width * L.U32 * big + (2.0 ** -20 * big if weight is not None else 0.0)
    tol = L.U16 * (mean_abs + 2 * out.abs()) + (2 * (d_s + width * L.U32) + n / 8 * L.U32) * (mean_abs + out.abs())
    if weight is not None:
        tol = tol + 2.0 ** -9 * 448 * weight[:, None]
    worst = float(((o - out).abs() / tol).max())
    off = float(((l - lse).abs() / (d_s + 8 * L.U32 * lse.abs() + n / 128 * 5 * L.U32 + 2.0 ** -20)).max())
    bias = float(((o - out).mean(dim=-1) / out.abs().mean(dim=-1)).abs().max())
    print(f"{what}: out {worst:.3f} of its bound, lse {off:.3f}, mean off by {bias:.5f}")
    assert worst <= 1.0 and off <= 1.0, f"{what}: out {worst:.3f}, lse {off:.3f} of their bounds"


def decode(q, ch, batch, scale, **kw):
    """The batch's outputs; q [q_len, H, width] for every sequence."""
    lens = torch.full((batch,), ch["n"], dtype=torch.int32, device="cuda")
    o, l = B.paged_latent_decode(q.expand(batch, *q.shape).contiguous(), ch["latent"], ch["rope"],
                                 ch["table"].expand(batch, -1).contiguous(), lens, scale=scale,
                                 latent_scales=ch["scales"], **kw)
    clear()
    return o.flatten(1, 2), l.flatten(1, 2)


# ---------------------------------------------------------------------------
# weights of very different sizes

def peak(n, p, at, sigma=0.0):
    """A flat tail (normally distributed scores) and one token of probability p."""
    t = sigma * torch.randn(n, generator=torch.Generator().manual_seed(3))
    t[at] = math.log(n * math.exp(sigma * sigma / 2) * p / (1 - p))
    return t


def combs(n):
    """Every fifth tile has a token 9 above the rest."""
    t = torch.zeros(n)
    t[77::640] = 9.0
    return t


def valley(n):
    """Scores that fall by 90 and rise by 110."""
    return torch.cat([torch.linspace(0, -90, n // 2), torch.linspace(-90, 20, n - n // 2)])


def stairs(n):
    """Ever smaller peaks over a flat floor."""
    t = torch.full((n,), -12.0)
    at = torch.arange(50, n, 997)
    t[at] = -torch.arange(len(at)) * 0.25
    return t.clamp(min=-12.0)


SCORES = [
    ("peak .8 first", 131072, lambda n: peak(n, 0.8, 0)),
    ("peak .8 last", 131072, lambda n: peak(n, 0.8, n - 1)),
    ("peak .8 in the middle", 131072, lambda n: peak(n, 0.8, n // 2, 0.35)),
    ("peak .9 first", 65536, lambda n: peak(n, 0.9, 5, 0.35)),
    ("peak .7 first", 65537, lambda n: peak(n, 0.7, 5)),
    ("combs", 50001, combs),
    ("valley", 30000, valley),
    ("stairs", 60000, stairs),
]


@pytest.mark.parametrize("uneven", [False, True], ids=["even", "uneven"])
@pytest.mark.parametrize("R,Dr,heads", [(512, 64, 128), (512, 64, 16), (256, 32, 32), (256, 64, 5)])
@pytest.mark.parametrize("case", range(len(SCORES)))
def test_fp8_decode_keeps_long_tails(case, R, Dr, heads, uneven):
    """Weights far below the largest count in full when there are enough of them."""
    name, n, scores = SCORES[case]
    ch = cache(n, R, Dr, True, 40 + case, scores(n), uneven)
    q = torch.zeros((1, heads, R + Dr), dtype=torch.bfloat16, device="cuda")
    q[0, :, R] = 1 - torch.arange(heads, device="cuda") / (16.0 * heads)   # peaks of 0.6 to 0.9
    o, l = decode(q, ch, batch_of(heads, True, 100), 1.0)
    ref = definition(q[0], ch, 1.0, torch.full((heads,), n - 1, device="cuda"))
    check(o, l, ref, n, R + Dr, f"{name}, {R}, {heads} heads")


# ---------------------------------------------------------------------------
# whole sequences of many tiles a CTA, in every variant of the kernel

VARIANTS = [  # FP8, latent_dim, rope_dim, heads: 16, 32, 64 (bf16) packed rows a CTA, one or two CTAs a team
    (False, 512, 64, 16), (False, 512, 64, 20), (False, 512, 32, 64), (False, 512, 64, 128),
    (False, 256, 64, 5), (False, 256, 32, 32), (False, 256, 64, 40),
    (True, 512, 64, 16), (True, 512, 64, 20), (True, 512, 32, 64),
    (True, 256, 64, 5), (True, 256, 32, 32), (True, 256, 64, 40),
]


@pytest.mark.parametrize("n", [2049, 6000, 20001])
@pytest.mark.parametrize("fp8,R,Dr,heads", VARIANTS)
def test_decode_walks_long_sequences(fp8, R, Dr, heads, n):
    ch = cache(n, R, Dr, fp8, n, uneven=True)
    g = torch.Generator(device="cuda").manual_seed(heads)
    q = torch.randn((1, heads, R + Dr), generator=g, device="cuda").to(torch.bfloat16)
    scale = (128 + Dr) ** -0.5 / 2
    o, l = decode(q, ch, batch_of(heads, fp8, 400), scale)
    ref = definition(q[0], ch, scale, torch.full((heads,), n - 1, device="cuda"))
    check(o, l, ref, n, R + Dr, f"{n}, {R}, {heads} heads")


def levels(n, seed):
    """Every tile at a level of its own, between 25 below and 5 above, more or less flat."""
    g = torch.Generator().manual_seed(seed)
    tiles = (n + 127) // 128
    at = torch.rand((tiles, 1), generator=g) * 30 - 25
    return (at + torch.rand((tiles, 1), generator=g) * 2 * torch.randn((tiles, 128), generator=g)).flatten()[:n]


@pytest.mark.parametrize("kind", ["rising", "falling", "waves", "flat", "levels 1", "levels 2", "levels 3"])
@pytest.mark.parametrize("fp8,R,Dr,heads", VARIANTS)
def test_decode_moves_its_reference_in_long_sequences(fp8, R, Dr, heads, kind):
    """Rising: by 8 a tile, so that the accumulators move in every tile."""
    n = 12000
    j = torch.arange(n).float()
    scores = {"rising": j / 16, "falling": -j / 16, "flat": torch.zeros(n),
              "waves": 30 * torch.sin(j / 500) + j / 1000}.get(kind)
    if scores is None:
        scores = levels(n, int(kind.split()[1]))
    ch = cache(n, R, Dr, fp8, 77, scores, uneven=True)
    q = torch.zeros((1, heads, R + Dr), dtype=torch.bfloat16, device="cuda")
    q[0, :, R] = 1 - torch.arange(heads, device="cuda") / (2.0 * heads)
    o, l = decode(q, ch, batch_of(heads, fp8, 400), 1.0)
    ref = definition(q[0], ch, 1.0, torch.full((heads,), n - 1, device="cuda"))
    check(o, l, ref, n, 2, f"{kind}, {R}, {heads} heads")   # (a score is one product, and scaled)


@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("fp8,R,Dr,heads", VARIANTS)
def test_decode_walks_long_sequences_of_many_lengths(fp8, R, Dr, heads, window):
    """Verify rows, and beginnings of one sequence: items of many sizes follow one another in a CTA."""
    n, q_len = 9000, 3
    ch = cache(n, R, Dr, fp8, 31, uneven=True)
    g = torch.Generator(device="cuda").manual_seed(heads)
    q = torch.randn((q_len, heads, R + Dr), generator=g, device="cuda").to(torch.bfloat16)
    scale = (128 + Dr) ** -0.5 / 2
    sizes = [9000, 2, 4097, 0, 130, 8999, 6400, 1]
    batch = batch_of(q_len * heads, fp8, 400) // 8 * 8
    lens = torch.tensor(sizes * (batch // 8), dtype=torch.int32)[torch.randperm(batch, generator=torch.Generator().manual_seed(2))]
    o, l = B.paged_latent_decode(q.expand(batch, *q.shape).contiguous(), ch["latent"], ch["rope"],
                                 ch["table"].expand(batch, -1).contiguous(), lens.cuda(), scale=scale,
                                 causal_offset=L.BOTTOM_RIGHT, window=window, latent_scales=ch["scales"])
    clear()
    for size in sizes:
        rows = (lens == size).cuda()
        keep = [i for i in range(q_len) if size - q_len + i >= 0]   # rows that see a key
        none = [i for i in range(q_len) if i not in keep]
        assert not bool(o[rows][:, none].any()) and bool(l[rows][:, none].isneginf().all())
        if keep:
            part = dict(ch, n=size, **{k: ch[k][:size] for k in ("c", "r", "exps") if ch[k] is not None})
            pos = torch.tensor([size - q_len + i for i in keep], device="cuda").repeat_interleave(heads)
            ref = definition(q[keep].flatten(0, 1), part, scale, pos, window)
            check(o[rows][:, keep].flatten(1, 2), l[rows][:, keep].flatten(1, 2), ref, size, R + Dr,
                  f"{size} of many, {R}, {heads} heads")
