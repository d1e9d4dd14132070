"""NaN and infinities that a row of latent attention sees reach its results; the
others keep theirs."""

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from tests import latent_util as L
from tests.test_latent_gpu import _decode, _decode_inputs, _fp8_of, _prefill_inputs, clear, cuda

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# lengths (sequence 1 is the one with the value), its token: in one CTA's range, cut in two
# to four, cut in many
RANGES = {"whole": ([40, 100, 7], 61), "few": ([3000] * 60 + [5], 200), "many": ([900, 20000], 12345)}


def slot(ch, b, j):
    return int(ch["page_table"][b, j // ch["page"]]) * ch["page"] + j % ch["page"]


def others(o, l, ref, rows, what, fp8):
    """The rows (mask [B, q_len, H]) that do not see the value are within their bounds."""
    pick = lambda t: t[rows]
    L.check(o.cpu()[rows], l.cpu()[rows], (pick(ref[0]), pick(ref[1]), pick(ref[2]), ref[3]), 576, what, fp8)


@pytest.mark.parametrize("where", ["latent", "rope nan", "rope inf"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("name", RANGES)
def test_decode_of_a_key_that_is_not_finite(name, fp8, where):
    """Every row of its sequence is NaN, however the sequence is cut; the others keep their results."""
    lens, j = RANGES[name]
    ch, q, scale = _decode_inputs(lens, 1, 20, 512, 64, 64, fp8, 5)
    ref = L.decode_reference(q, ch, scale, L.OFF, 0)
    at = slot(ch, 1, j)
    if where == "latent":
        ch["latent"].view(-1, 512)[at, 77] = 0x7F if fp8 else NAN
    else:
        ch["rope"].view(-1, 64)[at, 3] = INF if where == "rope inf" else NAN
        q[1, :, :, 512 + 3] = q[1, :, :, 512 + 3].abs() + 0.5   # the score is +inf
    o, l = _decode(cuda(ch), q, scale)
    clear()
    assert bool(o[1].isnan().all())
    assert not bool((l[1].isfinite() | l[1].isneginf()).any())
    rows = torch.ones(l.shape, dtype=torch.bool)
    rows[1] = False
    others(o, l, ref, rows, where, _fp8_of(ch) if fp8 else None)


@pytest.mark.parametrize("fp8,value", [(False, NAN), (False, INF), (True, NAN), (True, INF)])
@pytest.mark.parametrize("name", RANGES)
def test_decode_of_a_query_that_is_not_finite(name, fp8, value):
    """The row of that query is NaN (with an infinite element some keys' scores are +inf),
    the other heads are not."""
    lens, _ = RANGES[name]
    ch, q, scale = _decode_inputs(lens, 1, 20, 512, 64, 64, fp8, 6)
    ref = L.decode_reference(q, ch, scale, L.OFF, 0)
    q[1, 0, 5, 100] = value
    q[1, 0, 19, 512 + 40] = value
    o, l = _decode(cuda(ch), q, scale)
    clear()
    rows = torch.ones(l.shape, dtype=torch.bool)
    rows[1, 0, 5] = rows[1, 0, 19] = False
    assert bool(o.cpu()[~rows].isnan().all())
    assert not bool((l.cpu()[~rows].isfinite() | l.cpu()[~rows].isneginf()).any())
    others(o, l, ref, rows, "query", _fp8_of(ch) if fp8 else None)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_of_a_query_that_sees_nothing_and_is_not_finite(fp8):
    """A row without keys gives 0 and -inf whatever its query holds."""
    ch, q, scale = _decode_inputs([2, 0, 300], 4, 8, 512, 64, 64, fp8, 7)
    ref = L.decode_reference(q, ch, scale, L.BOTTOM_RIGHT, 0)
    q[0, :2] = NAN
    q[1] = INF
    o, l = _decode(cuda(ch), q, scale, causal_offset=L.BOTTOM_RIGHT)
    clear()
    L.check(o, l, ref, 576, "no keys", _fp8_of(ch))


@pytest.mark.parametrize("where", ["key nan", "rope nan", "rope inf", "query nan", "query inf"])
@pytest.mark.parametrize("q_lens,kv_lens,j", [([90, 5], [90, 5], 40), ([5, 700], [9, 1500], 1000)])
def test_prefill_of_values_that_are_not_finite(q_lens, kv_lens, j, where):
    """Rows that see such a score are NaN; rows before the key, other heads and sequences are not."""
    q, kv, r, scale = _prefill_inputs(q_lens, kv_lens, 3, 64, 9)
    ref = L.prefill_reference(q, kv, r, q_lens, kv_lens, scale, L.BOTTOM_RIGHT, 0)
    b = q_lens.index(max(q_lens))
    q0, k0 = sum(q_lens[:b]), sum(kv_lens[:b])
    hit = torch.zeros(ref[1].shape, dtype=torch.bool)
    sees = torch.arange(q_lens[b]) + kv_lens[b] - q_lens[b] >= j
    if where == "key nan":
        kv[k0 + j, 1, 7] = NAN
        hit[q0:q0 + q_lens[b], 1] = sees
    elif where.startswith("rope"):
        r[k0 + j, 9] = INF if where == "rope inf" else NAN
        q[q0:q0 + q_lens[b], :, 128 + 9] = 1.0
        ref = L.prefill_reference(q, kv, r.nan_to_num(0.0, 0.0), q_lens, kv_lens, scale, L.BOTTOM_RIGHT, 0)
        hit[q0:q0 + q_lens[b]] = sees[:, None]
    else:
        q[q0 + 33, 2, 11] = NAN if where == "query nan" else INF
        hit[q0 + 33, 2] = True
    o, l = (t.cpu() for t in B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), L.offsets(q_lens).cuda(),
                                                   L.offsets(kv_lens).cuda(), scale=scale))
    clear()
    assert bool(o[hit].isnan().all())
    assert not bool((l[hit].isfinite() | l[hit].isneginf()).any())
    L.check(o[~hit], l[~hit], (ref[0][~hit], ref[1][~hit], ref[2][~hit], ref[3]), 192, where)
