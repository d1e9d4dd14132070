"""Prefill of ragged batches with and without a bound on the rows of a sequence: the same
bits, a similar time, and bad offsets recorded whichever way the work is numbered."""

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from tests import latent_util as L
from tests.test_latent_gpu import BAD_PAGE, _prefill_inputs, bits, clear

pytestmark = pytest.mark.gpu


def run(lens, heads, first=0, behind=0, **kw):
    """Equal queries and keys; rows in front and behind that belong to no sequence."""
    q, kv, r, scale = _prefill_inputs([first, *lens, behind], [first, *lens, behind], heads, 64, len(lens))
    off = (L.offsets(lens) + first).cuda()
    out = torch.full((q.shape[0], heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
    q, kv, r = q.cuda(), kv.cuda(), r.cuda()
    call = lambda **kw: B.latent_prefill_attn(q, kv, r, off, off, scale=scale, out=out, lse=lse, **kw)
    return call, (q, kv, r, scale, out, lse)


@pytest.mark.parametrize("first,behind", [(0, 0), (300, 1000)])
@pytest.mark.parametrize("lens,heads", [
    ([500] * 64, 2),                              # ranked with and without a bound
    ([(i * 379) % 1200 for i in range(100)], 1),  # ranked without, in order of rows
    ([3] * 2000 + [700], 1),                      # a search of three steps
    ([0, 0, 256, 0, 512, 1, 0, 255, 257, 0], 3),
    ([0] * 40 + [1500] + [0] * 40, 2),
])
def test_prefill_without_a_bound_on_its_rows(lens, heads, first, behind):
    call, (q, kv, r, scale, out, lse) = run(lens, heads, first, behind)
    want = [t.clone() for t in call(max_q_len=max(lens))]
    out.fill_(7.0)
    lse.fill_(7.0)
    got = call()
    clear()
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, want))
    n = sum(lens)
    for t in got:
        assert bool((t[:first] == 7).all()) and bool((t[first + n:] == 7).all())
    some = [b for b in range(len(lens)) if lens[b]][:8] + [max(range(len(lens)), key=lambda b: lens[b])]
    off = [first + sum(lens[:b]) for b in range(len(lens) + 1)]
    cq, ck, cr = q.cpu(), kv.cpu(), r.cpu()
    for b in some:
        s = slice(off[b], off[b + 1])
        ref = L.prefill_reference(cq[s], ck[s], cr[s], [lens[b]], [lens[b]], scale, L.BOTTOM_RIGHT, 0)
        L.check(got[0][s], got[1][s], ref, 192, f"sequence {b}")


def test_prefill_without_a_bound_takes_no_longer_by_the_square():
    """64 prompts of 500 rows: 3024 CTAs of which 2048 have work, not 128 000. Half again as
    long as with the bound would be the idle ones' share if they cost what the others do."""
    call, _ = run([500] * 64, 16)
    times = {}
    for bound in (500, None):
        call(max_q_len=bound)
        each = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call(max_q_len=bound)
            b.record()
            torch.cuda.synchronize()
            each.append(a.elapsed_time(b))
        times[bound] = sorted(each)[4]
    clear()
    assert times[None] < 2 * times[500], times


@pytest.mark.parametrize("count", [300, 600])
@pytest.mark.parametrize("what", ["falling", "far", "negative", "keys"])
def test_prefill_reports_bad_offsets_of_any_sequence(what, count):
    q, kv, r, scale = _prefill_inputs([10] * count, [10] * count, 1, 64, 2)
    for at in (1, count // 2, count):
        qo, ko = L.offsets([10] * count), L.offsets([10] * count)
        if what == "falling":
            qo[at] = qo[at - 1] - 3
        elif what == "far":
            qo[at] = 1 << 30
        elif what == "negative":
            qo[at] = -(1 << 30)
        else:
            ko[at] = 10 * count + 1
        B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), qo.cuda(), ko.cuda(), scale=scale)
        torch.cuda.synchronize()
        assert B.last_device_error() == BAD_PAGE, (what, at)


def test_prefill_with_offsets_that_decrease_writes_no_rows_of_others():
    """Empty sequences far behind the units that a search of unordered offsets may give them: their
    rows would lie in front of them. No sequence has rows, so out holds what it held."""
    count = 640
    q, kv, r, scale = _prefill_inputs([20000], [20000], 1, 64, 3)
    qo = torch.full((count + 1,), 20000, dtype=torch.int32)
    qo[::7] = 1                      # up and down all the way; no sequence has rows
    qo[1::7] = 1
    ko = torch.zeros(count + 1, dtype=torch.int32)
    ko[:-1][(qo[:-1] == 1) & (qo[1:] > 1)] = 5   # those that go up have keys that go down
    assert not any(qo[b] < qo[b + 1] and ko[b] <= ko[b + 1] for b in range(count))
    out = torch.full((20000, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), qo.cuda(), ko.cuda(), scale=scale, out=out)
    torch.cuda.synchronize()
    assert B.last_device_error() == BAD_PAGE
    assert bool((out == 7.0).all())
