"""Latent-cache operators on the GPU against their 64-bit definitions."""

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from tests import latent_util as L

pytestmark = pytest.mark.gpu

BAD_PAGE = 6


def cuda(ch):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in ch.items()}


def clear():
    torch.cuda.synchronize()
    err = B.last_device_error()
    assert err == 0, B.STATUS.get(err, err)


# ---------------------------------------------------------------------------
# rows in and out

def _append_case(lens, before, page, R, Dr, fp8, seed, stride=None):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    table, num_pages = L.page_table([a + n for a, n in zip(before, lens)], page, g)
    x = torch.randn((total, stride or R + Dr), generator=g)
    x *= torch.exp2(torch.randint(-40, 41, (total, 1), generator=g).float())
    x = x.to(torch.bfloat16)
    fill = torch.randint(0, 255, (num_pages, page, R), generator=g)
    lat = fill.to(torch.uint8) if fp8 else fill.to(torch.int16).view(torch.bfloat16)
    rope = torch.randint(0, 255, (num_pages, page, Dr), generator=g).to(torch.int16).view(torch.bfloat16)
    sc = torch.randint(0, 255, (num_pages, page), generator=g).to(torch.uint8) if fp8 else None
    return dict(c=x[:, :R], r=x[:, x.shape[1] - Dr:], both=x, off=L.offsets(lens), table=table,
                before=torch.tensor(before, dtype=torch.int32), latent=lat, rope=rope, scales=sc, page=page)


def _append_reference(k):
    lat, rope = k["latent"].clone(), k["rope"].clone()
    sc = None if k["scales"] is None else k["scales"].clone()
    R, Dr, page = lat.shape[2], rope.shape[2], k["page"]
    for b in range(len(k["before"])):
        a, e = int(k["off"][b]), int(k["off"][b + 1])
        pos = int(k["before"][b]) + torch.arange(e - a)
        slot = k["table"][b].long()[pos // page] * page + pos % page
        rope.view(-1, Dr)[slot] = k["r"][a:e]
        if sc is None:
            lat.view(-1, R)[slot] = k["c"][a:e]
        else:
            codes, s = L.quantise(k["c"][a:e].float())
            lat.view(-1, R)[slot] = codes
            sc.view(-1)[slot] = s
    return lat, rope, sc


def _append_run(k):
    both = k["both"].cuda()
    R, Dr = k["latent"].shape[2], k["rope"].shape[2]
    lat, rope = k["latent"].cuda(), k["rope"].cuda()
    sc = None if k["scales"] is None else k["scales"].cuda()
    B.paged_latent_append(both[:, :R], both[:, both.shape[1] - Dr:], k["off"].cuda(), k["table"].cuda(),
                          k["before"].cuda(), lat, rope, latent_scales=sc)
    return lat, rope, sc


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("R,Dr,page,lens,before", [
    (512, 64, 64, [1], [0]),
    (256, 32, 8, [1, 1, 1, 1, 1], [0, 7, 8, 100, 63]),
    (512, 32, 16, [0, 5, 0, 17, 0], [3, 14, 0, 31, 9]),
    (256, 64, 256, [700, 0, 1], [255, 4, 256]),
    (512, 64, 128, [1500, 2501], [0, 1]),
    (512, 64, 32, [2] * 70, list(range(70))),
])
def test_append_bits(fp8, R, Dr, page, lens, before):
    k = _append_case(lens, before, page, R, Dr, fp8, 7 + R + page)
    got = _append_run(k)
    clear()
    for x, y in zip(got, _append_reference(k)):
        assert (x is None and y is None) or torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("count", [31, 32, 1023, 1024, 1500])
def test_append_many_sequences(count):
    """Each way of finding a row's sequence, at its ends; a third of them get no rows."""
    for most in (3, 6):   # few rows, and many
        lens = [i % most for i in range(count)]
        k = _append_case(lens, [(5 * i) % 11 for i in range(count)], 8, 256, 32, True, count)
        got = _append_run(k)
        clear()
        for x, y in zip(got, _append_reference(k)):
            assert torch.equal(bits(x), bits(y)), most


def test_append_fp8_borders():
    """Rows at the borders of the exponent rule, infinities, NaN, zeros and ties."""
    R = 256
    rows = torch.zeros((12, R))
    for i, v in enumerate([448.0, 450.0, 446.0, 0.0, 1e-38, 2.0 ** -60, 3e38, float("inf"), 2.0 ** 39, 1.75]):
        rows[i, 3] = v
    rows[8, 4:20] = torch.arange(16) * 2.0 ** 35
    rows[9, 5:37] = 1.0 + torch.arange(32) / 32.0 * 0.75   # ties at half steps
    rows[10, 0], rows[10, 255] = float("nan"), -7.0
    rows[11] = float("nan")
    k = _append_case([12], [5], 8, R, 32, True, 3)
    k["both"][:, :R] = rows.to(torch.bfloat16)
    k["c"] = k["both"][:, :R]
    got = _append_run(k)
    clear()
    want = _append_reference(k)
    assert torch.equal(got[2].cpu(), want[2])
    a, b = (t[0].cpu().view(torch.float8_e4m3fn).float() for t in (got, want))
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(bits(got[0])[~a.isnan()], bits(want[0])[~b.isnan()])


def test_append_wide_strides_and_rows_outside():
    """Slices of a wider projection; row_offsets that start behind the first row and
    end before the last one."""
    k = _append_case([3, 9], [30, 0], 16, 512, 64, False, 5, stride=1024)
    k["off"] = torch.tensor([2, 5, 11], dtype=torch.int32)
    got = _append_run(k)
    clear()
    for x, y in zip(got, _append_reference(k)):
        assert (x is None and y is None) or torch.equal(bits(x), bits(y))


def test_append_reports_bad_places():
    for what in ("page", "position", "length"):
        k = _append_case([4, 4], [0, 6], 8, 256, 32, True, 11)
        want = _append_reference(dict(k, off=torch.tensor([0, 4, 4], dtype=torch.int32)))
        if what == "page":
            k["table"][1, 0] = 1 << 20
            k["off"] = torch.tensor([0, 4, 6], dtype=torch.int32)
        elif what == "position":
            k["before"][1] = k["table"].shape[1] * 8
        else:
            k["before"][1] = -2
        got = _append_run(k)
        torch.cuda.synchronize()
        assert B.last_device_error() == BAD_PAGE, what
        for x, y in zip(got, want):
            assert torch.equal(bits(x), bits(y)), what


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("R,Dr,page,lens,starts", [
    (512, 64, 64, [1], [0]),
    (256, 32, 8, [0, 9, 33, 0, 1], [0, 0, 7, 3, 63]),
    (512, 64, 128, [2000, 1, 900], [100, 127, 0]),
    (256, 64, 16, [3] * 50, list(range(50))),
])
def test_gather(fp8, R, Dr, page, lens, starts):
    ch = L.cache([a + n for a, n in zip(starts, lens)], page, R, Dr, fp8, 23 + R, spread=6.0)
    d = cuda(ch)
    total = sum(lens)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    c, r = B.paged_latent_gather(d["latent"], d["rope"], d["page_table"], L.offsets(lens).cuda(),
                                 starts=st, total_rows=total, latent_scales=d["scales"])
    clear()
    want = [L.rows_of(ch, b, a + n) for b, (a, n) in enumerate(zip(starts, lens))]
    wc = torch.cat([x[0][a:] for x, a in zip(want, starts)])
    wr = torch.cat([x[1][a:] for x, a in zip(want, starts)])
    assert torch.equal(c.cpu().double(), wc) and torch.equal(r.cpu().double(), wr)


def test_gather_leaves_other_rows_alone():
    ch = cuda(L.cache([20, 11], 8, 256, 32, True, 2))
    out = torch.full((40, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([3, 13, 24], dtype=torch.int32, device="cuda")
    c, r = B.paged_latent_gather(ch["latent"], ch["rope"], ch["page_table"], off, latent_scales=ch["scales"],
                                 latent=out[:, :256], rope=out[:, 280:312])
    clear()
    seven = torch.full_like(out, 7.0)
    assert torch.equal(out[:3], seven[:3]) and torch.equal(out[24:], seven[24:])
    assert torch.equal(out[:, 256:280], seven[:, 256:280]) and torch.equal(out[:, 312:], seven[:, 312:])
    w = L.rows_of({k: v.cpu() if torch.is_tensor(v) else v for k, v in ch.items()}, 0, 10)
    assert torch.equal(c[3:13].cpu().double(), w[0]) and torch.equal(r[3:13].cpu().double(), w[1])


def test_gather_reports_bad_places():
    ch = cuda(L.cache([20, 11], 8, 256, 32, False, 2))
    ch["page_table"][1, 0] = -5
    out = torch.full((31, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    B.paged_latent_gather(ch["latent"], ch["rope"], ch["page_table"], L.offsets([20, 11]).cuda(),
                          latent=out, rope=torch.empty((31, 32), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert B.last_device_error() == BAD_PAGE
    assert bool((out[20:28] == 7.0).all()) and not bool((out[28:] == 7.0).all())


def test_rows_far_into_a_large_pool():
    """Rows whose byte offset in the pool passes 2^32."""
    page, num_pages = 256, 17000   # 4.35 M rows of 1024 bytes: 4.46 GB
    lat = torch.empty((num_pages, page, 512), dtype=torch.bfloat16, device="cuda")
    rope = torch.empty((num_pages, page, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[num_pages - 1, 16500]], dtype=torch.int32, device="cuda")
    x = torch.randn((300, 576), device="cuda").to(torch.bfloat16)
    off = L.offsets([300]).cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.paged_latent_append(x[:, :512], x[:, 512:], off, table, zero, lat, rope)
    c, r = B.paged_latent_gather(lat, rope, table, off, total_rows=300)
    q = torch.randn((1, 1, 16, 576), device="cuda").to(torch.bfloat16)
    o, l = B.paged_latent_decode(q, lat, rope, table, zero + 300, scale=0.07)
    clear()
    assert torch.equal(c, x[:, :512]) and torch.equal(r, x[:, 512:])
    assert torch.equal(lat[num_pages - 1, 5], x[5, :512]) and torch.equal(lat[16500, 0], x[256, :512])
    xd = x.double().cpu()
    ref = L.attend(q.view(16, 576).double().cpu(), xd, xd[:, :512], 0.07, torch.full((16,), 299), L.OFF, 0)
    L.check(o.view(16, 512), l.view(16), ref, 576, "far pages")


# ---------------------------------------------------------------------------
# decode

DECODE = [
    # lens, q_len, heads, R, Dr, page, causal, window
    ([1], 1, 1, 512, 64, 64, L.OFF, 0),
    ([777], 1, 20, 512, 64, 16, L.OFF, 0),
    ([0, 1, 127, 128, 129, 0], 1, 16, 512, 64, 64, L.OFF, 0),
    ([300, 5, 1000], 1, 128, 512, 64, 128, L.OFF, 0),
    ([511, 3, 0, 64], 1, 40, 256, 32, 8, L.OFF, 0),
    ([257, 900], 1, 64, 256, 64, 256, L.OFF, 0),
    ([130, 2, 0, 640], 3, 16, 512, 64, 128, L.BOTTOM_RIGHT, 0),
    ([130, 7, 0, 640], 8, 5, 512, 32, 32, L.BOTTOM_RIGHT, 100),
    ([400, 30], 2, 33, 512, 64, 64, 10, 0),
    ([400, 30], 4, 8, 256, 32, 16, 350, 77),
    ([1500], 1, 32, 512, 64, 64, L.OFF, 129),
    ([600, 64], 8, 20, 512, 64, 64, L.BOTTOM_RIGHT, 1),
    ([5000, 17, 1200], 1, 17, 512, 64, 64, L.OFF, 0),
    ([40] * 200, 1, 8, 512, 64, 16, L.OFF, 0),
    ([i % 7 for i in range(1500)], 1, 4, 256, 32, 8, L.OFF, 0),
    ([333, 70], 8, 256, 512, 64, 64, L.BOTTOM_RIGHT, 0),
    ([1300, 0, 1], 5, 23, 256, 64, 8, L.BOTTOM_RIGHT, 500),
    # several sequences a team: with up to 128 of them, more, and two CTAs a team
    ([(i * 397) % 1500 for i in range(100)], 1, 4, 256, 32, 32, L.OFF, 0),
    ([(i * 211) % 900 for i in range(180)], 2, 3, 256, 64, 64, L.BOTTOM_RIGHT, 0),
    ([(i * 397) % 1500 for i in range(60)], 1, 40, 512, 64, 64, L.OFF, 0),
]


def _decode_inputs(lens, q_len, heads, R, Dr, page, fp8, seed=0, gain=1.0):
    ch = L.cache(lens, page, R, Dr, fp8, 1000 + seed)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((len(lens), q_len, heads, R + Dr), generator=g) * gain).to(torch.bfloat16)
    return ch, q, (128 + Dr) ** -0.5


def _decode(d, q, scale, **kw):
    return B.paged_latent_decode(q.cuda(), d["latent"], d["rope"], d["page_table"], d["kv_lens"],
                                 scale=scale, latent_scales=d["scales"], **kw)


def _fp8_of(ch):
    return (int(ch["kv_lens"].max()) + 1, float(ch["values"].nan_to_num(0.0).abs().max())) \
        if ch["scales"] is not None else None


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case, fp8):
    lens, q_len, heads, R, Dr, page, causal, window = DECODE[case]
    ch, q, scale = _decode_inputs(lens, q_len, heads, R, Dr, page, fp8, case)
    o, l = _decode(cuda(ch), q, scale, causal_offset=causal, window=window)
    clear()
    ref = L.decode_reference(q, ch, scale, causal, window)
    L.check(o, l, ref, R + Dr, f"decode {case}", _fp8_of(ch))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_peaked_rising(fp8):
    """Scores that rise by hundreds along the keys: the running maximum moves in every tile."""
    ch, q, _ = _decode_inputs([1400, 390], 1, 24, 512, 64, 64, fp8, 3)
    n = ch["page"]
    for b in range(2):
        j = torch.arange(int(ch["kv_lens"][b]))
        slot = ch["page_table"][b].long()[j // n] * n + j % n
        ch["rope"].view(-1, 64)[slot, 0] = (j.float() / 4).to(torch.bfloat16)
    ch["rope_values"] = ch["rope"].view(-1, 64).double()
    q[..., 512] = 2.0
    o, l = _decode(cuda(ch), q, 0.5)
    clear()
    L.check(o, l, L.decode_reference(q, ch, 0.5, L.OFF, 0), 576, "peaked", _fp8_of(ch))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_does_not_depend_on_neighbours(fp8):
    """Each sequence alone gives what it gives in a batch, within both errors; and a
    repeated call gives the same bits."""
    lens = [900, 0, 33, 2100, 128]
    ch, q, scale = _decode_inputs(lens, 2, 48, 512, 64, 64, fp8, 5)
    d = cuda(ch)
    o, l = _decode(d, q, scale, causal_offset=L.BOTTOM_RIGHT)
    o2, l2 = _decode(d, q, scale, causal_offset=L.BOTTOM_RIGHT)
    assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(l), bits(l2))
    ref = L.decode_reference(q, ch, scale, L.BOTTOM_RIGHT, 0)
    for b in range(len(lens)):
        one = dict(d, page_table=d["page_table"][b:b + 1].contiguous(), kv_lens=d["kv_lens"][b:b + 1])
        ob, lb = _decode(one, q[b:b + 1], scale, causal_offset=L.BOTTOM_RIGHT)
        L.check(ob[0], lb[0], (ref[0][b], ref[1][b], ref[2][b], ref[3]), 576, f"alone {b}", _fp8_of(ch))
    clear()


def test_decode_scale_bytes_at_the_ends():
    """FP8 rows with the least and the greatest exponents side by side, and bytes
    outside the range, which read as its ends."""
    ch, q, scale = _decode_inputs([200], 1, 16, 256, 32, 16, True, 9)
    sc = ch["scales"].view(-1)
    slot = ch["page_table"][0].long()[torch.arange(200) // 16] * 16 + torch.arange(200) % 16
    sc[slot] = torch.randint(110, 128, (200,)).to(torch.uint8)
    sc[slot[::7]] = 97
    sc[slot[1::7]] = 0
    q = (q.float() / 64).to(torch.bfloat16)
    ch["values"] = L.values(ch["latent"].view(-1, 256), sc)
    o, l = _decode(cuda(ch), q, scale)
    clear()
    L.check(o, l, L.decode_reference(q, ch, scale, L.OFF, 0), 288, "ends", _fp8_of(ch))


def test_decode_without_lse_with_given_outputs_and_workspaces():
    ch, q, scale = _decode_inputs([1000, 70], 1, 32, 512, 64, 64, False, 6)
    d = cuda(ch)
    ref = L.decode_reference(q, ch, scale, L.OFF, 0)
    o, l = _decode(d, q, scale)
    out = torch.full_like(o, float("nan"))
    o1, l1 = _decode(d, q, scale, out=out, with_lse=False, library_workspace=True)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = _decode(d, q, scale, workspace=ws)
    o3, l3 = _decode(d, q, scale, flags=B.PDA_FLAG_NO_PDL)
    clear()
    assert l1 is None and o1 is out
    for x in (o1, o2, o3):
        assert torch.equal(bits(x), bits(o))
    L.check(o, l, ref, 576, "given")


def test_decode_workspace_too_small():
    ch, q, scale = _decode_inputs([1000, 70], 1, 32, 512, 64, 64, False, 6)
    p = B.PdaLatentParams(2, 1, 32, 512, 64, 64, ch["page_table"].shape[1], ch["latent"].shape[0], scale,
                          L.OFF, 0, 0, 0, None, None, 0)
    import ctypes
    need = B.load().paged_latent_decode_workspace_bytes(ctypes.byref(p))
    if need:
        with pytest.raises(B.PdaError) as e:
            _decode(cuda(ch), q, scale, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 4


def test_decode_workspace_elsewhere():
    ch, q, scale = _decode_inputs([1000, 70], 1, 32, 512, 64, 64, False, 6)
    d = cuda(ch)
    for ws in (torch.empty(64 << 20, dtype=torch.uint8),
               torch.empty(64 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            _decode(d, q, scale, workspace=ws)


def test_library_workspace_in_a_graph_is_refused():
    ch, q, scale = _decode_inputs([1000, 70], 1, 32, 512, 64, 64, False, 6)
    d, q = cuda(ch), q.cuda()
    o, l = _decode(d, q, scale, library_workspace=True)   # grown already
    x = torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(B.PdaError) as e:
            _decode(d, q, scale, out=o, lse=l, library_workspace=True)
        x += 1
    assert e.value.status == 4
    g.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1.0] * 4
    clear()


def test_two_graphs_of_one_call_at_once():
    """Two captures of the same call have workspaces of their own."""
    ch, q, scale = _decode_inputs([1900, 5, 640, 3000], 1, 64, 512, 64, 64, False, 33)
    d, q = cuda(ch), q.cuda()
    want = _decode(d, q, scale)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, torch.cuda.Stream(), _decode(d, q, scale)))
    for _ in range(20):
        for _, _, (o, l) in graphs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, _, (o, l) in graphs:
            assert torch.equal(bits(o), bits(want[0])) and torch.equal(bits(l), bits(want[1]))
    clear()


def test_outputs_of_another_stream():
    """A call on a given stream gets no block that the caller's stream is still to
    write: the results outlast the writes."""
    ch, q, scale = _decode_inputs([1000, 70], 1, 32, 512, 64, 64, False, 6)
    d, q = cuda(ch), q.cuda()
    want = _decode(d, q, scale)
    off = L.offsets([1000, 70]).cuda()
    rows = B.paged_latent_gather(d["latent"], d["rope"], d["page_table"], off, total_rows=1070)
    pq, kv, r, ps = (t.cuda() if torch.is_tensor(t) else t for t in _prefill_inputs([1000, 70], [1000, 70], 2, 64, 1))
    wide = B.latent_prefill_attn(pq, kv, r, off, off, scale=ps)
    s = torch.cuda.Stream()
    calls = [(lambda: _decode(d, q, scale, stream=s), want),
             (lambda: B.paged_latent_gather(d["latent"], d["rope"], d["page_table"], off, total_rows=1070, stream=s), rows),
             (lambda: B.latent_prefill_attn(pq, kv, r, off, off, scale=ps, stream=s), wide)]
    torch.cuda.synchronize()
    for call, results in calls:
        blocks = [torch.empty_like(t) for t in results]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for t in blocks:
            t.fill_(float("nan"))
        del blocks, t
        got = call()
        torch.cuda.synchronize()
        for x, y in zip(got, results):
            assert torch.equal(bits(x), bits(y))
    clear()


def test_calls_with_nothing_to_do():
    d = cuda(L.cache([20, 11], 8, 256, 32, False, 2))
    none = d["page_table"][:0], d["kv_lens"][:0]
    q = torch.zeros((0, 1, 4, 288), dtype=torch.bfloat16, device="cuda")
    o, l = B.paged_latent_decode(q, d["latent"], d["rope"], *none, scale=1.0)
    assert o.shape == (0, 1, 4, 256) and l.shape == (0, 1, 4)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    c, r = B.paged_latent_gather(d["latent"], d["rope"], d["page_table"], off, total_rows=0)
    assert c.shape == (0, 256) and r.shape == (0, 32)
    before = d["latent"].clone(), d["rope"].clone()
    B.paged_latent_append(c, r, off, d["page_table"], d["kv_lens"], d["latent"], d["rope"])
    q = torch.zeros((0, 2, 192), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((7, 2, 256), dtype=torch.bfloat16, device="cuda")
    o, l = B.latent_prefill_attn(q, kv, kv[:, 0, :64], off, off, scale=1.0)
    assert o.shape == (0, 2, 128) and l.shape == (0, 2)
    clear()
    assert torch.equal(bits(before[0]), bits(d["latent"])) and torch.equal(bits(before[1]), bits(d["rope"]))


def test_decode_reports_bad_places():
    for what in ("page", "long", "negative"):
        ch, q, scale = _decode_inputs([300, 50], 1, 16, 512, 64, 64, False, 8)
        d = cuda(ch)
        if what == "page":
            d["page_table"][0, 2] = 1 << 30
        else:
            d["kv_lens"][0] = 1 << 30 if what == "long" else -1
            d["page_table"].clamp_(min=0)
        o, l = _decode(d, q, scale)
        torch.cuda.synchronize()
        assert B.last_device_error() == BAD_PAGE, what
        ref = L.decode_reference(q, ch, scale, L.OFF, 0)
        L.check(o[1], l[1], (ref[0][1], ref[1][1], ref[2][1], ref[3]), 576, what)


def test_decode_on_streams_and_in_graphs():
    """Two calls at once on two streams; a captured call replayed on changed inputs;
    a captured call without a workspace of its own is refused."""
    cases = [_decode_inputs([1900, 5, 640], 1, 32, 512, 64, 64, fp8, 20 + fp8) for fp8 in (False, True)]
    ds = [cuda(c[0]) for c in cases]
    qs = [c[1].cuda() for c in cases]
    want = [_decode(d, q, c[2]) for d, q, c in zip(ds, qs, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for d, q, c, s in zip(ds, qs, cases, streams):
            with torch.cuda.stream(s):
                got.append(_decode(d, q, c[2]))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(bits(o), bits(wo)) and torch.equal(bits(l), bits(wl))
    o, l = B.paged_latent_decode(qs[0], ds[0]["latent"], ds[0]["rope"], ds[0]["page_table"],
                                 ds[0]["kv_lens"], scale=cases[0][2], stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(bits(o), bits(want[0][0]))
    graphs = []
    for d, q, c in zip(ds, qs, cases):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = _decode(d, q, c[2])
        graphs.append((g, res))
    lens = [d["kv_lens"].clone() for d in ds]
    for n in (1, 0):
        for d, ln in zip(ds, lens):
            d["kv_lens"].copy_(torch.tensor([100, 0, 640]) if n else ln)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (g, (o, l)), d, q, c in zip(graphs, ds, qs, cases):
            wo, wl = _decode(d, q, c[2])
            assert torch.equal(bits(o), bits(wo)) and torch.equal(bits(l), bits(wl))
    clear()


# ---------------------------------------------------------------------------
# prefill

PREFILL = [
    # q_lens, kv_lens, heads, Dr, causal, window
    ([1], [1], 1, 64, L.BOTTOM_RIGHT, 0),
    ([5, 0, 130], [5, 9, 131], 3, 64, L.BOTTOM_RIGHT, 0),
    ([128, 256, 257], [128, 256, 400], 2, 64, L.BOTTOM_RIGHT, 0),
    ([300, 7], [900, 0], 2, 32, L.BOTTOM_RIGHT, 0),
    ([40, 300], [10, 100], 2, 64, L.BOTTOM_RIGHT, 0),     # rows before the first key
    ([129, 64], [511, 640], 2, 64, L.OFF, 0),
    ([400, 3], [700, 3], 2, 64, L.BOTTOM_RIGHT, 150),
    ([400], [700], 1, 32, L.BOTTOM_RIGHT, 1),
    ([200, 100], [300, 50], 2, 64, 37, 0),
    ([260], [600], 1, 64, L.OFF, 33),
    ([1, 1, 1, 1], [1, 127, 128, 1025], 5, 64, L.BOTTOM_RIGHT, 0),
    ([700], [700], 1, 64, 650, 90),
    ([5, 0, 300], [0, 0, 0], 2, 64, L.BOTTOM_RIGHT, 0),                  # no keys at all
    ([1 + i % 7 for i in range(450)], [3 + i % 5 for i in range(450)], 2, 32, L.BOTTOM_RIGHT, 0),
    ([300, 1] + [2] * 190, [310, 400] + [9] * 190, 1, 64, L.BOTTOM_RIGHT, 0),   # 384 pairs of sequence and tile
]


def _prefill_inputs(q_lens, kv_lens, heads, Dr, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((sum(q_lens), heads, 128 + Dr), generator=g) * gain).to(torch.bfloat16)
    kv = torch.randn((sum(kv_lens), heads, 256), generator=g).to(torch.bfloat16)
    r = torch.randn((sum(kv_lens), Dr), generator=g).to(torch.bfloat16)
    return q, kv, r, (128 + Dr) ** -0.5


@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill(case):
    q_lens, kv_lens, heads, Dr, causal, window = PREFILL[case]
    q, kv, r, scale = _prefill_inputs(q_lens, kv_lens, heads, Dr, case)
    o, l = B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), L.offsets(q_lens).cuda(),
                                 L.offsets(kv_lens).cuda(), scale=scale, causal_offset=causal,
                                 window=window, max_q_len=max(q_lens))
    clear()
    ref = L.prefill_reference(q, kv, r, q_lens, kv_lens, scale, causal, window)
    L.check(o, l, ref, 128 + Dr, f"prefill {case}")


def test_prefill_peaked_rising():
    q, kv, r, _ = _prefill_inputs([300], [900], 2, 64, 77)
    r[:, 0] = (torch.arange(900) / 4).to(torch.bfloat16)
    q[..., 128] = 2.0
    off = [L.offsets([n]).cuda() for n in (300, 900)]
    o, l = B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), *off, scale=0.5)
    clear()
    L.check(o, l, L.prefill_reference(q, kv, r, [300], [900], 0.5, L.BOTTOM_RIGHT, 0), 192, "peaked")


def test_prefill_rows_outside_and_strided_rope():
    """Offsets that start behind the first row and end before the last, NaN in the rows
    between, k_rope as a slice of a wider tensor, and max_q_len that is not tight."""
    q_lens, kv_lens = [70, 0, 200], [90, 130, 333]
    q, kv, r, scale = _prefill_inputs(q_lens, kv_lens, 2, 64, 5)
    ref = L.prefill_reference(q, kv, r, q_lens, kv_lens, scale, L.BOTTOM_RIGHT, 0)
    nan = float("nan")
    pad = lambda t, n: torch.cat([torch.full((n, *t.shape[1:]), nan), t, torch.full((n + 200, *t.shape[1:]), nan)]).to(torch.bfloat16)
    wide = torch.full((sum(kv_lens) + 212, 576), nan, dtype=torch.bfloat16)
    wide[6:6 + sum(kv_lens), 512:] = r
    out = torch.full((sum(q_lens) + 206, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sum(q_lens) + 206, 2), 7.0, device="cuda")
    B.latent_prefill_attn(pad(q, 3).cuda(), pad(kv, 6).cuda(), wide.cuda()[:, 512:],
                          (L.offsets(q_lens) + 3).cuda(), (L.offsets(kv_lens) + 6).cuda(), scale=scale,
                          out=out, lse=lse)
    clear()
    n = sum(q_lens)
    L.check(out[3:3 + n], lse[3:3 + n], ref, 192, "outside")
    for t in (out, lse):
        assert bool((t[:3] == 7).all()) and bool((t[3 + n:] == 7).all())


def test_prefill_computes_the_rows_of_max_q_len():
    """Rows past max_q_len are not computed; rows behind it keep what they held."""
    q_lens, kv_lens = [300, 20], [400, 20]
    q, kv, r, scale = _prefill_inputs(q_lens, kv_lens, 2, 64, 8)
    ref = L.prefill_reference(q, kv, r, q_lens, kv_lens, scale, L.BOTTOM_RIGHT, 0)
    out = torch.full((320, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    o, l = B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), L.offsets(q_lens).cuda(),
                                 L.offsets(kv_lens).cuda(), scale=scale, max_q_len=150, out=out)
    clear()
    for a, e in ((0, 150), (300, 320)):
        L.check(o[a:e], l[a:e], (ref[0][a:e], ref[1][a:e], ref[2][a:e], ref[3]), 192, "bounded")
    assert bool((o[150:300] == 7.0).all())


def test_prefill_reports_bad_offsets():
    q, kv, r, scale = _prefill_inputs([20, 20], [20, 20], 1, 64, 2)
    for qo, ko in (([0, 20, 60], [0, 20, 40]), ([0, 20, 40], [0, 20, 41]), ([0, 20, 10], [0, 20, 40]),
                   ([0, 20, 40], [0, 20, -3])):
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        o, l = B.latent_prefill_attn(q.cuda(), kv.cuda(), r.cuda(), t(qo), t(ko), scale=scale)
        torch.cuda.synchronize()
        assert B.last_device_error() == BAD_PAGE
        ref = L.prefill_reference(q[:20], kv[:20], r[:20], [20], [20], scale, L.BOTTOM_RIGHT, 0)
        L.check(o[:20], l[:20], ref, 192, "beside bad offsets")


def test_prefill_in_a_graph():
    q, kv, r, scale = _prefill_inputs([300, 77], [512, 77], 2, 64, 12)
    q, kv, r = q.cuda(), kv.cuda(), r.cuda()
    qo, ko = L.offsets([300, 77]).cuda(), L.offsets([512, 77]).cuda()
    want = B.latent_prefill_attn(q, kv, r, qo, ko, scale=scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = B.latent_prefill_attn(q, kv, r, qo, ko, scale=scale)
    for _ in range(2):
        got[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(bits(got[1]), bits(want[1]))
    clear()


# ---------------------------------------------------------------------------
# together

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_append_gather_prefill_decode_together(fp8):
    """A prompt goes into the cache, is read back, expanded and attended to; then two
    more tokens are appended and decoded. The last token's absorbed output, taken through
    the value up-projection, is what the expanded form gives for it: the same attention
    computed in 64 bits from the cache's own rows."""
    R, Dr, D, H, page = 512, 64, 128, 4, 32
    g = torch.Generator().manual_seed(31)
    prompt, new = [75, 130, 1], 2
    wk = (torch.randn((H, D, R), generator=g) / R ** 0.5).to(torch.bfloat16)
    wv = (torch.randn((H, D, R), generator=g) / R ** 0.5).to(torch.bfloat16)
    table, num_pages = L.page_table([n + new for n in prompt], page, g)
    table = table.cuda()
    lat = torch.zeros((num_pages, page, R), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    rope = torch.zeros((num_pages, page, Dr), dtype=torch.bfloat16, device="cuda")
    sc = torch.zeros((num_pages, page), dtype=torch.uint8, device="cuda") if fp8 else None
    x = torch.randn((sum(prompt), R + Dr), generator=g).to(torch.bfloat16).cuda()
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    off = L.offsets(prompt).cuda()
    B.paged_latent_append(x[:, :R], x[:, R:], off, table, lens, lat, rope, latent_scales=sc)
    lens += torch.tensor(prompt, dtype=torch.int32, device="cuda")
    c, r = B.paged_latent_gather(lat, rope, table, off, total_rows=sum(prompt), latent_scales=sc)
    if not fp8:
        assert torch.equal(c, x[:, :R]) and torch.equal(r, x[:, R:])
    both = torch.cat([wk, wv], 1).cuda()                       # [H, 2D, R]
    kv = torch.einsum("tr,hdr->thd", c.float(), both.float()).to(torch.bfloat16)
    q = torch.randn((sum(prompt), H, D + Dr), generator=g).to(torch.bfloat16).cuda()
    o, l = B.latent_prefill_attn(q, kv, r, off, off, scale=0.07, max_q_len=max(prompt))
    ref = L.prefill_reference(q.cpu(), kv.cpu(), r.cpu(), prompt, prompt, 0.07, L.BOTTOM_RIGHT, 0)
    L.check(o, l, ref, D + Dr, "prompt")
    y = torch.randn((3 * new, R + Dr), generator=g).to(torch.bfloat16).cuda()
    B.paged_latent_append(y[:, :R], y[:, R:], L.offsets([new] * 3).cuda(), table, lens, lat, rope,
                          latent_scales=sc)
    lens += new
    qn = torch.randn((3, new, H, D), generator=g)
    qr = torch.randn((3, new, H, Dr), generator=g)
    qa = torch.cat([torch.einsum("bihd,hdr->bihr", qn, wk.float()), qr], -1).to(torch.bfloat16).cuda()
    o, l = B.paged_latent_decode(qa, lat, rope, table, lens, scale=0.07, causal_offset=L.BOTTOM_RIGHT,
                                 latent_scales=sc)
    clear()
    total = [n + new for n in prompt]
    c, r = B.paged_latent_gather(lat, rope, table, L.offsets(total).cuda(), total_rows=sum(total),
                                 latent_scales=sc)
    ch = dict(page_table=table.cpu(), kv_lens=lens.cpu(), page=page, scales=sc,
              rope_values=rope.cpu().view(-1, Dr).double(),
              values=L.values(lat.cpu().view(-1, R), sc.cpu().view(-1)) if fp8 else lat.cpu().view(-1, R).double())
    want = L.decode_reference(qa.cpu(), ch, 0.07, L.BOTTOM_RIGHT, 0)
    L.check(o, l, want, R + Dr, "new tokens", _fp8_of(ch))
    # the rows that gather returned give the same attention, expanded
    at = 0
    for b, n in enumerate(total):
        cb, rb = c[at:at + n].double().cpu(), r[at:at + n].double().cpu()
        at += n
        o64, l64, *_ = L.attend(qa[b].reshape(new * H, -1).double().cpu(), torch.cat([cb, rb], 1), cb, 0.07,
                                L.positions(new, n, L.BOTTOM_RIGHT).repeat_interleave(H), L.BOTTOM_RIGHT, 0)
        assert torch.allclose(o64.view(new, H, -1), want[0][b], rtol=1e-12, atol=1e-12)
