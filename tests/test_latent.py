"""Latent-cache entry points: what they refuse, on the host (no GPU needed)."""

import ctypes

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from paged_kv_decode_30_b200 import build as build_mod
from tests import latent_util as L

OK = ctypes.c_void_p(1 << 20)     # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD4 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def rows_params(**over):
    kw = dict(batch=2, total_rows=10, latent_dim=512, rope_dim=64, page_size=64, max_pages_per_seq=4,
              num_pages=9, kv_dtype=0, latent_stride=512, rope_stride=64, latent_scales=1 << 20)
    kw.update(over)
    p = B.PdaLatentRowsParams()
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def decode_params(**over):
    kw = dict(batch=2, q_len=1, num_heads=16, latent_dim=512, rope_dim=64, page_size=64,
              max_pages_per_seq=4, num_pages=9, scale=0.1, causal_offset=-1, window=0, kv_dtype=0,
              flags=0, latent_scales=1 << 20)
    kw.update(over)
    p = B.PdaLatentParams()
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def prefill_params(**over):
    kw = dict(batch=2, total_q=10, total_kv=20, max_q_len=10, num_heads=4, head_dim=128, rope_dim=64,
              k_rope_stride=64, scale=0.1, causal_offset=-2, window=0)
    kw.update(over)
    p = B.PdaLatentPrefillParams()
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def append(lib, p, latent=OK, rope=OK, ro=OK, pt=OK, kl=OK, lp=OK, rp=OK):
    return lib.paged_latent_append(latent, rope, ro, pt, kl, p and ctypes.byref(p), lp, rp, None)


def gather(lib, p, latent=OK, rope=OK, ro=OK, pt=OK, kl=OK, lp=OK, rp=OK):
    return lib.paged_latent_gather(lp, rp, pt, ro, kl, p and ctypes.byref(p), latent, rope, None)


def decode(lib, p, q=OK, lp=OK, rp=OK, pt=OK, kl=OK, out=OK, lse=OK):
    return lib.paged_latent_decode(q, lp, rp, pt, kl, p and ctypes.byref(p), out, lse, None)


def prefill(lib, p, q=OK, kv=OK, kr=OK, qo=OK, ko=OK, out=OK, lse=OK):
    return lib.latent_prefill_attn(q, kv, kr, qo, ko, p and ctypes.byref(p), out, lse, None)


@pytest.mark.parametrize("call", [append, gather])
@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), 1), (dict(total_rows=-1), 1), (dict(latent_dim=0), 1), (dict(rope_dim=0), 1),
    (dict(page_size=0), 1), (dict(max_pages_per_seq=0), 1), (dict(num_pages=0), 1),
    (dict(kv_dtype=3), 1), (dict(kv_dtype=-1), 1), (dict(max_pages_per_seq=1 << 26), 1),
    (dict(num_pages=1 << 26), 1), (dict(latent_stride=504), 1), (dict(rope_stride=56), 1),
    (dict(latent_dim=384), 2), (dict(latent_dim=128), 2), (dict(rope_dim=128), 2),
    (dict(page_size=4), 2), (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(kv_dtype=2), 2),
    (dict(latent_stride=516), 3), (dict(rope_stride=66), 3),
    (dict(kv_dtype=1, latent_scales=None), 1),
])
def test_rows_refusals(lib, call, over, status):
    assert call(lib, rows_params(**over)) == status


@pytest.mark.parametrize("call", [append, gather])
def test_rows_pointers(lib, call):
    assert call(lib, None) == 1
    for name in ("latent", "rope", "ro", "pt", "lp", "rp"):
        assert call(lib, rows_params(), **{name: None}) == 1, name
    for name in ("latent", "rope", "lp", "rp"):
        assert call(lib, rows_params(), **{name: ODD}) == 3, name
    for name in ("ro", "pt", "kl"):
        assert call(lib, rows_params(), **{name: ODD4}) == 3, name
    assert append(lib, rows_params(), kl=None) == 1
    for over in (dict(batch=0), dict(total_rows=0)):  # nothing to do, nothing looked at
        assert call(lib, rows_params(**over), None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), 1), (dict(q_len=0), 1), (dict(num_heads=0), 1), (dict(latent_dim=0), 1),
    (dict(rope_dim=-4), 1), (dict(page_size=0), 1), (dict(max_pages_per_seq=0), 1),
    (dict(num_pages=0), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(causal_offset=-3), 1), (dict(kv_dtype=7), 1),
    (dict(flags=2), 1), (dict(max_pages_per_seq=1 << 26), 1), (dict(num_pages=1 << 26), 1),
    (dict(kv_dtype=1, latent_scales=None), 1),
    (dict(latent_dim=384), 2), (dict(rope_dim=16), 2), (dict(page_size=4), 2), (dict(page_size=24), 2),
    (dict(kv_dtype=2), 2), (dict(q_len=9), 2), (dict(num_heads=257), 2), (dict(batch=65536), 2),
])
def test_decode_refusals(lib, over, status):
    p = decode_params(**over)
    assert decode(lib, p) == status
    pointer_only = over.keys() & {"latent_scales"}
    if not pointer_only:
        assert lib.paged_latent_decode_workspace_bytes(ctypes.byref(p)) == ctypes.c_size_t(-1).value


def test_decode_pointers(lib):
    assert decode(lib, None) == 1
    for name in ("q", "lp", "rp", "pt", "kl", "out"):
        assert decode(lib, decode_params(), **{name: None}) == 1, name
    for name in ("q", "lp", "rp", "out"):
        assert decode(lib, decode_params(), **{name: ODD}) == 3, name
    for name in ("pt", "kl", "lse"):
        assert decode(lib, decode_params(), **{name: ODD4}) == 3, name
    assert decode(lib, decode_params(workspace=(1 << 20) + 16, workspace_bytes=1 << 20)) == 3
    assert decode(lib, decode_params(batch=0), None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), 1), (dict(total_q=-1), 1), (dict(total_kv=-1), 1), (dict(max_q_len=-1), 1),
    (dict(num_heads=0), 1), (dict(head_dim=0), 1), (dict(rope_dim=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(causal_offset=-3), 1), (dict(k_rope_stride=56), 1),
    (dict(head_dim=64), 2), (dict(rope_dim=128), 2), (dict(num_heads=257), 2), (dict(batch=65536), 2),
    (dict(k_rope_stride=68), 3),
])
def test_prefill_refusals(lib, over, status):
    assert prefill(lib, prefill_params(**over)) == status


def test_prefill_pointers(lib):
    assert prefill(lib, None) == 1
    for name in ("q", "kv", "kr", "qo", "ko", "out"):
        assert prefill(lib, prefill_params(), **{name: None}) == 1, name
    for name in ("q", "kv", "kr", "out"):
        assert prefill(lib, prefill_params(), **{name: ODD}) == 3, name
    for name in ("qo", "ko", "lse"):
        assert prefill(lib, prefill_params(), **{name: ODD4}) == 3, name
    for over in (dict(batch=0), dict(total_q=0), dict(max_q_len=0)):
        assert prefill(lib, prefill_params(**over), None, None, None, None, None, None, None) == 0


def test_binding_refuses_host_tensors():
    ch = L.cache([5], 8, 256, 32, False, 1)
    row = torch.zeros((5, 256), dtype=torch.bfloat16)
    off = L.offsets([5])
    with pytest.raises(ValueError):
        B.paged_latent_append(row, row[:, :32], off, ch["page_table"], ch["kv_lens"], ch["latent"],
                              ch["rope"])
    with pytest.raises(ValueError):
        B.paged_latent_gather(ch["latent"], ch["rope"], ch["page_table"], off, total_rows=5)
    q = torch.zeros((1, 1, 4, 288), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.paged_latent_decode(q, ch["latent"], ch["rope"], ch["page_table"], ch["kv_lens"], scale=1.0)
    q = torch.zeros((5, 2, 192), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.latent_prefill_attn(q, torch.zeros((5, 2, 256), dtype=torch.bfloat16),
                              torch.zeros((5, 64), dtype=torch.bfloat16), off, off, scale=1.0)


def test_lengths_near_32_bits(lib):
    """A position and the tile behind it fit 32 bits, or the call is refused."""
    over = dict(page_size=8, num_pages=9)
    size = lambda n: lib.paged_latent_decode_workspace_bytes(ctypes.byref(
        decode_params(batch=1, max_pages_per_seq=n, **over)))
    assert size((2 ** 31 - 136) // 8) != ctypes.c_size_t(-1).value
    assert size((2 ** 31 - 120) // 8) == ctypes.c_size_t(-1).value
    assert decode(lib, decode_params(batch=1, max_pages_per_seq=(2 ** 31 - 120) // 8, **over)) == 1


@pytest.mark.parametrize("over", [dict(window=1 << 31), dict(window=(1 << 32) + 5),
                                  dict(causal_offset=1 << 31), dict(causal_offset=-(1 << 32) - 1)])
def test_binding_refuses_masks_past_32_bits(over):
    with pytest.raises(ValueError, match="32 bits"):
        ch = L.cache([5], 8, 256, 32, False, 1)
        B.paged_latent_decode(torch.zeros((1, 1, 4, 288), dtype=torch.bfloat16), ch["latent"], ch["rope"],
                              ch["page_table"], ch["kv_lens"], scale=1.0, **over)
    with pytest.raises(ValueError, match="32 bits"):
        off = L.offsets([5])
        B.latent_prefill_attn(torch.zeros((5, 2, 192), dtype=torch.bfloat16),
                              torch.zeros((5, 2, 256), dtype=torch.bfloat16),
                              torch.zeros((5, 64), dtype=torch.bfloat16), off, off, scale=1.0, **over)


def test_quantiser_of_the_tests_at_its_borders():
    """The rule's borders by hand: 448 fits exponent 0, the next bf16 does not; zero and tiny
    rows take the least exponent, infinity the greatest."""
    x = torch.tensor([[448.0, 1.0], [450.0, 1.0], [0.0, -0.0], [1e-30, 0.0], [float("inf"), 1.0],
                      [float("nan"), 3.5]])
    codes, s = L.quantise(x)
    assert s.tolist() == [127, 128, 97, 97, 157, 120]
    assert codes[0, 0] == 0x7E and codes[4, 0] == 0x7E and codes[5, 0] == 0x7F and codes[5, 1] == 0x7E
