"""The library-owned workspaces of paged_decode_attn and paged_latent_decode are two:
a latent call leaves that of a captured paged_decode_attn alone."""

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from paged_kv_decode_30_b200 import workloads as W
from tests import gpu_util as U
from tests.test_latent_gpu import _decode, _decode_inputs, bits, clear, cuda

pytestmark = pytest.mark.gpu


def test_a_latent_call_beside_a_captured_call_on_the_library_workspace():
    wl = W.Workload(name="beside_latent", batch=16, num_q_heads=32, num_kv_heads=8, head_dim=128,
                    page_size=16, kv_lens=("uniform", 300, 2500), seed=52)
    t = U.to_device(W.generate(wl))
    call = lambda: B.paged_decode_attn(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["kv_lens"],
                                       num_kv_heads=wl.num_kv_heads, scale=W.scale_of(wl), num_splits=4,
                                       library_workspace=True)
    want = [x.clone() for x in call()[:2]]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()[:2]
    ch, q, scale = _decode_inputs([3000, 70, 1500], 1, 64, 512, 64, 64, False, 6)   # a larger workspace
    d, q = cuda(ch), q.cuda()
    latent = _decode(d, q, scale)
    for _ in range(3):
        o, l = _decode(d, q, scale, library_workspace=True)
        junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")   # takes what was given back
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(o), bits(latent[0])) and torch.equal(bits(l), bits(latent[1]))
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, want))
        del junk
    clear()
