"""The binding without torch: loading and planning need none."""

import os
import subprocess
import sys

from paged_kv_decode_30_b200 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PLAN = """
params = B.make_params(batch=4, q_len=1, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                       max_pages_per_seq=8, num_pages=64, scale=0.1, max_kv_len=128)
assert B.load().pda_abi_version() == 3
assert B.choose_num_splits(params, 148) >= 1
assert B.status_string(0)
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_loads_and_plans_without_torch():
    build_mod.build()
    run("import sys; sys.modules['torch'] = None\n"
        "from paged_kv_decode_30_b200 import binding as B\n" + PLAN)


def test_importing_the_binding_does_not_import_torch():
    build_mod.build()
    run("import sys\nfrom paged_kv_decode_30_b200 import binding as B\n" + PLAN +
        "assert 'torch' not in sys.modules")


def test_latent_calls_after_an_import_before_torch():
    """Torch arrives after the binding: the calls' checks find it."""
    build_mod.build()
    run("""
from paged_kv_decode_30_b200 import binding as B
import torch
t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
i = torch.zeros(2, dtype=torch.int32)
for call in (lambda: B.latent_prefill_attn(t(5, 2, 192), t(5, 2, 256), t(5, 64), i, i, scale=1.0),
             lambda: B.paged_latent_decode(t(1, 1, 4, 288), t(3, 8, 256), t(3, 8, 32), i.view(1, 2), i[:1], scale=1.0),
             lambda: B.paged_latent_append(t(5, 256), t(5, 32), i, i.view(1, 2), i[:1], t(3, 8, 256), t(3, 8, 32)),
             lambda: B.paged_latent_gather(t(3, 8, 256), t(3, 8, 32), i.view(1, 2), i, total_rows=5)):
    B.torch = None
    try:
        call()
    except ValueError as e:
        assert "current CUDA device" in str(e), e
    else:
        raise AssertionError("host tensors were taken")
""")
