"""Calls of the latent entry points that their documentation allows or refuses, one by one."""

import pytest
import torch

from paged_kv_decode_30_b200 import binding as B
from tests import latent_util as L
from tests.test_latent_gpu import cuda

pytestmark = pytest.mark.gpu


def test_append_without_lengths_is_refused():
    d = cuda(L.cache([5], 8, 256, 32, False, 1))
    x = torch.zeros((5, 288), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.PdaError) as e:
        B.paged_latent_append(x[:, :256], x[:, 256:], L.offsets([5]).cuda(), d["page_table"], None,
                              d["latent"], d["rope"])
    assert e.value.status == 1
