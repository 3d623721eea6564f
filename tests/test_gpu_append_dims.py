"""mla_cache_append writes the same rows whatever the head count of its dims."""

import pytest
import torch

from head_latent_attention_absorb_b200 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d_c,d_r,heads", [(torch.bfloat16, 512, 64, (1, 16, 100)), (torch.float32, 40, 6, (1, 1024))])
def test_rows_do_not_depend_on_the_heads(dtype, d_c, d_r, heads):
    x = torch.randn((3, d_c + d_r), device="cuda").to(dtype)
    pos = torch.tensor([0, 7, 3], dtype=torch.int32, device="cuda")

    def rows(n_h, d_h):
        cache = torch.zeros((3, 8, d_c + d_r), dtype=dtype, device="cuda")
        api.mla_cache_append((n_h, d_c, d_r, d_h, d_h), x, pos, cache[..., :d_c], cache[..., d_c:])
        return cache

    want = rows(128, 128)
    assert all(bool((want[b, int(pos[b])] != 0).any()) for b in range(3))
    for n_h in heads:
        for d_h in (0, 128):
            assert torch.equal(rows(n_h, d_h), want)
