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


def test_rows_apart_from_positions_on_another_stream():
    x = torch.randn((3, 576), device="cuda").to(torch.bfloat16)
    pos, at = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([9000, 7, 3], [1, 0, 5]))
    want = torch.zeros((3, 8, 576), dtype=torch.bfloat16, device="cuda")
    api.mla_cache_append((16, 512, 64, 128, 128), x, pos, want[..., :512], want[..., 512:], rows=at)
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        got = torch.zeros_like(want)
        torch.cuda.synchronize()
        api.mla_cache_append((16, 512, 64, 128, 128), x, pos, got[..., :512], got[..., 512:], rows=at, stream=stream)
        st.synchronize()
        assert torch.equal(got, want) and bool((want[1, 0] != 0).any())
