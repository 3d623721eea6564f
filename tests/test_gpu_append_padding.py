"""Padding of a batch of prompts is not read by the 4-bit append: the rows need not exist."""

import pytest
import torch

from head_latent_attention_absorb_b200 import _capi, api

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype,d_c,d_r", [(torch.bfloat16, 512, 64), (torch.float32, 48, 10)])
def test_rows_behind_the_counts_need_not_exist(dtype, d_c, d_r):
    """Three sequences' rows lie one behind the other, two, none and three of them; T says 30000."""
    T, n_max, width = 30000, 8, d_c + d_r
    counts = [2, 0, 3]
    x = torch.randn((6, width), device=DEV).to(dtype)

    def cache():
        return (torch.zeros((3, n_max, d_c // 2), dtype=torch.uint8, device=DEV),
                torch.zeros((3, n_max, d_c // 16), dtype=torch.uint8, device=DEV), torch.zeros((3, n_max, d_r), dtype=dtype, device=DEV))

    padded = torch.zeros((3, 3, width), dtype=dtype, device=DEV)
    want = cache()
    for b in range(3):
        padded[b, :counts[b]] = x[2 * b:2 * b + counts[b]] if b < 2 else x[4:6].repeat(2, 1)[:3]
    # a batch stride of two rows: sequence 2 begins at row 4 and its third row is the buffer's row 6
    buf = torch.empty((7, width), dtype=dtype, device=DEV)
    buf[:6] = x
    buf[6] = x[4]
    api.mla_cache_append_fp4((4, d_c, d_r, 1, 1), padded, i32([0, 5, 2]), *want, counts=i32(counts))
    c4, sc, kr = got = cache()
    pos, n, err = i32([0, 5, 2]), i32(counts), i32([0])
    es = _capi.MLA_BF16 if dtype == torch.bfloat16 else _capi.MLA_F32
    status = _capi.lib().mla_cache_append_fp4(
        _capi.MLADims(4, d_c, d_r, 1, 1), es, 3, T, buf.data_ptr(), 2 * width, width, 0, 1e-6, 1e4, 1.0, pos.data_ptr(), 0,
        n.data_ptr(), n_max, c4.data_ptr(), c4.stride(0), c4.stride(1), sc.data_ptr(), sc.stride(0), sc.stride(1), kr.data_ptr(),
        kr.stride(0), kr.stride(1), err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and int(err) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((want[0][2, 2:5] != 0).any()) and bool((want[0][1] == 0).all())
