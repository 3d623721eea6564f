"""Caches of nearly 2^31 rows, which the 4-bit decode and the attention weights would count past 32 bits, are refused."""

import pytest

from head_latent_attention_absorb_b200 import _capi
from head_latent_attention_absorb_b200.build import build

P = 0x10000  # an aligned non-NULL address; no call below passes validation
F32, BF = _capi.MLA_F32, _capi.MLA_BF16
UNSUPPORTED, WORKSPACE = 2, 6
SMALL = _capi.MLADims(1, 16, 2, 1, 1)
WIDE = _capi.MLADims(1, 512, 64, 1, 1)
MOST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def L():
    build(quiet=True)
    return _capi.lib()


@pytest.mark.parametrize("dims,dt,w", [(SMALL, F32, (16, 2)), (WIDE, BF, (512, 64))])
@pytest.mark.parametrize("n_max", [MOST + 1, 2 ** 31 - 64, 2 ** 31 - 1])
def test_rows_past_the_limit(L, dims, dt, w, n_max):
    lead = (dims, dt, 1, 1, P, w[0], P, w[1])
    planes = (P, 0, w[0] // 2, P, 0, w[0] // 16 if dt == F32 else 32, P, 0, w[1], 1.0)
    assert L.mla_decode_absorb_fp4kv(*lead, *planes, n_max, P, 0.1, P, 0, P, 1 << 40, 0, 0) == UNSUPPORTED
    assert L.mla_cache_weights_fp4kv(*lead, *planes, n_max, P, 0.1, P, 0, n_max, 1.0, P, n_max, 0, 0) == UNSUPPORTED
    assert L.mla_cache_weights(*lead, P, 0, w[0], P, 0, w[1], n_max, P, 0.1, P, 0, n_max, 1.0, P, n_max, 0, 0) == UNSUPPORTED
    assert L.mla_decode_fp4kv_workspace_size(dims, dt, 1, 1, n_max) == 0


@pytest.mark.parametrize("dims,dt", [(SMALL, F32), (WIDE, BF)])
def test_rows_at_the_limit_have_a_workspace(L, dims, dt):
    assert 0 < L.mla_decode_fp4kv_workspace_size(dims, dt, 1, 1, MOST) < 1 << 30
