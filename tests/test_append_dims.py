"""Which dimensions mla_cache_append and mla_cache_append_at take: the heads do not enter, so a rank's share of them will do."""

import pytest
import torch

from head_latent_attention_absorb_b200 import _capi, api
from head_latent_attention_absorb_b200.build import build

P = 0x10000  # an aligned non-NULL address; no call below passes validation
BF, F32 = _capi.MLA_BF16, _capi.MLA_F32
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    build(quiet=True)
    return _capi.lib()


def call(L, at, dims, dt, eps=-1.0):
    """The eps of -1 is refused after the dimensions have been taken."""
    n_h, d_c, d_r = dims
    w = max(d_c, 8), max(d_r, 8)
    tail = (16, P, 16 * w[0], w[0], P, 16 * w[1], w[1], 0, 0)
    d = _capi.MLADims(n_h, d_c, d_r, 0, 0)
    lead = (d, dt, 2, P, w[0] + w[1], 0, eps, 1e4, P)
    return L.mla_cache_append_at(*lead, 0, *tail) if at else L.mla_cache_append(*lead, *tail)


@pytest.mark.parametrize("at", [False, True])
@pytest.mark.parametrize("dims,dt,want", [
    ((0, 512, 64), BF, "dimensions"), ((-1, 512, 64), BF, "dimensions"), ((129, 512, 64), BF, "n_h"), ((128, 256, 64), BF, "d_c"),
    ((128, 512, 32), BF, "d_r"), ((0, 64, 16), F32, "dimensions"), ((1025, 64, 16), F32, "n_h"), ((4, 1025, 16), F32, "d_c"),
    ((4, 64, 130), F32, "d_r"), ((4, 64, 15), F32, "d_r must be even"), ((4, 64, 16), 7, "dtype"),
    ((1, 512, 64), BF, "eps"), ((16, 512, 64), BF, "eps"), ((128, 512, 64), BF, "eps"),       # taken
    ((1, 7, 2), F32, "eps"), ((1024, 1024, 128), F32, "eps")])
def test_dimensions(L, at, dims, dt, want):
    status = call(L, at, dims, dt)
    assert status in (INVALID, UNSUPPORTED)
    assert want in L.mla_last_error_message().decode(), L.mla_last_error_message()


def _append_at(**kw):
    a = dict(x=torch.zeros((2, 80)), pos=torch.zeros(2, dtype=torch.int32), c=torch.zeros((2, 16, 64)), k=torch.zeros((2, 16, 16)),
             rows=torch.zeros(2, dtype=torch.int32), gain=None, err=None)
    a.update(kw)
    api.mla_cache_append((4, 64, 16, 32, 32), a["x"], a["pos"], a["c"], a["k"], gain=a["gain"], rows=a["rows"], dev_err=a["err"])


@pytest.mark.parametrize("kw,kind,match", [
    (dict(pos=torch.zeros(1, dtype=torch.int32)), TypeError, "positions"), (dict(rows=torch.zeros(1, dtype=torch.int32)), TypeError, "rows"),
    (dict(x=torch.zeros((2, 79))), ValueError, "kv_a"), (dict(x=torch.zeros((1, 80))), ValueError, "kv_a"),
    (dict(c=torch.zeros((2, 16, 48))), ValueError, "c_kv"), (dict(c=torch.zeros((2, 16, 64), dtype=torch.bfloat16)), TypeError, "c_kv"),
    (dict(k=torch.zeros((2, 15, 16))), ValueError, "k_r"), (dict(k=torch.zeros((1, 16, 16))), ValueError, "k_r"),
    (dict(k=torch.zeros((2, 16, 16), dtype=torch.bfloat16)), TypeError, "k_r"), (dict(gain=torch.ones(63)), ValueError, "gain"),
    (dict(err=torch.zeros(1)), TypeError, "dev_err"), (dict(), ValueError, "CUDA tensor")])
def test_binding_refuses_what_would_leave_its_arrays(kw, kind, match):
    with pytest.raises(kind, match=match):
        _append_at(**kw)
