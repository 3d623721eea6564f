"""Host-side refusals of the 4-bit cache, attention-weight and eviction calls: through the C ABI
(nothing here reaches a launch) and through the Python binding (no GPU needed)."""

import ctypes

import pytest
import torch

from head_latent_attention_absorb_b200 import _capi, api
from head_latent_attention_absorb_b200.build import build

DS = _capi.MLADims(128, 512, 64, 128, 128)
TINY = _capi.MLADims(4, 64, 16, 32, 32)
P = 0x10000  # an aligned non-NULL address; every call below fails validation before using it
BF, F32 = _capi.MLA_BF16, _capi.MLA_F32
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def L():
    build(quiet=True)
    return _capi.lib()


def _append(L, **kw):
    a = dict(dims=DS, dt=BF, B=2, T=1, kv_a=P, lda_b=576, lda=576, gain=0, eps=1e-6, base=1e4, ls=1.0, pos=P, rows=0,
             counts=0, n_max=16, c4=P, c4b=16 * 256, c4r=256, sc=P, scb=16 * 32, scr=32, kr=P, krb=16 * 64, krr=64)
    a.update(kw)
    return L.mla_cache_append_fp4(a["dims"], a["dt"], a["B"], a["T"], a["kv_a"], a["lda_b"], a["lda"], a["gain"],
                                  a["eps"], a["base"], a["ls"], a["pos"], a["rows"], a["counts"], a["n_max"], a["c4"],
                                  a["c4b"], a["c4r"], a["sc"], a["scb"], a["scr"], a["kr"], a["krb"], a["krr"], 0, 0)


def _decode(L, **kw):
    a = dict(dims=DS, dt=BF, B=2, T=1, q=P, ldq=512, qp=P, ldqp=64, c4=P, c4b=16 * 256, c4r=256, sc=P, scb=16 * 32,
             scr=32, kr=P, krb=16 * 64, krr=64, ls=1.0, n_max=16, lens=P, scale=0.07, ctx=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.mla_decode_absorb_fp4kv(a["dims"], a["dt"], a["B"], a["T"], a["q"], a["ldq"], a["qp"], a["ldqp"], a["c4"],
                                     a["c4b"], a["c4r"], a["sc"], a["scb"], a["scr"], a["kr"], a["krb"], a["krr"],
                                     a["ls"], a["n_max"], a["lens"], a["scale"], a["ctx"], 0, a["ws"], a["wsb"], 0, 0)


def _weights(L, **kw):
    a = dict(dims=DS, dt=BF, B=2, T=1, q=P, ldq=512, qp=P, ldqp=64, c=P, cb=16 * 512, cr=512, kr=P, krb=16 * 64,
             krr=64, n_max=16, lens=P, scale=0.07, lse=P, acc=P, accb=16, decay=1.0, out=P, outb=16)
    a.update(kw)
    return L.mla_cache_weights(a["dims"], a["dt"], a["B"], a["T"], a["q"], a["ldq"], a["qp"], a["ldqp"], a["c"],
                               a["cb"], a["cr"], a["kr"], a["krb"], a["krr"], a["n_max"], a["lens"], a["scale"],
                               a["lse"], a["acc"], a["accb"], a["decay"], a["out"], a["outb"], 0, 0)


def _evict(L, planes=((P, 16 * 64, 64, 64),), **kw):
    a = dict(B=2, n_max=16, acc=P, accb=16, lens=P, keep=8, sink=1, recent=2, new=P, map=P, n=None)
    a.update(kw)
    arr = (_capi.MLARows * max(1, len(planes)))(*[_capi.MLARows(*p) for p in planes])
    return L.mla_cache_evict(a["B"], a["n_max"], arr, len(planes) if a["n"] is None else a["n"], a["acc"], a["accb"],
                             a["lens"], a["keep"], a["sink"], a["recent"], a["new"], a["map"], 0, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(dims=_capi.MLADims(0, 512, 64, 1, 1)), INVALID), (dict(dims=_capi.MLADims(129, 512, 64, 1, 1)), UNSUPPORTED),
    (dict(dims=TINY), UNSUPPORTED), (dict(dims=_capi.MLADims(4, 72, 16, 1, 1), dt=F32), UNSUPPORTED),
    (dict(dims=_capi.MLADims(4, 64, 15, 1, 1), dt=F32), INVALID), (dict(dt=7), INVALID),
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(n_max=0), INVALID), (dict(kv_a=0), INVALID), (dict(pos=0), INVALID),
    (dict(c4=0), INVALID), (dict(sc=0), INVALID), (dict(kr=0), INVALID), (dict(lda=575), INVALID), (dict(lda=580), INVALID),
    (dict(kv_a=P + 8), INVALID), (dict(c4=P + 8), INVALID), (dict(sc=P + 4), INVALID), (dict(kr=P + 2), INVALID),
    (dict(c4r=248), INVALID), (dict(c4r=264), INVALID), (dict(scr=16), INVALID), (dict(scr=40), INVALID),
    (dict(c4b=15 * 256), INVALID), (dict(scb=15 * 32), INVALID), (dict(krb=15 * 64), INVALID), (dict(krr=60), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(base=0.0), INVALID), (dict(ls=0.0), INVALID),
    (dict(ls=3.0), INVALID), (dict(ls=-1.0), INVALID), (dict(ls=2.0 ** 65), INVALID), (dict(ls=float("nan")), INVALID)])
def test_append_refuses(L, kw, want):
    assert _append(L, **kw) == want, L.mla_last_error_message()


@pytest.mark.parametrize("kw,want", [
    (dict(dims=_capi.MLADims(200, 512, 64, 1, 1)), UNSUPPORTED), (dict(T=17), INVALID), (dict(T=0), INVALID),
    (dict(B=65536), UNSUPPORTED), (dict(q=0), INVALID), (dict(lens=0), INVALID), (dict(ctx=0), INVALID),
    (dict(ldq=504), INVALID), (dict(ldq=516), INVALID), (dict(ldqp=60), INVALID), (dict(q=P + 8), INVALID),
    (dict(ctx=P + 8), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(ls=0.3), INVALID),
    (dict(c4b=-256), INVALID), (dict(krr=56), INVALID), (dict(ws=0), WORKSPACE), (dict(wsb=8), WORKSPACE),
    (dict(ws=P + 8), INVALID)])
def test_decode_refuses(L, kw, want):
    assert _decode(L, **kw) == want, L.mla_last_error_message()


def test_workspace_size(L):
    assert L.mla_decode_fp4kv_workspace_size(DS, BF, 2, 1, 16) > 0
    for bad in ((DS, BF, 0, 1, 16), (DS, BF, 1, 0, 16), (DS, BF, 1, 17, 16), (TINY, BF, 1, 1, 16), (DS, BF, 65536, 1, 16)):
        assert L.mla_decode_fp4kv_workspace_size(*bad) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(lse=0), INVALID), (dict(out=0), INVALID), (dict(c=0), INVALID), (dict(cr=504), INVALID), (dict(cr=516), INVALID),
    (dict(c=P + 8), INVALID), (dict(accb=15), INVALID), (dict(outb=15), INVALID), (dict(accb=32), INVALID),
    (dict(decay=-1.0), INVALID), (dict(decay=float("inf")), INVALID), (dict(decay=float("nan")), INVALID),
    (dict(dims=TINY), UNSUPPORTED), (dict(T=20), INVALID)])
def test_weights_refuse(L, kw, want):
    assert _weights(L, **kw) == want, L.mla_last_error_message()


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INVALID), (dict(n_max=0), INVALID), (dict(keep=0), INVALID), (dict(keep=17), INVALID),
    (dict(sink=-1), INVALID), (dict(recent=-1), INVALID), (dict(sink=5, recent=4), INVALID),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID), (dict(acc=0), INVALID), (dict(lens=0), INVALID),
    (dict(new=0), INVALID), (dict(map=0), INVALID), (dict(accb=15), INVALID), (dict(n=0), INVALID), (dict(n=5), INVALID),
    (dict(planes=((0, 1024, 64, 64),)), INVALID), (dict(planes=((P, 1024, 32, 64),)), INVALID),
    (dict(planes=((P, 512, 64, 64),)), INVALID), (dict(planes=((P, 1024, 64, 0),)), INVALID)])
def test_evict_refuses(L, kw, want):
    assert _evict(L, **kw) == want, L.mla_last_error_message()


def _read(L, **kw):
    a = dict(dims=DS, dt=BF, B=2, n=16, n_max=16, c4=P, c4b=16 * 256, c4r=256, sc=P, scb=16 * 32, scr=32, ls=1.0, out=P,
             outb=16 * 512, outr=512)
    a.update(kw)
    return L.mla_cache_read_fp4(a["dims"], a["dt"], a["B"], a["n"], 0, 0, a["n_max"], a["c4"], a["c4b"], a["c4r"], a["sc"],
                                a["scb"], a["scr"], a["ls"], a["out"], a["outb"], a["outr"], 0, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INVALID), (dict(n=0), INVALID), (dict(n_max=0), INVALID), (dict(out=0), INVALID), (dict(c4=0), INVALID),
    (dict(out=P + 8), INVALID), (dict(outr=504), INVALID), (dict(outr=516), INVALID), (dict(outb=15 * 512), INVALID),
    (dict(c4r=264), INVALID), (dict(scr=16), INVALID), (dict(ls=3.0), INVALID), (dict(dims=TINY), UNSUPPORTED)])
def test_read_refuses(L, kw, want):
    assert _read(L, **kw) == want, L.mla_last_error_message()


def test_sizes_that_pass_32_bits_are_refused(L):
    assert _append(L, B=1 << 16, T=1 << 15, c4b=1 << 40, scb=1 << 40, krb=1 << 40) == UNSUPPORTED
    assert _decode(L, B=65535, n_max=1 << 30, c4b=0, scb=0, krb=0) == UNSUPPORTED
    assert _decode(L, B=32768, T=2, n_max=16) == UNSUPPORTED
    assert _weights(L, B=65536, accb=16, outb=16) == UNSUPPORTED
    assert _evict(L, B=65536) == UNSUPPORTED
    assert _evict(L, n_max=400001, accb=400001, planes=((P, 1 << 40, 64, 64),)) == UNSUPPORTED
    assert _evict(L, planes=((P, 1 << 40, 1 << 31, (1 << 31) - 1),)) == UNSUPPORTED
    assert _evict(L, planes=((P, 1 << 40, 1 << 30, 1 << 30), (P, 1 << 40, 16, 16))) == UNSUPPORTED


def test_append_at_refuses_like_append(L):
    assert L.mla_cache_append_at(DS, BF, 2, P, 575, 0, 1e-6, 1e4, P, P, 16, P, 16 * 512, 512, P, 16 * 64, 64, 0, 0) == INVALID


def _host(B=2, n_max=16, T=None):
    lead = (B,) if T is None else (B, T)
    q, qp = torch.zeros((*lead, 128, 512), dtype=torch.bfloat16), torch.zeros((*lead, 128, 64), dtype=torch.bfloat16)
    c4, sc = torch.zeros((B, n_max, 256), dtype=torch.uint8), torch.zeros((B, n_max, 32), dtype=torch.uint8)
    kr = torch.zeros((B, n_max, 64), dtype=torch.bfloat16)
    return q, qp, c4, sc, kr, torch.full((B,), n_max, dtype=torch.int32)


def test_binding_refuses_host_tensors():
    q, qp, c4, sc, kr, lens = _host()
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.mla_decode_absorb_fp4kv(DS, q, qp, c4, sc, kr, lens, 0.07)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.mla_cache_append_fp4(DS, torch.zeros((2, 576), dtype=torch.bfloat16), lens, c4, sc, kr)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.mla_cache_read_fp4(DS, c4, sc, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.mla_cache_evict([kr], torch.zeros((2, 16)), lens, 8)


def test_binding_refuses_wrong_shapes_and_types():
    q, qp, c4, sc, kr, lens = _host()
    with pytest.raises(ValueError, match="kv_scale"):
        api.mla_decode_absorb_fp4kv(DS, q, qp, c4, sc[:, :8], kr, lens, 0.07)
    with pytest.raises(TypeError, match="c4"):
        api.mla_decode_absorb_fp4kv(DS, q, qp, c4.to(torch.int32), sc, kr, lens, 0.07)
    with pytest.raises(TypeError, match="k_r"):
        api.mla_decode_absorb_fp4kv(DS, q, qp, c4, sc, kr.float(), lens, 0.07)
    with pytest.raises(ValueError, match="sequences"):
        api.mla_decode_absorb_fp4kv(DS, q[:1], qp[:1], c4, sc, kr, lens, 0.07)
    with pytest.raises(TypeError, match="lengths"):
        api.mla_decode_absorb_fp4kv(DS, q, qp, c4, sc, kr, lens[:1], 0.07)
    with pytest.raises(ValueError, match="ctx"):
        api.mla_decode_absorb_fp4kv(DS, q, qp, c4, sc, kr, lens, 0.07, ctx=torch.empty((2, 128, 256), dtype=q.dtype))
    qT, qpT = _host(T=3)[:2]
    with pytest.raises(ValueError, match="evenly strided"):
        api.mla_decode_absorb_fp4kv(DS, qT.transpose(0, 1).contiguous().transpose(0, 1), qpT, c4, sc, kr, lens, 0.07)
    with pytest.raises(ValueError, match="lse"):
        api.mla_cache_weights_fp4kv(DS, q, qp, c4, sc, kr, lens, 0.07, torch.zeros((2, 64)))
    with pytest.raises(ValueError, match="acc"):
        api.mla_cache_weights_fp4kv(DS, q, qp, c4, sc, kr, lens, 0.07, torch.zeros((2, 128)), acc=torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="kv_a"):
        api.mla_cache_append_fp4(DS, torch.zeros((2, 512), dtype=torch.bfloat16), lens, c4, sc, kr)
    with pytest.raises(TypeError, match="counts"):
        api.mla_cache_append_fp4(DS, torch.zeros((2, 3, 576), dtype=torch.bfloat16), lens, c4, sc, kr, counts=lens.long())
    with pytest.raises(ValueError, match="plane 0"):
        api.mla_cache_evict([kr[:, :8]], torch.zeros((2, 16)), lens, 8)
    with pytest.raises(ValueError, match="planes"):
        api.mla_cache_evict([], torch.zeros((2, 16)), lens, 8)
    with pytest.raises(TypeError, match="row_map"):
        api.mla_cache_evict([kr], torch.zeros((2, 16)), lens, 8, row_map=torch.zeros((2, 9), dtype=torch.int32))


def test_rows_struct_matches_the_header():
    assert ctypes.sizeof(_capi.MLARows) == 32
