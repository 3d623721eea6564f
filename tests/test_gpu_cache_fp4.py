"""The 4-bit latent cache on the GPU against its fp64 definition: append, read-back and decode."""

import numpy as np
import pytest
import torch

import oracle as O
from head_latent_attention_absorb_b200 import _capi, api

from _cache_util import DEV, V3, check_decode, pack, random_fp4, reference, values

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def dims(n_h=128, d_c=512, d_r=64):
    return (n_h, d_c, d_r, 128, 128)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------ append and read
def run_append(d_c, d_r, dtype, B, T, n_max, positions, rows=None, counts=None, gain=True, ls=1.0, seed=0, x=None,
               eps=1e-6):
    rng = np.random.default_rng(seed)
    if x is None:
        x = torch.from_numpy(rng.standard_normal((B, T, d_c + d_r), dtype=np.float32) * 3).to(dtype)
    g = torch.from_numpy(rng.uniform(0.5, 1.5, d_c).astype(np.float32)) * ls if gain else None
    c4, sc, kr = random_fp4(B, n_max, d_c, seed + 1, d_r, dtype)
    dc4, dsc, dkr = pack(c4, sc, kr) if d_c == 512 else (c4.to(DEV), sc.to(DEV), kr.to(DEV))
    err = i32([0])
    api.mla_cache_append_fp4((4, d_c, d_r, 32, 32), x.to(DEV), i32(positions), dc4, dsc, dkr,
                             rows=None if rows is None else i32(rows), counts=None if counts is None else i32(counts),
                             gain=None if g is None else g.to(DEV), eps=eps, latent_scale=ls, dev_err=err)
    got = (dc4.cpu(), dsc.cpu(), dkr.cpu())
    rows = positions if rows is None else rows
    counts = [T] * B if counts is None else counts
    touched = np.zeros((B, n_max), dtype=bool)
    for b in range(B):
        for i in range(counts[b] if 0 <= counts[b] <= T else 0):
            r, p = rows[b] + i, positions[b] + i
            if positions[b] < 0 or not 0 <= r < n_max:
                continue
            touched[b, r] = True
            xi = x[b, i:i + 1].double().numpy()
            wc, ws, wk = O.cache_append_fp4(xi, d_c, [p], None if g is None else g.double().numpy(),
                                            float(np.float32(eps)), latent_scale=ls)
            gv = O.fp4_values(got[0][b, r].numpy(), got[1][b, r].numpy(), ls)
            wv = O.fp4_values(wc[0], ws[0], ls)
            assert np.array_equal(gv, wv, equal_nan=True), (b, i, np.flatnonzero(gv != wv)[:4])
            # one rounding to the type, sincos of half a turn to a few 2^-24, and the rotation's two products
            bound = torch.finfo(dtype).eps / 2 * np.abs(wk[0]) + 2.0 ** -20 * np.abs(xi[0, d_c:]).reshape(-1, 2).sum(-1).repeat(2)
            diff = np.abs(got[2][b, r].double().numpy() - wk[0])
            assert (diff <= bound).all() or np.isnan(wk).any(), (b, i, (diff / bound).max())
    for a, w in zip(got, (c4, sc, kr)):  # every other row is as it was
        assert torch.equal(a[torch.from_numpy(~touched)], w[torch.from_numpy(~touched)])
    return int(err.item()), got


@pytest.mark.parametrize("dtype,d_c,d_r", [(BF, 512, 64), (F32, 512, 64), (F32, 16, 2), (F32, 528, 34), (F32, 1024, 128)])
@pytest.mark.parametrize("gain", [True, False])
def test_append_one_token(dtype, d_c, d_r, gain):
    err, _ = run_append(d_c, d_r, dtype, 5, 1, 9, [0, 8, 3, 3, 1], gain=gain, seed=d_c + d_r)
    assert err == 0


@pytest.mark.parametrize("ls", [1.0, 2.0 ** -12, 2.0 ** 20])
def test_append_prompts_padded_with_rows_apart_from_positions(ls):
    err, _ = run_append(512, 64, BF, 4, 70, 80, [0, 65000, 7, 1000000], rows=[10, 0, 5, 9], counts=[70, 1, 0, 33], ls=ls)
    assert err == 0


def test_append_many_rows_on_rounding_borders():
    """Inputs on a coarse grid with the norm fixed at one: quotients fall on and next to every border."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.integers(-24, 25, (3, 400, 576)).astype(np.float32) / 4).to(BF)
    err, _ = run_append(512, 64, BF, 3, 400, 400, [0, 0, 0], gain=False, x=x)
    assert err == 0


def test_append_zero_rows_extreme_sizes_and_nan():
    x = torch.zeros((1, 6, 576), dtype=F32)
    x[0, 1] = 1e-25
    x[0, 2] = torch.linspace(-1, 1, 576) * 1e30
    x[0, 3, 5] = 1e-30
    x[0, 4] = torch.linspace(-3, 3, 576)
    x[0, 4, 100] = float("nan")
    x[0, 5] = torch.linspace(0.1, 1e-3, 576)
    err, got = run_append(512, 64, F32, 1, 6, 6, [0], gain=False, x=x)
    assert err == 0
    assert (O.fp4_values(got[0][0, 0].numpy(), got[1][0, 0].numpy()) == 0).all()
    assert np.isnan(O.fp4_values(got[0][0, 4].numpy(), got[1][0, 4].numpy())).all()


@pytest.mark.parametrize("positions,rows,counts,code", [
    ([0, 9], None, None, 4), ([-1, 0], None, None, 4), ([0, 0], [0, -1], None, 4), ([0, 0], [7, 0], None, 4),
    ([0, 0], None, [4, 0], 7), ([0, 0], None, [-1, 2], 7)])
def test_append_bad_indices_are_flagged_and_write_nothing(positions, rows, counts, code):
    err, _ = run_append(512, 64, BF, 2, 3, 9, positions, rows=rows, counts=counts)
    assert err == code


@pytest.mark.parametrize("dtype,d_c", [(BF, 512), (F32, 512), (F32, 48), (F32, 1024)])
@pytest.mark.parametrize("ls", [1.0, 2.0 ** -9])
def test_read_returns_the_values(dtype, d_c, ls):
    B, n_max, n = 3, 41, 17
    c4, sc, kr = random_fp4(B, n_max, d_c, 3)
    sc[0, 3, 0], sc[1, 30, 1] = 0x7F, 0          # a NaN block and a zero block
    dc4, dsc, _ = pack(c4, sc, kr) if d_c == 512 else (c4.to(DEV), sc.to(DEV), None)
    first, counts = [0, 24, 40], [17, 5, 1]
    out = api.mla_cache_read_fp4(dims(4, d_c), dc4, dsc, n, first=i32(first), counts=i32(counts), latent_scale=ls, dtype=dtype)
    want = np.zeros((B, n, d_c))
    v = values(c4, sc, ls)
    for b in range(B):
        want[b, :counts[b]] = v[b, first[b]:first[b] + counts[b]]
    assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)
    whole = api.mla_cache_read_fp4(dims(4, d_c), dc4, dsc, n_max, latent_scale=ls, dtype=dtype)
    assert np.array_equal(whole.double().cpu().numpy(), v, equal_nan=True)


def test_read_flags_bad_rows_and_returns_zeros():
    c4, sc, kr = random_fp4(3, 8, 512, 4)
    dc4, dsc, _ = pack(c4, sc, kr)
    for first, counts, code in (([0, 7, 0], [2, 2, 2], 4), ([-1, 0, 0], [2, 2, 2], 4), ([0, 0, 0], [2, 3, 2], 7)):
        err = i32([0])
        out = api.mla_cache_read_fp4(dims(4), dc4, dsc, 2, first=i32(first), counts=i32(counts), dev_err=err)
        assert int(err.item()) == code
        assert torch.isfinite(out.float()).all()
    strided = torch.full((3, 5, 1024), -7.0, dtype=BF, device=DEV)
    api.mla_cache_read_fp4(dims(4), dc4, dsc, 5, out=strided[..., :512])
    assert np.array_equal(strided[..., :512].double().cpu().numpy(), values(c4, sc)[:, :5])
    assert (strided[..., 512:] == -7).all()


# ------------------------------------------------------------------------------------------ decode
def run_decode(n_h, T, n_max, lengths, dtype=BF, d_c=512, d_r=64, seed=0, ls=1.0, q_std=0.226, scale=0.0722, packed=True,
               garbage=True, q=None, edit=None):
    B = len(lengths)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, T, n_h, d_c), generator=g) * q_std / ls).to(dtype) if q is None else q
    qp = torch.randn((B, T, n_h, d_r), generator=g).to(dtype)
    c4, sc, kr = random_fp4(B, n_max, d_c, seed + 7, d_r, dtype)
    if edit is not None:
        edit(c4, sc, kr)
    ref = reference(q, qp, values(c4, sc, ls), kr, lengths, T, float(np.float32(scale)))
    if garbage:  # rows behind a sequence hold NaN
        for b, L in enumerate(lengths):
            if 0 <= L < n_max:
                sc[b, L:] = 0x7F
                kr[b, L:] = float("nan")
    planes = pack(c4, sc, kr) if packed and d_c == 512 else (c4.to(DEV), sc.to(DEV), kr.to(DEV))
    if T == 1:
        q, qp = q[:, 0], qp[:, 0]
    lse = torch.full(q.shape[:-1], 99.0, device=DEV)
    err = i32([0])
    ctx = api.mla_decode_absorb_fp4kv(dims(n_h, d_c, d_r), q.to(DEV), qp.to(DEV), *planes, i32(lengths), scale,
                                      latent_scale=ls, lse=lse, dev_err=err)
    torch.cuda.synchronize()
    return ctx, lse, ref, int(err.item())


@pytest.mark.parametrize("lengths", [[1], [2, 127, 128, 129], [255, 256, 257, 1], [1000, 63, 64, 65], [4096, 3001]])
def test_decode_lengths(lengths):
    ctx, lse, ref, err = run_decode(128, 1, max(lengths) + 3, lengths, seed=len(lengths))
    assert err == 0
    check_decode(ctx, lse, ref, BF)


@pytest.mark.parametrize("n_h", [1, 7, 16, 20, 32, 33, 64, 65, 100, 127, 128])
def test_decode_head_counts(n_h):
    ctx, lse, ref, err = run_decode(n_h, 1, 400, [400, 131, 260], seed=n_h)
    assert err == 0
    check_decode(ctx, lse, ref, BF)


@pytest.mark.parametrize("n_h,T", [(128, 2), (128, 3), (16, 2), (16, 4), (20, 3), (64, 2), (1, 5), (5, 40)])
def test_decode_several_tokens(n_h, T):
    ctx, lse, ref, err = run_decode(n_h, T, 300, [T, T + 1, 128, 130, 300], seed=n_h + T)
    assert err == 0
    check_decode(ctx, lse, ref, BF)


@pytest.mark.parametrize("d_c,d_r,n_h,T", [(64, 16, 4, 1), (16, 2, 1, 2), (512, 64, 3, 3), (528, 66, 9, 1), (1024, 128, 2, 2)])
def test_decode_fp32(d_c, d_r, n_h, T):
    ctx, lse, ref, err = run_decode(n_h, T, 700, [T, 257, 700], dtype=F32, d_c=d_c, d_r=d_r, seed=d_c)
    assert err == 0
    check_decode(ctx, lse, ref, F32)


@pytest.mark.parametrize("ls", [2.0 ** -30, 2.0 ** -7, 2.0 ** 11, 2.0 ** 40])
def test_decode_latent_scale(ls):
    ctx, lse, ref, err = run_decode(128, 1, 300, [300, 20], seed=3, ls=ls)
    assert err == 0
    check_decode(ctx, lse, ref, BF)


@pytest.mark.parametrize("q_std", [0.0, 1e-12, 20.0])
def test_decode_flat_and_peaked_softmax(q_std):
    """Zero and tiny queries (uniform weights over the rotary scores alone) and scores that span hundreds."""
    ctx, lse, ref, err = run_decode(128, 1, 900, [900, 513], seed=4, q_std=q_std)
    assert err == 0
    check_decode(ctx, lse, ref, BF)


def test_decode_heads_of_very_different_size():
    g = torch.Generator().manual_seed(8)
    q = torch.randn((2, 1, 128, 512), generator=g) * (2.0 ** torch.arange(-60, 4, 0.5))[:128, None]
    q[:, :, 127] = 0.0
    ctx, lse, ref, err = run_decode(128, 1, 300, [300, 129], q=q.to(BF))
    check_decode(ctx, lse, ref, BF)


def test_decode_rising_scores_and_extreme_scales():
    """Later rows outscore the earlier ones by far (the running maximum moves in every tile); the largest
    and smallest scales, and zero blocks."""
    def edit(c4, sc, kr):
        sc[0] = torch.linspace(0x10, 0x40, sc.shape[1]).to(torch.uint8)[:, None]
        sc[1, ::3] = 0
        sc[1, 1::3] = 1
        sc[2, :, :16] = 0x7E
    ctx, lse, ref, err = run_decode(128, 1, 1100, [1100, 700, 200], seed=5, edit=edit, q_std=0.02)
    check_decode(ctx, lse, ref, BF)


def test_decode_nan_stays_in_its_sequence_and_head():
    def edit(c4, sc, kr):
        sc[1, 17, 3] = 0x7F
    q = (torch.randn((3, 1, 128, 512), generator=torch.Generator().manual_seed(2)) * 0.2).to(BF)
    q[2, 0, 9, 4] = float("nan")
    q[2, 0, 70, 4] = float("inf")
    with np.errstate(invalid="ignore"):
        ctx, lse, ref, err = run_decode(128, 1, 300, [300, 290, 280], q=q, edit=edit)
    bad = torch.isnan(ctx.float()).any(-1).cpu()
    assert bad[1].all() and not bad[0].any()
    assert bad[2].nonzero().flatten().tolist() == [9, 70]
    keep = ~bad.numpy()[:, None]
    check_decode(torch.from_numpy(np.where(keep[..., None], ctx.double().cpu().numpy()[:, None], 0)), None,
                 tuple(np.where(keep[..., None] if r.ndim == 4 else keep, r, 0) for r in ref), BF)


def test_decode_bad_lengths_are_flagged_and_zero():
    for lengths in ([0, 300], [300, 301], [-5, 4]):
        ctx, lse, ref, err = run_decode(128, 1, 300, lengths, garbage=False)
        assert err == 7
        check_decode(ctx, lse, ref, BF)
    ctx, lse, ref, err = run_decode(16, 4, 300, [3, 200], garbage=False)
    assert err == 7
    check_decode(ctx, lse, ref, BF)
    ctx, lse, ref, err = run_decode(3, 2, 300, [1, 200], dtype=F32, d_c=64, d_r=16, garbage=False)
    assert err == 7
    check_decode(ctx, lse, ref, F32)


def test_decode_many_sequences_and_separate_planes():
    lengths = [int(v) for v in np.random.default_rng(3).integers(1, 200, 170)]
    ctx, lse, ref, err = run_decode(128, 1, 200, lengths, seed=6, packed=False)
    check_decode(ctx, lse, ref, BF)


def test_decode_equals_the_bf16_decode_on_the_values():
    """code * scale is exact in bf16, so the bf16 decode over the read-back sees the same cache."""
    B, n = 4, 1000
    c4, sc, kr = random_fp4(B, n, 512, 9)
    planes = pack(c4, sc, kr)
    q = (torch.randn((B, 128, 512), device=DEV) * 0.226).to(BF)
    qp = torch.randn((B, 128, 64), device=DEV).to(BF)
    lens = i32([1000, 1, 640, 127])
    a = api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, lens, 0.0722).float()
    c = api.mla_cache_read_fp4(dims(), planes[0], planes[1], n)
    b = api.mla_decode_absorb(dims(), q, qp, c, planes[2].contiguous(), lens, 0.0722).float()
    assert (a - b).abs().max() <= 2e-2 and (a - b).norm() / b.norm() <= 1e-2


def test_decode_offsets_past_32_bits():
    """Row and batch offsets beyond 2^32 bytes: two sequences whose rows lie 1.5 MB apart."""
    n, stride = 2000, 1572864
    if torch.cuda.mem_get_info()[0] < 3 * n * stride:
        pytest.skip("not enough memory")
    c4, sc, kr = random_fp4(2, n, 512, 11)
    base = torch.empty((2 * n * stride,), dtype=torch.uint8, device=DEV)
    views = []
    for t, off in ((c4, 0), (sc, 256), (kr.view(torch.uint8), 288)):
        v = base.as_strided((2, n, t.shape[-1]), (n * stride, stride, 1), off)
        v.copy_(t)
        views.append(v)
    views[2] = base.view(BF).as_strided((2, n, 64), (n * stride // 2, stride // 2, 1), 144)
    q, qp = torch.randn((2, 1, 128, 512)) * 0.2, torch.randn((2, 1, 128, 64))
    q, qp = q.to(BF), qp.to(BF)
    ctx = api.mla_decode_absorb_fp4kv(dims(), q[:, 0].to(DEV), qp[:, 0].to(DEV), *views, i32([n, n - 77]), 0.0722)
    check_decode(ctx, None, reference(q, qp, values(c4, sc), kr, [n, n - 77], 1, float(np.float32(0.0722))), BF)


def test_decode_repeats_bit_for_bit_on_streams_and_in_graphs():
    B, n = 6, 3000
    c4, sc, kr = random_fp4(B, n, 512, 12)
    planes = pack(c4, sc, kr)
    q = (torch.randn((B, 2, 128, 512), device=DEV) * 0.226).to(BF)
    qp = torch.randn((B, 2, 128, 64), device=DEV).to(BF)
    lens = i32([3000, 5, 1500, 2999, 128, 640])
    first = api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, lens, 0.0722)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, lens, 0.0722, stream=s) for s in (s1, s2) * 4]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    graphs = []
    for _ in range(2):
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
        with torch.cuda.graph(g):
            api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, lens, 0.0722, ctx=out)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out, first)
    lens.fill_(77)  # a replay reads the lengths that are there
    graphs[0][0].replay()
    want = api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, lens, 0.0722)
    assert torch.equal(graphs[0][1], want)


def test_a_small_workspace_is_refused():
    c4, sc, kr = random_fp4(1, 64, 512, 13)
    planes = pack(c4, sc, kr)
    q, qp = torch.zeros((1, 128, 512), dtype=BF, device=DEV), torch.zeros((1, 128, 64), dtype=BF, device=DEV)
    with pytest.raises(_capi.MLAError, match="WORKSPACE"):
        api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, i32([64]), 0.07, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_v3_widths():
    assert V3 == (512, 64)
