"""Accumulated attention weights and eviction on the GPU, and a serving run of them together."""

import numpy as np
import pytest
import torch

import oracle as O
from head_latent_attention_absorb_b200 import api

from _cache_util import DEV, pack, random_fp4, reference, values

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def dims(n_h=128, d_c=512, d_r=64):
    return (n_h, d_c, d_r, 128, 128)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------ weights
def run_weights(n_h, T, n_max, lengths, dtype=BF, d_c=512, d_r=64, fp4=False, seed=0, ls=1.0, acc=True, decay=1.0,
                in_place=False, scale=0.0722, q_std=0.226, drop=()):
    B = len(lengths)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, T, n_h, d_c), generator=g) * q_std / ls).to(dtype)
    qp = torch.randn((B, T, n_h, d_r), generator=g).to(dtype)
    c4, sc, kr = random_fp4(B, n_max, d_c, seed + 7, d_r, dtype)
    plain = torch.randn((B, n_max, d_c), generator=g).to(dtype)
    c = values(c4, sc, ls) if fp4 else plain.double().numpy()
    _, lse, _, ez = reference(q, qp, c, kr, lengths, T, float(np.float32(scale)))
    lse32 = torch.from_numpy(lse).float()
    for b, s, h in drop:
        lse32[b, s, h] = float("-inf")
    a = torch.rand((B, n_max + 5), generator=g)[:, :n_max] * 4
    want = np.full((B, n_max), -3.0)
    if in_place:
        want = a.double().numpy().copy()
    bound = np.zeros((B, n_max))
    for b, L in enumerate(lengths):
        if not T <= L <= n_max:
            continue
        w = O.token_weights(q[b].double(), qp[b].double(), c[b, :L], kr[b, :L].double(), float(np.float32(scale)), lse32[b].numpy())
        old = np.zeros(L)
        if acc:
            old[:L - T] = decay * a[b, :L - T].double().numpy()
        want[b, :L] = w + old
        # exp of a score off by ez, of a lse rounded to fp32, a sum of T n_h positive terms, one product and one sum
        bound[b, :L] = w * (2 * ez[b].max() + 2.0 ** -18 + T * n_h * 2.0 ** -23) + 2.0 ** -22 * np.abs(want[b, :L]) + 1e-30
        # ex2.approx flushes denormals: each of the T n_h terms may lose 2^-126
        bound[b, :L] += T * n_h * 2.0 ** -125
    if fp4:
        for b, L in enumerate(lengths):
            if 0 <= L < n_max:
                sc[b, L:], kr[b, L:] = 0x7F, float("nan")
        planes = pack(c4, sc, kr) if d_c == 512 else (c4.to(DEV), sc.to(DEV), kr.to(DEV))
    else:
        rows = torch.cat((plain, kr), -1)
        for b, L in enumerate(lengths):
            if 0 <= L < n_max:
                rows[b, L:] = float("nan")
        rows = rows.to(DEV)
        planes = (rows[..., :d_c], rows[..., d_c:])
    da = torch.empty((B, n_max + 5), device=DEV)[:, :n_max]
    da.copy_(a)
    out = da if in_place else torch.full((B, n_max), -3.0, device=DEV)
    if T == 1:
        q, qp, lse32 = q[:, 0], qp[:, 0], lse32[:, 0]
    err = i32([0])
    kw = dict(acc=da if acc else None, decay=decay, out=out, dev_err=err)
    if fp4:
        kw["latent_scale"] = ls
    f = api.mla_cache_weights_fp4kv if fp4 else api.mla_cache_weights
    got = f(dims(n_h, d_c, d_r), q.to(DEV), qp.to(DEV), *planes, i32(lengths), scale, lse32.to(DEV).contiguous(), **kw)
    diff = np.abs(got.double().cpu().numpy() - want)
    assert (diff <= bound).all(), (np.argwhere(diff > bound)[:4], (diff / np.maximum(bound, 1e-300)).max())
    return int(err.item())


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("lengths", [[1], [2, 127, 128, 129], [255, 256, 257, 1], [1000, 63, 64, 65], [2500, 3001]])
def test_weights_lengths(lengths, fp4):
    assert run_weights(128, 1, max(lengths) + 3, lengths, fp4=fp4, seed=len(lengths)) == 0


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("n_h,T", [(1, 1), (7, 1), (16, 2), (20, 3), (64, 1), (65, 1), (100, 2), (128, 2), (128, 3), (5, 40)])
def test_weights_heads_and_tokens(n_h, T, fp4):
    assert run_weights(n_h, T, 300, [T, T + 1, 128, 130, 300], fp4=fp4, seed=n_h + T) == 0


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("kw", [dict(acc=False), dict(decay=0.0), dict(decay=0.97), dict(in_place=True),
                                dict(in_place=True, decay=0.5, T=3), dict(drop=[(0, 0, 3), (1, 0, 77)]), dict(q_std=20.0)])
def test_weights_accumulation(kw, fp4):
    T = kw.pop("T", 1)
    assert run_weights(128, T, 300, [300, 200, 4], fp4=fp4, seed=21, **kw) == 0


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("d_c,d_r,n_h,T", [(64, 16, 4, 1), (16, 2, 1, 2), (528, 66, 9, 1), (1024, 128, 2, 2)])
def test_weights_fp32(d_c, d_r, n_h, T, fp4):
    assert run_weights(n_h, T, 100, [T, 100, 33], dtype=F32, d_c=d_c, d_r=d_r, fp4=fp4, seed=d_c) == 0


def test_weights_fp32_odd_width():
    assert run_weights(3, 1, 50, [50, 7], dtype=F32, d_c=16, d_r=5) == 0


@pytest.mark.parametrize("ls", [2.0 ** -30, 2.0 ** 11])
def test_weights_latent_scale(ls):
    assert run_weights(128, 1, 300, [300, 20], fp4=True, ls=ls) == 0


@pytest.mark.parametrize("fp4", [False, True])
def test_weights_bad_lengths_write_nothing(fp4):
    assert run_weights(128, 1, 300, [0, 300, 301], fp4=fp4) == 7
    assert run_weights(16, 4, 300, [3, 200], fp4=fp4) == 7


def test_weights_sum_to_one_per_head():
    B, n = 3, 2000
    c4, sc, kr = random_fp4(B, n, 512, 31)
    planes = pack(c4, sc, kr)
    q = (torch.randn((B, 2, 128, 512), device=DEV) * 0.226).to(BF)
    qp = torch.randn((B, 2, 128, 64), device=DEV).to(BF)
    lens = i32([2000, 2, 1111])
    lse = torch.empty((B, 2, 128), device=DEV)
    api.mla_decode_absorb_fp4kv(dims(), q, qp, *planes, lens, 0.0722, lse=lse)
    w = api.mla_cache_weights_fp4kv(dims(), q, qp, *planes, lens, 0.0722, lse)
    assert torch.allclose(w.double().sum(-1), torch.full((B,), 256.0, dtype=torch.float64, device=DEV), rtol=1e-3)


# ------------------------------------------------------------------------------------------ evict
def run_evict(lengths, n_max, keep, sink, recent, widths=((576, BF),), acc=None, seed=0, alias=False, stride_pad=0):
    B = len(lengths)
    g = torch.Generator().manual_seed(seed)
    if acc is None:
        acc = torch.exp(2 * torch.randn((B, n_max), generator=g)) * (torch.rand((B, n_max), generator=g) > 0.2)
    planes = []
    for w, dt in widths:
        p = torch.randint(0, 256, (B, n_max, w * dt.itemsize + stride_pad), generator=g, dtype=torch.uint8).to(DEV)
        planes.append(p[..., :w * dt.itemsize].view(dt) if stride_pad % dt.itemsize == 0 else p[..., :w])
    before = [p.cpu().contiguous().view(torch.uint8).clone() for p in planes]
    lens = i32(lengths)
    err = i32([0])
    new, row_map = api.mla_cache_evict(planes, acc.to(DEV), lens, keep, sink=sink, recent=recent,
                                       new_lengths=lens if alias else None, dev_err=err)
    code = int(err.item())
    row_map, new = row_map.cpu(), new.cpu()
    for b, L in enumerate(lengths):
        want = O.evict_map(acc[b].numpy(), L, keep, sink, recent) if 0 <= L <= n_max else []
        assert row_map[b].tolist() == want + [-1] * (keep - len(want)), b
        assert int(new[b]) == len(want)
        for p, old in zip(planes, before):
            exp = old[b].clone()
            exp[:len(want)] = old[b][torch.tensor(want, dtype=torch.long)]
            assert torch.equal(p[b].cpu().contiguous().view(torch.uint8), exp)
    return code


@pytest.mark.parametrize("n_max,keep,sink,recent", [(1, 1, 0, 0), (5, 3, 1, 1), (40, 40, 3, 3), (40, 39, 0, 39), (300, 100, 4, 32),
                                                    (1025, 1024, 0, 0), (5000, 37, 30, 7), (5000, 4000, 0, 1), (20000, 9999, 4, 128)])
def test_evict_shapes(n_max, keep, sink, recent):
    lengths = [n_max, max(1, n_max // 2), 0, keep, min(keep + 1, n_max), max(1, n_max - 1)]
    assert run_evict(lengths, n_max, keep, sink, recent, seed=n_max) == 0


@pytest.mark.parametrize("widths,pad", [(((576, BF),), 0), (((256, torch.uint8), (32, torch.uint8), (64, BF)), 0),
                                        (((512, torch.uint8), (4, F32), (64, BF), (1, F32)), 0), (((7, torch.uint8),), 0),
                                        (((7, torch.uint8), (3, F32)), 4), (((512, BF), (64, BF)), 1024), (((3, BF),), 2)])
def test_evict_planes(widths, pad):
    assert run_evict([700, 333, 90], 700, 200, 4, 50, widths=widths, stride_pad=pad, alias=True) == 0


@pytest.mark.parametrize("kind", ["equal", "zeros", "two", "nan", "inf", "negative", "rising", "falling", "low_bits", "denormal"])
def test_evict_scores(kind):
    n, g = 3000, torch.Generator().manual_seed(1)
    acc = {"equal": torch.full((2, n), 0.7), "zeros": torch.zeros((2, n)) * -1.0,
           "two": (torch.rand((2, n), generator=g) > 0.5).float(),
           "rising": torch.arange(n).float().expand(2, n).contiguous(), "falling": -torch.arange(n).float().expand(2, n).contiguous(),
           "negative": torch.randn((2, n), generator=g),
           "low_bits": (1.0 + torch.randint(0, 40, (2, n), generator=g) * 2.0 ** -23),
           "denormal": torch.randint(0, 50, (2, n), generator=g) * 1e-45}.get(kind)
    if kind in ("nan", "inf"):
        acc = torch.randn((2, n), generator=g)
        acc[:, ::3] = float(kind)
        acc[1, ::7] = float("-inf")
    if kind == "zeros":
        acc[:, ::2] = 0.0
    assert run_evict([n, n - 11], n, 1200, 3, 64, acc=acc, widths=((16, torch.uint8),)) == 0


def test_evict_bad_lengths_move_nothing():
    assert run_evict([50, -1, 41, 30], 40, 20, 1, 2) == 7


def test_evict_everything_protected_and_nothing_protected():
    assert run_evict([500, 77], 500, 64, 32, 32) == 0
    assert run_evict([500, 77], 500, 64, 0, 0) == 0


def test_evict_long_sequences():
    assert run_evict([100000, 60001, 5], 100000, 40000, 4, 1024, widths=((8, torch.uint8),), seed=3) == 0


@pytest.mark.parametrize("B,n_max", [(2, 8192), (2, 8193), (40, 8193), (40, 32768), (40, 32769), (2, 32769), (12, 12288), (12, 13312)])
def test_evict_one_cta_and_cluster(B, n_max):
    lengths = [n_max - 37 * b for b in range(B)]
    assert run_evict(lengths, n_max, n_max // 2 + 1, 5, 333, widths=((4, torch.uint8),), seed=B + n_max) == 0


@pytest.mark.parametrize("kind", ["equal", "two", "nan", "low_bits"])
@pytest.mark.parametrize("keep,sink,recent", [(7000, 2500, 2600), (11999, 0, 0), (5000, 2000, 3000), (1, 0, 0)])
def test_evict_ties_in_a_cluster(kind, keep, sink, recent):
    n, g = 12000, torch.Generator().manual_seed(2)
    acc = {"equal": torch.full((2, n), -0.3), "two": (torch.rand((2, n), generator=g) > 0.5).float(),
           "nan": torch.where(torch.rand((2, n), generator=g) > 0.4, float("nan"), 1.0),
           "low_bits": 1.0 + torch.randint(0, 40, (2, n), generator=g) * 2.0 ** -23}[kind]
    assert run_evict([n, n - 1777], n, keep, sink, recent, acc=acc, widths=((16, torch.uint8),)) == 0


def test_evict_repeats_in_a_graph():
    n, keep = 4000, 1500
    acc = torch.rand((3, n), device=DEV)
    cache = torch.randn((3, n, 64), device=DEV)
    lens = i32([4000, 3999, 1200])
    want = cache.clone()
    new, row_map = api.mla_cache_evict([want], acc, lens, keep, sink=4, recent=100)
    out, m = torch.empty_like(new), torch.empty_like(row_map)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        api.mla_cache_evict([cache], acc, lens, keep, sink=4, recent=100, new_lengths=out, row_map=m)
    for _ in range(2):  # the second replay selects and moves the same rows again
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache, want) and torch.equal(out, new) and torch.equal(m, row_map)


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fp4", [True, False])
def test_serving_run(fp4):
    """Prompts appended, tokens decoded with their weights accumulated, the cache cut whenever it is full: the
    decode over the evicted cache equals the fp64 attention over exactly the rows that the oracle keeps."""
    B, n_max, keep, sink, recent, n_h = 3, 96, 64, 2, 16, 16
    d = dims(n_h)
    g = torch.Generator().manual_seed(7)
    cache = torch.zeros((B, n_max, 576), dtype=BF, device=DEV)
    planes = pack(torch.zeros((B, n_max, 256), dtype=torch.uint8), torch.zeros((B, n_max, 32), dtype=torch.uint8),
                  torch.zeros((B, n_max, 64), dtype=BF)) if fp4 else (cache[..., :512], cache[..., 512:])
    acc = torch.zeros((B, n_max), device=DEV)
    prompt = [40, 64, 17]
    x = torch.randn((B, 64, 576), generator=g).to(BF)
    held = [list(range(p)) for p in prompt]          # positions of each cached row
    store = [{} for _ in range(B)]                   # position -> (latent, key) as read back
    if fp4:
        api.mla_cache_append_fp4(d, x.to(DEV), i32([0] * B), *planes, counts=i32(prompt))
    else:
        for i in range(64):  # one token at a time; a finished prompt rewrites its last row
            j = [min(i, p - 1) for p in prompt]
            api.mla_cache_append(d, x[torch.arange(B), torch.tensor(j)].to(DEV), i32(j), *planes)
    pos, rows = list(prompt), list(prompt)
    ref_acc = [np.zeros(p) for p in prompt]

    def latent():
        return api.mla_cache_read_fp4(d, planes[0], planes[1], n_max).double().cpu() if fp4 else planes[0].double().cpu()

    for step in range(50):
        kv = torch.randn((B, 576), generator=g).to(BF).to(DEV)
        if fp4:
            api.mla_cache_append_fp4(d, kv, i32(pos), *planes, rows=i32(rows))
        else:
            api.mla_cache_append(d, kv, i32(pos), *planes, rows=i32(rows))
        for b in range(B):
            held[b].append(pos[b])
            pos[b] += 1
            rows[b] += 1
        lens = i32(rows)
        q = (torch.randn((B, n_h, 512), generator=g) * 0.3).to(BF)
        qp = torch.randn((B, n_h, 64), generator=g).to(BF)
        lse = torch.empty((B, n_h), device=DEV)
        if fp4:
            ctx = api.mla_decode_absorb_fp4kv(d, q.to(DEV), qp.to(DEV), *planes, lens, 0.0722, lse=lse)
            api.mla_cache_weights_fp4kv(d, q.to(DEV), qp.to(DEV), *planes, lens, 0.0722, lse, acc=acc, out=acc)
        else:
            lat, key = latent(), planes[1].double().cpu()
            for b in range(B):
                _, l, _ = O.latent_attention(q[b], qp[b], lat[b, :rows[b]], key[b, :rows[b]], 0.0722)
                lse[b] = torch.from_numpy(l).to(DEV)
            api.mla_cache_weights(d, q.to(DEV), qp.to(DEV), *planes, lens, 0.0722, lse, acc=acc, out=acc)
        if step % 10 == 0 or max(rows) == n_max:
            lat, key = latent(), planes[-1].double().cpu()
            for b in range(B):
                L = rows[b]
                for r in range(L):  # each row still holds the token that the bookkeeping says
                    p = held[b][r]
                    row = (lat[b, r], key[b, r])
                    if p in store[b]:
                        assert torch.equal(row[0], store[b][p][0]) and torch.equal(row[1], store[b][p][1])
                    store[b][p] = row
                if fp4:
                    want, _, _ = O.latent_attention(q[b], qp[b], lat[b, :L], key[b, :L], 0.0722)
                    assert np.abs(ctx[b].double().cpu().numpy() - want).max() <= 2e-2
        if max(rows) == n_max:
            a = acc.cpu()
            moved = [*planes, acc.unsqueeze(-1)]
            new, row_map = api.mla_cache_evict(moved, acc, lens, keep, sink=sink, recent=recent, new_lengths=lens)
            for b in range(B):
                want = O.evict_map(a[b].numpy(), rows[b], keep, sink, recent)
                assert row_map[b, :len(want)].tolist() == want
                held[b] = [held[b][t] for t in want]
                rows[b] = len(want)
                assert torch.equal(acc[b, :rows[b]].cpu(), a[b][torch.tensor(want)])
            assert lens.tolist() == rows
    assert max(pos) > n_max and all(len(h) == r for h, r in zip(held, rows))
    assert all(0 in h and 1 in h for h in held)      # the sinks stay
    del ref_acc
