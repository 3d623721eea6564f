"""Eviction by token age on the GPU: single cuts against the oracle, repeated cuts against sets of positions, and a serving
run whose weights are accumulated apart."""

import numpy as np
import pytest
import torch

import oracle as O
from head_latent_attention_absorb_b200 import api

from _cache_util import DEV, pack, reference

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SCALE = 0.0722


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------ one cut
def run_evict(lengths, n_max, keep, sink, recent, positions, acc=None, seed=0, pad=0):
    """positions: numpy int32 [B, n_max]."""
    B = len(lengths)
    g = torch.Generator().manual_seed(seed)
    if acc is None:
        acc = torch.exp(2 * torch.randn((B, n_max), generator=g)) * (torch.rand((B, n_max), generator=g) > 0.2)
    plane = torch.randint(0, 256, (B, n_max, 12), generator=g, dtype=torch.uint8)
    dp = plane.to(DEV)
    pos = torch.full((B, n_max + pad), -77, dtype=torch.int32, device=DEV)[:, :n_max]
    pos.copy_(torch.from_numpy(positions))
    lens, err = i32(lengths), i32([0])
    new, row_map = api.mla_cache_evict([dp], acc.to(DEV), lens, keep, sink=sink, recent=recent, new_lengths=lens, dev_err=err,
                                       positions=pos)
    for b, L in enumerate(lengths):
        want = O.evict_map(acc[b].numpy(), L, keep, sink, recent, positions[b]) if 0 <= L <= n_max else []
        assert row_map[b].tolist() == want + [-1] * (keep - len(want)), b
        assert int(new[b]) == len(want)
        src = torch.tensor(want + list(range(len(want), n_max)), dtype=torch.long)
        assert torch.equal(dp[b].cpu(), plane[b][src])
        assert pos[b].tolist() == positions[b][src.numpy()].tolist()
    return int(err.item())


def order(kind, B, n, seed):
    rng = np.random.default_rng(seed)
    if kind == "in order":
        p = np.arange(n) + 1000 * np.arange(B)[:, None]
    elif kind == "shuffled":
        p = np.stack([rng.permutation(n) for _ in range(B)])
    elif kind == "falling":
        p = np.broadcast_to(n - np.arange(n), (B, n))
    elif kind == "ties":
        p = rng.integers(0, 7, (B, n))
    elif kind == "equal":
        p = np.full((B, n), 123456789)
    elif kind == "whole range":
        p = rng.integers(-2 ** 31, 2 ** 31, (B, n))
        p[:, 0], p[:, -1] = -2 ** 31, 2 ** 31 - 1
    else:  # two clusters of positions far apart
        p = rng.permutation(2 * n)[:n] % n + (rng.random((B, n)) > 0.5) * 1000000
    return np.ascontiguousarray(p).astype(np.int32)


ORDERS = ["in order", "shuffled", "falling", "ties", "equal", "whole range", "two"]


@pytest.mark.parametrize("kind", ORDERS)
@pytest.mark.parametrize("n_max,keep,sink,recent", [(1, 1, 0, 0), (5, 3, 1, 1), (40, 39, 0, 39), (300, 100, 4, 32), (300, 64, 64, 0),
                                                    (1025, 1024, 0, 1), (5000, 37, 30, 7), (20000, 9999, 4, 128)])
def test_one_cut(n_max, keep, sink, recent, kind):
    lengths = [n_max, max(1, n_max // 2), 0, keep, min(keep + 1, n_max), max(1, n_max - 1)]
    assert run_evict(lengths, n_max, keep, sink, recent, order(kind, 6, n_max, n_max)) == 0


@pytest.mark.parametrize("kind", ORDERS)
@pytest.mark.parametrize("keep,sink,recent", [(7000, 2500, 2600), (5000, 2000, 3000), (6000, 0, 6000), (11999, 0, 1), (1, 0, 1)])
def test_one_cut_in_a_cluster(keep, sink, recent, kind):
    n, g = 12000, torch.Generator().manual_seed(2)
    acc = torch.where(torch.rand((2, n), generator=g) > 0.4, float("inf"), torch.rand((2, n), generator=g))
    acc[:, ::5] = float("nan")
    assert run_evict([n, n - 1777], n, keep, sink, recent, order(kind, 2, n, keep), acc=acc, pad=9) == 0


@pytest.mark.parametrize("B,n_max", [(2, 8192), (2, 8193), (40, 8193), (33, 32768), (2, 32769), (1, 100001), (1, 400000)])
def test_one_cut_of_long_sequences(B, n_max):
    lengths = [n_max - 37 * b for b in range(B)]
    assert run_evict(lengths, n_max, n_max // 2 + 1, 5, 333, order("two", B, n_max, B + n_max), seed=B) == 0


def test_bad_lengths_leave_positions_alone():
    assert run_evict([50, -1, 41, 30], 40, 20, 1, 2, order("shuffled", 4, 40, 1)) == 7


def test_without_recent_rows_positions_still_move():
    assert run_evict([500, 77], 500, 64, 8, 0, order("shuffled", 2, 500, 2)) == 0


# ------------------------------------------------------------------------------------------ many cuts
def content(b, p):
    """Five numbers that tell a sequence's token at position p from every other."""
    return torch.from_numpy((np.asarray(p)[:, None] * 31 + b * 7 + np.arange(5) * 1009) % 32749).to(torch.int16)


@pytest.mark.parametrize("B,n_max,keep,sink,recent,news", [
    (3, 80, 64, 4, 16, [1, 1, 1, 3, 16, 1, 7, 2, 1, 15, 9, 1]),
    (3, 80, 40, 0, 40, [1, 2, 1, 5, 1, 1, 1, 3, 1, 1]),
    (2, 9000, 8900, 4, 1024, [100, 1, 30, 1, 77, 1, 99, 5, 1, 100, 1]),       # a cluster for each sequence
    (12, 9000, 8300, 4, 512, [700, 1, 30, 1, 300, 1, 99, 5, 1, 600, 1])])     # one CTA
def test_repeated_cuts_keep_the_newest_tokens(B, n_max, keep, sink, recent, news):
    """A cache cut after every few tokens.  What it should hold is kept as sets of positions with their weights and
    contents, apart from rows."""
    rng = np.random.default_rng(n_max)
    start = [keep - b for b in range(B)]
    plane = torch.zeros((B, n_max, 5), dtype=torch.int16, device=DEV)
    acc = torch.zeros((B, n_max), device=DEV)
    positions = torch.full((B, n_max), -1, dtype=torch.int32, device=DEV)
    held = []
    for b in range(B):
        w = rng.permutation(keep)[:start[b]].astype(np.float32) + 1
        held.append(dict(enumerate(w.tolist())))
        acc[b, :start[b]] = torch.from_numpy(w)
        positions[b, :start[b]] = torch.arange(start[b], dtype=torch.int32)
        plane[b, :start[b]] = content(b, np.arange(start[b])).to(DEV)
    lens, pos = list(start), list(start)
    for cut, new in enumerate(news):
        for b in range(B):
            p = list(range(pos[b], pos[b] + new))
            w = ((cut * 1000 + np.arange(new)) * 1e-5 + 1e-6).astype(np.float32)  # less than every older token's
            rows = slice(lens[b], lens[b] + new)
            acc[b, rows], positions[b, rows] = torch.from_numpy(w).to(DEV), i32(p)
            plane[b, rows] = content(b, p).to(DEV)
            held[b].update(zip(p, w.tolist()))
            pos[b] += new
            lens[b] += new
        length = i32(lens)
        api.mla_cache_evict([plane, acc.unsqueeze(-1)], acc, length, keep, sink=sink, recent=recent, new_lengths=length,
                            positions=positions)
        lens = length.tolist()
        got_pos, got_acc, got = positions.cpu(), acc.cpu(), plane.cpu()
        for b in range(B):
            age = sorted(held[b])
            if len(age) > keep:
                rest = sorted(age[sink:len(age) - recent], key=lambda p: -held[b][p])[:keep - sink - recent]
                held[b] = {p: held[b][p] for p in age[:sink] + age[len(age) - recent:] + rest}
            assert lens[b] == len(held[b])
            now = got_pos[b, :lens[b]].tolist()
            assert sorted(now) == sorted(held[b]), (cut, b)
            assert got_acc[b, :lens[b]].tolist() == [held[b][p] for p in now]
            assert torch.equal(got[b, :lens[b]], content(b, now))


def evict_state(n_max=3000):
    g = torch.Generator().manual_seed(n_max)
    pos = torch.stack([torch.randperm(n_max, generator=g) for _ in range(3)]).to(torch.int32)
    return dict(plane=torch.randn((3, n_max, 6), generator=g).to(DEV), acc=torch.rand((3, n_max), generator=g).to(DEV),
                lens=i32([n_max, n_max - 5, 900]), pos=pos.to(DEV), new=i32([0] * 3),
                row_map=torch.zeros((3, 1000), dtype=torch.int32, device=DEV))


def cut(s, **kw):
    api.mla_cache_evict([s["plane"], s["acc"].unsqueeze(-1)], s["acc"], s["lens"], 1000, sink=4, recent=200, positions=s["pos"],
                        new_lengths=s["new"], row_map=s["row_map"], **kw)


@pytest.mark.parametrize("n_max", [3000, 20000])
def test_streams_and_captured_cuts(n_max):
    want, start = evict_state(n_max), evict_state(n_max)
    cut(want)
    torch.cuda.synchronize()
    for as_handle in (False, True):
        s, st = evict_state(n_max), torch.cuda.Stream()
        torch.cuda.synchronize()
        cut(s, stream=st.cuda_stream if as_handle else st)
        st.synchronize()
        assert all(torch.equal(s[k], want[k]) for k in s)
    s, graph = evict_state(n_max), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cut(s)
    for _ in range(3):
        for k in s:
            s[k].copy_(start[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[k], want[k]) for k in s)


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fp4", [True, False])
def test_serving_run_by_position(fp4):
    """The serving loop with a cut after every eight tokens or fewer, a window of 16: the newest 16 tokens stay, and each row's
    weight is the sum over its token's steps in 64 bits, kept by position."""
    B, n_max, keep, sink, recent, n_h, decay = 3, 72, 64, 2, 16, 16, 0.97
    d = (n_h, 512, 64, 128, 128)
    g = torch.Generator().manual_seed(11)
    if fp4:
        planes = pack(torch.zeros((B, n_max, 256), dtype=torch.uint8), torch.zeros((B, n_max, 32), dtype=torch.uint8),
                      torch.zeros((B, n_max, 64), dtype=BF))
    else:
        cache = torch.zeros((B, n_max, 576), dtype=BF, device=DEV)
        planes = (cache[..., :512], cache[..., 512:])
    acc = torch.full((B, n_max), 7.0, device=DEV)  # an earlier user's weights: a new token's row starts from nothing
    positions = torch.full((B, n_max), -1, dtype=torch.int32, device=DEV)
    lengths, pos = i32([0] * B), i32([0, 500, 9])
    token = [{} for _ in range(B)]   # position -> [latent, key, weight in 64 bits, its bound]
    cuts = 0
    for step in range(120):
        kv = torch.randn((B, 576), generator=g).to(BF).to(DEV)
        if fp4:
            api.mla_cache_append_fp4(d, kv, pos, *planes, rows=lengths)
        else:
            api.mla_cache_append(d, kv, pos, *planes, rows=lengths)
        positions.scatter_(1, lengths.long()[:, None], pos[:, None])
        lengths += 1
        q = (torch.randn((B, n_h, 512), generator=g) * 0.3).to(BF)
        qp = torch.randn((B, n_h, 64), generator=g).to(BF)
        lse = torch.empty((B, n_h), device=DEV)
        if fp4:
            api.mla_decode_absorb_fp4kv(d, q.to(DEV), qp.to(DEV), *planes, lengths, SCALE, lse=lse)
            api.mla_cache_weights_fp4kv(d, q.to(DEV), qp.to(DEV), *planes, lengths, SCALE, lse, acc=acc, out=acc, decay=decay)
            lat = api.mla_cache_read_fp4(d, planes[0], planes[1], n_max).double().cpu()
        else:
            lat = planes[0].double().cpu()
        key, now, lens = planes[-1].double().cpu(), positions.tolist(), lengths.tolist()
        for b in range(B):
            L, p = lens[b], int(pos[b])
            token[b][p] = [lat[b, L - 1].clone(), key[b, L - 1].clone(), 0.0, 0.0]
            assert sorted(now[b][:L]) == sorted(token[b])
            # the tokens' own contents, in the cache's order of rows
            c = torch.stack([token[b][r][0] for r in now[b][:L]])
            k = torch.stack([token[b][r][1] for r in now[b][:L]])
            assert torch.equal(c, lat[b, :L]) and torch.equal(k, key[b, :L])
            if not fp4:
                lse[b] = torch.from_numpy(O.latent_attention(q[b], qp[b], c, k, SCALE)[1]).to(DEV)
            _, _, _, ez = reference(q[b:b + 1, None], qp[b:b + 1, None], c[None].numpy(), k[None], [L], 1, float(np.float32(SCALE)))
            w = O.token_weights(q[b:b + 1].double(), qp[b:b + 1].double(), c, k, float(np.float32(SCALE)), lse[b:b + 1].cpu().numpy())
            for r, wr in zip(now[b][:L], w):
                t = token[b][r]
                fresh = r == p
                t[2] = wr + (0.0 if fresh else float(np.float32(decay)) * t[2])
                # a step's own error as for one step of weights, and what the earlier ones left
                t[3] = wr * (2 * ez.max() + 2.0 ** -18 + n_h * 2.0 ** -23) + 2.0 ** -22 * t[2] + t[3] + n_h * 2.0 ** -125
        if not fp4:
            api.mla_cache_weights(d, q.to(DEV), qp.to(DEV), *planes, lengths, SCALE, lse, acc=acc, out=acc, decay=decay)
        a = acc.cpu()
        for b in range(B):
            for row, r in enumerate(now[b][:lens[b]]):
                assert abs(float(a[b, row]) - token[b][r][2]) <= token[b][r][3], (step, b, r)
        before = [now[b][:lens[b]] for b in range(B)]
        pos += 1
        if lens[0] == n_max or (step > 70 and step % 3 == 0):
            api.mla_cache_evict([*planes, acc.unsqueeze(-1)], acc, lengths, keep, sink=sink, recent=recent, new_lengths=lengths,
                                positions=positions)
            cuts += 1
            now, lens = positions.tolist(), lengths.tolist()
            for b in range(B):
                age = sorted(token[b])
                kept = now[b][:lens[b]]
                assert lens[b] == min(len(age), keep)
                assert set(age[:sink]) | set(age[-recent:]) <= set(kept)
                if len(age) > keep:  # the others by their weight on the GPU, which may round two of them together
                    weight = dict(zip(before[b], a[b].tolist()))
                    rest = set(kept) - set(age[:sink]) - set(age[-recent:])
                    gone = set(age) - set(kept)
                    assert min(weight[r] for r in rest) >= max(weight[r] for r in gone)
                token[b] = {r: token[b][r] for r in kept}
    assert cuts >= 10
