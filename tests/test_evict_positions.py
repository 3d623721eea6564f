"""Eviction by token age on the CPU: the oracle over repeated cuts, and what the calls refuse."""

import numpy as np
import pytest
import torch

import oracle as O
from head_latent_attention_absorb_b200 import _capi, api
from head_latent_attention_absorb_b200.build import build

P = 0x10000  # an aligned non-NULL address; every call below fails validation before using it
INVALID, UNSUPPORTED = 1, 2


@pytest.mark.parametrize("every", [1, 3, 16, 40])
def test_the_newest_tokens_survive_repeated_cuts(every):
    """A full cache cut after every few tokens, whose weights are small: what stays are the sinks, the newest tokens
    and the heaviest of the others, told apart by position alone."""
    rng = np.random.default_rng(every)
    keep, sink, recent = 64, 4, 16
    held = {p: float(w) for p, w in enumerate(rng.random(64) * 4)}     # position -> weight
    positions, acc = list(held), list(held.values())
    for cut in range(200 // every):
        for _ in range(every):
            p = max(positions) + 1
            w = float(rng.random() * 0.05)
            positions.append(p)
            acc.append(w)
            held[p] = w
        m = O.evict_map(np.array(acc), len(acc), keep, sink, recent, positions)
        positions, acc = [positions[t] for t in m], [acc[t] for t in m]
        order = sorted(held)
        newest = order[-recent:]
        rest = sorted((p for p in order[sink:-recent]), key=lambda p: -held[p])[:keep - sink - recent]
        held = {p: held[p] for p in order[:sink] + newest + rest}
        assert sorted(positions) == sorted(held), cut
        assert all(held[p] == w for p, w in zip(positions, acc))
        assert positions[:sink] == [0, 1, 2, 3]


def test_rows_in_order_of_age_need_no_positions():
    rng = np.random.default_rng(0)
    acc = rng.random(100)
    for n, keep, sink, recent in ((100, 40, 3, 12), (100, 40, 0, 40), (100, 40, 40, 0), (60, 59, 5, 0)):
        want = O.evict_map(acc, n, keep, sink, recent)
        assert O.evict_map(acc, n, keep, sink, recent, 7 * np.arange(100) - 300) == want
        assert O.evict_map(acc, n, keep, sink, recent, np.full(100, 5)) == want  # equal positions: the higher row


def test_evict_map_by_position_on_a_worked_case():
    acc = [9, 1, 5, 1, 7, 3, 1, 8]
    # sink row 0; the newest of rows 1..7 is row 3; of the others the heaviest two are 7 and 4
    assert O.evict_map(acc, 8, 4, 1, 1, [0, 1, 2, 99, 4, 5, 6, 7]) == [0, 4, 7, 3]
    # the sink is kept whatever its position, and is not among the newest of the others
    assert O.evict_map(acc, 8, 3, 1, 1, [50, 1, 2, 40, 4, 5, 6, 7]) == [0, 3, 7]


@pytest.fixture(scope="module")
def L():
    build(quiet=True)
    return _capi.lib()


@pytest.mark.parametrize("kw,want", [
    (dict(posb=15), INVALID), (dict(keep=0), INVALID), (dict(sink=5, recent=4), INVALID), (dict(acc=0), INVALID),
    (dict(map=0), INVALID), (dict(n=5), INVALID), (dict(B=65536), UNSUPPORTED), (dict(n_max=400001, accb=1 << 20, posb=1 << 20), UNSUPPORTED)])
def test_evict_at_refuses(L, kw, want):
    a = dict(B=2, n_max=16, acc=P, accb=16, lens=P, keep=8, sink=1, recent=2, pos=P, posb=16, new=P, map=P, n=1)
    a.update(kw)
    arr = (_capi.MLARows * 1)(_capi.MLARows(P, 1 << 40, 64, 64))
    assert L.mla_cache_evict_at(a["B"], a["n_max"], arr, a["n"], a["acc"], a["accb"], a["lens"], a["keep"], a["sink"], a["recent"],
                                a["pos"], a["posb"], a["new"], a["map"], 0, 0) == want, L.mla_last_error_message()


def test_binding_refuses_wrong_positions():
    plane, acc, lens = torch.zeros((2, 16, 8)), torch.zeros((2, 16)), torch.full((2,), 16, dtype=torch.int32)
    for bad, kind in ((torch.zeros((2, 15), dtype=torch.int32), ValueError), (torch.zeros((2, 16)), TypeError),
                      (torch.zeros((2, 16), dtype=torch.int64), TypeError), (torch.zeros((2, 16, 1), dtype=torch.int32), ValueError),
                      (torch.zeros((2, 32), dtype=torch.int32)[:, ::2], ValueError)):
        with pytest.raises(kind, match="positions"):
            api.mla_cache_evict([plane], acc, lens, 8, positions=bad)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.mla_cache_evict([plane], acc, lens, 8, positions=torch.zeros((2, 16), dtype=torch.int32))
