"""Rows of a 4-bit cache that only some of the new tokens see, holding NaN: a token that does not see them is not touched by
them, one that does is NaN."""

import numpy as np
import pytest
import torch

from head_latent_attention_absorb_b200 import api

from _cache_util import DEV, check_decode, pack, random_fp4, reference, values

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCALE = 0.0722


def run(n_h, T, L, hidden, what, dtype=BF, d_c=512, d_r=64, seed=0):
    """Sequence 0 has its row L - 1 - hidden spoilt, sequence 1 is clean and one row longer."""
    lengths = [L, L + 1]
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((2, T, n_h, d_c), generator=g) * 0.226).to(dtype)
    qp = torch.randn((2, T, n_h, d_r), generator=g).to(dtype)
    c4, sc, kr = random_fp4(2, L + 3, d_c, seed + 1, d_r, dtype)
    ref = reference(q, qp, values(c4, sc), kr, lengths, T, float(np.float32(SCALE)))
    row = L - 1 - hidden
    if what == "key":
        kr[0, row, 5] = float("nan")
    elif what == "key inf":
        kr[0, row] = float("inf")
    else:
        sc[0, row, what] = 0x7F
    planes = pack(c4, sc, kr) if d_c == 512 else (c4.to(DEV), sc.to(DEV), kr.to(DEV))
    lse = torch.empty((2, T, n_h), device=DEV)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    ctx = api.mla_decode_absorb_fp4kv((n_h, d_c, d_r, 1, 1), q.to(DEV), qp.to(DEV), *planes, lens, SCALE, lse=lse)
    seeing = T - 1 - hidden  # the first token that sees the row
    assert torch.isnan(ctx[0, seeing:].float()).all() and torch.isnan(lse[0, seeing:]).all()
    clean = torch.ones((2, T), dtype=torch.bool)
    clean[0, seeing:] = False
    m = clean.numpy()[..., None]
    check_decode(torch.from_numpy(np.where(m[..., None], ctx.double().cpu().numpy(), 0)),
                 torch.from_numpy(np.where(m, lse.double().cpu().numpy(), 0)),
                 tuple(np.where(m[..., None] if r.ndim == 4 else m, r, 0) for r in ref), dtype)
    if what not in ("key", "key inf") or dtype == F32:
        w = api.mla_cache_weights_fp4kv((n_h, d_c, d_r, 1, 1), q.to(DEV), qp.to(DEV), *planes, lens, SCALE, lse)
        assert not torch.isnan(w[1]).any() and torch.isnan(w[0, row])


@pytest.mark.parametrize("what", [0, 9, 15, 16, 31, "key", "key inf"])
@pytest.mark.parametrize("n_h,T", [(128, 2), (128, 3), (16, 4), (100, 3), (1, 9)])
def test_hidden_rows(n_h, T, what):
    for hidden in {0, T - 2}:
        run(n_h, T, 300, hidden, what, seed=n_h)


@pytest.mark.parametrize("L", [3, 64, 65, 127, 128, 129, 130, 192, 256, 257, 385, 1000, 5000])
def test_hidden_rows_by_length(L):
    run(16, 3, L, 0, 7, seed=L)
    run(128, 3, L, 1, 20, seed=L)


@pytest.mark.parametrize("hidden", [0, 1, 70, 127, 128, 149, 258])
def test_many_tokens(hidden):
    run(5, 260, 700, hidden, 3, seed=hidden)     # eleven groups of query rows, hidden rows in four tiles


@pytest.mark.parametrize("what", [0, 2, "key", "key inf"])
def test_fp32(what):
    run(3, 4, 90, 1, what, dtype=F32, d_c=48, d_r=10)
