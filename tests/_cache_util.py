"""Inputs and element-wise bounds of the 4-bit cache and attention-weight tests."""

import numpy as np
import torch

import oracle as O

DEV = "cuda"
V3 = (512, 64)


def random_fp4(B, n, d_c, seed, packed_r=0, dtype=torch.bfloat16):
    """A 4-bit cache with every code and scales over a wide range; with packed_r rotary features the planes
    are views of one packed row."""
    rng = np.random.default_rng(seed)
    c4 = torch.from_numpy(rng.integers(0, 256, (B, n, d_c // 2), dtype=np.uint8))
    sc = torch.from_numpy(rng.integers(0x20, 0x34, (B, n, d_c // 16), dtype=np.uint8))  # 2^-3 .. 0.6
    kr = torch.from_numpy(rng.standard_normal((B, n, packed_r or 64), dtype=np.float32)).to(dtype)
    return c4, sc, kr


def pack(c4, sc, kr):
    """One packed device row per token; returns its three views."""
    w = (c4.shape[-1], sc.shape[-1], kr.shape[-1] * kr.element_size())
    rows = torch.cat((c4, sc, kr.contiguous().view(torch.uint8)), -1).to(DEV)
    a, b, c = rows.split(w, -1)
    return a, b, c.view(kr.dtype)


def values(c4, sc, latent_scale=1.0):
    return O.fp4_values(c4.numpy(), sc.numpy(), latent_scale)


def reference(q, qp, c, kr, lengths, T, scale):
    """fp64 decode: ctx, lse, the mean |c| under the softmax weights and the bound on a score's error.

    The mean holds 2^-21 of the plain sum of |c| besides: fp16 probabilities have no steps below 2^-24, so each is off
    by up to 2^-25 beyond its relative rounding, while their sum is at least 2^7 (they are taken relative to 2^-7 of
    the largest).  That is 2^-32 of the weights' sum per key, and the mean is weighed by at least 2^-11 below.

    Scores: products of at most 11-bit by 8-bit factors are exact in fp32, and a sum of 576 of them in any order, with
    truncating adds of 2^-23, is off by at most 576 * 2^-23 of the sum of magnitudes; the scale, the base-2
    exponent and its offset add a few 2^-24 of |z|."""
    B = len(lengths)
    n_h = q.shape[-2]
    qf = np.concatenate((q.double().numpy(), qp.double().numpy()), -1).reshape(B, T, n_h, -1)
    ctx = np.zeros((B, T, n_h, c.shape[-1]))
    mean_abs = np.zeros_like(ctx)
    lse = np.full((B, T, n_h), -np.inf)
    ez = np.zeros((B, T, n_h))
    for b, L in enumerate(lengths):
        if not T <= L <= c.shape[1]:
            continue
        keys = np.concatenate((c[b, :L], kr[b, :L].double().numpy()), -1)
        for s in range(T):
            n = L - T + s + 1
            z = scale * (qf[b, s] @ keys[:n].T)
            mag = scale * (np.abs(qf[b, s]) @ np.abs(keys[:n]).T)
            m = z.max(-1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(-1, keepdims=True)
            p /= l
            ctx[b, s] = p @ keys[:n, :c.shape[-1]]
            mean_abs[b, s] = (p + 2.0 ** -21) @ np.abs(keys[:n, :c.shape[-1]])
            lse[b, s] = (m + np.log(l))[:, 0]
            ez[b, s] = (mag * 576 * 2.0 ** -23 + np.abs(z) * 2.0 ** -21).max(-1)
    return ctx, lse, mean_abs, ez


def check_decode(got, got_lse, ref, dtype):
    """|ctx error| <= one rounding to the output type, half a step (eps / 2) of the value, plus the weights' error
    times the mean |c|: a score's error ez moves a weight by 2 ez at most (itself and the normalisation), fp16
    probabilities round to 2^-11 each, and sums of up to 2^16 fp32 terms stay below 2^-12.
    fp32: no fp16 rounding, sums below 2^-14."""
    ctx, lse, mean_abs, ez = ref
    g = got.double().cpu().numpy().reshape(ctx.shape)
    half = torch.finfo(dtype).eps / 2
    own = 2.0 ** -11 + 2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -14
    bound = half * np.abs(ctx) + (own + 2 * ez[..., None]) * mean_abs * (1 + half) + 1e-30
    bad = np.abs(g - ctx) > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {(np.abs(g - ctx) / bound).max():.2f} bounds"
    if got_lse is not None:
        gl = got_lse.double().cpu().numpy().reshape(lse.shape)
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty)
        with np.errstate(invalid="ignore"):
            off = np.abs(gl - lse) > ez + 2.0 ** -12 + np.abs(lse) * 2.0 ** -22
        assert not off[~empty].any(), np.abs(gl - lse)[~empty].max()
