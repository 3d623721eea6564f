"""Oracle of the 4-bit latent cache, of the accumulated attention weights and of the eviction (fp64)."""

from __future__ import annotations

import numpy as np

from .mla_oracle import e4m3_value, rms_norm, rope_interleaved

# the E2M1 magnitudes by code: S.EE.M with bias 1, subnormal at exponent 0
E2M1 = np.array([m / 2.0 if e == 0 else (1 + m / 2.0) * 2.0 ** (e - 1) for e in range(4) for m in range(2)])
# the E4M3 magnitudes by code, without the NaN
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def nearest_code(v: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Code of the nearest magnitude of an ascending grid, ties to the even code, saturating."""
    v = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def fp4_quantise(y: np.ndarray, latent_scale: float = 1.0):
    """Rows y [..., d] to (c4 uint8 [..., d / 2], scale uint8 [..., d / 16])."""
    y = np.asarray(y, dtype=np.float64) / latent_scale
    blocks = y.reshape(*y.shape[:-1], -1, 16)
    with np.errstate(invalid="ignore"):
        amax = np.abs(blocks).max(-1)
        s8 = nearest_code(np.nan_to_num(amax) / 6.0, E4M3)
        nan = np.isnan(amax)
        s = E4M3[s8][..., None]
        r = np.where((s > 0) & ~nan[..., None], blocks / np.where(s > 0, s, 1.0), 0.0)
    code = nearest_code(r, E2M1) | np.where(r < 0, 8, 0)
    s8 = np.where(nan, 0x7F, s8)
    code = code.reshape(y.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), s8.astype(np.uint8)


def fp4_values(c4: np.ndarray, s8: np.ndarray, latent_scale: float = 1.0) -> np.ndarray:
    """The values [..., d] of 4-bit rows."""
    c4 = np.asarray(c4).astype(np.int64)
    code = np.stack((c4 & 15, c4 >> 4), -1).reshape(*c4.shape[:-1], -1)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(e4m3_value(np.asarray(s8)), 16, -1) * latent_scale


def cache_append_fp4(kv_a, d_c: int, positions, gain=None, eps: float = 1e-6, base: float = 10000.0,
                     latent_scale: float = 1.0):
    """Token rows kv_a [n, d_c + d_r] at positions [n]: (c4, scale, rotated keys [n, d_r])."""
    x = np.asarray(kv_a, dtype=np.float64)
    g = np.ones(d_c) if gain is None else np.asarray(gain, dtype=np.float64)
    c4, s8 = fp4_quantise(rms_norm(x[:, :d_c], g, eps), latent_scale)
    return c4, s8, rope_interleaved(x[:, d_c:], positions, base)


def token_weights(q_tilde, q_pe, c_kv, k_r, scale: float, lse):
    """Attention weight of each of L rows, summed over T tokens and their heads.  q_tilde [T, n_h, d_c],
    lse [T, n_h] (-inf: no softmax); token s sees rows t <= L - T + s."""
    q = np.concatenate((np.asarray(q_tilde, np.float64), np.asarray(q_pe, np.float64)), -1)
    keys = np.concatenate((np.asarray(c_kv, np.float64), np.asarray(k_r, np.float64)), -1)
    T, L = q.shape[0], keys.shape[0]
    w = np.zeros(L)
    for s in range(T):
        for h in range(q.shape[1]):
            n = L - T + s + 1
            if np.isneginf(lse[s][h]):
                continue
            w[:n] += np.exp(scale * (keys[:n] @ q[s, h]) - float(lse[s][h]))
    return w


def evict_map(acc, length: int, keep: int, sink: int, recent: int, positions=None):
    """The rows that rows 0 .. min(length, keep) - 1 held before the eviction.  positions: of each row's token
    (None: rows in order of age)."""
    if length <= keep:
        return list(range(length))
    w = [float(v) for v in acc[:length]]
    age = range(length) if positions is None else [int(p) for p in positions[:length]]
    by_age = sorted(range(sink, length), key=lambda t: (age[t], t))
    newest, rest = by_age[len(by_age) - recent:], by_age[:len(by_age) - recent]
    rank = sorted(rest, key=lambda t: (np.isnan(w[t]), -w[t] if w[t] == w[t] else 0.0, t))
    held = set(range(sink)) | set(newest) | set(rank[:keep - sink - recent])
    late = [t for t in range(keep, length) if t in held]
    holes = [i for i in range(keep) if i not in held]
    assert len(late) == len(holes)
    out = list(range(keep))
    for i, t in zip(holes, late):
        out[i] = t
    return out
