"""Timed cases of the 4-bit latent cache and of eviction by attention weight.

Five operators that let a latent cache hold longer contexts in less memory:

* append   ``mla_cache_append_fp4`` (new tokens normalised, quantised and written) followed by
           ``mla_cache_read_fp4`` (the written rows as the values they stand for)
* decode   ``mla_decode_absorb_fp4kv``: the absorbed decode over the 4-bit cache
* weights  ``mla_cache_weights`` / ``mla_cache_weights_fp4kv``: the attention weight that each cached
           row received, summed over heads and new tokens and accumulated
* evict    ``mla_cache_evict``: the rows of least accumulated weight leave the cache

With ``own`` false, ``run`` computes the plain form in elementary torch operations; with ``own`` true it
makes the library's calls.

The 4-bit format: a latent row is cut into blocks of 16 features; a block holds sixteen E2M1 codes
(0, .5, 1, 1.5, 2, 3, 4, 6 and a sign; feature 2i in the low half of byte i) and one E4M3 scale,
value = code * scale * latent_scale with a power of two latent_scale for the whole cache.
"""

import math

import torch

own = False

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_V3 = {"d_c": 512, "d_r": 64, "d_h": 128, "d_v": 128}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token for each sequence of a batch: what every decode step of a server does first
        dict(name="append_token_b32", kind="append", dtype="bf16", B=32, T=1, n_max=4096, gain=True, lo=1, hi=1, **_V3),
        # a padded batch of prompts written at once after their prefill; prompts of odd lengths
        dict(name="append_prompts_b4", kind="append", dtype="bf16", B=4, T=4095, n_max=4096, gain=True, lo=777,
             hi=4095, **_V3),
        # one short conversation, one new token: latency
        dict(name="decode_b1_n1000", kind="decode", dtype="bf16", B=1, T=1, n_h=128, n_max=1024, lo=1000, hi=1000,
             **_V3),
        # the batch decode at the size of the bench's decode step
        dict(name="decode_b32_n4096", kind="decode", dtype="bf16", B=32, T=1, n_h=128, n_max=4096, lo=4096, hi=4096,
             **_V3),
        # long and short contexts in one batch, the bench's ragged range
        dict(name="decode_ragged_b8_64k", kind="decode", dtype="bf16", B=8, T=1, n_h=128, n_max=65536, lo=1024,
             hi=65536, **_V3),
        # a rank of eight with 16 of the 128 heads, two new tokens per sequence (speculative decoding)
        dict(name="decode_heads16_t2_b32", kind="decode", dtype="bf16", B=32, T=2, n_h=16, n_max=8192, lo=500,
             hi=8191, **_V3),
        # fp32 at small, odd widths: the type and sizes of the library's any-dimension path
        dict(name="decode_f32_small", kind="decode", dtype="f32", B=3, T=1, n_h=4, n_max=200, lo=64, hi=193, d_c=64,
             d_r=16, d_h=32, d_v=32),
        # the weights of a bf16 cache at the bench's decode size
        dict(name="weights_b32_n4096", kind="weights", dtype="bf16", cache="plain", B=32, T=1, n_h=128, n_max=4096,
             lo=4096, hi=4096, **_V3),
        # the same over a 4-bit cache with ragged lengths
        dict(name="weights_fp4_b8_16k", kind="weights", dtype="bf16", cache="fp4", B=8, T=1, n_h=128, n_max=16384,
             lo=1000, hi=16384, **_V3),
        # a bf16 cache of long contexts cut to half its rows
        dict(name="evict_b4_32k", kind="evict", dtype="bf16", cache="plain", B=4, n_max=32768, lo=20001, hi=32768,
             keep=16384, sink=4, recent=1024, **_V3),
        # a 4-bit cache that makes room for its next tokens: a few rows leave each sequence
        dict(name="evict_fp4_b32_4k", kind="evict", dtype="bf16", cache="fp4", B=32, n_max=4096, lo=3900, hi=4096,
             keep=3840, sink=4, recent=256, **_V3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "append", "decode", "decode", "decode", "weights", "weights", "evict", "evict"])
    if kind == "append":
        B = _log(rng, 1, 64)
        T = rng.choice([1, _log(rng, 1, max(1, 16384 // B))])
        n_max = T + _log(rng, 1, 4096)
        small = rng.random() < 0.2
        dims = dict(d_c=16 * rng.randint(1, 40), d_r=2 * rng.randint(1, 48), d_h=32, d_v=32) if small else dict(_V3)
        return dict(kind=kind, dtype="f32" if small else "bf16", B=B, T=T, n_max=n_max, gain=rng.random() < 0.7,
                    lo=rng.randint(1, T), hi=T, **dims)
    if kind == "evict":
        B = _log(rng, 1, 16)
        n_max = _log(rng, 32, 98304 // B)
        hi = rng.randint(max(1, n_max // 2), n_max)
        keep = rng.randint(1, max(1, hi))
        sink = rng.randint(0, min(keep, 8))
        return dict(kind=kind, dtype="bf16", cache=rng.choice(["plain", "fp4"]), B=B, n_max=n_max,
                    lo=rng.randint(1, hi), hi=hi, keep=keep, sink=sink, recent=rng.randint(0, (keep - sink) // 2),
                    **_V3)
    T = rng.choice([1, 1, 1, 2, 3, 4])
    if rng.random() < 0.15:
        B = rng.randint(1, 4)
        n_max = rng.randint(T, 500)
        dims = dict(d_c=16 * rng.randint(1, 40), d_r=2 * rng.randint(1, 48), d_h=32, d_v=32)
        n_h, dtype = rng.randint(1, 9), "f32"
    else:
        B, n_h = _log(rng, 1, 48), rng.choice([128, 128, 128, 64, 32, 16, 20])
        n_max = max(T, _log(rng, 16, min(65536, 262144 // (B * T))))
        dims, dtype = dict(_V3), "bf16"
    hi = rng.randint(max(T, n_max // 2), n_max)
    c = dict(kind=kind, dtype=dtype, B=B, T=T, n_h=n_h, n_max=n_max, lo=rng.randint(T, hi), hi=hi, **dims)
    if kind == "weights":
        c["cache"] = rng.choice(["plain", "fp4"])
    return c


def _lengths(case):
    """Lengths of the batch, spread over [lo, hi] with both ends taken, the longest first."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if b == 0 else lo if b == B - 1 else lo + ((hi - lo) * ((b * 7919) % 1009)) // 1009 for b in range(B)]


def _row_bytes(case):
    d_c, d_r = case["d_c"], case["d_r"]
    es = 2 if case["dtype"] == "bf16" else 4
    fp4 = case["kind"] in ("append", "decode") or case["cache"] == "fp4"
    return (d_c // 2 + d_c // 16 if fp4 else d_c * es) + d_r * es


def work(case):
    d_c, d_r, n = case["d_c"], case["d_r"], sum(_lengths(case))
    es = 2 if case["dtype"] == "bf16" else 4
    row = _row_bytes(case)
    if case["kind"] == "append":
        # rows in, cache rows out, and the read-back of the 4-bit part (padding comes back as zeros)
        quant = d_c // 2 + d_c // 16
        return {"bytes": n * ((d_c + d_r) * es + row + quant) + case["B"] * case["T"] * d_c * es + d_c * 4,
                "flops": n * (10 * d_c + 6 * d_r)}
    if case["kind"] == "evict":
        keep, sink, recent = case["keep"], case["sink"], case["recent"]
        moved = 0.0
        for L in _lengths(case):
            if L > keep:
                free = max(1, L - sink - recent)
                moved += max(0, min(keep, L - recent) - sink) * (1.0 - (keep - sink - recent) / free)
        return {"bytes": int(4 * n + 2 * moved * row + 4 * case["B"] * keep), "flops": 4 * n}
    rows = case["B"] * case["T"] * case["n_h"]
    if case["kind"] == "weights":
        return {"bytes": n * (row + 8) + rows * ((d_c + d_r) * es + 4),
                "flops": 2 * n * case["T"] * case["n_h"] * (d_c + d_r)}
    return {"bytes": n * row + rows * ((2 * d_c + d_r) * es + 4),
            "flops": 2 * n * case["T"] * case["n_h"] * (2 * d_c + d_r)}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _make_fp4(shape, g):
    """A 4-bit cache as an earlier fill left it: RMS-normalised rows, block scale amax / 6."""
    B, n, d = shape
    c4 = torch.empty((B, n, d // 2), dtype=torch.uint8, device="cuda")
    sc = torch.empty((B, n, d // 16), dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for b in range(B):
        x = torch.randn((n, d), generator=g, device="cuda").reshape(n, d // 16, 16)
        s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        r = x / s.float().clamp_min(2.0 ** -9)[..., None]
        code = torch.bucketize(r.abs(), edges).to(torch.uint8) | ((r < 0).to(torch.uint8) << 3)
        code = code.reshape(n, d // 2, 2)
        c4[b] = code[..., 0] | (code[..., 1] << 4)
        sc[b] = s.view(torch.uint8)
    return c4, sc


def prepare(case, seed):
    g = _gen(seed)
    dt, B, n_max, d_c, d_r = _DT[case["dtype"]], case["B"], case["n_max"], case["d_c"], case["d_r"]
    lens = _lengths(case)
    s = {"case": case, "dims": (case.get("n_h", 128), d_c, d_r, case["d_h"], case["d_v"])}
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["kind"] == "append":
        T = case["T"]
        s["kv_a"] = torch.randn((B, T, d_c + d_r), generator=g, device="cuda").to(dt)
        s["gain"] = (0.5 + torch.rand(d_c, generator=g, device="cuda")) if case["gain"] else None
        # each sequence goes on where it stands: its next free row is its next position
        start = torch.randint(0, n_max - T + 1, (B,), generator=g, device="cuda")
        s["positions"] = start.to(torch.int32)
        s["counts"] = torch.tensor(lens, **i32)
        s["c4"] = torch.zeros((B, n_max, d_c // 2), dtype=torch.uint8, device="cuda")
        s["sc"] = torch.zeros((B, n_max, d_c // 16), dtype=torch.uint8, device="cuda")
        s["k_r"] = torch.zeros((B, n_max, d_r), dtype=dt, device="cuda")
        s["out"] = torch.empty((B, T, d_c), dtype=dt, device="cuda")
        return s
    s["lengths"] = torch.tensor(lens, **i32)
    fp4 = case["kind"] == "decode" or case["cache"] == "fp4"
    if fp4:
        s["c4"], s["sc"] = _make_fp4((B, n_max, d_c), g)
        s["k_r"] = torch.randn((B, n_max, d_r), generator=g, device="cuda").to(dt)
    else:
        # one packed row per token, the latent first
        cache = torch.empty((B, n_max, d_c + d_r), dtype=dt, device="cuda")
        for b in range(B):
            cache[b] = torch.randn((n_max, d_c + d_r), generator=g, device="cuda").to(dt)
        s["c_kv"], s["k_r"] = cache[..., :d_c], cache[..., d_c:]
    if case["kind"] == "evict":
        # accumulated weights are heavy-tailed; rows that no query looked at hold exact zeros (ties)
        acc = torch.exp(2.0 * torch.randn((B, n_max), generator=g, device="cuda"))
        s["acc"] = acc * (torch.rand((B, n_max), generator=g, device="cuda") > 0.1)
        return s
    T, n_h = case["T"], case["n_h"]
    # absorbed queries: 128 content features of unit variance through weights of deviation 0.02
    s["q_tilde"] = (torch.randn((B, T, n_h, d_c), generator=g, device="cuda") * 0.226).to(dt)
    s["q_pe"] = torch.randn((B, T, n_h, d_r), generator=g, device="cuda").to(dt)
    s["scale"] = 1.0 / math.sqrt(case["d_h"] + d_r)
    if case["kind"] == "weights":
        s["acc"] = torch.rand((B, n_max), generator=g, device="cuda")
        s["out"] = torch.zeros((B, n_max), dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty((B, T, n_h), dtype=torch.float32, device="cuda")
        for b in range(B):
            s["lse"][b] = torch.logsumexp(_scores(s, b, lens[b]), -1)
    else:
        s["lse"] = torch.empty((B, T, n_h), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------
def _e4m3(v):
    """v >= 0 (float64) to the nearest E4M3 value, ties to even, saturating at 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.where(torch.isnan(v), v, (torch.round(v / step) * step).clamp_max(448.0))


def _e2m1(r):
    """|r| (float64) to the index of the nearest E2M1 magnitude, ties to the even index."""
    a = r.abs()
    up = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    idx = torch.zeros_like(a, dtype=torch.uint8)
    for i, edge in enumerate(up):
        idx += ((a > edge) if i % 2 == 0 else (a >= edge)).to(torch.uint8)
    return idx


def _values(c4, sc, latent_scale=1.0):
    """The fp32 values of 4-bit rows."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float32, device=c4.device)
    code = torch.stack((c4 & 15, c4 >> 4), -1).flatten(-2)
    s = sc.view(torch.float8_e4m3fn).float() * latent_scale
    v = grid[code.int()].reshape(*sc.shape, 16) * s[..., None]
    return v.flatten(-2)


def _latent(s, b, L):
    if "c4" in s:
        return _values(s["c4"][b, :L], s["sc"][b, :L])
    return s["c_kv"][b, :L].float()


def _scores(s, b, L, c=None):
    """Scaled scores [T, n_h, L] of sequence b, -inf where a new token does not see a row."""
    c = _latent(s, b, L) if c is None else c
    T = s["q_tilde"].shape[1]
    z = s["q_tilde"][b].float() @ c.t() + s["q_pe"][b].float() @ s["k_r"][b, :L].float().t()
    z = z * s["scale"]
    if T > 1:
        t = torch.arange(L, device=z.device)
        last = L - T + torch.arange(T, device=z.device)
        z = z.masked_fill((t[None, :] > last[:, None])[:, None, :], float("-inf"))
    return z


def _plain_append(s):
    case = s["case"]
    B, T, d_c, d_r = case["B"], case["T"], case["d_c"], case["d_r"]
    x = s["kv_a"].double()
    y = x[..., :d_c]
    y = y * (1.0 / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6))
    if s["gain"] is not None:
        y = y * s["gain"].double()
    y = y.reshape(B, T, d_c // 16, 16)
    scale = _e4m3(y.abs().amax(-1) / 6.0)
    r = y / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    r = torch.where(scale[..., None] > 0, r, torch.zeros_like(r))
    code = (_e2m1(r) | ((r < 0).to(torch.uint8) << 3)).reshape(B, T, d_c // 2, 2)
    c4 = code[..., 0] | (code[..., 1] << 4)
    sc = scale.float().to(torch.float8_e4m3fn).view(torch.uint8)
    pos = s["positions"].long()[:, None] + torch.arange(T, device=x.device)
    theta = 10000.0 ** (-torch.arange(0, d_r, 2, dtype=torch.float64, device=x.device) / d_r)
    ang = pos.double()[..., None] * theta
    cos, sin = torch.cos(ang), torch.sin(ang)
    k = x[..., d_c:]
    rot = torch.stack((k[..., 0::2] * cos - k[..., 1::2] * sin, k[..., 0::2] * sin + k[..., 1::2] * cos), -1)
    rot = rot.flatten(-2).to(s["k_r"].dtype)
    live = torch.arange(T, device=x.device)[None, :] < s["counts"][:, None]
    bi, ti = torch.nonzero(live, as_tuple=True)
    row = pos[bi, ti]
    s["c4"][bi, row], s["sc"][bi, row], s["k_r"][bi, row] = c4[bi, ti], sc[bi, ti], rot[bi, ti]
    bb = torch.arange(B, device=x.device)[:, None]
    v = _values(s["c4"][bb, pos], s["sc"][bb, pos]) * live[..., None]
    return v.to(s["k_r"].dtype), s["k_r"]


def _plain_decode(s):
    case = s["case"]
    ctx = torch.empty_like(s["q_tilde"])
    for b, L in enumerate(_lengths(case)):
        c = _latent(s, b, L)
        z = _scores(s, b, L, c)
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        l = p.sum(-1, keepdim=True)
        ctx[b] = ((p @ c) / l).to(ctx.dtype)
        s["lse"][b] = (m + torch.log(l))[..., 0]
    return ctx, s["lse"]


def _plain_weights(s):
    T = s["case"]["T"]
    for b, L in enumerate(_lengths(s["case"])):
        w = torch.exp(_scores(s, b, L) - s["lse"][b][..., None]).sum((0, 1))
        old = s["acc"][b, :L].clone()
        old[L - T:] = 0.0
        s["out"][b, :L] = old + w
    return s["out"]


def _planes(s):
    """The row arrays of the cache: rows move byte for byte, so codes and scales count as whole numbers."""
    return [s["c4"], s["sc"], s["k_r"]] if "c4" in s else [s["c_kv"], s["k_r"]]


def _plain_evict(s):
    case = s["case"]
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    lens, dev = _lengths(case), s["acc"].device
    new = torch.tensor([min(L, keep) for L in lens], dtype=torch.int32, device=dev)
    row_map = torch.full((case["B"], keep), -1, dtype=torch.int32, device=dev)
    for b, L in enumerate(lens):
        if L <= keep:
            row_map[b, :L] = torch.arange(L, dtype=torch.int32, device=dev)
            continue
        order = torch.sort(s["acc"][b, sink:L - recent], descending=True, stable=True).indices + sink
        kept = torch.zeros(L, dtype=torch.bool, device=dev)
        kept[order[:keep - sink - recent]] = True
        kept[:sink] = True
        kept[L - recent:] = True
        holes = torch.nonzero(~kept[:keep])[:, 0]
        moved = torch.nonzero(kept[keep:])[:, 0] + keep
        row_map[b] = torch.arange(keep, dtype=torch.int32, device=dev)
        row_map[b, holes] = moved.to(torch.int32)
        for p in _planes(s):
            p[b, holes] = p[b, moved]
    return [*_planes(s), new, row_map]


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(state):
    s = state
    kind = s["case"]["kind"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "weights": _plain_weights,
                "evict": _plain_evict}[kind](s)
    from head_latent_attention_absorb_b200 import api

    if kind == "append":
        api.mla_cache_append_fp4(s["dims"], s["kv_a"], s["positions"], s["c4"], s["sc"], s["k_r"],
                                 counts=s["counts"], gain=s["gain"])
        v = api.mla_cache_read_fp4(s["dims"], s["c4"], s["sc"], s["case"]["T"], first=s["positions"],
                                   counts=s["counts"], out=s["out"])
        return v, s["k_r"]
    if kind == "decode":
        ctx = api.mla_decode_absorb_fp4kv(s["dims"], s["q_tilde"], s["q_pe"], s["c4"], s["sc"], s["k_r"],
                                          s["lengths"], s["scale"], lse=s["lse"])
        return ctx, s["lse"]
    if kind == "weights":
        if "c4" in s:
            return api.mla_cache_weights_fp4kv(s["dims"], s["q_tilde"], s["q_pe"], s["c4"], s["sc"], s["k_r"],
                                               s["lengths"], s["scale"], s["lse"], acc=s["acc"], out=s["out"])
        return api.mla_cache_weights(s["dims"], s["q_tilde"], s["q_pe"], s["c_kv"], s["k_r"], s["lengths"],
                                     s["scale"], s["lse"], acc=s["acc"], out=s["out"])
    case = s["case"]
    new, row_map = api.mla_cache_evict(_planes(s), s["acc"], s["lengths"], case["keep"], sink=case["sink"],
                                       recent=case["recent"])
    return [*_planes(s), new, row_map]


# ------------------------------------------------------------------------------------------
# the definition in 64 bits, on the same inputs
# ------------------------------------------------------------------------------------------
def _nearest(v, table):
    """Nearest entry of an ascending table whose even entries win ties (float64)."""
    hi = torch.searchsorted(table, v.contiguous()).clamp(1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(take_hi, table[hi], table[lo])


def _decoded(s, b, L):
    if "c4" not in s:
        return s["c_kv"][b, :L].double()
    byte = s["c4"][b, :L].long()
    code = torch.empty((L, 2 * byte.shape[1]), dtype=torch.long, device=byte.device)
    code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
    mag, exp, man = code % 8, code % 8 // 2, code % 2
    val = torch.where(exp == 0, 0.5 * man.double(), (1.0 + 0.5 * man) * torch.exp2(exp.double() - 1))
    val = torch.where(code >= 8, -val, val)
    sb = s["sc"][b, :L].long()
    se, sm = sb // 8 % 16, sb % 8
    sv = torch.where(se == 0, sm.double() * 2.0 ** -9, (1.0 + sm / 8.0) * torch.exp2(se.double() - 7))
    return val * sv.repeat_interleave(16, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "evict":
        return _exact_evict(s)
    if case["kind"] == "append":
        d_c, d_r, T, B = case["d_c"], case["d_r"], case["T"], case["B"]
        e4 = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
                          [:127], dtype=torch.float64, device="cuda")
        e2 = torch.tensor(_GRID, dtype=torch.float64, device="cuda")
        val = torch.zeros((B, T, d_c), dtype=torch.float64, device="cuda")
        k_r = s["k_r"].double()
        freq = torch.exp(-math.log(10000.0) * 2.0 / d_r * torch.arange(d_r // 2, dtype=torch.float64, device="cuda"))
        for b, n in enumerate(_lengths(case)):
            x = s["kv_a"][b, :n, :d_c].double()
            y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d_c + 1e-6)
            y = (y if s["gain"] is None else y * s["gain"].double()).view(n, -1, 16)
            sv = _nearest(y.abs().max(-1).values / 6.0, e4)[..., None]
            mag = _nearest(y.abs() / sv.clamp_min(2.0 ** -9), e2) * sv
            val[b, :n] = torch.where(y < 0, -mag, mag).view(n, d_c)
            p0 = int(s["positions"][b])
            z = torch.view_as_complex(s["kv_a"][b, :n, d_c:].double().reshape(n, d_r // 2, 2).contiguous())
            pos = torch.arange(p0, p0 + n, dtype=torch.float64, device="cuda")
            turn = pos[:, None] * freq
            z = z * torch.complex(torch.cos(turn), torch.sin(turn))
            k_r[b, p0:p0 + n] = torch.view_as_real(z).reshape(n, d_r)
        return val, k_r
    n_h, T = case["n_h"], case["T"]
    ctx, lse = [], []
    out = s["out"].double() if case["kind"] == "weights" else None
    for b, L in enumerate(_lengths(case)):
        c, k = _decoded(s, b, L), s["k_r"][b, :L].double()
        keys = torch.cat((c, k), 1)
        q = torch.cat((s["q_tilde"][b], s["q_pe"][b]), -1).double().reshape(T * n_h, -1)
        tok = torch.arange(T * n_h, device="cuda") // n_h
        z = torch.mm(q, keys.t()) * s["scale"]
        seen = torch.arange(L, device="cuda")[None, :] <= (L - T + tok)[:, None]
        z = torch.where(seen, z, torch.full_like(z, -math.inf))
        if case["kind"] == "weights":
            w = torch.exp(z - s["lse"][b].double().reshape(-1, 1)).sum(0)
            out[b, :L] = w
            out[b, :L - T] += s["acc"][b, :L - T].double()
        else:
            ctx.append(torch.mm(torch.softmax(z, -1), c).view(T, n_h, -1))
            lse.append(torch.logsumexp(z, -1).view(T, n_h))
    return out if case["kind"] == "weights" else (torch.stack(ctx), torch.stack(lse))


def _exact_evict(s):
    """Brute selection on the host: rank by (weight descending, position ascending)."""
    case = s["case"]
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    new, maps = [], []
    for b, L in enumerate(_lengths(case)):
        if L <= keep:
            new.append(L)
            maps.append(list(range(L)) + [-1] * (keep - L))
            continue
        w = s["acc"][b].tolist()
        free = sorted(range(sink, L - recent), key=lambda t: (-w[t], t))[:keep - sink - recent]
        held = set(range(sink)) | set(range(L - recent, L)) | set(free)
        late = iter(t for t in range(keep, L) if t in held)
        maps.append([i if i in held else next(late) for i in range(keep)])
        new.append(keep)
        src = torch.tensor(maps[-1], device="cuda")
        for p in _planes(s):
            p[b, :keep] = p[b].index_select(0, src)
    return [*_planes(s), torch.tensor(new, dtype=torch.int32), torch.tensor(maps, dtype=torch.int32)]
