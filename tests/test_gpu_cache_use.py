"""The cache operators as a server calls them: shared caches, strided inputs, other streams, several calls at once,
and a step of all of them captured and replayed."""

import numpy as np
import pytest
import torch

from head_latent_attention_absorb_b200 import api

from _cache_util import DEV, check_decode, pack, random_fp4, reference, values

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCALE = 0.0722


def dims(n_h=128, d_c=512, d_r=64):
    return (n_h, d_c, d_r, 128, 128)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def queries(B, T, n_h, seed, d_c=512, d_r=64, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, T, n_h, d_c), generator=g) * 0.226).to(dtype), torch.randn((B, T, n_h, d_r), generator=g).to(dtype)


def decode(q, qp, planes, lens, n_h=128, d=None, **kw):
    lse = torch.empty(q.shape[:-1], device=DEV)
    return api.mla_decode_absorb_fp4kv(d or dims(n_h), q, qp, *planes, lens, SCALE, lse=lse, **kw), lse


def weights(q, qp, planes, lens, lse, n_h=128, d=None, **kw):
    return api.mla_cache_weights_fp4kv(d or dims(n_h), q, qp, *planes, lens, SCALE, lse, **kw)


@pytest.mark.parametrize("n_h,T,lengths", [
    (16, 1, [int(v) for v in np.random.default_rng(1).integers(1, 700, 230)]),   # several sequences for each pair of CTAs
    (128, 3, [3000, 3, 1500, 259]),                                              # groups of query rows, each split
    (40, 4, [1100, 4, 129]),                                                     # a last group of 32 rows
    (16, 1, [1] * 100 + [5000]),                                                 # one long among many short
])
def test_decode_and_weights_over_uneven_batches(n_h, T, lengths):
    B, n_max = len(lengths), max(lengths)
    q, qp = queries(B, T, n_h, 5)
    c4, sc, kr = random_fp4(B, n_max, 512, 6)
    planes = pack(c4, sc, kr)
    ref = reference(q, qp, values(c4, sc), kr, lengths, T, float(np.float32(SCALE)))
    lens = i32(lengths)
    ctx, lse = decode(q.to(DEV), qp.to(DEV), planes, lens, n_h)
    check_decode(ctx, lse, ref, BF)
    # a head's weights sum to one: each is off by its score's error and that of lse, twice ez and 2^-12 at most
    w = weights(q.to(DEV), qp.to(DEV), planes, lens, lse, n_h).double().sum(-1).cpu().numpy()
    tol = (2 * ref[3] + 2.0 ** -11 + 2.0 ** -16).sum((1, 2))
    assert (np.abs(w - T * n_h) <= tol).all(), (np.abs(w - T * n_h) / tol).max()


def test_sequences_that_share_one_cache():
    B, n = 5, 700
    q, qp = (t.to(DEV) for t in queries(B, 2, 128, 7))
    c4, sc, kr = random_fp4(1, n, 512, 8)
    one = pack(c4, sc, kr)
    shared = tuple(p.expand(B, -1, -1) for p in one)
    apart = tuple(p.expand(B, -1, -1).contiguous() for p in one)
    lens = i32([700, 2, 333, 128, 699])
    a, lse = decode(q, qp, shared, lens)
    b, lse_b = decode(q, qp, apart, lens)
    assert torch.equal(a, b) and torch.equal(lse, lse_b)
    assert torch.equal(weights(q, qp, shared, lens, lse), weights(q, qp, apart, lens, lse))
    assert torch.equal(api.mla_cache_read_fp4(dims(), *shared[:2], n), api.mla_cache_read_fp4(dims(), *apart[:2], n))
    rows = api.mla_cache_read_fp4(dims(), *one[:2], n)
    k = apart[2][:1].contiguous()
    w = api.mla_cache_weights(dims(), q, qp, rows.expand(B, -1, -1), k.expand(B, -1, -1), lens, SCALE, lse)
    v = api.mla_cache_weights(dims(), q, qp, rows.expand(B, -1, -1).contiguous(), apart[2], lens, SCALE, lse)
    assert torch.equal(w, v)


@pytest.mark.parametrize("dtype,d_c,d_r", [(BF, 512, 64), (F32, 48, 18)])
def test_strided_queries(dtype, d_c, d_r):
    """Heads out of a wider projection: rows further apart than they are wide."""
    B, T, n_h, n = 3, 2, 16, 300
    d = dims(n_h, d_c, d_r)
    q, qp = queries(B, T, n_h, 9, d_c, d_r, dtype)
    both = torch.full((B, T, n_h, d_c + d_r + 32), float("nan"), dtype=dtype, device=DEV)
    both[..., :d_c], both[..., d_c:d_c + d_r] = q.to(DEV), qp.to(DEV)
    c4, sc, kr = random_fp4(B, n, d_c, 10, d_r, dtype)
    planes = (c4.to(DEV), sc.to(DEV), kr.to(DEV))
    lens = i32([300, 2, 111])
    a, lse = decode(both[..., :d_c], both[..., d_c:d_c + d_r], planes, lens, d=d)
    b, lse_b = decode(q.to(DEV), qp.to(DEV), planes, lens, d=d)
    assert torch.equal(a, b) and torch.equal(lse, lse_b)
    assert torch.equal(weights(both[..., :d_c], both[..., d_c:d_c + d_r], planes, lens, lse, d=d),
                       weights(q.to(DEV), qp.to(DEV), planes, lens, lse, d=d))
    # one token of two: the sequences' rows are not evenly spaced, which the row strides cannot say
    with pytest.raises(ValueError, match="q_tilde"):
        decode(both[:, 1, :, :d_c], both[:, 1, :, d_c:d_c + d_r], planes, lens, d=d)


def test_weights_offsets_past_32_bits():
    n, stride = 1500, 1572864
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
    near = pack(c4, sc, kr)
    q, qp = (t[:, 0].to(DEV) for t in queries(2, 1, 128, 12))
    lens = i32([n, n - 77])
    ctx, lse = decode(q, qp, near, lens)
    assert torch.equal(weights(q, qp, views, lens, lse), weights(q, qp, near, lens, lse))
    acc = torch.rand((2, n), device=DEV)
    got = api.mla_cache_evict(views, acc, lens, 500, sink=4, recent=64)
    want = api.mla_cache_evict(near, acc, lens, 500, sink=4, recent=64)
    assert torch.equal(got[1], want[1]) and all(torch.equal(a, b) for a, b in zip(views, near))
    x = torch.randn((2, 3, 576), device=DEV).to(BF)
    for p in (views, near):
        api.mla_cache_append_fp4(dims(), x, i32([5000, 9]), *p, rows=i32([n - 3, n - 90]))
    assert all(torch.equal(a, b) for a, b in zip(views, near))


def step(x, q, qp, planes, acc, lens, pos, out, lse, new, row_map):
    """One serving step: append, decode, accumulate, evict."""
    d = dims(16)
    api.mla_cache_append_fp4(d, x, pos, *planes, rows=lens - 1)
    api.mla_decode_absorb_fp4kv(d, q, qp, *planes, lens, SCALE, ctx=out, lse=lse)
    api.mla_cache_weights_fp4kv(d, q, qp, *planes, lens, SCALE, lse, acc=acc, out=acc, decay=0.9)
    api.mla_cache_evict([*planes, acc.unsqueeze(-1)], acc, lens, 200, sink=4, recent=32, new_lengths=new, row_map=row_map)


def step_state(seed, n_max=400):
    B = 3
    q, qp = (t[:, 0].to(DEV) for t in queries(B, 1, 16, seed))
    g = torch.Generator().manual_seed(seed)
    return dict(x=torch.randn((B, 576), generator=g).to(BF).to(DEV), q=q, qp=qp, planes=pack(*random_fp4(B, n_max, 512, seed)),
                acc=torch.rand((B, n_max), generator=g).to(DEV), lens=i32([400, 201, 77]), pos=i32([1000, 5, 76]),
                out=torch.empty_like(q), lse=torch.empty((B, 16), device=DEV), new=i32([0] * B),
                row_map=torch.empty((B, 200), dtype=torch.int32, device=DEV))


def copies(s):
    return {k: tuple(t.clone() for t in v) if isinstance(v, tuple) else v.clone() for k, v in s.items()}


def packed_copies(s):
    """A copy whose planes are views of packed rows again."""
    c = copies(s)
    c["planes"] = pack(*(p.cpu() for p in s["planes"]))
    return c


def same(a, b):
    return all(all(torch.equal(x, y) for x, y in zip(a[k], b[k])) if isinstance(a[k], tuple) else torch.equal(a[k], b[k]) for k in a)


def test_a_captured_step_replays_like_eager_calls():
    start = step_state(20)
    want = packed_copies(start)
    step(**want)
    s = packed_copies(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(**s)
    for _ in range(3):
        for k, v in start.items():
            for dst, src in zip(s[k], v) if isinstance(v, tuple) else ((s[k], v),):
                dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert same(s, want)


def test_steps_of_several_batches_at_once():
    """Steps on four streams beside one another, each eager and as two graphs of one memory pool in turn."""
    starts = [step_state(30 + i) for i in range(4)]
    want = [packed_copies(s) for s in starts]
    for w in want:
        step(**w)
    got = [packed_copies(s) for s in starts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in got]
    for s, st in zip(got, streams):
        with torch.cuda.stream(st):
            step(**s)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))
    got = [packed_copies(s) for s in starts]
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for s in got[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            step(**s)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got[:2], want))


def test_stream_arguments():
    """Every operator on a stream that is not the current one, as an object and as a handle."""
    start = step_state(40)
    want = packed_copies(start)
    d = dims(16)
    step(**want)
    for as_handle in (False, True):
        s = packed_copies(start)
        rows = s["lens"] - 1
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        k = dict(stream=st.cuda_stream if as_handle else st)
        api.mla_cache_append_fp4(d, s["x"], s["pos"], *s["planes"], rows=rows, **k)
        s["out"] = api.mla_decode_absorb_fp4kv(d, s["q"], s["qp"], *s["planes"], s["lens"], SCALE, lse=s["lse"], **k)
        api.mla_cache_weights_fp4kv(d, s["q"], s["qp"], *s["planes"], s["lens"], SCALE, s["lse"], acc=s["acc"], out=s["acc"],
                                    decay=0.9, **k)
        s["new"], s["row_map"] = api.mla_cache_evict([*s["planes"], s["acc"].unsqueeze(-1)], s["acc"], s["lens"], 200, sink=4,
                                                     recent=32, **k)
        st.synchronize()
        assert same(s, want)
        rows = api.mla_cache_read_fp4(d, *s["planes"][:2], 50, stream=k["stream"])
        st.synchronize()
        assert torch.equal(rows, api.mla_cache_read_fp4(d, *s["planes"][:2], 50))


def test_evict_of_sequences_that_fit():
    acc = torch.rand((2, 50), device=DEV)
    plane = torch.randint(0, 256, (2, 50, 8), dtype=torch.uint8, device=DEV)
    before = plane.clone()
    for lens in ([50, 3], [0, 0]):
        new, row_map = api.mla_cache_evict([plane], acc, i32(lens), 50, sink=0, recent=0)
        assert new.tolist() == lens and torch.equal(plane, before)
        assert row_map[0].tolist() == [i if i < lens[0] else -1 for i in range(50)]


@pytest.mark.parametrize("dtype,d_c,d_r", [(BF, 512, 64), (F32, 40, 6)])
def test_append_at_writes_the_row_that_append_writes(dtype, d_c, d_r):
    d, B, far, near = dims(4, d_c, d_r), 4, 4001, 8
    x = torch.randn((B, d_c + d_r), device=DEV).to(dtype)
    gain = torch.rand((d_c,), device=DEV) + 0.5
    pos, rows = [4000, 3, 0, 1234], [5, 0, 7, 2]
    a = torch.full((B, far, d_c + d_r), 3.0, dtype=dtype, device=DEV)
    b = torch.full((B, near, d_c + d_r), 3.0, dtype=dtype, device=DEV)
    api.mla_cache_append(d, x, i32(pos), a[..., :d_c], a[..., d_c:], gain=gain)
    api.mla_cache_append(d, x, i32(pos), b[..., :d_c], b[..., d_c:], gain=gain, rows=i32(rows))
    want = torch.full_like(b, 3.0)
    for s in range(B):
        want[s, rows[s]] = a[s, pos[s]]
    assert torch.equal(b, want)
    # a row behind the cache, before it, and a negative position: reported, nothing written
    for p, r in (([1] * B, [0, 8, 1, 2]), ([1] * B, [0, -1, 1, 2]), ([1, -1, 1, 1], [0, 1, 1, 2])):
        b.fill_(3.0)
        err = i32([0])
        api.mla_cache_append(d, x, i32(p), b[..., :d_c], b[..., d_c:], gain=gain, rows=i32(r), dev_err=err)
        assert int(err) == 4 and bool((b[1] == 3.0).all()) and bool((b[0, 0] != 3.0).any())


def test_caches_that_end_with_their_rows():
    """The last sequence fills its cache to the end of the allocation, at lengths inside and at the end of a tile."""
    for n in (1, 63, 64, 65, 127, 128, 129, 255, 256, 300):
        c4, sc, kr = random_fp4(2, n, 512, n)
        planes = (c4.to(DEV), sc.to(DEV), kr.to(DEV))
        q, qp = queries(2, 1, 128, n)
        lens = [n, n]
        ctx, lse = decode(q[:, 0].to(DEV), qp[:, 0].to(DEV), planes, i32(lens))
        check_decode(ctx, lse, reference(q, qp, values(c4, sc), kr, lens, 1, float(np.float32(SCALE))), BF)
        w = weights(q[:, 0].to(DEV), qp[:, 0].to(DEV), planes, i32(lens), lse)
        rows = api.mla_cache_read_fp4(dims(), *planes[:2], n)
        v = api.mla_cache_weights(dims(), q[:, 0].to(DEV), qp[:, 0].to(DEV), rows, planes[2], i32(lens), SCALE, lse)
        assert torch.equal(w, v)  # the same bf16 operands, in the same order
