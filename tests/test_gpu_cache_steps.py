"""Many serving steps one after the other without a word from the host, where each kernel may start while the one before
it runs: the same bits as with a synchronisation after every call, eager and captured."""

import pytest
import torch

from head_latent_attention_absorb_b200 import api

from _cache_util import DEV, pack

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCALE = 0.0722


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(kind, steps, B=5, n_max=70):
    """A server's state with every sequence at another length, and the inputs of all steps."""
    n_h, d_c, d_r, dt = (128, 512, 64, BF) if kind != "fp32" else (3, 48, 10, F32)
    g = torch.Generator().manual_seed(3)
    s = dict(d=(n_h, d_c, d_r, 128, 128), kv=(torch.randn((steps, B, d_c + d_r), generator=g)).to(dt).to(DEV),
             q=(torch.randn((steps, B, n_h, d_c), generator=g) * 0.3).to(dt).to(DEV),
             qp=torch.randn((steps, B, n_h, d_r), generator=g).to(dt).to(DEV))
    if kind == "bf16":
        cache = torch.zeros((B, n_max, d_c + d_r), dtype=dt, device=DEV)
        s["planes"] = (cache[..., :d_c], cache[..., d_c:])
    else:
        planes = (torch.zeros((B, n_max, d_c // 2), dtype=torch.uint8), torch.zeros((B, n_max, d_c // 16), dtype=torch.uint8),
                  torch.zeros((B, n_max, d_r), dtype=dt))
        s["planes"] = pack(*planes) if kind == "fp4" else tuple(p.to(DEV) for p in planes)
    s.update(acc=torch.zeros((B, n_max), device=DEV), row_pos=torch.full((B, n_max), -1, dtype=torch.int32, device=DEV),
             lens=i32([0, 60, 13, 69, 64][:B]), pos=i32([0, 60, 13, 69, 64][:B]), lse=torch.zeros((steps, B, n_h), device=DEV),
             ctx=torch.zeros((steps, B, n_h, d_c), dtype=dt, device=DEV), row_map=torch.zeros((B, 64), dtype=torch.int32, device=DEV))
    return s


def step(s, i, kind, after):
    d, p = s["d"], s["planes"]
    if kind == "bf16":
        api.mla_cache_append(d, s["kv"][i], s["pos"], *p, rows=s["lens"])
    else:
        api.mla_cache_append_fp4(d, s["kv"][i], s["pos"], *p, rows=s["lens"])
    after()
    s["row_pos"].scatter_(1, s["lens"].long()[:, None], s["pos"][:, None])
    s["lens"] += 1
    s["pos"] += 1
    after()
    if kind == "bf16":
        api.mla_decode_absorb(d, s["q"][i], s["qp"][i], *p, s["lens"], SCALE, ctx=s["ctx"][i], lse=s["lse"][i])
    else:
        api.mla_decode_absorb_fp4kv(d, s["q"][i], s["qp"][i], *p, s["lens"], SCALE, ctx=s["ctx"][i], lse=s["lse"][i])
    after()
    f = api.mla_cache_weights if kind == "bf16" else api.mla_cache_weights_fp4kv
    f(d, s["q"][i], s["qp"][i], *p, s["lens"], SCALE, s["lse"][i], acc=s["acc"], out=s["acc"], decay=0.98)
    after()
    api.mla_cache_evict([*p, s["acc"].unsqueeze(-1)], s["acc"], s["lens"], 64, sink=2, recent=16, new_lengths=s["lens"],
                        row_map=s["row_map"], positions=s["row_pos"])
    after()


def tensors(s):
    return [t for k in ("planes", "acc", "row_pos", "lens", "pos", "lse", "ctx", "row_map") for t in (s[k] if k == "planes" else [s[k]])]


@pytest.mark.parametrize("kind", ["fp4", "bf16", "fp32"])
def test_steps_without_synchronisation(kind):
    steps = 40
    want = make(kind, steps)
    for i in range(steps):
        step(want, i, kind, torch.cuda.synchronize)
    assert want["lens"].tolist() == [40, 64, 53, 64, 64] and bool(torch.isfinite(want["ctx"].float()).all())
    for _ in range(3):
        got = make(kind, steps)
        for i in range(steps):
            step(got, i, kind, lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(tensors(got), tensors(want)))
    got, graph = make(kind, steps), torch.cuda.CUDAGraph()
    for i in range(2):
        step(got, i, kind, lambda: None)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for i in range(2, steps):
            step(got, i, kind, lambda: None)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(tensors(got), tensors(want)))
