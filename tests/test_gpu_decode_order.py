"""Steps of one layer in a row: cache write and decode over the same pools again
and again, with nothing between them, give the bits of the same calls with the
device idle in between."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


@pytest.mark.parametrize("B,ctx", [(1, 40), (4, 300), (64, 700)])
@pytest.mark.parametrize("fp8", [False, True])
def test_steps_in_a_row(pa, fp8, B, ctx):
    hq, hkv, d, bs, steps = 16, 4, 256, 16, 40
    width = -(-(ctx + steps) // bs)
    nb = B * width
    g = torch.Generator(device=DEV).manual_seed(B)

    def rand(*s):
        return torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)

    kp, vp = rand(nb, bs, hkv, d), rand(nb, bs, hkv, d)
    if fp8:
        kp, vp = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (kp, vp))
    tab = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).view(B, width)
    q, k, v = rand(steps, B, hq, d), rand(steps, B, hkv, d), rand(steps, B, hkv, d)
    pos = ctx + torch.arange(steps, device=DEV)
    lens = (pos[:, None] + 1).to(torch.int32).expand(steps, B).contiguous()
    slots = tab.long()[:, pos // bs].T.contiguous() * bs + (pos % bs)[:, None]
    outs = torch.zeros(steps, B, hq, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(pa.pa_decode_workspace_bytes(B, hq, hkv, d, ctx + steps), dtype=torch.uint8,
                     device=DEV)
    pools, status = [kp, vp], torch.zeros(1, dtype=torch.int32, device=DEV)

    def step(i, wait):
        if fp8:
            pa.pa_reshape_and_cache_fp8(k[i], v[i], *pools, slots[i], 1.0, 1.0, status)
        else:
            pa.pa_reshape_and_cache(k[i], v[i], *pools, slots[i], status)
        if wait:
            torch.cuda.synchronize()
        if fp8:
            pa.pa_decode_attention_fp8(outs[i], q[i], *pools, tab, lens[i], ctx + steps, d ** -0.5,
                                       1.0, 1.0, ws, status)
        else:
            pa.pa_decode_attention(outs[i], q[i], *pools, tab, lens[i], ctx + steps, d ** -0.5, ws,
                                   status)
        if wait:
            torch.cuda.synchronize()

    start = [x.clone() for x in pools]
    for i in range(steps):
        step(i, True)
    want, want_pools = outs.clone(), [x.clone() for x in pools]

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        for i in range(steps):
            step(i, False)
    for _ in range(3):
        for x, y in zip(pools, start):
            x.copy_(y)
        outs.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert torch.equal(outs, want)
        for x, y in zip(pools, want_pools):
            assert torch.equal(x, y)
    del graph
