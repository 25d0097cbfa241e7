"""Block-scaled decode directly behind the kernel that wrote its inputs: a chunk's
append, a block copy, kernels that raise the lengths and change the tables.  The
outputs must have the bits of the same calls with the device idle between them."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import Case, _dev

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _twice(steps, state, start, rounds=6):
    """Runs `steps` (callables) round after round from the same state, once with
    a device synchronisation behind each and once in a row; both runs' outputs."""
    outs = []
    for sync in (True, False):
        for x, y in zip(state, start):
            x.copy_(y)
        torch.cuda.synchronize()
        got = []
        for i in range(rounds):
            for s in steps:
                r = s(i)
                if sync:
                    torch.cuda.synchronize()
                if r is not None:
                    got.append(r)
        torch.cuda.synchronize()
        outs.append(got + [x.clone() for x in state])
    return outs


@pytest.mark.parametrize("lens,hq,hkv,d,bs", [
    ([400] * 64, 16, 4, 256, 16),            # many ranges of several tiles
    ([3000, 2000], 16, 4, 256, 16),          # pieces joined by a kernel of their own
    ([90], 8, 1, 128, 32),
])
def test_every_input_written_by_the_kernel_ahead(pa, lens, hq, hkv, d, bs):
    c = Case(61, lens, hq, hkv, d, bs)
    B, T = len(lens), 70
    pools = [_dev(x) for x in (c.kp, c.vp, c.ks, c.vs)]
    pools[0][pools[0] == 0x7F] = 0
    pools[1][pools[1] == 0x7F] = 0
    g = torch.Generator(device=DEV).manual_seed(3)
    n = np.minimum(np.asarray(lens), T)
    cu = _dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    total = int(n.sum())
    k, v = (torch.randn(6, total, hkv, d, generator=g, device=DEV).to(torch.bfloat16)
            for _ in range(2))
    tab, full = _dev(c.tab), _dev(c.lens)
    # (two tables and lengths to change between)
    other = tab.flip(0).contiguous() if all(x == lens[0] for x in lens) else tab
    table, length = tab.clone(), full.clone()
    state = (*pools, table, length)
    start = [x.clone() for x in state]
    short = torch.clamp(full - 33, min=1)
    ids = torch.from_numpy(c.tab[c.tab >= 0].astype(np.int64)).to(DEV)
    half = len(ids) // 2
    pairs = torch.stack([ids[:half], ids[len(ids) - half:]], dim=1).contiguous()
    ws = torch.empty(pa.pa_decode_workspace_bytes(B, hq, hkv, d, max(lens)), dtype=torch.uint8,
                     device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def decode(_):
        out = torch.empty_like(c.q)
        pa.pa_decode_attention_q8(out, c.q, *pools, table, length, max(lens), c.scale, ws, status)
        return out

    def append(i):
        pa.pa_rope_and_cache_q8(None, None, k[i], v[i], *pools, cu, T, table, length,
                                dev_status=status)

    def copy(_):
        pa.pa_copy_blocks_q8(*pools, *pools, pairs, status)

    def shorten(_):
        length.copy_(short)

    def lengthen(_):
        length.copy_(full)

    def retable(i):
        table.copy_(other if i % 2 else tab)

    steps = [lengthen, append, decode, copy, decode, shorten, decode, lengthen, decode, retable, decode]
    apart, row = _twice(steps, state, start)
    assert int(status.item()) == 0
    for x, y in zip(apart, row):
        assert torch.equal(x, y)
