"""The block-scaled append that rotates nothing: queries are copied to
query_out, keys are quantised as they come, and positions, which are not
given, are not read."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from paged_kv_cache_455_b200 import workloads as W
from test_gpu_rope import _Cache, _dev, _f32, _qkv, _tables

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _case(counts, hq, hkv, d, bs, pad, fused):
    rng = np.random.default_rng(sum(counts) + d)
    counts = np.asarray(counts)
    lens = (counts + rng.integers(0, 3, len(counts)) * bs).astype(np.int32)
    tab, nb = _tables(rng, lens, bs)
    cache = _Cache(rng, nb, bs, hkv, d)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q, k, v = _qkv(rng, int(cu[-1]) + pad, hq, hkv, d, torch.bfloat16, fused)
    return cache, q, k, v, cu, tab, lens


def _expect(cache, k, v, cu, tab, lens):
    real = int(cu[-1])
    cache.kp, cache.ks = O.append_q8_np(cache.kp, cache.ks, _f32(k)[:real], cu, tab, lens)
    cache.vp, cache.vs = O.append_q8_np(cache.vp, cache.vs, _f32(v)[:real], cu, tab, lens)


@pytest.mark.parametrize("counts,hq,hkv,d,bs,pad,fused", [
    ([1, 1, 1, 0, 1], 8, 2, 128, 16, 0, True),
    ([1] * 9, 16, 4, 256, 32, 3, False),
    ([30, 0, 17, 64], 6, 3, 256, 16, 5, True),
])
def test_queries_are_copied(pa, counts, hq, hkv, d, bs, pad, fused):
    cache, q, k, v, cu, tab, lens = _case(counts, hq, hkv, d, bs, pad, fused)
    real = int(cu[-1])
    out = torch.full((q.shape[0], hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    _expect(cache, k, v, cu, tab, lens)
    pa.pa_rope_and_cache_q8(out, q, k, v, *cache.dev, _dev(cu), max(counts), _dev(tab), _dev(lens),
                            dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    cache.check()
    assert torch.equal(out[:real], q[:real]) and (out[real:] == 9.0).all()


def test_positions_without_a_table_are_ignored(pa):
    # through the C entry: positions beyond any table, max_position 0
    cache, q, k, v, cu, tab, lens = _case([2, 5], 8, 2, 128, 16, 0, False)
    out = torch.full_like(q, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.full((7,), 1 << 40, device=DEV)
    keep = [_dev(cu), _dev(tab), _dev(lens)]
    _expect(cache, k, v, cu, tab, lens)
    st = pa.lib.pa_rope_and_cache_q8(
        out.data_ptr(), 8 * 128, q.data_ptr(), 8 * 128, k.data_ptr(), 2 * 128, v.data_ptr(), 2 * 128,
        *[x.data_ptr() for x in cache.dev], keep[0].data_ptr(), 7, 5, keep[1].data_ptr(),
        tab.shape[1], keep[2].data_ptr(), 2, pos.data_ptr(), None, 0, 0, 0, 8, 2, 128, 16,
        cache.kp.shape[0], status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and int(status.item()) == 0
    cache.check()
    assert torch.equal(out, q)


def test_queries_in_place_are_left_alone(pa):
    cache, q, k, v, cu, tab, lens = _case([3, 1], 8, 2, 128, 16, 2, True)
    want = W.to_numpy_elems(q.contiguous())
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    _expect(cache, k, v, cu, tab, lens)
    pa.pa_rope_and_cache_q8(q, q, k, v, *cache.dev, _dev(cu), 3, _dev(tab), _dev(lens),
                            dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    cache.check()
    assert np.array_equal(W.to_numpy_elems(q.contiguous()), want)
