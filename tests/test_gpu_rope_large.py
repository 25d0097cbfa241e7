"""Rotary cache writes past the sizes from which a thread takes four rows, bit for
bit against the oracle.  The sizes follow from the thresholds in the source, so
that a changed threshold does not leave these kernels untested."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_455_b200 as pkg
from oracle import oracle as O
from paged_kv_cache_455_b200 import workloads as W
from test_gpu_rope import _append, _Cache, _dev, _f32, _qkv, _raw, _tables

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SOURCE = os.path.join(os.path.dirname(pkg.__file__), "csrc", "pa_rope.cu")


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _threshold(pattern):
    with open(SOURCE) as f:
        found = re.findall(pattern + r"[^;?]*?>= ([0-9 *]+)[;?]", f.read())
    assert len(found) == 1, (pattern, found)
    return int(np.prod([int(x) for x in found[0].split("*")]))


@pytest.mark.parametrize("dtype,hq,hkv,d,rot,bs,inter,fused,inplace", [
    (torch.bfloat16, 16, 4, 256, 256, 16, False, True, False),
    (torch.bfloat16, 5, 5, 128, 48, 32, True, False, True),      # 15 rows: the last group is short
    (torch.float32, 1, 2, 64, 64, 8, False, True, True),         # 5 rows
    (torch.bfloat16, 0, 3, 128, 128, 16, False, True, False),    # 6 rows, keys and values only
])
def test_rope_and_cache_four_rows_a_thread(pa, dtype, hq, hkv, d, rot, bs, inter, fused, inplace):
    units, rows = d * (4 if dtype == torch.float32 else 2) // 32, hq + 2 * hkv
    T = -(-_threshold("bool many =") // (units * -(-rows // 4))) + 1
    rng = np.random.default_rng(d + rows)
    maxpos = 900
    table = rng.uniform(-1, 1, (maxpos, rot)).astype(np.float32)
    pos = rng.integers(0, maxpos, T)
    nb = -(-T // bs) + 3
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[rng.random(T) < 0.05] = -1
    q, k, v = _qkv(rng, T, max(hq, 1), hkv, d, dtype, fused)
    kp = torch.full((nb, bs, hkv, d), 7.5, dtype=dtype, device=DEV)
    vp = kp.clone()
    want_q = _raw(O.rotate_f32(_f32(q), pos, table, rot, inter), dtype)
    want_k = _raw(O.rotate_f32(_f32(k), pos, table, rot, inter), dtype)
    k_ref, v_ref = O.reshape_and_cache_np(want_k, W.to_numpy_elems(v.contiguous()),
                                          W.to_numpy_elems(kp), W.to_numpy_elems(vp), slots)
    out = None if hq == 0 else (q if inplace else torch.full((T, hq, d), 3.0, dtype=dtype, device=DEV))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache(out, None if hq == 0 else q, k, v, kp, vp, _dev(slots), _dev(pos),
                         _dev(table), inter, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    if hq:
        assert W.to_numpy_elems(out.contiguous()).tobytes() == want_q.tobytes()
    assert W.to_numpy_elems(kp).tobytes() == k_ref.tobytes()
    assert W.to_numpy_elems(vp).tobytes() == v_ref.tobytes()


@pytest.mark.parametrize("hq,hkv,d,rot,bs,inter,fused,inplace", [
    (16, 4, 256, 64, 16, False, True, False),
    (5, 5, 128, 128, 32, True, False, False),
    (12, 3, 128, 0, 16, False, True, False),
    (8, 1, 256, 256, 32, False, True, True),
])
def test_append_four_query_rows_a_thread(pa, hq, hkv, d, rot, bs, inter, fused, inplace):
    need = -(-_threshold("p.query_rows = query_ctas") * (128 // (d // 16)) // hq) + 1
    rng = np.random.default_rng(d + hq)
    counts = []
    while sum(counts) < need:
        counts.append(int(rng.integers(0, 700)))
    counts = np.asarray(counts)
    lens = counts + rng.integers(0, 3, len(counts)) * bs
    tab, nb = _tables(rng, lens, bs)
    cache = _Cache(rng, nb, bs, hkv, d)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    real, T = int(cu[-1]), int(cu[-1]) + 3
    table = rng.uniform(-1, 1, (int(lens.max()) + 1, max(rot, 16))).astype(np.float32)[:, :rot]
    pos = np.zeros(T, np.int64)
    pos[:real] = np.concatenate([np.arange(l - m, l) for l, m in zip(lens, counts)])
    q, k, v = _qkv(rng, T, hq, hkv, d, torch.bfloat16, fused)
    out = q if inplace else torch.full((T, hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    before = W.to_numpy_elems(out.contiguous())
    want = O.f32_to_bf16_raw(O.rotate_f32(_f32(q), pos, table, rot, inter))
    want[real:] = before[real:]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    _append(pa, cache, q, k, v, cu, int(counts.max()), tab, lens, pos, table, rot, inter, status, out)
    assert int(status.item()) == 0
    cache.check()
    assert W.to_numpy_elems(out.contiguous()).tobytes() == want.tobytes()
