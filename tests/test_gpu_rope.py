"""Rotary cache writes and block copies of the block-scaled cache on the GPU,
bit for bit against the numpy oracle.

The oracle rotates in binary32 with every product and sum rounded once, rounds
to bf16 (or keeps binary32), and settles a block's scale, its requantised rows
and its new codes from the definition; the kernels promise the same numbers,
so nothing here has a tolerance.
"""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from paged_kv_cache_455_b200 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _f32(t):
    return t.float().cpu().numpy()


def _qkv(rng, T, hq, hkv, d, dtype, fused):
    x = rng.standard_normal((T, (hq + 2 * hkv) * d)).astype(np.float32)
    t = _dev(x).to(dtype)
    q, k, v = t.split([hq * d, hkv * d, hkv * d], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q.view(T, hq, d), k.view(T, hkv, d), v.view(T, hkv, d)


def _raw(x, dtype):
    return O.f32_to_bf16_raw(x) if dtype == torch.bfloat16 else x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hq,hkv,d,rot,bs,inter,fused,inplace", [
    (1, 1, 1, 64, 64, 4, False, False, False),
    (5, 8, 2, 64, 16, 8, True, True, True),
    (67, 16, 4, 256, 64, 16, False, True, False),
    (33, 16, 4, 256, 256, 32, True, False, True),
    (130, 6, 3, 128, 48, 16, False, True, True),
    (2500, 16, 4, 128, 128, 16, False, True, False),   # four rows per thread
    (40, 0, 5, 128, 96, 16, True, True, False),        # keys only
])
def test_rope_and_cache_is_bit_exact(pa, dtype, T, hq, hkv, d, rot, bs, inter, fused, inplace):
    rng = np.random.default_rng(T * 7 + d + rot)
    maxpos = 5000
    table = rng.uniform(-1, 1, (maxpos, rot)).astype(np.float32)
    pos = rng.integers(0, maxpos, T)
    pos[0] = maxpos - 1
    nb = -(-T // bs) + 3
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1                    # padding
    q, k, v = _qkv(rng, T, max(hq, 1), hkv, d, dtype, fused)
    kp = torch.full((nb, bs, hkv, d), 7.5, dtype=dtype, device=DEV)
    vp = kp.clone()
    qf, kf = _f32(q), _f32(k)
    v_in = W.to_numpy_elems(v.contiguous())
    q_out = None if hq == 0 else (q if inplace else torch.full((T, hq, d), 3.0, dtype=dtype,
                                                               device=DEV))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want_q = _raw(O.rotate_f32(qf, pos, table, rot, inter), dtype)
    want_k = _raw(O.rotate_f32(kf, pos, table, rot, inter), dtype)
    k_ref, v_ref = O.reshape_and_cache_np(want_k, v_in, W.to_numpy_elems(kp), W.to_numpy_elems(vp),
                                          slots)
    pa.pa_rope_and_cache(q_out, None if hq == 0 else q, k, v, kp, vp, _dev(slots), _dev(pos),
                         _dev(table), inter, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    if hq:
        assert W.to_numpy_elems(q_out.contiguous()).tobytes() == want_q.tobytes()
    assert W.to_numpy_elems(kp).tobytes() == k_ref.tobytes()
    assert W.to_numpy_elems(vp).tobytes() == v_ref.tobytes()


def test_rope_without_a_table_only_caches(pa):
    rng = np.random.default_rng(5)
    q, k, v = _qkv(rng, 9, 4, 2, 128, torch.bfloat16, True)
    kp = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    out = torch.zeros(9, 4, 128, dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(9, device=DEV) * 3
    pa.pa_rope_and_cache(out, q, k, v, kp, vp, slots)
    assert torch.equal(out, q)
    assert torch.equal(kp.view(-1, 2, 128)[slots], k)
    assert torch.equal(vp.view(-1, 2, 128)[slots], v)


def test_rope_reports_bad_positions_and_slots(pa):
    rng = np.random.default_rng(6)
    T, hq, hkv, d, rot, bs = 6, 4, 2, 128, 64, 16
    q, k, v = _qkv(rng, T, hq, hkv, d, torch.bfloat16, False)
    table = torch.randn(10, rot, device=DEV)
    kp = torch.full((2, bs, hkv, d), 2.0, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    out = torch.full_like(q, 5.0)
    pos = torch.tensor([0, 9, 10, -1, 3, 4], device=DEV)
    slots = torch.tensor([0, 1, 2, 3, 32, -5], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache(out, q, k, v, kp, vp, slots, pos, table, False, status)
    assert int(status.item()) == pa.PA_DEV_BAD_POSITION | pa.PA_DEV_BAD_SLOT
    assert (out[2:4] == 0).all() and (out[[0, 1, 4, 5]] != 5.0).any(dim=-1).all()
    flat = kp.view(-1, hkv, d)
    assert (flat[2:] == 2.0).all() and not (flat[:2] == 2.0).all(dim=-1).any()
    assert (vp.view(-1, hkv, d)[2:] == 2.0).all()


# ------------------------------------------------------- block-scaled appends
def _tables(rng, lens, bs, spare=3):
    need = [-(-int(c) // bs) for c in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb)
    tab = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        tab[b, :n] = perm[at:at + n]
        at += n
    return tab, nb


class _Cache:
    """Device pools with their oracle copies."""

    def __init__(self, rng, nb, bs, hkv, d):
        self.kp = rng.integers(0, 256, (nb, bs, hkv, d)).astype(np.uint8)
        self.vp = rng.integers(0, 256, (nb, bs, hkv, d)).astype(np.uint8)
        self.ks = np.exp2(rng.integers(-4, 5, (nb, hkv))).astype(np.float32)
        self.vs = np.exp2(rng.integers(-4, 5, (nb, hkv))).astype(np.float32)
        self.dev = [_dev(x) for x in (self.kp, self.vp, self.ks, self.vs)]

    def check(self):
        for name, got, want in zip(("k", "v", "ks", "vs"), self.dev,
                                   (self.kp, self.vp, self.ks, self.vs)):
            got = got.cpu().numpy()
            if got.tobytes() != want.tobytes():
                bad = np.argwhere(got != want)
                raise AssertionError(f"{name}: {len(bad)} differ, first {bad[:3].tolist()}")


def _append(pa, cache, q, k, v, cu, maxq, tab, lens, pos, table, rot, inter, status, q_out):
    """One call and the oracle's step; k, v: device tensors."""
    hkv, d = cache.kp.shape[2:]
    real = int(cu[-1])
    kf = O.rotate_f32(_f32(k)[:real], pos[:real], table, rot, inter)
    cache.kp, cache.ks = O.append_q8_np(cache.kp, cache.ks, kf, cu, tab, lens)
    cache.vp, cache.vs = O.append_q8_np(cache.vp, cache.vs, _f32(v)[:real], cu, tab, lens)
    args = (_dev(pos), _dev(table)) if rot else (None, None)
    pa.pa_rope_and_cache_q8(q_out, q, k, v, *cache.dev, _dev(cu), maxq, _dev(tab),
                            _dev(np.asarray(lens, np.int32)), *args, inter, status)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("hq,hkv,d,rot,inter,fused", [
    (16, 4, 256, 64, False, True),
    (8, 1, 128, 128, True, False),
    (6, 3, 128, 48, False, True),
    (2, 2, 256, 256, False, False),
])
def test_append_q8_chunks_then_tokens(pa, bs, hq, hkv, d, rot, inter, fused):
    # three ragged chunks per sequence (some empty), then single tokens whose
    # size keeps growing, so that blocks are requantised
    rng = np.random.default_rng(bs + d + rot)
    B, maxpos = 7, 400
    table = rng.uniform(-1, 1, (maxpos, rot)).astype(np.float32)
    steps = [np.array([1, 5, 16, 33, 0, 64, 17]), np.array([15, 0, 31, 2, 40, 1, 100]),
             np.array([1, 12, 1, 0, 3, 2, 7])]
    final = sum(steps) + 20
    tab, nb = _tables(rng, final, bs)
    cache = _Cache(rng, nb, bs, hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = np.zeros(B, np.int64)
    for i in range(3 + 6):
        n = steps[i] if i < 3 else np.ones(B, np.int64)
        lens = lens + n
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        pad = 2 if i % 2 else 0
        T = int(cu[-1]) + pad
        q, k, v = _qkv(rng, T, hq, hkv, d, torch.bfloat16, fused)
        grow = 2.0 ** (i - 2) if i >= 3 else 1.0
        k, v = k * grow, v * (grow * rng.uniform(0.1, 1))
        pos = np.zeros(T, np.int64)
        pos[:int(cu[-1])] = np.concatenate([np.arange(l - m, l) for l, m in zip(lens, n)])
        q_out = torch.full((T, hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
        want_q = O.f32_to_bf16_raw(O.rotate_f32(_f32(q), pos, table, rot, inter))
        want_q[int(cu[-1]):] = O.f32_to_bf16_raw(np.float32(9.0))
        _append(pa, cache, q, k, v, cu, int(n.max()), tab, lens, pos, table, rot, inter, status,
                q_out)
        assert int(status.item()) == 0
        cache.check()
        assert W.to_numpy_elems(q_out).tobytes() == want_q.tobytes()


def test_append_q8_values_at_the_borders(pa):
    # zeros, the format's ends, infinities, NaN, subnormal bf16, a scale that
    # is no power of two, and the exponent limits
    rng = np.random.default_rng(3)
    B, hkv, d, bs = 9, 2, 128, 16
    tab, nb = _tables(rng, np.full(B, 20), bs)
    cache = _Cache(rng, nb, bs, hkv, d)
    cache.ks[tab[3, 1]] = 0.3
    cache.dev[2].copy_(_dev(cache.ks))
    lens = np.array([1, 17, 16, 20, 1, 2, 1, 18, 1], np.int32)
    k = rng.standard_normal((B, hkv, d)).astype(np.float32)
    k[0] = 0.0
    k[1, 0] = 448.0
    k[2, :, 3] = np.inf
    k[3, :, 5] = 40.0
    k[4, :, 7] = np.nan
    k[5] = 1e-39
    k[6] = 3e38
    k[7, 0, 0] = 449.0 * 2.0 ** 7
    k[8] = 1e-30
    kt = _dev(k).to(torch.bfloat16)
    vt = (kt * 0.5).contiguous()
    cu = np.arange(B + 1).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    _append(pa, cache, None, kt, vt, cu, 1, tab, lens, np.zeros(B, np.int64),
            np.zeros((1, 16), np.float32), 0, False, status, None)
    assert int(status.item()) == 0
    cache.check()


def test_append_q8_refuses_bad_rows_on_the_device(pa):
    rng = np.random.default_rng(8)
    hkv, d, bs, rot = 2, 128, 16, 16
    lens = np.array([5, 9, 40, 3, 6, 33], np.int32)
    tab, nb = _tables(rng, lens, bs)
    tab[4, 0] = nb                         # outside the pool
    cache = _Cache(rng, nb, bs, hkv, d)
    cu = np.array([0, 2, 12, 14, 15, 17, 20], np.int32)   # sequence 1: 10 rows, 9 cached
    T = 20
    q, k, v = _qkv(rng, T, 4, hkv, d, torch.bfloat16, True)
    table = rng.uniform(-1, 1, (50, rot)).astype(np.float32)
    pos = np.arange(T).astype(np.int64)
    pos[14] = 50                           # sequence 3's only token
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.empty_like(q).contiguous()
    pa.pa_rope_and_cache_q8(q_out, q, k, v, *cache.dev, _dev(cu), 10, _dev(tab), _dev(lens),
                            _dev(pos), _dev(table), False, status)
    torch.cuda.synchronize()
    assert int(status.item()) == (pa.PA_DEV_BAD_CONTEXT | pa.PA_DEV_BAD_BLOCK |
                                  pa.PA_DEV_BAD_POSITION)
    # sequences 0, 2 and 5 are stored; 1, 4 and the token of 3 are not, and
    # their blocks keep codes and scales (3's block was begun before this call)
    kf = O.rotate_f32(_f32(k), np.minimum(pos, 49), table, rot, False)
    for pool, scales, x, name in ((cache.kp, cache.ks, kf, "kp"), (cache.vp, cache.vs, _f32(v), "vp")):
        for b in (0, 2, 5):
            part = np.array([0, cu[b + 1] - cu[b]], np.int32)
            new, sc = O.append_q8_np(pool, scales, x[cu[b]:cu[b + 1]], part, tab[b:b + 1],
                                     lens[b:b + 1])
            pool[...], scales[...] = new, sc
    cache.check()
    assert (q_out[14] == 0).all()


def test_copy_q8_inside_a_pool_and_to_the_host(pa):
    rng = np.random.default_rng(4)
    nb, bs, hkv, d = 40, 32, 3, 128
    cache = _Cache(rng, nb, bs, hkv, d)
    perm = rng.permutation(nb)
    pairs = np.stack([perm[rng.integers(0, 20, 15)], perm[25:40]], axis=1).astype(np.int64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_copy_blocks_q8(*cache.dev, *cache.dev, _dev(pairs), status)
    for x in (cache.kp, cache.vp, cache.ks, cache.vs):
        x[pairs[:, 1]] = x[pairs[:, 0]]
    torch.cuda.synchronize()
    cache.check()
    # out to pinned memory and back into other blocks, with one pair outside
    host = [torch.zeros(6, *x.shape[1:], dtype=x.dtype).pin_memory() for x in cache.dev]
    out = np.array([[perm[1], 5], [perm[2], 0], [nb, 1], [perm[3], 6]], np.int64)
    pa.pa_copy_blocks_q8(*host, *cache.dev, _dev(out), status)
    torch.cuda.synchronize()
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK
    back = np.array([[5, perm[30]], [0, perm[31]]], np.int64)
    pa.pa_copy_blocks_q8(*cache.dev, *host, _dev(back), None)
    torch.cuda.synchronize()
    for x in (cache.kp, cache.vp, cache.ks, cache.vs):
        x[perm[30]], x[perm[31]] = x[perm[1]], x[perm[2]]
    cache.check()
