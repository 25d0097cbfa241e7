"""The oracle's rotation and block-scaled cache, pinned to facts outside it."""
import numpy as np
import pytest
import torch

from oracle import oracle as O


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_by_a_quarter_turn_and_none(inter):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 32)).astype(np.float32)
    table = np.zeros((2, 16), np.float32)
    table[0, :8] = 1.0                       # position 0: angle 0
    table[1, 8:] = 1.0                       # position 1: a quarter turn
    y = O.rotate_f32(x, [0, 1], table, 16, inter)
    assert np.array_equal(y[0], x[0])
    assert np.array_equal(y[:, :, 16:], x[:, :, 16:])
    a, b = (x[1, :, 0:16:2], x[1, :, 1:16:2]) if inter else (x[1, :, :8], x[1, :, 8:16])
    ya, yb = (y[1, :, 0:16:2], y[1, :, 1:16:2]) if inter else (y[1, :, :8], y[1, :, 8:16])
    assert np.array_equal(ya, -b) and np.array_equal(yb, a)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_complex_multiplication_and_keeps_scores_relative(inter):
    # q at p and k at s give the same score as q at p - s and k at 0: the
    # products of unit complex numbers; binary32 rounding, 64 terms
    d = 64
    rng = np.random.default_rng(1)
    inv = 100.0 ** (-np.arange(d // 2) / (d / 2))
    ang = np.arange(40)[:, None] * inv
    table = np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)
    q, k = rng.standard_normal((2, 1, 1, d)).astype(np.float32)
    dot = lambda p, s: float((O.rotate_f32(q, [p], table, d, inter).astype(np.float64) *  # noqa: E731
                              O.rotate_f32(k, [s], table, d, inter)).sum())
    tol = 6 * 2.0 ** -24 * float((np.abs(q) * np.abs(k)).sum() + 2 * np.linalg.norm(q) * np.linalg.norm(k))
    assert abs(dot(30, 21) - dot(9, 0)) <= tol
    z = (q[..., ::2] + 1j * q[..., 1::2]) if inter else (q[..., :d // 2] + 1j * q[..., d // 2:])
    w = z * np.exp(1j * ang[7])
    y = O.rotate_f32(q, [7], table, d, inter)
    got = (y[..., ::2] + 1j * y[..., 1::2]) if inter else (y[..., :d // 2] + 1j * y[..., d // 2:])
    assert np.abs(got - w).max() <= 8 * 2.0 ** -24 * np.abs(z).max()


def test_bf16_rounding_matches_torch():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal(4096) * np.exp2(rng.integers(-30, 30, 4096))).astype(np.float32)
    x[:4] = [0.0, -0.0, np.inf, 3.4e38]
    want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(O.f32_to_bf16_raw(x), want)


def test_block_scale_closed_forms():
    assert O.block_scale(0.0) == 2.0 ** -64
    assert O.block_scale(448.0) == 1.0
    assert O.block_scale(np.nextafter(np.float32(448), np.float32(1e9))) == 2.0
    assert O.block_scale(1.0) == 2.0 ** -8
    assert O.block_scale(3.38e38) == 2.0 ** 120


def _pools(rng, nb, bs, hkv, d):
    return rng.integers(0, 255, (nb, bs, hkv, d)).astype(np.uint8), \
        rng.uniform(0.5, 2, (nb, hkv)).astype(np.float32)


def test_append_in_steps_equals_append_at_once_when_the_scale_holds():
    # the first token carries the largest value, so no later one raises the
    # scale and the codes do not depend on how the rows were cut
    rng = np.random.default_rng(3)
    nb, bs, hkv, d = 6, 16, 2, 32
    x = rng.uniform(-1, 1, (40, hkv, d)).astype(np.float32)
    x[0::16, :, 0] = 1.5
    tab = np.array([[4, 1, 3]], np.int32)
    pool, sc = _pools(rng, nb, bs, hkv, d)
    once, s1 = O.append_q8_np(pool, sc, x, [0, 40], tab, [40])
    cut, s2 = pool, sc
    for a, b in ((0, 5), (5, 16), (16, 17), (17, 39), (39, 40)):
        cut, s2 = O.append_q8_np(cut, s2, x[a:b], [0, b - a], tab, [b])
    assert np.array_equal(once, cut) and np.array_equal(s1, s2)
    # rows that hold no token and other blocks keep their bytes
    assert np.array_equal(once[3, 8:], pool[3, 8:])
    for other in (0, 2, 5):
        assert np.array_equal(once[other], pool[other]) and np.array_equal(s1[other], sc[other])


def test_append_error_is_half_a_step_of_e4m3():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((32, 3, 64)) * np.exp2(rng.integers(-6, 6, (1, 3, 1)))).astype(np.float32)
    tab = np.array([[1, 0]], np.int32)
    pool, sc = _pools(rng, 2, 16, 3, 64)
    codes, s = O.append_q8_np(pool, sc, x, [0, 32], tab, [32])
    back = O.dequantize_q8(codes, s)[[1, 0]].reshape(32, 3, 64)
    step = np.repeat(s[[1, 0]].astype(np.float64), 16, axis=0)[:, :, None]
    # 2^-4 of the value, or half the subnormal quantum 2^-9 of the scale
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)).all()
    assert (np.abs(x).reshape(2, 16, 3, 64).max(axis=(1, 3)) > 224 * s[[1, 0]]).all()


def test_growth_requantises_exactly_above_the_subnormals():
    rng = np.random.default_rng(5)
    small = rng.uniform(0.5, 1, (5, 1, 32)).astype(np.float32)
    big = (small[:1] * 2.0 ** 5).astype(np.float32)
    tab = np.array([[0]], np.int32)
    pool, sc = _pools(rng, 1, 16, 1, 32)
    a, s1 = O.append_q8_np(pool, sc, small, [0, 5], tab, [5])
    b, s2 = O.append_q8_np(a, s1, big, [0, 1], tab, [6])
    assert s2[0, 0] == s1[0, 0] * 32
    assert np.array_equal(O.dequantize_q8(a, s1)[0, :5], O.dequantize_q8(b, s2)[0, :5])


def test_attention_over_codes_equals_attention_over_their_values():
    rng = np.random.default_rng(6)
    kp, ks = _pools(rng, 4, 16, 2, 32)
    vp, vs = _pools(rng, 4, 16, 2, 32)
    kp[kp & 0x7f == 0x7f] = 0
    vp[vp & 0x7f == 0x7f] = 0
    q = O.f32_to_bf16_raw(rng.standard_normal((2, 4, 32)).astype(np.float32))
    tab = np.array([[2, 0], [3, -1]], np.int32)
    val = lambda c, s: torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy() * \
        s[:, None, :, None].astype(np.float64)                                # noqa: E731
    want = O.paged_attention_np(O.to_f64(q, "bf16"), val(kp, ks), val(vp, vs), tab, [30, 7], 0.1, "f64")
    got = O.paged_attention_q8_np(q, kp, vp, ks, vs, tab, [30, 7], 0.1)
    assert np.array_equal(got, want)
    pre = O.prefill_attention_q8_np(q, kp, vp, ks, vs, tab, [30, 7], [0, 1, 2], 0.1)
    # (one query row per sequence is a decode step; the sums run in another order)
    assert np.abs(pre - want).max() <= 1e-9 * np.abs(want).max()
