"""Many small softmax weights next to a large one, over the block-scaled cache:
the first token (an attention sink) takes the largest weight of a row, and
thousands of tokens far below it share a sizeable part of the sum.  The error is
measured against the output.

Token 0 has V = 0, every other token t has V_t = c (a vector), so that
    out = c T / (1 + T),   T = the sum of the tail's weights, the sink's being 1.
The queries are powers of two, which the kernels carry exactly, so what is off
is the weights (1 + T comes from fp32 sums), fp32 sums (2^-12 at most, as in
tests/q8_reference.py) and the output's rounding to bf16, 2^-8.

A weight x in units in which the row's largest is 2^L is off by at most
  chunks (L = 5): hi of 4 bits, half a step 2^-4, half its quantum 2^-10; the
          rest of 3 bits, half a step 2^-3, half its quantum 2^-17:
          2^-7 x + min(2^-13, 2^-3 x + 2^-17)
  decode (L = 0): three parts of 3 bits, the last with half a quantum of 2^-23:
          2^-9 x + 2^-23
"""
import numpy as np
import pytest
import torch

from test_gpu_q8 import Case, _dev

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FP32_AND_BF16 = 2.0 ** -12 + 2.0 ** -8
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _weight_error(x, chunks):
    """The most that a weight x (the row's largest is 1) is off, relative to it."""
    if not chunks:
        return 2.0 ** -9 + 2.0 ** -23 / x
    x = x * 2.0 ** 5
    return 2.0 ** -7 + np.minimum(2.0 ** -13, 2.0 ** -3 * x + 2.0 ** -17) / x


def _case(level, sigma, L, d, bs, chunks, seed, copies=1):
    """Tail weights 2^(level + sigma z), z standard normal; returns the case,
    the weights and the values c.  `copies` sequences share the blocks: with one
    a cluster's CTAs, or a decode's, take parts of it, each with a reference of
    its own; with 149 every row block has one CTA (there are more row blocks
    than SMs), whose reference is the first token's."""
    rng = np.random.default_rng(seed)
    c = Case(seed, [L], 4, 1, d, bs, chunks=chunks, spread=0.0)
    c.scale = 1.0
    c.q[:] = 1.0
    # logit_t = 2^-4 sum_i code_ti
    mean, dev = level / LOG2E * 16 / d, sigma / LOG2E * 16 / d ** 0.5
    x = (mean + dev * rng.standard_normal((L, d))).astype(np.float32)
    x[0] = 0.0
    code = torch.from_numpy(x).to(torch.float8_e4m3fn)
    logit = code.double().numpy().sum(axis=1) / 16
    vals = np.exp2(rng.integers(-2, 3, d)).astype(np.float32) * rng.choice([1.0, 1.25, 1.5], d)
    t = np.arange(L)
    rows = (c.tab[0, t // bs], t % bs, 0)
    c.kp[rows] = code.view(torch.uint8).numpy()
    c.vp[rows] = torch.from_numpy(vals.astype(np.float32)).to(torch.float8_e4m3fn) \
        .view(torch.uint8).numpy()
    c.vp[c.tab[0, 0], 0, 0] = 0
    c.ks[:], c.vs[:] = 2.0 ** -4, 1.0
    rows = 1 if chunks is None else chunks[0]
    c.tab = np.repeat(c.tab, copies, axis=0)
    c.lens = np.repeat(c.lens, copies)
    c.chunks = np.repeat(c.chunks, copies)
    c.cu = (np.arange(copies + 1) * rows).astype(np.int32)
    c.q = c.q[:rows].repeat(copies, 1, 1)
    return c, np.exp(logit[1:]), vals


def _check(pa, c, w, vals, chunks, off):
    """`off`: bound of the relative error of the tail's sum."""
    out = (c.prefill(pa) if chunks else c.decode(pa)).double().cpu().numpy()
    n = 1 if chunks is None else chunks[0]
    for j in range(n):                     # row j sees all but the last n - 1 - j tokens
        T = w[:len(w) - (n - 1 - j)].sum()
        want = vals * T / (1 + T)
        err = np.abs(out[j::n] - want).max(axis=(0, 1)) / want
        assert err.max() <= off + FP32_AND_BF16, (j, T, err.max(), off)


@pytest.mark.parametrize("copies", [1, 149])
@pytest.mark.parametrize("chunks", [None, [2]])
@pytest.mark.parametrize("d,bs", [(128, 32), (256, 16)])
@pytest.mark.parametrize("level,L", [(-9.3, 1200), (-11.8, 6000), (-12.6, 9000)])
def test_equal_small_weights(pa, level, L, d, bs, chunks, copies):
    # (codes of one value: every tail weight is the same number)
    c, w, vals = _case(level, 0.0, L, d, bs, chunks, 51, copies)
    assert w.min() == w.max() and 0.2 < w.sum() < 8
    _check(pa, c, w, vals, chunks, float(_weight_error(w[0], chunks)))


@pytest.mark.parametrize("copies", [1, 149])
@pytest.mark.parametrize("chunks", [None, [2]])
@pytest.mark.parametrize("d,bs", [(128, 32), (256, 16)])
@pytest.mark.parametrize("level,L", [(-13.0, 6000), (-15.0, 20000), (-17.0, 32768), (-17.5, 100000)])
def test_spread_small_weights(pa, level, L, d, bs, chunks, copies):
    """Weights that spread over binades are rounded up as often as down.  What
    is left of a cell [a - h, a + h] that is rounded to a is the density's
    slope over it: (h / a)^2 / 3 (1 + |d ln p / d ln x|) of it, h / a <= 1 / 8
    where only the lower part has bits.  With the spread of one binade (0.69
    nats) and the sum's weight one standard deviation from the mean at most,
    1 + slope <= 1 + 1 / 0.69: 1.3 % = 2^-6.3; six standard deviations of the
    random part (each weight off by an eighth of itself) are 6 / 8 / N^0.5."""
    c, w, vals = _case(level, 1.0, L, d, bs, chunks, 52, copies)
    assert w.max() < 2.0 ** -8 and w.sum() > 0.1
    n_eff = w.sum() ** 2 / (w ** 2).sum()
    off = 2.0 ** -6.3 + 0.75 / n_eff ** 0.5 if chunks else 2.0 ** -9 + 2.0 ** -23 / w.mean()
    _check(pa, c, w, vals, chunks, off)
