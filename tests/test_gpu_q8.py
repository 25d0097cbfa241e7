"""Attention over the block-scaled E4M3 cache on the GPU, through the C ABI,
against fp64 attention over the dequantised values.  The tolerance of every
element is the bound that tests/q8_reference.py derives from the kernels'
roundings."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from paged_kv_cache_455_b200 import workloads as W
from q8_reference import attention_with_bound

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case:
    """Pools with codes 0x7f (NaN) in every row that no sequence holds, block
    scales that differ by several binades, tables of -1 past each sequence."""

    def __init__(self, seed, lens, hq, hkv, d, bs, chunks=None, spread=2.0, odd_scales=False):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        need = -(-self.lens // bs)
        nb = int(need.sum()) + 5
        perm = rng.permutation(nb)
        self.tab = np.full((len(lens), max(1, int(need.max()))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tab[b, :n] = perm[at:at + n]
            at += n
        n = np.ones(len(lens), np.int64) if chunks is None else np.asarray(chunks)
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.chunks = n
        held = np.zeros((nb, bs), bool)
        for b, c in enumerate(self.lens):
            t = np.arange(c)
            held[self.tab[b, t // bs], t % bs] = True
        pools, scales = [], []
        for _ in range(2):
            x = rng.standard_normal((nb, bs, hkv, d)).astype(np.float32)
            x *= np.exp2(rng.uniform(-spread, spread, (nb, 1, hkv, 1))).astype(np.float32)
            amax = np.abs(x).max(axis=(1, 3))
            s = np.exp2(np.ceil(np.log2(amax / 448))).astype(np.float32)
            if odd_scales:
                s = (s * rng.uniform(1.0, 1.9, s.shape)).astype(np.float32)
            codes = torch.from_numpy(x / s[:, None, :, None]).to(torch.float8_e4m3fn)
            codes = codes.view(torch.uint8).numpy().copy()
            codes[~held] = 0x7F
            pools.append(codes)
            scales.append(s)
        self.kp, self.vp = pools
        self.ks, self.vs = scales
        self.q = _dev(rng.standard_normal((int(self.cu[-1]), hq, d)).astype(np.float32)) \
            .to(torch.bfloat16)
        self.scale = d ** -0.5
        self.bs, self.nb = bs, nb

    def device(self):
        return [_dev(x) for x in (self.kp, self.vp, self.ks, self.vs)]

    def decode(self, pa, workspace=True, status=None, scale=None, max_ctx=None, ws=None):
        out = torch.full_like(self.q, float("nan"))
        B, hq, d = self.q.shape
        mc = int(self.lens.max()) if max_ctx is None else max_ctx
        if workspace and ws is None:
            ws = torch.full((pa.pa_decode_workspace_bytes(B, hq, self.kp.shape[2], d, mc),), 255,
                            dtype=torch.uint8, device=DEV)
        pa.pa_decode_attention_q8(out, self.q, *self.device(), _dev(self.tab), _dev(self.lens), mc,
                                  self.scale if scale is None else scale, ws, status)
        torch.cuda.synchronize()
        return out

    def prefill(self, pa, status=None, scale=None):
        out = torch.full_like(self.q, float("nan"))
        pa.pa_prefill_attention_q8(out, self.q, _dev(self.cu), int(self.chunks.max()),
                                   *self.device(), _dev(self.tab), _dev(self.lens),
                                   int(self.lens.max()), self.scale if scale is None else scale,
                                   status)
        torch.cuda.synchronize()
        return out

    def check(self, out, prefill, scale=None):
        ref, tol = attention_with_bound(W.to_numpy_elems(self.q), self.kp, self.vp, self.ks,
                                        self.vs, self.tab, self.lens, self.cu,
                                        self.scale if scale is None else scale, prefill)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        over = np.abs(got - ref) - tol
        assert over.max() <= 0, f"{(over > 0).mean():.3g} of the elements over, by {over.max():.3g}"
        return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


HEADS = [(1, 1, 128, 16), (8, 1, 256, 32), (2, 2, 256, 16), (8, 2, 128, 32), (16, 4, 256, 16),
         (32, 4, 256, 32), (12, 3, 128, 16), (64, 8, 128, 32), (4, 4, 128, 16), (20, 5, 256, 16)]


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("hq,hkv,d,bs", HEADS)
def test_decode_every_tail(pa, hq, hkv, d, bs, workspace):
    # every length around the tile (32 to 128 tokens) and block borders
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 0, 100, 127, 128, 129, 160, 255, 257]
    c = Case(hq * d + bs, lens, hq, hkv, d, bs)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.decode(pa, workspace, status)
    assert int(status.item()) == 0
    assert (out[13] == 0).all()
    c.check(out, False)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,d,bs", [
    ([3000], 16, 4, 256, 16),
    ([5000, 1, 700], 8, 1, 128, 32),
    ([1234, 4321, 77, 0, 2000], 16, 2, 256, 16),
    ([9000], 64, 8, 128, 16),
])
def test_decode_long_contexts(pa, lens, hq, hkv, d, bs, workspace):
    c = Case(sum(lens), lens, hq, hkv, d, bs)
    out = c.decode(pa, workspace)
    err = c.check(out, False)
    assert err < 4e-3      # bf16 rounds by 2^-8 / sqrt(3) of a value at most


def test_decode_many_short_sequences(pa):
    rng = np.random.default_rng(1)
    for hq, hkv, d, bs in ((8, 4, 128, 16), (16, 4, 256, 16), (32, 4, 256, 32), (8, 1, 128, 32)):
        c = Case(2, rng.integers(0, 90, 700), hq, hkv, d, bs)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = c.decode(pa, status=status)
        assert int(status.item()) == 0
        c.check(out, False)


@pytest.mark.parametrize("scale", [-0.06, 0.0, 3.0])
def test_any_softmax_scale(pa, scale):
    c = Case(11, [70, 300], 8, 2, 256, 16)
    c.check(c.decode(pa, scale=scale), False, scale)
    c = Case(12, [70, 300], 8, 2, 256, 16, chunks=[3, 150])
    c.check(c.prefill(pa, scale=scale), True, scale)


@pytest.mark.parametrize("spread,odd", [(12.0, False), (3.0, True)])
def test_scales_far_apart_and_no_powers_of_two(pa, spread, odd):
    # the softmax is dominated by few tokens here; V scales span 24 binades
    c = Case(13, [40, 900, 333], 16, 4, 256, 16, spread=spread, odd_scales=odd)
    c.check(c.decode(pa), False)
    c = Case(14, [40, 900, 333], 16, 4, 256, 16, chunks=[40, 10, 200], spread=spread,
             odd_scales=odd)
    c.check(c.prefill(pa), True)


def test_growing_logits_rescale_again_and_again(pa):
    # keys that point further and further along the query: the reference of
    # the weights grows with almost every tile
    for chunks in (None, [64]):
        c = Case(15, [1500], 4, 1, 256, 16, chunks=chunks, spread=0.0)
        q = c.q.float().cpu().numpy()
        q[:] = np.abs(q)
        c.q = _dev(q).to(torch.bfloat16)
        c.kp[:] = 0x38                      # 1.0
        t = np.arange(-(-1500 // 16))
        c.ks[c.tab[0, t], 0] = np.exp2(-9 + 8 * t / len(t)).astype(np.float32)
        if chunks is None:
            c.check(c.decode(pa), False)
        else:
            c.check(c.prefill(pa), True)


def test_many_small_weights_next_to_a_large_one(pa):
    # one token with most of the weight, thousands that share the rest
    for chunks in (None, [2]):
        c = Case(16, [8000], 4, 1, 128, 32, chunks=chunks, spread=0.0)
        c.kp[:] = 0x38
        c.ks[:] = 2.0 ** -12
        c.ks[c.tab[0, 0], 0] = 8.2 / 8 ** 0.5
        c.kp[c.tab[0, 0], 1:] = 0
        c.q[:] = 0.0884
        c.scale = 1.0
        c.vp[c.tab[0, 0], 0] = 0x30
        if chunks is None:
            err = c.check(c.decode(pa), False)
        else:
            err = c.check(c.prefill(pa), True)
        assert err < 1e-2


def test_bad_blocks_and_lengths(pa):
    c = Case(17, [40, 300, 5, 64, 200], 8, 4, 128, 16, chunks=None)
    c.tab[1, 3] = c.nb
    c.lens[2] = c.tab.shape[1] * 16 + 1
    c.lens[3] = -4
    want = Case(17, [40, 300, 5, 64, 200], 8, 4, 128, 16).decode(pa)
    for workspace in (True, False):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = c.decode(pa, workspace, status, max_ctx=300)
        assert int(status.item()) == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
        assert (out[1:4] == 0).all()
    # (the same tiles, cut elsewhere: the sums may round differently)
    assert (out[[0, 4]].float() - want[[0, 4]].float()).abs().max() <= 2.0 ** -6


def test_a_non_finite_query_row_gives_nan_and_nothing_else(pa):
    for chunks in (None, [20, 30]):
        c = Case(18, [100, 90], 8, 2, 256, 16, chunks=chunks)
        clean = c.decode(pa) if chunks is None else c.prefill(pa)
        c.q[1, 3, 7] = float("inf")
        got = c.decode(pa) if chunks is None else c.prefill(pa)
        assert torch.isnan(got[1, 3]).all()
        got[1, 3], clean[1, 3] = 0, 0
        assert torch.equal(got, clean)


def test_decode_is_the_same_on_every_run(pa):
    c = Case(19, [3000, 20, 1700, 900], 16, 4, 256, 16)
    outs = [c.decode(pa) for _ in range(3)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])


PREFILL = [([7], [7]), ([64], [64]), ([65, 128, 1], [1, 128, 1]), ([300, 200, 97, 33], [77, 200, 5, 0]),
           ([1000, 40], [130, 33])]


@pytest.mark.parametrize("lens,chunks", PREFILL)
@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 4, 256, 16), (8, 1, 256, 32), (2, 2, 128, 32),
                                         (6, 3, 128, 16)])
def test_prefill(pa, lens, chunks, hq, hkv, d, bs):
    c = Case(sum(lens) + d, lens, hq, hkv, d, bs, chunks=chunks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.prefill(pa, status)
    assert int(status.item()) == 0
    c.check(out, True)


def test_prefill_bad_blocks_and_lengths(pa):
    c = Case(21, [40, 300, 50, 64], 8, 4, 128, 16, chunks=[10, 200, 20, 64])
    want = c.prefill(pa)
    c.tab[1, 3] = -7
    c.lens[2] = 19
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.prefill(pa, status)
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK | pa.PA_DEV_BAD_CONTEXT
    cu = c.cu
    assert (out[cu[1]:cu[3]] == 0).all()
    assert torch.equal(out[:cu[1]], want[:cu[1]]) and torch.equal(out[cu[3]:], want[cu[3]:])


def test_decode_captured_once_and_replayed(pa):
    # one call per graph, two graphs that share the workspace, replayed in turn
    cases = [Case(22, [3000, 20, 1700, 900], 16, 4, 256, 16), Case(23, [5000, 640], 8, 1, 128, 32)]
    want = [c.decode(pa) for c in cases]
    ws = torch.full((max(pa.pa_decode_workspace_bytes(4, 16, 4, 256, 3000),
                         pa.pa_decode_workspace_bytes(2, 8, 1, 128, 5000)),), 255,
                    dtype=torch.uint8, device=DEV)
    side, graphs, outs, keep = torch.cuda.Stream(DEV), [], [], []
    for c in cases:
        args = (*c.device(), _dev(c.tab), _dev(c.lens))
        out = torch.zeros_like(c.q)
        keep.append(args)
        outs.append(out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            pa.pa_decode_attention_q8(out, c.q, *args, int(c.lens.max()), c.scale, ws)
        graphs.append(g)
    for which in (0, 0, 1, 0, 1, 1):
        outs[which].fill_(float("nan"))
        graphs[which].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[which], want[which])
    del graphs


@pytest.mark.parametrize("cta", [0, 70, 147])
def test_decode_wait_that_runs_out(pa, cta):
    # CTA `cta` never gets its second tile: its waits end after the limit, the
    # sequences it held from there on are zeros, the rest is right, and the
    # workspace serves the next call
    c = Case(24, [3000] * 12, 16, 4, 256, 16)
    want = c.decode(pa)
    ws = torch.zeros(pa.pa_decode_workspace_bytes(12, 16, 4, 256, 3000), dtype=torch.uint8,
                     device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.testing_set_wait_limit_ns(20_000_000)
    pa.testing_withhold_copy(cta)
    try:
        out = c.decode(pa, status=status, ws=ws)
    finally:
        pa.testing_withhold_copy(-1)
        pa.testing_set_wait_limit_ns(0)
    assert int(status.item()) == pa.PA_DEV_WAIT_TIMEOUT
    # (a range is an equal share of every sequence's tiles and one unit more)
    tiles = -(-3000 // 32)
    r0, r1 = (x * 12 * (tiles + 1) // 148 for x in (cta, cta + 1))
    lost = {v // (tiles + 1) for v in range(r0, r1) if v % (tiles + 1) < tiles}
    for b in range(12):
        assert (out[b] == 0).all() if b in lost else torch.equal(out[b], want[b])
    assert torch.equal(c.decode(pa, ws=ws), want)


@pytest.mark.parametrize("lens,chunks,hq,hkv,d,bs", [
    ([4000], [5], 4, 1, 256, 16),                       # clusters of eight
    ([3000, 40, 900, 2111], [5, 5, 1, 17], 16, 4, 256, 16),
    ([70] * 20 + [2600], [3] * 21, 8, 1, 128, 32),      # parts without a tile
    ([1500, 1400], [200, 33], 16, 2, 128, 16),
])
def test_prefill_of_few_rows_over_long_contexts(pa, lens, chunks, hq, hkv, d, bs):
    c = Case(sum(lens) + d, lens, hq, hkv, d, bs, chunks=chunks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.prefill(pa, status)
    assert int(status.item()) == 0
    c.check(out, True)
    c.tab[0, -1 if len(lens) == 1 else 0] = -1
    out = c.prefill(pa, status)
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK
    assert (out[:c.cu[1]] == 0).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("n,hq,hkv,d,bs", [
    (40, 12, 3, 128, 16),       # row blocks in pairs of CTAs, more sequences than are sorted
    (32, 16, 4, 256, 16),       # the most that are, many of one length, some without rows
    (33, 5, 5, 128, 32),        # single CTAs
])
def test_prefill_of_many_sequences(pa, n, hq, hkv, d, bs):
    rng = np.random.default_rng(n)
    lens = np.where(rng.random(n) < 0.4, 512, rng.integers(1, 900, n))
    chunks = np.minimum(lens, rng.integers(0, 9, n))
    c = Case(n, lens, hq, hkv, d, bs, chunks=chunks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.prefill(pa, status)
    assert int(status.item()) == 0
    c.check(out, True)
