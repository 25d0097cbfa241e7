"""Lengths as a caller holds them: context_lens as a column of a table of
per-sequence numbers, and one length for every sequence, give the block-scaled
cache's calls the same bits as a dense copy of them."""
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


def _column(lens):
    """The lengths as the second of three columns, the others absurd."""
    t = torch.full((len(lens), 3), 1 << 30, dtype=torch.int32, device=DEV)
    t[:, 1] = _dev(np.asarray(lens, np.int32))
    return t[:, 1]


def _decode(pa, c, lens, workspace):
    B, hq, d = c.q.shape
    out = torch.full_like(c.q, float("nan"))
    ws = None
    if workspace:
        ws = torch.empty(pa.pa_decode_workspace_bytes(B, hq, c.kp.shape[2], d, int(c.lens.max())),
                         dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_decode_attention_q8(out, c.q, *c.device(), _dev(c.tab), lens, int(c.lens.max()), c.scale,
                              ws, status)
    assert int(status.item()) == 0
    return out


def _prefill(pa, c, lens):
    out = torch.full_like(c.q, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_prefill_attention_q8(out, c.q, _dev(c.cu), int(c.chunks.max()), *c.device(), _dev(c.tab),
                               lens, int(c.lens.max()), c.scale, status)
    assert int(status.item()) == 0
    return out


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens", [[70, 0, 300, 1, 129], [4000, 3000, 3500], list(range(1, 60))])
def test_decode(pa, lens, workspace):
    # (the second case's pieces are joined by a kernel of their own)
    c = Case(41, lens, 16, 4, 256, 16)
    want = _decode(pa, c, _dev(c.lens), workspace)
    assert torch.equal(_decode(pa, c, _column(lens), workspace), want)
    c.check(want, False)


@pytest.mark.parametrize("lens,chunks", [([70, 300, 129], [20, 300, 1]), ([3000, 2500], [5, 3]),
                                         ([64] * 40, [3] * 40)])
def test_prefill(pa, lens, chunks):
    c = Case(42, lens, 8, 2, 128, 16, chunks=chunks)
    want = _prefill(pa, c, _dev(c.lens))
    assert torch.equal(_prefill(pa, c, _column(lens)), want)
    c.check(want, True)


@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [40, 0, 17, 1]])
def test_append(pa, counts):
    lens = [65, 32, 90, 1]
    c = Case(43, lens, 8, 2, 128, 16, chunks=counts)
    T = int(c.cu[-1])
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(T, 2, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    pos = torch.arange(T, device=DEV)
    table = pa.rope_table(T, 32)
    got = []
    for lengths in (_dev(c.lens), _column(lens)):
        pools, q_out = c.device(), torch.empty_like(c.q)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        pa.pa_rope_and_cache_q8(q_out, c.q, k, v, *pools, _dev(c.cu), max(counts), _dev(c.tab),
                                lengths, pos, table, False, status)
        assert int(status.item()) == 0
        got.append((q_out, *pools))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert not torch.equal(got[0][1], _dev(c.kp))


def test_one_length_for_every_sequence(pa):
    c = Case(44, [77] * 6, 8, 2, 128, 16)
    same = torch.tensor([77], dtype=torch.int32, device=DEV).expand(6)
    assert torch.equal(_decode(pa, c, same, True), _decode(pa, c, _dev(c.lens), True))
