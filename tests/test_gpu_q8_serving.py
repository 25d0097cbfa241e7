"""The block-scaled cache as a serving loop uses it: prompts in chunks, single
tokens, sharing with copy-on-write, paging out, drafted tokens, one captured
step.  The cache must equal the oracle's to the bit after every call, and every
attention stay within the bound that tests/q8_reference.py derives."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from paged_kv_cache_455_b200 import workloads as W
from paged_kv_cache_455_b200.blocks import BlockManager
from q8_reference import attention_with_bound

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Server:
    def __init__(self, pa, hq, hkv, d, bs, nb, seed, host_blocks=0, max_pos=4096):
        self.pa, self.hq, self.hkv, self.d, self.bs, self.nb = pa, hq, hkv, d, bs, nb
        self.rng = np.random.default_rng(seed)
        self.mgr = BlockManager(nb, bs, self.rng.permutation(nb), host_blocks)
        rot = d // 2
        ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))[None]
        self.table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.rot = rot
        codes = self.rng.integers(0, 255, (2, nb, bs, hkv, d), dtype=np.uint8)
        codes[(codes & 0x7f) == 0x7f] = 0
        scales = np.exp2(self.rng.integers(-9, -5, (2, nb, hkv))).astype(np.float32)
        self.np_k, self.np_v = codes
        self.np_ks, self.np_vs = scales
        self.kp, self.vp, self.ks, self.vs = (_dev(x) for x in (*codes, *scales))
        self.host = [torch.zeros((host_blocks, *x.shape[1:]), dtype=x.dtype).pin_memory()
                     for x in (self.kp, self.vp, self.ks, self.vs)] if host_blocks else None
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.scale = d ** -0.5
        self.tab = _dev(self.table)

    def pools(self):
        return self.kp, self.vp, self.ks, self.vs

    def new_rows(self, T):
        # (sizes that change from token to token: scales have to grow)
        x = self.rng.standard_normal((T, self.hq + 2 * self.hkv, self.d)).astype(np.float32)
        x *= np.exp2(self.rng.uniform(-1.5, 1.5, (T, 1, 1))).astype(np.float32)
        return _dev(x).to(torch.bfloat16)

    def step(self, seqs, counts):
        """Appends counts[i] tokens to sequence seqs[i] (blocks and lengths of the
        manager already include them) and returns what the attention needs."""
        tab, lens = self.mgr.block_tables(seqs)
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        pos = np.concatenate([np.arange(l - n, l) for l, n in zip(lens, counts)])
        qkv = self.new_rows(int(cu[-1]))
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], dim=1)
        qr = torch.empty_like(q.contiguous())
        args = (_dev(cu), int(max(counts)), _dev(tab), _dev(lens))
        self.pa.pa_rope_and_cache_q8(qr, q, k, v, *self.pools(), *args, _dev(pos), self.tab,
                                     False, self.status)
        kf, vf, qf = (x.float().cpu().numpy() for x in (k, v, q))
        kf = O.rotate_f32(kf, pos, self.table, self.rot, False)
        self.np_k, self.np_ks = O.append_q8_np(self.np_k, self.np_ks, kf, cu, tab, lens)
        self.np_v, self.np_vs = O.append_q8_np(self.np_v, self.np_vs, vf, cu, tab, lens)
        want = O.f32_to_bf16_raw(O.rotate_f32(qf, pos, self.table, self.rot, False))
        assert np.array_equal(W.to_numpy_elems(qr), want)
        return qr, args, tab, lens, cu

    def check_pools(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        for got, want in zip(self.pools(), (self.np_k, self.np_v, self.np_ks, self.np_vs)):
            assert np.array_equal(got.cpu().numpy(), want)

    def check(self, out, qr, tab, lens, cu, prefill):
        ref, tol = attention_with_bound(W.to_numpy_elems(qr), self.np_k, self.np_v, self.np_ks,
                                        self.np_vs, tab, lens, cu, self.scale, prefill)
        over = np.abs(out.double().cpu().numpy() - ref) - tol
        assert np.isfinite(over).all() and over.max() <= 0

    def prefill(self, qr, args, tab, lens, cu):
        out = torch.full_like(qr, float("nan"))
        self.pa.pa_prefill_attention_q8(out, qr, args[0], args[1], *self.pools(), args[2], args[3],
                                        int(lens.max()), self.scale, self.status)
        self.check_pools()
        self.check(out, qr, tab, lens, cu, True)

    def decode(self, qr, args, tab, lens, cu, ws=None, check=True):
        out = torch.full_like(qr, float("nan"))
        if ws is None:
            ws = torch.full((self.pa.pa_decode_workspace_bytes(
                len(lens), self.hq, self.hkv, self.d, int(lens.max())),), 255, dtype=torch.uint8,
                device=DEV)
        self.pa.pa_decode_attention_q8(out, qr, *self.pools(), args[2], args[3], int(lens.max()),
                                       self.scale, ws, self.status)
        if check:
            self.check_pools()
            self.check(out, qr, tab, lens, cu, False)
        return out

    def copy(self, pairs):
        self.pa.pa_copy_blocks_q8(*self.pools(), *self.pools(),
                                  _dev(np.asarray(pairs, np.int64).reshape(-1, 2)), self.status)
        for s, t in pairs:
            for x in (self.np_k, self.np_v, self.np_ks, self.np_vs):
                x[t] = x[s]

    def append(self, seqs):
        copies = [c for c in (self.mgr.append_slot(s)[1] for s in seqs) if c]
        if copies:
            self.copy(copies)
        return self.step(seqs, [1] * len(seqs))


@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 4, 256, 16), (16, 2, 128, 32), (5, 5, 128, 16)])
def test_prompts_tokens_forks_paging_and_drafts(pa, hq, hkv, d, bs):
    s = Server(pa, hq, hkv, d, bs, 160, hq + d, host_blocks=40)
    m = s.mgr
    # prompts in two chunks, the first of ragged sizes
    full, first = [300, 90, 17, 200], [129, 90, 1, 64]
    for i, n in enumerate(first):
        m.allocate(i, n)
    s.prefill(*s.step([0, 1, 2, 3], first))
    left = {i: full[i] - first[i] for i in range(4) if full[i] > first[i]}
    for i, n in left.items():
        for _ in range(n):
            assert m.append_slot(i)[1] is None
    s.prefill(*s.step(list(left), list(left.values())))
    # single tokens, past a block's border, next to an empty row's neighbours
    seqs = [0, 1, 2, 3]
    for _ in range(3):
        s.decode(*s.append(seqs))
    # two branches of sequence 0: the first to write takes a copy of the block
    m.fork(0, 10)
    m.fork(0, 11)
    seqs = [10, 3, 0, 11, 1]
    for _ in range(2):
        s.decode(*s.append(seqs))
    # sequence 3 out to host memory and back into other blocks
    before = [x[m.tables[3]].clone() for x in s.pools()]
    pairs = m.swap_out(3)
    s.pa.pa_copy_blocks_q8(*s.host, *s.pools(), torch.tensor(pairs, dtype=torch.int64, device=DEV),
                           s.status)
    torch.cuda.synchronize()
    pairs = m.swap_in(3)
    s.pa.pa_copy_blocks_q8(*s.pools(), *s.host, torch.tensor(pairs, dtype=torch.int64, device=DEV),
                           s.status)
    torch.cuda.synchronize()
    for x, y, z in zip(s.pools(), before, (s.np_k, s.np_v, s.np_ks, s.np_vs)):
        assert torch.equal(x[m.tables[3]], y)
        z[m.tables[3]] = y.cpu().numpy()
    s.decode(*s.append(seqs))
    # five drafted tokens for some, scored at once
    for i in (3, 10):
        for _ in range(5):
            copy = m.append_slot(i)[1]
            if copy:
                s.copy([copy])
    s.prefill(*s.step([3, 10], [5, 5]))
    s.decode(*s.append([3, 10, 2]))


def test_appends_in_a_row_across_block_borders(pa):
    """Two single-token appends follow each other, then a decode whose last block
    is the second one's: the first one's rows must be in, however early the
    kernels behind it start."""
    s = Server(pa, 16, 4, 256, 16, 700, 5)
    n = 40
    for i in range(n):
        s.mgr.allocate(i, 15 + 16 * (i % 12))          # one row left in the block
    s.step(list(range(n)), [s.mgr.lens[i] for i in range(n)])
    for _ in range(20):
        s.append(range(n))
        s.decode(*s.append(range(n)), check=False)
    s.decode(*s.append(range(n)))


def test_a_captured_step_replayed_over_growing_contexts(pa):
    """One graph of append and decode over static buffers, replayed while host
    code grows lengths and tables, equals the same calls made one by one."""
    hq, hkv, d, bs, B, steps = 16, 4, 256, 16, 6, 20
    lens0 = np.array([1, 15, 16, 100, 0, 300], np.int32)          # 0: a padded row
    width = 24
    rng = np.random.default_rng(0)
    tab = _dev(rng.permutation(B * width).reshape(B, width).astype(np.int32))
    s = Server(pa, hq, hkv, d, bs, B * width, 9)
    start = [x.clone() for x in s.pools()]
    live = lens0 > 0
    cu = _dev(np.concatenate([[0], np.cumsum(live)]).astype(np.int32))
    T = B
    inputs = [s.new_rows(T) for _ in range(steps)]
    buf = torch.zeros_like(inputs[0])
    q, k, v = buf.split([hq, hkv, hkv], dim=1)
    qr = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEV)
    qd = torch.zeros(B, hq, d, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(qd)
    lens = _dev(lens0)
    pos = torch.zeros(T, dtype=torch.int64, device=DEV)
    row = _dev(np.flatnonzero(live))
    ws = torch.empty(pa.pa_decode_workspace_bytes(B, hq, hkv, d, width * bs), dtype=torch.uint8,
                     device=DEV)

    def one():
        pa.pa_rope_and_cache_q8(qr, q, k, v, *s.pools(), cu, 1, tab, lens, pos, s.tab, False,
                                s.status)
        qd.index_copy_(0, row, qr[:len(row)])
        pa.pa_decode_attention_q8(out, qd, *s.pools(), tab, lens, width * bs, s.scale, ws,
                                  s.status)

    def run(call):
        for x, y in zip(s.pools(), start):
            x.copy_(y)
        lens.copy_(_dev(lens0))
        outs = []
        for i in range(steps):
            buf.copy_(inputs[i])
            lens.add_(_dev(live.astype(np.int32)))
            pos[:len(row)].copy_(lens[row].long() - 1)
            call()
            outs.append(out.clone())
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        return outs, [x.clone() for x in s.pools()]

    eager, pools = run(one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            one()
    torch.cuda.current_stream().wait_stream(side)
    replayed, after = run(graph.replay)
    for x, y in zip(pools, after):
        assert torch.equal(x, y)
    for x, y in zip(eager, replayed):
        assert torch.equal(x, y)
        assert (x[4] == 0).all()
