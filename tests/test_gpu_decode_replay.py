"""A graph that holds one decode call, replayed again and again: cut segments
are counted and merged on every replay, also when graphs of other shapes use
the same workspace in between."""
import numpy as np
import pytest
import torch

from paged_kv_cache_455_b200 import workloads as W
from oracle import oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL = {torch.float32: 1e-5, torch.bfloat16: 2e-2}     # as everywhere in these tests


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


class Call:
    """One decode call over its own pools; `kind`: bf16, f32, fp8 or static."""

    def __init__(self, pa, seed, kind, lens, hq, hkv, d, bs):
        rng = np.random.default_rng(seed)
        self.pa, self.kind = pa, kind
        self.lens = np.asarray(lens, np.int32)
        need = -(-self.lens // bs)
        nb = int(need.sum()) + 2
        perm = rng.permutation(nb)
        self.tab = np.full((len(lens), int(need.max())), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tab[b, :n] = perm[at:at + n]
            at += n
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.dtype = torch.float32 if kind == "f32" else torch.bfloat16

        def rand(*s):
            return torch.randn(*s, generator=g, device=DEV).to(self.dtype)

        self.q, self.kp, self.vp = rand(len(lens), hq, d), rand(nb, bs, hkv, d), rand(nb, bs, hkv, d)
        if kind == "fp8":
            self.kp, self.vp = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (self.kp, self.vp))
        self.scale = d ** -0.5
        self.args = (torch.from_numpy(self.tab).to(DEV), torch.from_numpy(self.lens).to(DEV),
                     int(self.lens.max()), self.scale)
        self.ws_bytes = pa.pa_decode_workspace_bytes(len(lens), hq, hkv, d, self.args[2])
        self.out = torch.zeros_like(self.q)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def __call__(self, ws):
        pa, a = self.pa, self.args
        if self.kind == "fp8":
            pa.pa_decode_attention_fp8(self.out, self.q, self.kp, self.vp, *a, 1.0, 1.0, ws,
                                       self.status)
        elif self.kind == "static":
            pa.pa_decode_attention_static(self.out, self.q, self.kp, self.vp, *a, self.status)
        else:
            pa.pa_decode_attention(self.out, self.q, self.kp, self.vp, *a, ws, self.status)

    def check_oracle(self):
        if self.kind == "fp8":
            return                        # (tests/test_gpu_fp8.py pins the eager call)
        ref = O.paged_attention(W.to_numpy_elems(self.q), W.to_numpy_elems(self.kp),
                                W.to_numpy_elems(self.vp), self.tab, self.lens, self.scale,
                                "f32" if self.kind == "f32" else "bf16")
        got = self.out.double().cpu().numpy()
        assert np.abs(got - ref).max() <= TOL[self.dtype]


SHAPES = {
    "bf16": [([3000, 20, 1700, 900], 16, 4, 256, 16), ([5000, 640], 8, 1, 128, 32),
             ([2000] * 3, 2, 2, 64, 8)],
    "f32": [([1500, 20, 700], 4, 2, 128, 16), ([2100], 8, 1, 64, 4)],
    "fp8": [([3000, 20, 1700, 900], 16, 4, 256, 16), ([5000, 640], 8, 1, 128, 32)],
    "static": [([3000, 20, 1700, 900], 16, 4, 256, 16), ([4000, 640], 8, 2, 128, 16)],
}


@pytest.mark.parametrize("kind", list(SHAPES))
def test_one_call_captured_and_replayed(pa, kind):
    calls = [Call(pa, 70 + i, kind, *s) for i, s in enumerate(SHAPES[kind])]
    ws = torch.full((max(c.ws_bytes for c in calls),), 255, dtype=torch.uint8, device=DEV)
    want = []
    for c in calls:
        c(ws)
        torch.cuda.synchronize()
        c.check_oracle()
        want.append(c.out.clone())
    side, graphs = torch.cuda.Stream(DEV), []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            c(ws)
        graphs.append(g)
    order = [0, 0, 0, 1, 0, 1, 1, 0]
    if len(calls) > 2:
        order += [2, 2, 0, 2, 1, 2]
    for i in order:
        calls[i].out.fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        assert int(calls[i].status.item()) == 0
        assert torch.equal(calls[i].out, want[i]), (i, order)
    # an eager call behind the replays
    for c, w in zip(calls, want):
        c.out.fill_(float("nan"))
        c(ws)
        assert torch.equal(c.out, w)
    del graphs
