"""Argument checks of the rotary cache writes and of the block-scaled cache's
calls: every refusal happens on the host, before any CUDA call, so fake
addresses are never dereferenced.  Runs without a GPU."""
import pytest
import torch

A = 0x10000          # 16-byte aligned
M = 0x10008          # misaligned


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import build
    build.build()
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _rope(pa, **kw):
    a = dict(qo=A, qos=2048, q=A, qs=2048, k=A, ks=256, v=A, vs=256, kp=A, vp=A, slots=A, pos=A,
             cs=A, rot=64, maxpos=100, inter=0, T=3, hq=8, hkv=2, d=128, bs=16, nb=8, dt=1)
    assert set(kw) <= set(a)
    a.update(kw)
    return pa.lib.pa_rope_and_cache(a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                    a["vs"], a["kp"], a["vp"], a["slots"], a["pos"], a["cs"],
                                    a["rot"], a["maxpos"], a["inter"], a["T"], a["hq"], a["hkv"],
                                    a["d"], a["bs"], a["nb"], a["dt"], None, None)


ROPE_SHARED = [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1),
    (dict(vp=None), 1), (dict(pos=None), 1), (dict(cs=None), 1), (dict(q=M), 1), (dict(qo=M), 1),
    (dict(k=M), 1), (dict(v=M), 1), (dict(kp=M), 1), (dict(cs=M), 1), (dict(rot=-16), 1),
    (dict(rot=24), 1), (dict(rot=144), 1), (dict(maxpos=0), 1), (dict(hq=-1), 1), (dict(hkv=0), 1),
    (dict(nb=0), 1), (dict(qs=1016), 1), (dict(qos=1016), 1), (dict(ks=248), 1), (dict(vs=248), 1),
    (dict(ks=260), 1), (dict(qs=2052), 1), (dict(d=96), 2), (dict(d=512), 2), (dict(bs=24), 2),
    (dict(bs=64), 2),
]


@pytest.mark.parametrize("kw,want", ROPE_SHARED + [
    (dict(slots=None), 1), (dict(T=-1), 1), (dict(dt=2), 2), (dict(dt=9), 2), (dict(bs=2), 2)])
def test_rope_refusals(pa, kw, want):
    assert _rope(pa, **kw) == want


def test_rope_with_nothing_to_do(pa):
    assert _rope(pa, T=0, k=None, q=None, kp=None) == 0


def _append(pa, **kw):
    a = dict(qo=A, qos=2048, q=A, qs=2048, k=A, ks=256, v=A, vs=256, kp=A, vp=A, ksc=A, vsc=A, cu=A,
             T=9, maxq=4, tab=A, maxb=4, lens=A, B=3, pos=A, cs=A, rot=64, maxpos=100, inter=0, hq=8,
             hkv=2, d=128, bs=16, nb=8)
    assert set(kw) <= set(a)
    a.update(kw)
    return pa.lib.pa_rope_and_cache_q8(a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                       a["vs"], a["kp"], a["vp"], a["ksc"], a["vsc"], a["cu"],
                                       a["T"], a["maxq"], a["tab"], a["maxb"], a["lens"], a["B"],
                                       a["pos"], a["cs"], a["rot"], a["maxpos"], a["inter"],
                                       a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], None, None)


@pytest.mark.parametrize("kw,want", ROPE_SHARED + [
    (dict(ksc=None), 1), (dict(vsc=None), 1), (dict(cu=None), 1), (dict(tab=None), 1),
    (dict(lens=None), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(maxq=-1), 1), (dict(maxb=0), 1),
    (dict(d=64), 2), (dict(bs=8), 2)])
def test_append_refusals(pa, kw, want):
    assert _append(pa, **kw) == want


@pytest.mark.parametrize("kw", [dict(T=0), dict(B=0), dict(maxq=0)])
def test_append_with_nothing_to_do(pa, kw):
    assert _append(pa, k=None, q=None, kp=None, cu=None, **kw) == 0


def _decode(pa, **kw):
    a = dict(out=A, q=A, kp=A, vp=A, ks=A, vs=A, tab=A, maxb=4, lens=A, B=3, mc=64, hq=8, hkv=2,
             d=128, bs=16, nb=16)
    assert set(kw) <= set(a)
    a.update(kw)
    return pa.lib.pa_decode_attention_q8(a["out"], a["q"], a["kp"], a["vp"], a["ks"], a["vs"],
                                         a["tab"], a["maxb"], a["lens"], a["B"], a["mc"], a["hq"],
                                         a["hkv"], a["d"], a["bs"], a["nb"], 0.1, None, 0, None,
                                         None)


ATTENTION = [
    (dict(out=None), 1), (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(tab=None), 1), (dict(lens=None), 1),
    (dict(out=M), 1), (dict(q=M), 1), (dict(kp=M), 1), (dict(vp=M), 1), (dict(B=-1), 1),
    (dict(mc=65), 1), (dict(mc=-1), 1), (dict(hq=6, hkv=4), 1), (dict(hq=12, hkv=4), 2),
    (dict(hq=32, hkv=2), 2), (dict(d=64), 2), (dict(d=96), 2), (dict(bs=8), 2), (dict(bs=64), 2),
    (dict(nb=0), 1), (dict(maxb=0), 1), (dict(nb=1 << 40), 1),
]


@pytest.mark.parametrize("kw,want", ATTENTION + [(dict(B=16385), 2)])
def test_decode_refusals(pa, kw, want):
    assert _decode(pa, **kw) == want


def test_decode_without_sequences(pa):
    assert _decode(pa, B=0, out=None, q=None, ks=None) == 0


def _prefill(pa, **kw):
    a = dict(out=A, q=A, cu=A, T=10, maxq=8, kp=A, vp=A, ks=A, vs=A, tab=A, maxb=4, lens=A, B=2,
             mc=64, hq=8, hkv=2, d=128, bs=16, nb=32)
    assert set(kw) <= set(a)
    a.update(kw)
    return pa.lib.pa_prefill_attention_q8(a["out"], a["q"], a["cu"], a["T"], a["maxq"], a["kp"],
                                          a["vp"], a["ks"], a["vs"], a["tab"], a["maxb"],
                                          a["lens"], a["B"], a["mc"], a["hq"], a["hkv"], a["d"],
                                          a["bs"], a["nb"], 0.1, None, None)


@pytest.mark.parametrize("kw,want", ATTENTION + [
    (dict(cu=None), 1), (dict(T=-1), 1), (dict(maxq=-1), 1), (dict(maxq=64, mc=60), 1)])
def test_prefill_refusals(pa, kw, want):
    assert _prefill(pa, **kw) == want


@pytest.mark.parametrize("kw", [dict(T=0), dict(B=0), dict(maxq=0)])
def test_prefill_with_nothing_to_do(pa, kw):
    assert _prefill(pa, out=None, q=None, cu=None, ks=None, **kw) == 0


def _copy(pa, **kw):
    a = dict(dk=A, dv=A, dks=A, dvs=A, dnb=8, sk=A, sv=A, sks=A, svs=A, snb=8, map=A, n=2, bs=16,
             hkv=2, d=128)
    assert set(kw) <= set(a)
    a.update(kw)
    return pa.lib.pa_copy_blocks_q8(a["dk"], a["dv"], a["dks"], a["dvs"], a["dnb"], a["sk"],
                                    a["sv"], a["sks"], a["svs"], a["snb"], a["map"], a["n"],
                                    a["bs"], a["hkv"], a["d"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dk=None), 1), (dict(dv=None), 1), (dict(dks=None), 1), (dict(dvs=None), 1),
    (dict(sk=None), 1), (dict(sv=None), 1), (dict(sks=None), 1), (dict(svs=None), 1),
    (dict(map=None), 1), (dict(dk=M), 1), (dict(sv=M), 1), (dict(n=-1), 1), (dict(dnb=0), 1),
    (dict(snb=0), 1), (dict(hkv=0), 1), (dict(d=64), 2), (dict(bs=8), 2)])
def test_copy_refusals(pa, kw, want):
    assert _copy(pa, **kw) == want


def test_copy_of_no_pairs(pa):
    assert _copy(pa, n=0, dk=None, sks=None, map=None) == 0


def test_bindings_reject_cpu_tensors(pa):
    x = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 16, 2, 128, dtype=torch.uint8)
    sc = torch.ones(4, 2)
    i32 = torch.zeros(3, dtype=torch.int32)
    tab = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(x, x, kv, kv, pool.bfloat16(), pool.bfloat16(), torch.arange(3))
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache_q8(x, x, kv, kv, pool, pool, sc, sc, torch.zeros(4, dtype=torch.int32),
                                1, tab, i32)
    with pytest.raises(ValueError):
        pa.pa_decode_attention_q8(x, x, pool, pool, sc, sc, tab, i32, 8, 0.1)
    with pytest.raises(ValueError):
        pa.pa_prefill_attention_q8(x, x, torch.zeros(4, dtype=torch.int32), 1, pool, pool, sc, sc,
                                   tab, i32, 8, 0.1)
    with pytest.raises(ValueError):
        pa.pa_copy_blocks_q8(pool, pool, sc, sc, pool, pool, sc, sc,
                             torch.zeros(1, 2, dtype=torch.int64))


def test_rope_table(pa):
    t = pa.rope_table(50, 32, 10000.0, device="cpu").double()
    assert t.shape == (50, 32)
    inv = 10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    ang = 49 * inv
    # one rounding to fp32: half a step of values up to 1
    assert (t[49, :16] - ang.cos()).abs().max() <= 2.0 ** -25
    assert (t[49, 16:] - ang.sin()).abs().max() <= 2.0 ** -25
