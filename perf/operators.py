"""Timed cases of the rotary cache writes and of the block-scaled 8-bit cache.

Five operators of the library are called here, each with the state a serving
loop holds between steps:

  rope         pa_rope_and_cache        rotate queries and keys, store K/V in a
                                        bf16 or fp32 paged cache
  rope_q8      pa_rope_and_cache_q8     the same into E4M3 pools with one scale
                                        per (block, KV head)
  decode_q8    pa_decode_attention_q8   one query token per sequence over those
                                        pools
  prefill_q8   pa_prefill_attention_q8  a chunk of query tokens per sequence
  copy_q8      pa_copy_blocks_q8        whole blocks with their scales (sharing
                                        with copy-on-write, defragmentation)

`run` gives each operator in its plain form (elementary torch operations in
32 bits) or, where `own` is true, through the library.  Pools hold E4M3 codes
in uint8 tensors; they are returned as float8_e4m3fn views, next to the
scales that multiply them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
SCALE_MIN, SCALE_MAX = -64, 120      # exponents of a block's scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's cache write: 60 sequences in a batch padded to 64,
        # partial rotation, as between the QKV product and attention
        dict(name="rope_decode_64", op="rope", seqs=60, lo=1, hi=1, pad=4, ctx=4096, hq=16, hkv=4,
             d=256, rot=64, bs=16, dtype="bf16", interleaved=False, fused=True),
        # prompts entering the cache: 16 ragged prompts, the whole head rotated
        dict(name="rope_prompts", op="rope", seqs=16, lo=1, hi=2048, pad=0, ctx=4096, hq=16, hkv=4,
             d=256, rot=256, bs=16, dtype="bf16", interleaved=False, fused=True),
        # one decode step into the 8-bit cache, a large batch
        dict(name="rope_q8_decode_256", op="rope_q8", seqs=256, lo=1, hi=1, pad=0, ctx=1024, hq=16,
             hkv=4, d=256, rot=64, bs=16, interleaved=False, fused=True),
        # prompt chunks of up to 512 tokens into the 8-bit cache
        dict(name="rope_q8_chunks", op="rope_q8", seqs=32, lo=1, hi=512, pad=3, ctx=2048, hq=16,
             hkv=4, d=256, rot=256, bs=16, interleaved=False, fused=True),
        # a single user's short conversation: latency alone counts
        dict(name="decode_q8_one", op="decode_q8", seqs=1, lo=100, hi=100, empty=0, hq=16, hkv=4,
             d=256, bs=16),
        # the qwen-shaped layer of the benchmark
        dict(name="decode_q8_qwen", op="decode_q8", seqs=64, lo=128, hi=4096, empty=0, hq=16,
             hkv=4, d=256, bs=16),
        # the long-context layer of the benchmark: few rows, a long axis
        dict(name="decode_q8_long", op="decode_q8", seqs=8, lo=8192, hi=8192, empty=0, hq=16,
             hkv=4, d=256, bs=16),
        # another head layout: eight query heads per KV head, d 128, blocks of
        # 32, ragged lengths from one token, three empty rows of a padded batch
        dict(name="decode_q8_wide", op="decode_q8", seqs=45, lo=1, hi=6000, empty=3, hq=64, hkv=8,
             d=128, bs=32),
        # five drafted tokens per sequence, scored against the whole context
        dict(name="prefill_q8_draft", op="prefill_q8", seqs=32, qlo=5, qhi=5, lo=500, hi=4000,
             hq=16, hkv=4, d=256, bs=16),
        # chunked prefill: 512-token chunks over contexts of 1-4K tokens
        dict(name="prefill_q8_chunk512", op="prefill_q8", seqs=16, qlo=512, qhi=512, lo=1024,
             hi=4096, hq=16, hkv=4, d=256, bs=16),
        # the last blocks of forked sequences, cloned on their first divergence
        dict(name="copy_q8_fork", op="copy_q8", pairs=48, blocks=2048, hkv=4, d=256, bs=16),
        # compaction of a fragmented pool
        dict(name="copy_q8_compact", op="copy_q8", pairs=3000, blocks=7000, hkv=8, d=128, bs=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_q8", "decode_q8", "decode_q8", "prefill_q8", "copy_q8"])
    d = rng.choice([128, 256])
    hkv = rng.choice([1, 2, 3, 4, 5, 8]) if d == 128 else rng.choice([1, 2, 3, 4])
    hq = hkv * rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32])
    if op in ("rope", "rope_q8"):
        c = dict(op=op, hkv=hkv, hq=hq, d=d, bs=bs)
        if op == "rope":
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            c["bs"] = rng.choice([4, 8, 16, 32])
            c["d"] = d = rng.choice([64, 128, 256])
        if rng.random() < 0.4:
            c.update(seqs=_log(rng, 1, 400), lo=1, hi=1)
        else:
            hi = _log(rng, 2, 1500)
            c.update(seqs=_log(rng, 1, max(2, 12000 // hi)), lo=1, hi=hi)
        c.update(pad=rng.choice([0, 0, 1, 5]), ctx=c["hi"] + _log(rng, 1, 700),
                 rot=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.4,
                 fused=rng.random() < 0.5)
        return c
    if op == "decode_q8":
        hi = _log(rng, 1, 12000)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(300, 100000 // hi))),
                    lo=max(1, int(hi * rng.random())), hi=hi, empty=rng.choice([0, 0, 1, 2]),
                    hq=hq, hkv=hkv, d=d, bs=bs)
    if op == "prefill_q8":
        qhi = _log(rng, 1, 700)
        hi = qhi + _log(rng, 1, 2500)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(40, 6000 // qhi))), qlo=rng.randint(1, qhi),
                    qhi=qhi, lo=qhi, hi=hi, hq=hkv * min(hq // hkv, 8 if hkv <= 2 else 2),
                    hkv=hkv, d=d, bs=bs)
    blocks = _log(rng, 40, 6000)
    return dict(op=op, pairs=rng.randint(1, blocks // 3), blocks=blocks, hkv=hkv, d=d, bs=bs)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(case):
    """(new tokens, context length) of each sequence, by the case alone: a seed
    shuffles them among the sequences."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    if case["op"] in ("rope", "rope_q8"):
        new = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(n - 1)]
        return [(x, x + rng.randint(0, case["ctx"] - case["hi"])) for x in new]
    lens = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(n - 1)]
    if case["op"] == "decode_q8":
        return [(1, x) for x in lens]
    return [(case["qhi"] if i == 0 else rng.randint(case["qlo"], case["qhi"]), x)
            for i, x in enumerate(lens)]


def _shuffled(case, g):
    """Both of _lengths as int32 tensors, in the seed's order."""
    x = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    return x[torch.randperm(x.shape[0], generator=g, device=DEV)].unbind(1)


def _tables(lens, bs, g, spare):
    """Block tables drawn from a shuffled free list: -1 past each sequence."""
    need = (lens + bs - 1) // bs
    total, width = int(need.sum()), max(1, int(need.max()))
    nb = total + spare
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)
    used = col[None, :] < need[:, None]
    tables = torch.full((lens.numel(), width), -1, dtype=torch.int32, device=DEV)
    tables[used] = perm[:total]
    return tables, nb


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, in the exponent range."""
    m, e = torch.frexp(amax)
    e = e.to(torch.int32)
    s = torch.where(m <= 0.875, e - 9, e - 8)
    s = torch.where(amax > 0, s, torch.full_like(s, SCALE_MIN)).clamp(SCALE_MIN, SCALE_MAX)
    return torch.ldexp(torch.ones_like(amax), s)


def _quantised(nb, bs, hkv, d, g):
    """Pools as a serving loop holds them: normal values whose size varies from
    channel to channel and from block to block, quantised block by block."""
    codes = torch.empty(nb, bs, hkv, d, dtype=torch.uint8, device=DEV)
    scales = torch.empty(nb, hkv, device=DEV)
    chan = torch.exp(0.4 * torch.randn(hkv, d, generator=g, device=DEV))
    step = max(1, (1 << 26) // (bs * hkv * d))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        x = torch.randn(n, bs, hkv, d, generator=g, device=DEV) * chan
        x *= torch.exp(0.5 * torch.randn(n, 1, hkv, 1, generator=g, device=DEV))
        s = _pow2_scale(x.abs().amax(dim=(1, 3)))
        codes[i:i + n] = (x / s[:, None, :, None]).to(F8).view(torch.uint8)
        scales[i:i + n] = s
    return codes, scales


def _rope_table(rows, rot):
    """[rows, rot] fp32: cos then sin of position * 10000^(-2 i / rot)."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    g = _gen(seed)
    op, hkv, d, bs = case["op"], case["hkv"], case["d"], case["bs"]
    st = dict(case=case, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if op in ("rope", "rope_q8"):
        dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
        B, hq = case["seqs"], case["hq"]
        n, lens = _shuffled(case, g)
        tables, nb = _tables(lens, bs, g, 8)
        cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        cu[1:] = torch.cumsum(n, 0)
        real = int(cu[-1])
        T = real + case["pad"]
        seq = torch.repeat_interleave(torch.arange(B, device=DEV), n.long())
        pos = torch.zeros(T, dtype=torch.int64, device=DEV)
        pos[:real] = (lens - n)[seq] + torch.arange(real, device=DEV) - cu[:-1][seq]
        width = (hq + 2 * hkv) * d
        chan = torch.exp(0.4 * torch.randn(width, generator=g, device=DEV))
        qkv = (torch.randn(T, width, generator=g, device=DEV) * chan).to(dt)
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        st.update(q=q.view(T, hq, d), k=k.view(T, hkv, d), v=v.view(T, hkv, d), pos=pos,
                  table=_rope_table(case["ctx"], case["rot"]), lens=lens, tables=tables, cu=cu,
                  q_out=torch.empty(T, hq, d, dtype=dt, device=DEV), max_q=case["hi"])
        if op == "rope":
            slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
            p = pos[:real]
            slots[:real] = tables[seq, p // bs].long() * bs + p % bs
            st.update(slots=slots, kp=torch.zeros(nb, bs, hkv, d, dtype=dt, device=DEV),
                      vp=torch.zeros(nb, bs, hkv, d, dtype=dt, device=DEV))
        else:
            st["kp"], st["ks"] = _quantised(nb, bs, hkv, d, g)
            st["vp"], st["vs"] = _quantised(nb, bs, hkv, d, g)
            st["q_out"][real:] = 0
    elif op in ("decode_q8", "prefill_q8"):
        B, hq = case["seqs"], case["hq"]
        n, lens = _shuffled(case, g)
        if op == "decode_q8":
            # the empty rows of a batch padded to the size of a captured graph
            lens = torch.cat([lens, lens.new_zeros(case["empty"])])
            B += case["empty"]
            T = B
        else:
            cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
            cu[1:] = torch.cumsum(n, 0)
            T = int(cu[-1])
            st.update(cu=cu, max_q=case["qhi"])
        tables, nb = _tables(lens, bs, g, 16)
        q = (1.5 * torch.randn(T, hq, d, generator=g, device=DEV)).to(torch.bfloat16)
        st["kp"], st["ks"] = _quantised(nb, bs, hkv, d, g)
        st["vp"], st["vs"] = _quantised(nb, bs, hkv, d, g)
        st.update(q=q, lens=lens, tables=tables, max_ctx=case["hi"], scale=d ** -0.5,
                  out=torch.empty_like(q))
    else:
        nb, P = case["blocks"], case["pairs"]
        perm = torch.randperm(nb, generator=g, device=DEV)
        src = perm[torch.randint(0, nb - P, (P,), generator=g, device=DEV)]
        st["map"] = torch.stack([src, perm[nb - P:]], dim=1).contiguous()
        st["kp"], st["ks"] = _quantised(nb, bs, hkv, d, g)
        st["vp"], st["vs"] = _quantised(nb, bs, hkv, d, g)
    return st


# ----------------------------------------------------- the operators, plain
def _rotate(x, cos, sin, rot, interleaved):
    """Rotates the first `rot` elements of x [T, H, d] (fp32) by the angles
    whose cosines and sines are [T, rot / 2]."""
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(st):
    c = st["case"]
    cs = st["table"][st["pos"]]
    cos, sin = cs.chunk(2, dim=1)
    dt = st["q"].dtype
    q = _rotate(st["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(dt)
    k = _rotate(st["k"].float(), cos, sin, c["rot"], c["interleaved"]).to(dt)
    keep = st["slots"] >= 0
    at = st["slots"][keep]
    st["kp"].view(-1, c["hkv"], c["d"])[at] = k[keep]
    st["vp"].view(-1, c["hkv"], c["d"])[at] = st["v"][keep]
    return dict(q=q, k=st["kp"], v=st["vp"])


def _append_q8(pool, scales, x, blk, off):
    """Stores rows x [T, hkv, d] (fp32) at rows `off` of blocks `blk`: a
    block's scale grows to hold its new rows, its older rows are requantised
    by the ratio, and a block written from its first row starts afresh."""
    ub, at = torch.unique(blk, return_inverse=True)
    n, bs = ub.numel(), pool.shape[1]
    mag = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=-1)
    amax = torch.zeros(n, x.shape[1], device=x.device).index_reduce_(0, at, mag, "amax")
    first = torch.full((n,), bs, device=x.device).index_reduce_(0, at, off, "amin")
    want, old = _pow2_scale(amax), scales[ub]
    fresh = (first == 0)[:, None]
    new = torch.where(fresh, want, torch.maximum(old, want))
    ratio = torch.where(fresh, torch.ones_like(old), old / new)
    rows = pool[ub]
    was = torch.arange(bs, device=x.device)[None, :] < first[:, None]
    moved = (rows.view(F8).float() * ratio[:, None, :, None]).to(F8).view(torch.uint8)
    rows = torch.where(was[:, :, None, None], moved, rows)
    rows[at, off] = (x / new[at][:, :, None]).clamp(-448, 448).to(F8).view(torch.uint8)
    pool[ub] = rows
    scales[ub] = new


def _plain_rope_q8(st):
    c = st["case"]
    cu, lens, bs = st["cu"].long(), st["lens"].long(), c["bs"]
    real = st["k"].shape[0] - c["pad"]
    t = torch.arange(real, device=DEV)
    seq = torch.bucketize(t, cu[1:], right=True)
    place = lens[seq] - (cu[seq + 1] - t)
    blk, off = st["tables"][seq, place // bs].long(), place % bs
    cos, sin = st["table"][st["pos"][:real]].chunk(2, dim=1)
    q = torch.zeros_like(st["q_out"])
    q[:real] = _rotate(st["q"][:real].float(), cos, sin, c["rot"], c["interleaved"]).to(q.dtype)
    k = _rotate(st["k"][:real].float(), cos, sin, c["rot"], c["interleaved"])
    _append_q8(st["kp"], st["ks"], k, blk, off)
    _append_q8(st["vp"], st["vs"], st["v"][:real].float(), blk, off)
    return dict(q=q, k=st["kp"].view(F8), v=st["vp"].view(F8), ks=st["ks"], vs=st["vs"])


def _gathered(pool, scales, tables):
    """[B, max_blocks * bs, hkv, d] fp32: the cache through the block tables."""
    at = tables.clamp(min=0).long()
    x = pool[at].view(F8).float() * scales[at][:, :, None, :, None]
    return x.flatten(1, 2)


def _softmax_weights(s, seen):
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(dim=-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(st):
    c = st["case"]
    B, hkv, d = st["q"].shape[0], c["hkv"], c["d"]
    K = _gathered(st["kp"], st["ks"], st["tables"]).permute(0, 2, 3, 1)
    V = _gathered(st["vp"], st["vs"], st["tables"]).permute(0, 2, 1, 3)
    s = torch.matmul(st["q"].float().view(B, hkv, -1, d), K) * st["scale"]
    seen = torch.arange(s.shape[-1], device=DEV) < st["lens"][:, None, None, None]
    # (a column without a token has weight 0, whatever the gathered row holds)
    V = torch.where(seen.transpose(-1, -2), V, torch.zeros_like(V))
    out = torch.matmul(_softmax_weights(s, seen), V)
    return out.reshape(B, c["hq"], d).to(torch.bfloat16)


def _plain_prefill(st):
    c = st["case"]
    B, hkv, d, n = st["lens"].numel(), c["hkv"], c["d"], st["max_q"]
    cu, lens, G = st["cu"].long(), st["lens"].long(), c["hq"] // c["hkv"]
    K = _gathered(st["kp"], st["ks"], st["tables"]).permute(0, 2, 3, 1)
    V = _gathered(st["vp"], st["vs"], st["tables"]).permute(0, 2, 1, 3)
    j = torch.arange(n, device=DEV)[None, :]
    count = (cu[1:] - cu[:-1])[:, None]
    row = (cu[:-1, None] + torch.minimum(j, count - 1)).flatten()
    q = st["q"][row].float().view(B, n, hkv, G, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, K) * st["scale"]
    place = lens[:, None] - count + torch.minimum(j, count - 1)
    seen = torch.arange(s.shape[-1], device=DEV) <= place[:, :, None]
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    held = torch.arange(s.shape[-1], device=DEV)[None, :] < lens[:, None]
    V = torch.where(held[:, None, :, None], V, torch.zeros_like(V))
    o = torch.matmul(_softmax_weights(s, seen), V)
    o = o.view(B, hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(B * n, c["hq"], d)
    out = torch.zeros_like(st["q"])
    out[row] = o.to(out.dtype)
    return out


def _plain_copy(st):
    src, dst = st["map"].unbind(1)
    st["kp"][dst], st["vp"][dst] = st["kp"][src], st["vp"][src]
    st["ks"][dst], st["vs"][dst] = st["ks"][src], st["vs"][src]
    return dict(k=st["kp"].view(F8), v=st["vp"].view(F8), ks=st["ks"], vs=st["vs"])


# --------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return {"rope": _plain_rope, "rope_q8": _plain_rope_q8, "decode_q8": _plain_decode,
                "prefill_q8": _plain_prefill, "copy_q8": _plain_copy}[op](st)
    from paged_kv_cache_455_b200 import pa
    if op == "rope":
        pa.pa_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["kp"], st["vp"],
                             st["slots"], st["pos"], st["table"], c["interleaved"], st["status"])
        return dict(q=st["q_out"], k=st["kp"], v=st["vp"])
    if op == "rope_q8":
        pa.pa_rope_and_cache_q8(st["q_out"], st["q"], st["k"], st["v"], st["kp"], st["vp"],
                                st["ks"], st["vs"], st["cu"], st["max_q"], st["tables"],
                                st["lens"], st["pos"], st["table"], c["interleaved"],
                                st["status"])
        return dict(q=st["q_out"], k=st["kp"].view(F8), v=st["vp"].view(F8), ks=st["ks"],
                    vs=st["vs"])
    if op == "decode_q8":
        if "ws" not in st:      # allocated once, as a serving loop does
            st["ws"] = torch.empty(
                pa.pa_decode_workspace_bytes(st["q"].shape[0], c["hq"], c["hkv"], c["d"],
                                             st["max_ctx"]), dtype=torch.uint8, device=DEV)
        pa.pa_decode_attention_q8(st["out"], st["q"], st["kp"], st["vp"], st["ks"], st["vs"],
                                  st["tables"], st["lens"], st["max_ctx"], st["scale"], st["ws"],
                                  st["status"])
        return st["out"]
    if op == "prefill_q8":
        pa.pa_prefill_attention_q8(st["out"], st["q"], st["cu"], st["max_q"], st["kp"], st["vp"],
                                   st["ks"], st["vs"], st["tables"], st["lens"], st["max_ctx"],
                                   st["scale"], st["status"])
        return st["out"]
    pa.pa_copy_blocks_q8(st["kp"], st["vp"], st["ks"], st["vs"], st["kp"], st["vp"], st["ks"],
                         st["vs"], st["map"], st["status"])
    return dict(k=st["kp"].view(F8), v=st["vp"].view(F8), ks=st["ks"], vs=st["vs"])


# ---------------------------------------------------- what a pass cannot avoid
def work(case):
    op, hkv, d, bs = case["op"], case["hkv"], case["d"], case["bs"]
    if op == "copy_q8":
        return dict(bytes=case["pairs"] * (4 * bs * hkv * d + 4 * hkv * 4 + 16), flops=0)
    lens, hq = _lengths(case), case["hq"]
    rows = sum(n for n, _ in lens)
    if op in ("rope", "rope_q8"):
        es = 4 if case.get("dtype") == "f32" else 2
        # q, k and v read, q written; a row of the table, a position and a slot
        # for each token; k and v written in the cache's type
        n = rows * ((2 * hq + 2 * hkv) * d * es + case["rot"] * 4 + 16)
        n += rows * 2 * hkv * d * (es if op == "rope" else 1)
        if op == "rope_q8":
            n += sum((x - 1) // bs - (x - m) // bs + 1 for m, x in lens) * (2 * hkv * 8 + 4)
        return dict(bytes=n, flops=rows * (hq + hkv) * case["rot"] * 3)
    # the cache and its scales once, a table entry per block; q and out
    n = sum(x * 2 * hkv * d + -(-x // bs) * (2 * hkv * 4 + 4) for _, x in lens)
    n += 2 * (rows + case.get("empty", 0)) * hq * d * 2
    seen = sum(m * x - m * (m - 1) // 2 for m, x in lens)
    return dict(bytes=n, flops=4 * seen * hq * d)


# ------------------------------------------------- the definitions, in 64 bits
def _e4m3(x):
    """The E4M3 value nearest to x (ties to even), within +-448."""
    x = x.clamp(-448, 448)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_rotation(x, pos, table, rot, interleaved):
    y = x.double().clone()
    ang = table[pos].double()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = ang[:, i, None], ang[:, rot // 2 + i, None]
        y[..., a], y[..., b] = (x[..., a].double() * c - x[..., b].double() * s,
                                x[..., a].double() * s + x[..., b].double() * c)
    return y


def _exact_scale(amax):
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448))
    # log2 may be one rounding off at a power of two: settle it by comparison
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(SCALE_MIN, SCALE_MAX))


def exact(case, seed):
    if case["op"] in ("decode_q8", "prefill_q8") and case["seqs"] > 320:
        return None
    st = prepare(case, seed)
    op, hkv, d, bs = case["op"], case["hkv"], case["d"], case["bs"]
    if op in ("rope", "rope_q8"):
        args = (st["pos"], st["table"], case["rot"], case["interleaved"])
        q, k = _exact_rotation(st["q"], *args), _exact_rotation(st["k"], *args)
        v = st["v"].double()
        if op == "rope":
            kp, vp = st["kp"].double(), st["vp"].double()
            for pool, x in ((kp, k), (vp, v)):
                rows = pool.view(-1, hkv, d)
                at = st["slots"]
                rows.index_copy_(0, at[at >= 0], x[at >= 0])
            return dict(q=q, k=kp, v=vp)
        cu, lens = st["cu"].tolist(), st["lens"].tolist()
        q[cu[-1]:] = 0
        kp, vp = st["kp"].view(F8).double(), st["vp"].view(F8).double()
        ks, vs = st["ks"].double(), st["vs"].double()
        for b in range(case["seqs"]):
            n = cu[b + 1] - cu[b]
            start = lens[b] - n
            b0, b1 = start // bs, (lens[b] - 1) // bs + 1
            ids = st["tables"][b, b0:b1].long()
            lead, tail = start - b0 * bs, b1 * bs - lens[b]
            for pool, scales, x in ((kp, ks, k), (vp, vs, v)):
                new = x[cu[b]:cu[b + 1]]
                grid = torch.cat([new.new_zeros(lead, hkv, d), new, new.new_zeros(tail, hkv, d)])
                grid = grid.view(b1 - b0, bs, hkv, d)
                s = _exact_scale(grid.abs().amax(dim=(1, 3)))
                held = pool[ids]
                if lead:
                    s[0] = torch.maximum(s[0], scales[ids[0]])
                    held[0, :lead] = _e4m3(held[0, :lead] * (scales[ids[0]] / s[0])[:, None])
                codes = _e4m3(grid / s[:, None, :, None]).view(-1, hkv, d)
                flat = held.view(-1, hkv, d)
                flat[lead:lead + n] = codes[lead:lead + n]
                pool[ids], scales[ids] = held, s
        return dict(q=q, k=kp, v=vp, ks=ks, vs=vs)
    if op == "copy_q8":
        got = dict(k=st["kp"].view(F8).double(), v=st["vp"].view(F8).double(),
                   ks=st["ks"].double(), vs=st["vs"].double())
        src, dst = st["map"][:, 0], st["map"][:, 1]
        return {n: x.index_copy(0, dst, x[src]) for n, x in got.items()}
    G = case["hq"] // hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    cu = st["cu"].tolist() if op == "prefill_q8" else list(range(st["q"].shape[0] + 1))
    for b, L in enumerate(st["lens"].tolist()):
        if L == 0:
            continue
        ids = st["tables"][b, :(L + bs - 1) // bs].long()
        K = (st["kp"][ids].view(F8).double() * st["ks"][ids].double()[:, None, :, None])
        V = (st["vp"][ids].view(F8).double() * st["vs"][ids].double()[:, None, :, None])
        K, V = K.flatten(0, 1)[:L], V.flatten(0, 1)[:L]
        q = st["q"][cu[b]:cu[b + 1]].double()
        n = q.shape[0]
        later = (torch.arange(L, device=DEV)[None, :] >
                 torch.arange(L - n, L, device=DEV)[:, None])
        for h in range(hkv):
            for g in range(G):
                s = (q[:, h * G + g] @ K[:, h].T) * st["scale"]
                w = torch.softmax(s.masked_fill(later, -math.inf), dim=-1)
                out[cu[b]:cu[b + 1], h * G + g] = w @ V[:, h]
    return out
