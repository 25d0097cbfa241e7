"""fp64 attention over a block-scaled cache with the error bound of the
kernels' arithmetic, for the GPU tests.

What the kernels round, for a query row and a head with softmax weights p_t,
logits s_t and values V_t (everything else is fp32 or exact):

  query     scaled to a largest element in [128, 256) and split into two E4M3
            parts of 4 bits: exact down to the subnormal quantum 2^-9, so each
            element is off by at most 2^-10, that is 2^-17 of the row's
            largest, and s_t by d_t = |scale| 2^-17 max|q| sum_i |K_ti|.
            Numerator and sum move by at most that share: 2 max_t d_t in all.
  weights   x_t = p_t vs_t, scaled.  Decode: three E5M2 parts of 3 bits, half a
            step each, 2^-9 of x_t, or half the quantum 2^-16 of the last part,
            which counts 2^-6: 2^-23, where the largest x_t is at least 1.
            Prefill: hi of 4 bits (half a step 2^-4, or half the quantum 2^-9),
            lo the rest with 3 bits (half a step 2^-3): 2^-7 of x_t or 2^-13,
            where the largest x_t is at least 1.
  output    bf16, half a step: 2^-8 of it.

fp32 accumulation and the exponential add less than 2^-12 of sum p |V|.
"""
import numpy as np

from oracle import oracle as O

EXTRA = 2.0 ** -12


def attention_with_bound(q, kp, vp, ks, vs, tab, lens, cu, scale, prefill):
    """(reference, bound), both [rows, Hq, d] float64.  q: raw bf16 rows; row
    j of sequence b sits at position lens[b] - n_b + j (decode: n_b = 1)."""
    qf = O.to_f64(q, "bf16")
    hq, d = qf.shape[1:]
    bs, hkv = kp.shape[1:3]
    G = hq // hkv
    ref = np.zeros(qf.shape)
    tol = np.zeros(qf.shape)
    for b in range(len(lens)):
        L, q0, n = int(lens[b]), int(cu[b]), int(cu[b + 1] - cu[b])
        if L == 0 or n == 0:
            continue
        ids = tab[b, :-(-L // bs)].astype(np.int64)
        K = O.dequantize_q8(kp[ids], ks[ids]).reshape(-1, hkv, d)[:L]
        V = O.dequantize_q8(vp[ids], vs[ids]).reshape(-1, hkv, d)[:L]
        sc = np.repeat(vs[ids].astype(np.float64), bs, axis=0)[:L]
        seen = np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]
        for h in range(hq):
            g = h // G
            rows = qf[q0:q0 + n, h]
            s = np.where(seen, scale * (rows @ K[:, g].T), -np.inf)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            ref[q0:q0 + n, h] = p @ V[:, g]
            dt = abs(scale) * 2.0 ** -17 * np.abs(rows).max(axis=1)[:, None] * \
                np.abs(K[:, g]).sum(axis=1)[None, :]
            shift = 2 * np.where(seen, dt, 0).max(axis=1, keepdims=True)
            x = p * sc[None, :, g]
            rel, least = (2.0 ** -7, 2.0 ** -13) if prefill else (2.0 ** -9, 2.0 ** -23)
            off = least * x.max(axis=1, keepdims=True) / sc[None, :, g]
            w = p * (rel + shift + EXTRA) + np.where(seen, off, 0)
            tol[q0:q0 + n, h] = w @ np.abs(V[:, g])
    return ref, tol + 2.0 ** -8 * np.abs(ref)
