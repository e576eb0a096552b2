"""Attention over the 8-bit paged cache in 64 bits, with an error bound that belongs to each token:
a token's score is off by what its own key and the query allow, weighted by its softmax weight, so
that a few large keys do not widen what is admitted for the others.  Test infrastructure only; works on
the model cache of tests/cache8_ref.py."""
import numpy as np

LN2, LOG2E = np.log(2.0), 1 / np.log(2.0)


def attend(ref, q, scale, n_q=None, absent=None):
    """q [L, B, Hq, n, d] float64 -> out, lse, and bounds on |out - exact| and |lse - exact|.

    absent [B, tokens] (or None): tokens that do not count, at positions that still do.

    A token's logit in base 2 with its value scale 2^e is x = log2(e) scale q.k + e; the weights are
    2^(x - M) for a reference M that is at most the largest x and at most 2^15 below it.
      dz, the error of a logit in natural units:
        d products (exact in fp32) summed in fp32, and the scaling: (d + 8) steps of sum |q k|, whole
        ones (2^-23), since a tensor core may truncate;
        q is held to 11 significant bits or to 2^-25 of its row's largest: 2^-25 |q|max sum |k|;
        x and x - M, each rounded in fp32, and M's own roundings: 2^-23 of |e| + |x| + |x|max + 32;
        the exponential's own error: 2^-21.
      A weight is off by e^dz - 1 and its rounding to 11 bits (2^-11), and, where fp16's steps end
      (2^-24), by 2^-25 of the largest weight times scale, times the code.
      The sums over T tokens are fp32 (T 2^-23), parts are joined (2^-20).
      The denominator's weights are fp32.  The output is rounded to bf16, half a step: 2^-8.
      lse = (M + log2 sum) ln 2: the denominator's error, and fp32's of |x|max, the sum's logarithm
      (at most 64 + 32 beyond) and the result."""
    L, B, Hq, n, d = q.shape
    G = Hq // ref.H
    out, lse = np.zeros(q.shape), np.full(q.shape[:4], -np.inf)
    tol, ltol = np.zeros(q.shape), np.zeros(q.shape[:4])
    for l in range(L):
        for b in range(B):
            m = int(ref.len[b])
            nq = n if n_q is None else int(n_q[b])
            there = np.ones(m, bool) if absent is None else ~absent[b, :m]
            if nq == 0 or not there.any():
                continue
            pos = np.flatnonzero(there)
            for h in range(ref.H):
                k, v, vs = _rows(ref, l, b, h, pos)
                e = np.log2(vs)
                for g in range(h * G, (h + 1) * G):
                    for j in range(nq):
                        see = int(np.searchsorted(pos, m - nq + j, side="right"))
                        if see == 0:
                            continue
                        at = l, b, g, j
                        out[at], lse[at], tol[at], ltol[at] = _row(q[at], k[:see], v[:see], vs[:see],
                                                                   e[:see], scale)
    return out, lse, tol, ltol


def _rows(ref, l, b, h, pos):
    blk = ref.table[b, pos // ref.bs]
    from tests.cache8_ref import decode
    got = []
    for w in (0, 1):
        s = ref.scale[w][l, blk, h].astype(np.float64)
        got += [decode(ref.pool[w][l, blk, h, pos % ref.bs], ref.fmt) * s[:, None], s]
    return got[0], got[2], got[3]


def _row(q, k, v, vs, e, scale):
    T, d = k.shape
    z = k @ q * scale
    top = z.max()
    w = np.exp(z - top)
    p = w / w.sum()
    out, lse = p @ v, top + np.log(w.sum())
    x = z * LOG2E + e
    xmax = x.max()
    dz = (2.0 ** -23 * (d + 8) * scale * (np.abs(k) @ np.abs(q)) +
          2.0 ** -25 * scale * np.abs(q).max() * np.abs(k).sum(1) +
          2.0 ** -23 * LN2 * (np.abs(e) + np.abs(x) + abs(xmax) + 32) + 2.0 ** -21)
    de = np.expm1(np.minimum(dz, 50.0))
    sums = T * 2.0 ** -23 + 2.0 ** -20
    low = p @ de + sums
    num = (p * (de + 2.0 ** -11 * (1 + de) + sums)) @ np.abs(v) + \
        2.0 ** -25 * (p * vs).max() * (np.abs(v) / vs[:, None]).sum(0)
    err = (num + low * np.abs(out)) * (1 + 2 * min(low, 1.0))
    return (out, lse, err + 2.0 ** -8 * (np.abs(out) + err) + 1e-30,
            low * (1 + low) + 2.0 ** -23 * LN2 * (abs(xmax) + 96) + 2.0 ** -23 * abs(lse))
