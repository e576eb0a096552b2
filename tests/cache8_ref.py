"""A plain 64-bit model of the 8-bit paged cache (include/kvc.h, "8-bit paged cache"): numpy and
loops, from the definitions, sharing no code with the library. Test infrastructure only."""
from __future__ import annotations

import numpy as np

E4M3, INT8 = "e4m3", "int8"
TOP = {E4M3: 448.0, INT8: 127.0}
BAD_INDEX, EXHAUSTED, NONFINITE = 0x2, 0x4, 0x8


def e4m3_value(code: int) -> float:
    """sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0 is subnormal; 0x7f is NaN."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


E4M3_VALUES = np.array([e4m3_value(c) for c in range(256)])
_UP = E4M3_VALUES[:127]                      # 0 .. 448, ascending
_MID = (_UP[1:] + _UP[:-1]) / 2


def decode(codes, fmt):
    codes = np.asarray(codes, np.uint8)
    return E4M3_VALUES[codes] if fmt == E4M3 else codes.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """Nearest code of x (in units of the scale), ties to even; NaN is 0, too large the largest."""
    x = np.where(np.isnan(x), 0.0, x)
    if fmt == INT8:
        return np.clip(np.rint(np.clip(x, -200, 200)), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    lo = np.searchsorted(_MID, a, side="left")      # number of midpoints below a
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def scale_of(x, fmt):
    """Smallest power of two (2^-64 .. 2^64) with max finite |x| / scale <= TOP."""
    a = np.abs(x[np.isfinite(x)]).max(initial=0.0)
    e = -64
    while e < 64 and a > TOP[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


class RefCache:
    """kvc_cache8 with numpy arrays; methods mirror the entry points and return status bits."""

    def __init__(self, L, B, H, d, n_blocks, bs, max_blocks, fmt):
        self.L, self.B, self.H, self.d, self.bs, self.M, self.N = L, B, H, d, bs, max_blocks, n_blocks
        self.fmt = fmt
        self.pool = [np.zeros((L, n_blocks, H, bs, d), np.uint8) for _ in "kv"]
        self.scale = [np.ones((L, n_blocks, H), np.float32) for _ in "kv"]
        self.table = np.full((B, max_blocks), -1, np.int32)
        self.len = np.zeros(B, np.int32)
        self.free_list = np.arange(n_blocks, dtype=np.int32)
        self.top = n_blocks
        self.ref = np.zeros(n_blocks, np.int32)

    def sibling(self, B=None):
        """Other sequences on the same pools and stack (shared arrays)."""
        o = object.__new__(RefCache)
        o.__dict__.update(self.__dict__)
        o.table = np.full_like(self.table, -1)
        o.len = np.zeros_like(self.len)
        return o

    def blocks(self, n):
        return -(-int(n) // self.bs)

    # -- pages --
    def grow(self, n_new):
        need = []
        for b, n in enumerate(n_new):
            n, m = int(n), int(self.len[b])
            if n < 0 or m < 0 or m + n > self.M * self.bs:
                return BAD_INDEX
            if n and m % self.bs and self.ref[self.table[b, m // self.bs]] != 1:
                return BAD_INDEX
            need.append(self.blocks(m + n) - self.blocks(m))
        S = sum(need)
        if S > self.top:
            return EXHAUSTED
        at = self.top - S
        if any(not 0 <= x < self.N or self.ref[x] for x in self.free_list[at:self.top]):
            return BAD_INDEX
        self.top = at
        for b, k in enumerate(need):
            have = self.blocks(self.len[b])
            for i in range(k):
                blk = self.free_list[at]
                self.table[b, have + i] = blk
                self.ref[blk] = 1
                at += 1
            self.len[b] += n_new[b]
        return 0

    def free(self, seqs):
        seqs = [int(s) for s in seqs]
        if len(set(seqs)) < len(seqs) or any(not 0 <= s < self.B for s in seqs):
            return BAD_INDEX
        held = [(s, self.table[s, i]) for s in seqs for i in range(self.blocks(self.len[s]))]
        if any(not 0 <= x < self.N for _, x in held):
            return BAD_INDEX
        times = {}
        for _, x in held:
            times[x] = times.get(x, 0) + 1
        if any(self.ref[x] < k for x, k in times.items()):
            return BAD_INDEX
        gone = {x for x, k in times.items() if self.ref[x] == k}
        if self.top + len(gone) > self.N:
            return BAD_INDEX
        for s, x in held:
            self.ref[x] -= 1
            if self.ref[x] == 0:
                self.free_list[self.top] = x
                self.top += 1
        for s in seqs:
            self.table[s, :self.blocks(self.len[s])] = -1
            self.len[s] = 0
        return 0

    def fork(self, src, dst):
        src, dst = [int(s) for s in src], [int(s) for s in dst]
        if any(not 0 <= s < self.B for s in src + dst) or len(set(dst)) < len(dst):
            return BAD_INDEX
        if set(src) & set(dst) or any(self.len[x] for x in dst):
            return BAD_INDEX
        for s in src:
            for x in self.table[s, :self.blocks(self.len[s])]:
                if not 0 <= x < self.N or self.ref[x] < 1:
                    return BAD_INDEX
        started = [s for s in src if self.len[s] % self.bs]
        if len(started) > self.top:
            return EXHAUSTED
        taken = self.free_list[self.top - len(started):self.top]
        if any(not 0 <= x < self.N or self.ref[x] for x in taken):
            return BAD_INDEX
        at = self.top = self.top - len(started)
        for s, x in zip(src, dst):
            full, part = divmod(int(self.len[s]), self.bs)
            for i in range(full):
                self.table[x, i] = self.table[s, i]
                self.ref[self.table[s, i]] += 1
            if part:
                old, new = self.table[s, full], self.free_list[at]
                at += 1
                self.table[x, full] = new
                self.ref[new] = 1
                for p, sc in zip(self.pool, self.scale):
                    p[:, new, :, :part] = p[:, old, :, :part]
                    sc[:, new] = sc[:, old]
            self.len[x] = self.len[s]
        return 0

    # -- rows --
    def append(self, k, v, n_new):
        """k, v [L, B, H, n, d] float64 (bf16 values)."""
        status = 0
        for b, n in enumerate(n_new):
            n = int(n)
            if n < 0 or n > k.shape[3] or n > self.len[b]:
                status |= BAD_INDEX
                continue
            start, end = int(self.len[b]) - n, int(self.len[b])
            for i in range(start // self.bs, self.blocks(end) if n else 0):
                lo, hi = max(i * self.bs, start), min(end, (i + 1) * self.bs)
                blk = self.table[b, i]
                if not 0 <= blk < self.N or self.ref[blk] != 1:
                    status |= BAD_INDEX
                    continue
                for l in range(self.L):
                    for h in range(self.H):
                        for x, p, sc in zip((k, v), self.pool, self.scale):
                            x = x[l, b, h, lo - start:hi - start]
                            if not np.isfinite(x).all():
                                status |= NONFINITE
                            s = scale_of(x, self.fmt)
                            r = lo - i * self.bs
                            if r:
                                old = float(sc[l, blk, h])
                                s = max(s, old)
                                p[l, blk, h, :r] = encode(decode(p[l, blk, h, :r], self.fmt) * (old / s),
                                                          self.fmt)
                            p[l, blk, h, r:hi - i * self.bs] = encode(x / s, self.fmt)
                            sc[l, blk, h] = s
        return status

    def rows(self, which, l, b, h, upto=None):
        """The values [len, d] that one sequence's head holds."""
        n = int(self.len[b]) if upto is None else upto
        out = np.zeros((n, self.d))
        for t in range(n):
            blk = self.table[b, t // self.bs]
            out[t] = decode(self.pool[which][l, blk, h, t % self.bs], self.fmt) * float(
                self.scale[which][l, blk, h])
        return out

    def gather(self, T):
        got = [np.zeros((self.L, self.B, self.H, T, self.d)) for _ in "kv"]
        pad = np.full(self.B, T, np.int32)
        status = 0
        for b in range(self.B):
            n = int(self.len[b])
            if n > T:
                status |= BAD_INDEX
                continue
            pad[b] = T - n
            for w in (0, 1):
                for l in range(self.L):
                    for h in range(self.H):
                        got[w][l, b, h, T - n:] = self.rows(w, l, b, h)
        return got[0], got[1], pad, status

    def compact(self, dst, pad, kept, n_kept):
        """kept [L, B, H, K], n_kept [L, B, H]; dst is grown."""
        status = 0
        for l in range(self.L):
            for b in range(self.B):
                for h in range(self.H):
                    nk = int(n_kept[l, b, h])
                    if nk != dst.len[b] or not 0 <= nk <= kept.shape[3]:
                        status |= BAD_INDEX
                        continue
                    for w in (0, 1):
                        src = self.rows(w, l, b, h)
                        x = np.zeros((nk, self.d))
                        for j in range(nk):
                            t = int(kept[l, b, h, j]) - int(pad[b])
                            if kept[l, b, h, j] >= 0 and 0 <= t < len(src):
                                x[j] = src[t]
                            else:
                                status |= BAD_INDEX
                        for i in range(dst.blocks(nk)):
                            r = x[i * dst.bs:(i + 1) * dst.bs]
                            s = scale_of(r, dst.fmt)
                            blk = dst.table[b, i]
                            if not 0 <= blk < dst.N or dst.ref[blk] != 1:
                                status |= BAD_INDEX
                                continue
                            dst.pool[w][l, blk, h, :len(r)] = encode(r / s, dst.fmt)
                            dst.scale[w][l, blk, h] = s
        return status

    # -- attention --
    def attend(self, q, scale, n_q=None):
        """q [L, B, Hq, n, d] float64 -> out, lse, and the bounds that the tests use: |out - exact|
        and |lse - exact| of a kernel that keeps its promises (tolerances())."""
        L, B, Hq, n, d = q.shape
        G = Hq // self.H
        out, lse = np.zeros(q.shape), np.full(q.shape[:4], -np.inf)
        tol, ltol = np.zeros(q.shape), np.zeros(q.shape[:4])
        for l in range(L):
            for b in range(B):
                m = int(self.len[b])
                nq = n if n_q is None else int(n_q[b])
                for h in range(self.H):
                    k, v = self.rows(0, l, b, h), self.rows(1, l, b, h)
                    vs = np.array([self.scale[1][l, self.table[b, t // self.bs], h] for t in range(m)],
                                  np.float64)
                    for g in range(h * G, (h + 1) * G):
                        for j in range(nq):
                            end = m - nq + j + 1
                            if end <= 0:
                                continue
                            z = k[:end] @ q[l, b, g, j] * scale
                            top = z.max()
                            e = np.exp(z - top)
                            p = e / e.sum()
                            out[l, b, g, j] = p @ v[:end]
                            lse[l, b, g, j] = top + np.log(e.sum())
                            zabs = (np.abs(k[:end]) @ np.abs(q[l, b, g, j])).max() * scale
                            qabs = np.abs(q[l, b, g, j]).max() * np.abs(k[:end]).sum(1).max() * scale
                            tol[l, b, g, j], ltol[l, b, g, j] = tolerances(
                                out[l, b, g, j], p @ np.abs(v[:end]),
                                (p * vs[:end]).max() * (np.abs(v[:end]) / vs[:end, None]).sum(0),
                                lse[l, b, g, j], zabs, qabs, end, d)
        return out, lse, tol, ltol


def tolerances(out, weight, least, lse, zabs, qabs, T, d):
    """What fp32 accumulation and rounded operands can be off by.

    A score's error dz: d products and additions, the scaling and the exponential's argument in fp32,
    each half a step (2^-24) of a sum of at most zabs; q is a bf16 value held exactly, or to 2^-25 of its
    row's largest where 11 significant bits do not reach (qabs = largest |q| times the sum of |k|); the
    exponential itself 2^-21.  A softmax weight is then off by 2 dz (its own and the sum's) and its
    rounding to 11 bits (2^-11); sums over T tokens by T 2^-24, the joining of parts by 2^-20.  The
    result is rounded to bf16, half a step: 2^-8 of it.
    Weights are rounded in fp16, whose steps end at 2^-24: with the largest weight times scale taken as
    1 or more, a smaller one is off by up to 2^-25 of that, times its token's codes; `least` is the
    largest weight times scale, times the sum of the codes' magnitudes.  (A column of values that is
    zero wherever the softmax has weight showed that this term was missing: its result, 2e-8 of the
    other columns', comes from weights below fp16's last step.)"""
    dz = (d + 8) * 2.0 ** -24 * zabs + 2.0 ** -25 * qabs + 2.0 ** -21
    err = weight * (2 * dz + 2.0 ** -11 + T * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -25 * least
    return (err + 2.0 ** -8 * (np.abs(out) + err) + 1e-30,
            dz + T * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * abs(lse))
