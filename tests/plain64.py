"""Plain 64-bit forms of the 8-bit store, the attention over it, block weights and eviction, in numpy.

One unit at a time; nothing here shares code with the library.
"""
import numpy as np

D, BLOCK, SUB = 128, 64, 16
TOP = {"int8": 127, "e4m3": 448}


def bf16(bits):
    """bf16 bit patterns as float64 (exact)."""
    return (np.ascontiguousarray(bits).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16_bits(x):
    """Nearest bf16 (ties to even) of finite float32 values, infinities kept."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def e4m3(y):
    """Nearest e4m3 value (ties to even, saturating) of float64 y."""
    with np.errstate(divide="ignore"):
        ex = np.floor(np.log2(np.abs(y)))
    step = np.exp2(np.maximum(ex, -6) - 3)
    return np.clip(np.rint(y / step) * step, -448, 448)


def code_half(x, fmt):
    """x [64][128] float64 (bf16 values): (codes' values, scale) of a block's keys or values."""
    a = np.float32(np.abs(x).max())
    if not np.isfinite(a):
        return np.zeros_like(x), np.float32(np.nan)
    if a < np.float32(2.0 ** -100):
        return np.zeros_like(x), np.float32(0)
    top = np.float32(TOP[fmt])
    s = a * (np.float32(1) / top)
    r = (np.float32(1) / a) * top
    if fmt == "int8":
        return np.rint(x * np.float64(r)), s  # 8 + 24 bits: the product is exact
    return e4m3((x * np.float64(r)).astype(np.float32).astype(np.float64)), s


class Unit:
    """A unit's tokens: k, v float64 [L][128] (bf16 values), e float64 [L]; what its store stands for."""

    def __init__(self, k, v, e, fmt, G, scale):
        self.L, self.fmt, self.G, self.scale = len(k), fmt, G, scale
        self.local = (self.L - 1) // BLOCK if self.L else -1
        self.e = e
        self.codes, self.scales = {}, {}
        self.k, self.v = k.copy(), v.copy()
        if fmt != "bf16":
            for b in range(max(self.local, 0)):
                rows = slice(b * BLOCK, (b + 1) * BLOCK)
                ck, sk = code_half(k[rows], fmt)
                cv, sv = code_half(v[rows], fmt)
                self.codes[b], self.scales[b] = np.stack([ck, cv]), np.array([sk, sv], np.float32)
                self.k[rows], self.v[rows] = ck * np.float64(sk), cv * np.float64(sv)

    def attend(self, q, blocks):
        """q float64 [G][128]: (out [G][128], its tolerance, weight per block, its tolerance)."""
        blocks = [b for b in blocks if 0 <= b <= self.local]
        rows = np.concatenate([np.arange(b * BLOCK, min((b + 1) * BLOCK, self.L)) for b in blocks]) if blocks else np.zeros(0, int)
        if not len(rows):
            z = np.zeros((self.G, D))
            return z, z, np.zeros(0), np.zeros(0)
        k, v, e = self.k[rows], self.v[rows], self.e[rows]
        with np.errstate(invalid="ignore", over="ignore"):
            z = q @ k.T * self.scale + e[None]
            m = z.max(1, keepdims=True)
            p = np.exp(z - np.where(m == -np.inf, 0, m))
            tot = p.sum(1, keepdims=True)
            p = np.where(tot == 0, 0, p / np.where(tot == 0, 1, tot))
            out = p @ v
        # Tolerance.  A logit is a sum of 128 products in 32 bits (at most 8 + 2 additions of matrix
        # instructions, each off by at most a step 2^-23 of what it has summed, two more roundings, the
        # logit's own and the reference maximum's): dz <= 2^-23 * 14 * (sum |q k| scale + |e|) <= 2^-19 of it.
        # P is rounded to f16 (2^-11 of it) over codes and to bf16 (2^-8) over bf16 rows, in the numerator
        # and in the denominator; the output to bf16 (2^-8).  exp2 and the final sums: 2^-20.  Over int8
        # codes P is a multiple of 1/65535 of the block's largest weight: off by at most half of that,
        # 2^-17 of the largest, for each of the block's tokens, whatever the token's own weight.
        fin = np.isfinite(e)
        mag = np.abs(q) @ np.abs(k).T * self.scale + np.where(fin, np.abs(np.where(fin, e, 0)), 0)[None]
        seen = p > 0
        dz = 2.0 ** -19 * np.where(seen, mag, 0).max(1, keepdims=True)
        half = np.ones(len(rows), bool) if self.fmt == "bf16" else rows >= self.local * BLOCK
        dp = 2.0 ** -8 * (p * half).sum(1, keepdims=True) + 2.0 ** -11 * (p * ~half).sum(1, keepdims=True)
        tol = 2.0 ** -8 * np.abs(out) + 2 * (dp + dz + 2.0 ** -20) * (p @ np.abs(v)) + 1e-38
        at = np.searchsorted(blocks, rows // BLOCK)
        if self.fmt == "int8":
            top = np.zeros((self.G, len(blocks)))
            np.maximum.at(top.T, at, np.where(half, 0, p).T)
            tol += 2.0 ** -17 * top[:, at] @ np.abs(v)
        w, wt = np.zeros(len(blocks)), np.zeros(len(blocks))
        np.add.at(w, at, p.sum(0))
        np.add.at(wt, at, (p * (2 * dz + 2.0 ** -18)).sum(0))  # log2, exp2 and sums beside the logits' error
        return out, tol, w, wt


def keep_blocks(weights, nb, keep, sink, recent):
    """Candidates of a unit that eviction keeps, ascending."""
    def rank(b):
        if b < sink or b >= nb - recent:
            return (0, 0.0, b)
        w = float(weights[b])
        return (1, 0.0, b) if np.isnan(w) else (2, -w, b)
    return sorted(sorted(range(nb), key=rank)[:keep])
