"""Layers of the 8-bit (and bf16) store with known tokens, and their comparison with tests/plain64.py."""
import numpy as np
import torch

import block_sparse_offloadable_b200 as nosa
from tests import plain64 as P

D, BLOCK = 128, 64


class Tokens:
    """Seeded keys, values (bf16 bits [units][n][128]), logits and queries of a batch."""

    def __init__(self, B, Hq, Hkv, n, seed, k_scale=1.0, v_scale=1.0):
        r = np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.G, self.units = B, Hq, Hkv, Hq // Hkv, B * Hkv
        chan = np.where(r.random((self.units, 1, D)) < 0.05, 5.0, 1.0)
        self.k = P.to_bf16_bits(r.standard_normal((self.units, n, D)) * chan * k_scale)
        self.v = P.to_bf16_bits(r.standard_normal((self.units, n, D)) * v_scale)
        self.e = (0.5 * r.standard_normal((self.units, n))).astype(np.float32)
        self.r = r

    def q(self, scale=1.0):
        return P.to_bf16_bits(self.r.standard_normal((self.B, self.Hq, D)) * scale)

    def unit(self, u, L, fmt, scale=D ** -0.5):
        return P.Unit(P.bf16(self.k[u, :L]), P.bf16(self.v[u, :L]), self.e[u, :L].astype(np.float64), fmt, self.G,
                      float(np.float32(scale)))

    def prefill(self, lay, T, lens=None):
        """The first T tokens (lens[b] of sequence b) into the empty layer."""
        if T < 1:
            return
        if T == 1 and lens is None:
            self.append(lay, np.zeros(self.units, int))
            return
        lay.append(dev16(self.k[:, :T]), dev16(self.v[:, :T]), dev32(self.e[:, :T]), T,
                   None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))

    def new(self, at):
        """The token at position at[u] of every unit: k, v, e on the device."""
        u = np.arange(self.units)
        return dev16(self.k[u, at][:, None]), dev16(self.v[u, at][:, None]), dev32(self.e[u, at][:, None])

    def append(self, lay, at):
        lay.append(*self.new(at), 1)


def dev16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def dev32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def layer(t, max_ctx, fmt, k_q=4, k_e=12, weights=False, **kw):
    return nosa.NosaLayer(nosa.make_config(t.B, t.Hq, t.Hkv, k_q, k_e, max_ctx, kv_format=fmt, **kw), weights=weights)


def out_of(out):
    return P.bf16(out.cpu().numpy())


def check_out(t, out, q, units, blocks):
    """out [B][Hq][128] against the plain form of each unit over blocks[u]."""
    got = out_of(out).reshape(t.units, t.G, D)
    qq = P.bf16(q).reshape(t.units, t.G, D)
    for u, ref in enumerate(units):
        want, tol = ref.attend(qq[u], blocks[u])[:2]
        assert np.array_equal(np.isnan(got[u]), np.isnan(want)), u
        bad = np.abs(got[u] - want) > tol
        assert not bad[~np.isnan(want)].any(), (u, np.abs(got[u] - want)[bad].max(), tol[bad].min())


def check_store(lay, t, units, fmt):
    """Codes, scales and tails of a device-store layer against the plain form, bit for bit."""
    codes, scales, tail = (x.cpu() for x in lay.kv8_views())
    for u, ref in enumerate(units):
        for b in ref.codes:
            assert np.array_equal(codes[u, b].float().numpy().astype(np.float64), ref.codes[b]), (u, b)
            got = scales[u, b].numpy()
            assert np.array_equal(got, ref.scales[b], equal_nan=True), (u, b, got, ref.scales[b])
        if ref.local >= 0:
            n = ref.L - ref.local * BLOCK
            rows = slice(ref.local * BLOCK, ref.L)
            assert np.array_equal(tail[u, 0, :n].view(torch.int16).numpy().view(np.uint16), t.k[u, rows])
            assert np.array_equal(tail[u, 1, :n].view(torch.int16).numpy().view(np.uint16), t.v[u, rows])


def sels(lay):
    s, n = lay.sel.cpu().numpy(), lay.nsel.cpu().numpy()
    return [list(s[u, :n[u]]) for u in range(len(n))]
