"""Logits that are large or not finite: common offsets, masks by the lowest finite value, NaN.

Every unit's block weights have to add up to its number of query heads, and `out` and the weights have to
be of the same softmax, whatever lies on all of its logits.
"""
import numpy as np
import pytest
import torch

from tests import kv8_harness as H
from tests import plain64 as P
from tests.test_gpu_weights import check_weights

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "int8", "e4m3"]
LOWEST = np.finfo(np.float32).min

# How far a unit's weights may be from adding up to its number of heads, relative to it.  A block's weight is
# 2^(v - M) / l with v the log2 of its sum.  With q = 0, |v| relative to the block's largest logit is below 8: half a
# step is 2^-22; log2, exp2, the 64 terms of the sum and 1 / l take 2^-22 each, the running sum l (up to 15 additions
# of a warp, 13 states) 2^-20: below 2^-18.  With other queries |v| < 84, half a step 2^-18, ln 2 of it: below 2^-17.
ZERO_Q, ANY_Q = 2.0 ** -18, 2.0 ** -17


def offset_tokens(B, Hq, Hkv, L, offset, seed):
    t = H.Tokens(B, Hq, Hkv, L, seed=seed)
    t.e[:] = offset
    return t


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offset", [-1e4, -1e5, -1e6, -1e7, -1e9, 1e6, 1e9, LOWEST])
def test_weights_add_up_under_a_common_offset(fmt, offset):
    # units over many CTAs, one CTA a unit; all blocks and a selection
    for B, L in ((1, 64 * 70 + 10), (100, 64 * 5 + 10)):
        t = offset_tokens(B, 16, 2, L, offset, 41)
        nblk = L // 64 + 2
        lay = H.layer(t, nblk * 64, fmt, k_q=4, k_e=12, weights=True)
        t.prefill(lay, L)
        rows = np.append(np.full(L // 64, 64), [L % 64, 0])
        out = torch.empty((B, 16, 128), dtype=torch.int16, device="cuda")
        for zero in (True, False):
            q = H.dev16(np.zeros_like(t.q()) if zero else t.q())
            lay.weights.zero_()
            lay.dense_decode_weights(q, out)
            w = lay.weights.cpu().numpy().astype(np.float64)
            assert np.abs(w.sum(1) - t.G).max() <= t.G * (ZERO_Q if zero else ANY_Q)
            if zero:  # every token weighs the same
                want = t.G * rows / L
                assert (np.abs(w - want) <= ZERO_Q * want).all()
            lay.weights.zero_()
            lay.select(q)
            lay.sparse_decode_weights(q, out)
            w = lay.weights.cpu().numpy().astype(np.float64)
            assert np.abs(w.sum(1) - t.G).max() <= t.G * (ZERO_Q if zero else ANY_Q)
        assert lay.read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mask", [-1e9, -1e4, LOWEST, -np.inf])
def test_weights_beside_masked_stretches(fmt, mask):
    # the oldest blocks, the newest one, every other block, single tokens: what is left decides, to the usual bound
    L = 64 * 21 + 30
    t = H.Tokens(5, 8, 1, L, seed=42)
    t.e[0, :64 * 9] = mask
    t.e[1, 64 * 21:] = mask
    t.e[2].reshape(-1)[:64 * 20].reshape(10, 128)[:, :64] = mask
    t.e[3, 3::5] = mask
    t.e[4, :L - 1] = mask
    lay = H.layer(t, 64 * 23, fmt, weights=True)
    t.prefill(lay, L)
    units = [t.unit(u, L, fmt) for u in range(5)]
    q = t.q()
    q[:, 1] = P.to_bf16_bits(P.bf16(q[:, 1]) * 30)  # a head with logits far from the others'
    out = torch.empty((5, 8, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode_weights(H.dev16(q), out)
    got = lay.weights.cpu().numpy()
    check_weights(t, got, np.zeros_like(got), q, units, [range(22)] * 5, 23)
    H.check_out(t, out, q, units, [range(22)] * 5)
    assert np.abs(got.sum(1) - 8).max() <= 8 * 2.0 ** -15  # the far head: |v| < 1024, half a step 2^-15


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("how", ["dense", "sparse"])
def test_small_weights_under_a_large_one_in_the_newest_block(fmt, how):
    # one CTA attends a whole unit, the newest block first; the other tokens are 2^-26 of its largest, and alone
    # have values.  Halves of f16 against that largest would lose them.
    B, nb = 150, 16
    L = 64 * nb + 10
    t = H.Tokens(B, 1, 1, 1, seed=43)
    t.k = np.zeros((B, L, 128), np.uint16)
    t.e = np.full((B, L), -26 * np.log(2), np.float32)
    t.e[:, L - 1] = 0
    t.v = np.broadcast_to(P.to_bf16_bits(np.full(128, 64.0)), (B, L, 128)).copy()
    t.v[:, 64 * nb:] = 0
    lay = H.layer(t, 64 * (nb + 2), fmt, k_q=0, k_e=nb, weights=True)
    t.prefill(lay, L)
    q = t.q()
    out = torch.empty((B, 1, 128), dtype=torch.int16, device="cuda")
    if how == "dense":
        lay.dense_decode(H.dev16(q), out)
    else:
        lay.select(H.dev16(q))
        lay.sparse_decode(H.dev16(q), out)
    got = H.out_of(out)
    # 1024 weights of 2^-26 against 1 + 9 * 2^-26 + themselves.  P in 8, 11 or 16 bits of the same value: off by at
    # most 2^-8 of it, as is the output's own rounding; the rest is below 2^-16.
    p = np.exp(np.float64(t.e[0, 0]))
    want = 64 * 64 * nb * p / (1 + (L - 1) * p)
    assert np.abs(got - want).max() <= (2.0 ** -7 + 2.0 ** -16) * want
    if how == "dense":
        lay.dense_decode_weights(H.dev16(q), out)
        assert np.abs(H.out_of(out) - want).max() <= (2.0 ** -7 + 2.0 ** -16) * want


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B", [1, 150])
def test_nan_reaches_out_and_weights_alike(fmt, B):
    # a key that is NaN: its unit's out and weights are; a value of the newest block: that dim of out alone; the
    # other units as ever.  One CTA a unit, and many.
    nb = 40 if B == 1 else 6
    L = 64 * nb + 20
    for where in ("none", "key", "newest key", "query", "newest value"):
        t = H.Tokens(B, 4, 1, L, seed=44)
        q = t.q()
        if where == "key":
            t.k[0, 70, 5] = 0x7FC0
        elif where == "newest key":
            t.k[0, L - 1, 5] = 0x7FC0
        elif where == "newest value":
            t.v[0, L - 1, 5] = 0x7FC0
        elif where == "query":
            q[0, :, 3] = 0x7FC0
        lay = H.layer(t, 64 * (nb + 2), fmt, weights=True)
        t.prefill(lay, L)
        out = torch.empty((B, 4, 128), dtype=torch.int16, device="cuda")
        lay.dense_decode_weights(H.dev16(q), out)
        got, w = H.out_of(out), lay.weights.cpu().numpy()
        if where in ("key", "newest key", "query"):
            assert np.isnan(got[0]).all() and np.isnan(w[0, :nb + 1]).all(), where
        else:
            assert np.isnan(got[0, :, 5]).all() == (where == "newest value")
            assert not np.isnan(np.delete(got[0], 5, 1)).any() and abs(w[0].sum() - 4) <= 4 * ANY_Q, where
        assert not np.isnan(got[1:]).any() and not np.isnan(w[1:]).any()
        assert not w[0, nb + 1:].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B", [1, 150])
def test_every_call_takes_a_mask_of_the_lowest_value_alike(fmt, B):
    # a unit whose logits all are the lowest finite value is the mean of its values, whichever call attends it; with
    # -inf beside it, of what is not -inf; -inf alone gives zeros.  tokens at the lowest value beside others: nothing.
    nb = 40 if B == 1 else 5
    L = 64 * nb + 20
    for kind in ("lowest", "lowest and -inf", "-inf", "lowest and others"):
        t = H.Tokens(B, 4, 1, L, seed=45)
        t.e[:] = -np.inf if kind == "-inf" else LOWEST
        seen = np.ones(L, bool)
        if kind == "lowest and -inf":
            seen[1::3] = False
            t.e[:, ~seen] = -np.inf
        if kind == "lowest and others":
            seen[:] = np.arange(L) >= 64 * (nb - 1)
            t.e[:, seen] = 0.5
        q = t.q()
        if kind == "lowest and others":
            q[:] = 0  # every seen token weighs the same
        lay = H.layer(t, 64 * (nb + 2), fmt, k_q=0, k_e=nb, weights=True)
        t.prefill(lay, L)
        units = [t.unit(u, L, fmt) for u in range(B)]
        # equal weights: P is the same for all, the output is rounded once, the sums are off by 2^-16 of the mean |v|
        want, size = (np.stack([f(r.v)[seen].mean(0) for r in units])[:, None] for f in (lambda x: x, np.abs))
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * size
        lay.select(H.dev16(q))
        lay.decode_resident(H.dev16(q))
        calls = {"dense": lay.dense_decode, "sparse": lay.sparse_decode, "split": lay.decode_rest,
                 "dense weights": lay.dense_decode_weights, "sparse weights": lay.sparse_decode_weights}
        for name, call in calls.items():
            out = torch.full((B, 4, 128), 0x4242, dtype=torch.int16, device="cuda")
            lay.weights.zero_()
            call(H.dev16(q), out)
            got = H.out_of(out)
            if kind == "-inf":
                assert not got.any() and not lay.weights.any(), name
                continue
            assert (np.abs(got - want) <= tol).all(), (kind, name, np.abs(got - want).max())
            if name.endswith("weights"):
                assert (lay.weights.sum(1) - 4).abs().max() <= 4 * ANY_Q, (kind, name)
        assert lay.read_error() == 0


def test_the_fused_step_takes_a_mask_of_the_lowest_value():
    for B in (1, 150):
        L = 64 * 9 + 20
        t = H.Tokens(B, 4, 1, L + 1, seed=46)
        t.e[:] = LOWEST
        lay = H.layer(t, 64 * 11, "bf16", k_q=0, k_e=9)
        t.prefill(lay, L)
        out = torch.empty((B, 4, 128), dtype=torch.int16, device="cuda")
        lay.fused_step(*t.new(np.full(B, L)), H.dev16(t.q()), out)
        v = np.stack([t.unit(u, L + 1, "bf16").v for u in range(B)])
        want = v.mean(1)[:, None]
        assert (np.abs(H.out_of(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * np.abs(v).mean(1)[:, None]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("top", [2.5e38, np.finfo(np.float32).max])
def test_a_logit_of_the_largest_values_takes_it_all(fmt, top):
    L = 64 * 5 + 9
    for at in (70, L - 2):
        t = H.Tokens(3, 4, 1, L, seed=48)
        t.e[0, at] = top
        t.e[1] = LOWEST
        t.e[1, at] = top
        lay = H.layer(t, 64 * 7, fmt, k_q=0, k_e=5, weights=True)
        t.prefill(lay, L)
        units = [t.unit(u, L, fmt) for u in range(3)]
        q = t.q()
        lay.select(H.dev16(q))
        for call in (lay.dense_decode, lay.sparse_decode, lay.dense_decode_weights):
            out = torch.empty((3, 4, 128), dtype=torch.int16, device="cuda")
            call(H.dev16(q), out)
            for u in range(2):  # the value itself, rounded once (a code's: 2^-16 for its product and its weight)
                want = units[u].v[at]
                assert (np.abs(H.out_of(out)[u] - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want)).all(), (at, u)
        w = lay.weights.cpu().numpy()
        assert (np.abs(w[:2, at // 64] - 4) <= 4 * ANY_Q).all() and np.abs(w.sum(1) - 4).max() <= 4 * ANY_Q


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("L", [5, 64 * 3 + 7])
def test_split_attention_carries_nan(fmt, L):
    # all that the unit attends is resident and NaN, and the second pass has nothing to add: NaN, as in one pass
    t = H.Tokens(2, 4, 1, L, seed=47)
    q = t.q()
    q[0, :, 3] = 0x7FC0
    lay = H.layer(t, 64 * 5, fmt, k_q=2, k_e=4)
    t.prefill(lay, L)
    one, two = (torch.empty((2, 4, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    lay.decode_resident(H.dev16(q))
    lay.select(H.dev16(q))
    lay.decode_rest(H.dev16(q), two)
    lay.sparse_decode(H.dev16(q), one)
    assert np.isnan(H.out_of(one)[0]).all() and np.isnan(H.out_of(two)[0]).all()
    assert not np.isnan(H.out_of(two)[1]).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offset", [-1e9, LOWEST])
def test_weights_add_up_over_the_block_cache(fmt, offset):
    # the same under an offset where the blocks' logits lie in cache slots, and replayed from a graph
    L, steps = 64 * 9 + 62, 4
    t = offset_tokens(3, 8, 2, L + steps, offset, 49)
    lay = H.layer(t, 64 * 12, fmt, k_q=2, k_e=3, offload=True, weights=True)
    t.prefill(lay, L)
    q = H.dev16(t.q())
    k, v, e = t.new(np.full(t.units, L))
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        lay.decode_step(k, v, e, q, out)
    for i in range(steps):  # over the border at 64 * 10
        for dst, src in zip((k, v, e), t.new(np.full(t.units, L + i))):
            dst.copy_(src)
        before = lay.weights.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        gain = (lay.weights - before).cpu().numpy().astype(np.float64)
        # a total's own addition: half a step of it for each of at most 6 blocks
        assert np.abs(gain.sum(1) - t.G).max() <= t.G * ANY_Q + 6 * 2.0 ** -24 * float(lay.weights.max()), i
    assert lay.read_error() == 0
