"""Accumulated block weights and eviction by them, on the GPU, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import block_sparse_offloadable_b200 as nosa
from tests import kv8_harness as H
from tests import plain64 as P

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "int8", "e4m3"]


def check_weights(t, got, before, q, units, blocks, nblk):
    """got [units][nblk] = before + the blocks' weights of q; the blocks not attended untouched."""
    qq = P.bf16(q).reshape(t.units, t.G, 128)
    for u, ref in enumerate(units):
        bl = [b for b in blocks[u] if 0 <= b <= ref.local]
        w, tol = ref.attend(qq[u], bl)[2:]
        want, lim = before[u].astype(np.float64).copy(), np.zeros(nblk)
        np.add.at(want, np.array(bl, int), w)
        np.add.at(lim, np.array(bl, int), tol)
        lim[bl] += 2.0 ** -23 * np.abs(want[bl])  # the addition
        assert (np.abs(got[u] - want) <= lim).all(), (u, np.abs(got[u] - want).max())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,Hq,Hkv,lens", [(1, 1, 1, [1]), (1, 8, 1, [65]), (3, 7, 1, [0, 1000, 63]),
                                           (1, 10, 2, [64 * 70 + 1]), (24, 8, 2, [64 * 60 - 100 * i for i in range(24)]), (1, 16, 2, [64 * 300]),
                                           (40, 16, 4, [65 + 7 * i for i in range(40)]),
                                           (24, 4, 1, [64 * 700] + [1 + i for i in range(23)]),  # one long, many short
                                           (6, 8, 2, [0, 64 * 90, 64, 0, 1, 64 * 33 + 1]),
                                           (2048, 2, 1, [1 + i % 130 for i in range(2048)])])  # the most units
def test_dense_weights(fmt, B, Hq, Hkv, lens):
    T = max(lens)
    t = H.Tokens(B, Hq, Hkv, T, seed=B + T)
    nblk = (T + 63) // 64 + 1
    lay = H.layer(t, nblk * 64, fmt, weights=True)
    t.prefill(lay, T, lens if T > 1 else None)
    units = [t.unit(u, lens[u // Hkv], fmt) for u in range(t.units)]
    blocks = [range(r.local + 1) for r in units]
    out, plain = (torch.empty((B, Hq, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    for _ in range(2):  # a second token adds to the first's
        q, before = t.q(), lay.weights.cpu().numpy()
        lay.dense_decode_weights(H.dev16(q), out)
        got = lay.weights.cpu().numpy()
        check_weights(t, got, before, q, units, blocks, nblk)
        total = (got - before).sum(1)
        for u, r in enumerate(units):  # G heads' weights, each summing to one
            assert abs(total[u] - (t.G if r.L else 0)) <= 1e-4 * t.G
        H.check_out(t, out, q, units, blocks)
    assert lay.read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offload", [False, True])
def test_step_weights(fmt, offload):
    # the layer's step, device and offload store, more units than SMs and few; weights of the selection alone
    for B, L, steps in ((2, 64 * 11 + 60, 6), (80, 64 * 6 + 63, 2)):
        t = H.Tokens(B, 8, 2, L + steps, seed=B)
        lay = H.layer(t, L // 64 * 64 + 192, fmt, k_q=2, k_e=3, offload=offload, weights=True)
        t.prefill(lay, L)
        lay.weights.uniform_(0, 3)
        out = torch.empty((B, 8, 128), dtype=torch.int16, device="cuda")
        for i in range(steps):
            q, before = t.q(), lay.weights.cpu().numpy()
            lay.decode_step(*t.new(np.full(t.units, L + i)), H.dev16(q), out)
            units = [t.unit(u, L + i + 1, fmt) for u in range(t.units)]
            s = H.sels(lay)
            check_weights(t, lay.weights.cpu().numpy(), before, q, units, s, lay.weights.shape[1])
            H.check_out(t, out, q, units, s)
        assert lay.read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_masked_and_repeated(fmt):
    L = 64 * 4 + 10
    t = H.Tokens(4, 2, 1, L, seed=21)
    t.e[0, :100] = -np.inf
    t.e[1] = -np.inf  # nothing seen: no weight at all
    t.e[2, 64:128] = np.finfo(np.float32).min
    lay = H.layer(t, 64 * 6, fmt, weights=True)
    t.prefill(lay, L)
    units = [t.unit(u, L, fmt) for u in range(4)]
    q = t.q()
    out = torch.empty((4, 2, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode_weights(H.dev16(q), out)
    got = lay.weights.cpu().numpy()
    check_weights(t, got, np.zeros_like(got), q, units, [range(5)] * 4, 6)
    assert not got[1].any() and got[0, 0] == 0
    # a list that names a block twice: both entries' weight is added
    lay.weights.zero_()
    lay.sel.fill_(-1)
    lay.sel[:, :4] = torch.tensor([2, 2, 3, 4])
    lay.nsel.fill_(4)
    lay.sparse_decode_weights(H.dev16(q), out)
    w = lay.weights.cpu().numpy()
    assert abs(w[3].sum() - 2) < 1e-4 and not w[:, :2].any()
    once = units[3].attend(P.bf16(q)[3], [2, 3, 4])[2]
    # block 2 counted twice in the sums as well: w2' = 2 w2 / (1 + w2) of a head's share; checked on the total
    assert w[3, 2] > once[0]


def test_results_do_not_vary():
    t = H.Tokens(1, 16, 2, 64 * 200, seed=22)
    lay = H.layer(t, 64 * 201, "int8", weights=True)
    t.prefill(lay, 64 * 200)
    q = H.dev16(t.q())
    out = torch.empty((1, 16, 128), dtype=torch.int16, device="cuda")
    seen = []
    for _ in range(5):
        lay.weights.zero_()
        lay.dense_decode_weights(q, out)
        seen.append((out.clone(), lay.weights.clone()))
    assert all(torch.equal(a, seen[0][0]) and torch.equal(b, seen[0][1]) for a, b in seen)


# ---- eviction ----------------------------------------------------------------------------------------

def check_evicted(src, dst, kept, w, lens, keep, sink, recent, fmt, fill=False):
    """dst's whole state against the plain rule, bit for bit; unreached parts untouched (0x5A bytes)."""
    units = len(lens)
    kept, w = kept.cpu().numpy(), w.cpu().numpy()
    sn, dn = src.cfg.max_ctx // 64, dst.cfg.max_ctx // 64
    get = lambda lay, name, n: getattr(lay, name).cpu().view(units, n, -1)  # noqa: E731
    dwt = dst.weights.cpu().numpy()
    for u in range(units):
        L = lens[u]
        nb = (L - 1) // 64 if L else 0
        ids = P.keep_blocks(w[u], nb, keep, sink, recent)
        want = (ids + [nb] if L else [])
        assert kept[u].tolist() == want + [-1] * (keep + 1 - len(want)), u
        assert int(dst.seq_len[u]) == (len(ids) * 64 + L - nb * 64 if L else 0)
        full = np.zeros(dn, np.float32)
        full[:len(want)] = w[u, want]
        assert np.array_equal(dwt[u], full, equal_nan=True)
        new = {b: i for i, b in enumerate(ids)}
        ge = [new[b] for b in src.gamma_e.cpu().view(units, -1)[u, :int(src.gamma_n[u])].tolist() if b in new]
        assert dst.gamma_e.cpu().view(units, -1)[u, :int(dst.gamma_n[u])].tolist() == ge
        if fill:
            pool = [new[b] for b in src.pool.cpu().view(units, -1)[u, :int(src.pool_n[u])].tolist() if b in new]
            assert dst.pool.cpu().view(units, -1)[u, :int(dst.pool_n[u])].tolist() == pool
        e, ck, E = (get(dst, n, dn)[u] for n in ("evict_logit", "ck", "blk_evict"))
        e0, ck0, E0 = (get(src, n, sn)[u] for n in ("evict_logit", "ck", "blk_evict"))
        stale = lambda x: bool((x.contiguous().view(torch.uint8) == 0x5A).all())  # noqa: E731
        for i in range(dn):
            b = want[i] if i < len(want) else None
            rows = 0 if b is None else min(64, L - b * 64)
            if b is not None:
                assert torch.equal(e[i, :rows], e0[b, :rows])
                m = rows // 16 * 128
                assert torch.equal(ck[i, :m], ck0[b, :m]) and stale(ck[i, m:])
                assert torch.equal(E[i], E0[b]) if rows == 64 else stale(E[i])
            assert stale(e[i, rows:])
            if fmt == "bf16":
                kv, kv0 = (lay.kv_store.cpu().view(torch.int16).view(units, n, 2, 64, 128)[u]
                           for lay, n in ((dst, dn), (src, sn)))
                if b is not None:
                    assert torch.equal(kv[i, :, :rows], kv0[b, :, :rows])
                assert stale(kv[i, :, rows:])
            else:
                (c, s, _), (c0, s0, _) = ([x.cpu() for x in lay.kv8_views()] for lay in (dst, src))
                if b is not None and b != nb:
                    assert torch.equal(c[u, i].view(torch.uint8), c0[u, b].view(torch.uint8))
                    assert torch.equal(s[u, i], s0[u, b])
                else:
                    assert stale(c[u, i]) and stale(s[u, i])
        if fmt != "bf16":
            rows = L - nb * 64 if L else 0
            tail, tail0 = (lay.kv8_views()[2].cpu().view(torch.int16)[u] for lay in (dst, src))
            assert torch.equal(tail[:, :rows], tail0[:, :rows]) and stale(tail[:, rows:])


def spoiled(lay):
    """Fill what eviction writes with 0x5A bytes: what it leaves is seen."""
    for x in (lay.kv_store, lay.evict_logit, lay.ck, lay.blk_evict, lay.gamma_e, lay.weights, lay.pool):
        if x is not None:
            x.view(torch.uint8).fill_(0x5A)
    return lay


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("keep,sink,recent", [(0, 0, 0), (1, 0, 1), (5, 1, 1), (7, 7, 0), (12, 0, 12), (40, 3, 2)])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_evict(fmt, keep, sink, recent, kind):
    lens = [64 * 30 + 17, 64 * 9, 1, 64 * 22 + 63, 0]
    t = H.Tokens(5, 4, 2, max(lens), seed=keep)
    src = H.layer(t, 64 * 33, fmt, k_q=2, k_e=7, weights=True)
    dst = spoiled(H.layer(t, 64 * (keep + 2), fmt, k_q=2, k_e=7, weights=True))
    t.prefill(src, max(lens), lens)
    w = torch.rand(src.weights.shape, generator=torch.Generator().manual_seed(keep))
    if kind == "ties":
        w = (w * 3).floor()
    if kind == "odd":
        w = torch.where(w < 0.1, float("nan"), torch.where(w < 0.2, float("inf"), torch.where(w < 0.3, -0.0, w - 0.6)))
        w = torch.where((w > 0.3) & (w < 0.33), 0.0, w)
    src.weights.copy_(w)
    kept = src.evict(dst, keep, sink, recent)
    torch.cuda.synchronize()
    check_evicted(src, dst, kept, w, np.repeat(lens, 2), keep, sink, recent, fmt)
    assert src.read_error() == 0


def test_evict_fill_and_bf16_keys():
    t = H.Tokens(2, 4, 2, 64 * 50 + 3, seed=31)
    make = lambda n: H.layer(t, n, "int8", k_q=3, k_e=6, weights=True, fill=True, ck_bf16=True)  # noqa: E731
    src, dst = make(64 * 52), spoiled(make(64 * 24))
    t.prefill(src, 64 * 50)
    out = torch.empty((2, 4, 128), dtype=torch.int16, device="cuda")
    for i in range(3):  # drops pool entries, orders Gamma_e by rank
        src.decode_step(*t.new(np.full(4, 64 * 50 + i)), H.dev16(t.q()), out)
    src.dense_decode_weights(H.dev16(t.q()), out)
    w = src.weights.clone()
    kept = src.evict(dst, 19, 1, 2)
    check_evicted(src, dst, kept, w, [64 * 50 + 3] * 4, 19, 1, 2, "int8", fill=True)
    for i in range(70):  # and goes on
        dst.decode_step(*t.new(np.full(4, i)), H.dev16(t.q()), out)
    assert dst.read_error() == 0 and dst.seq_len.tolist() == [64 * 19 + 3 + 70] * 4


def test_evict_large():
    # units of 2^20 tokens (16383 candidates), many equal weights, offsets past 2^32 bytes
    t = H.Tokens(3, 8, 8, 64, seed=32)
    src = H.layer(t, 1 << 20, "int8", k_q=2, k_e=4, weights=True)
    dst = H.layer(t, 1 << 19, "int8", k_q=2, k_e=4, weights=True)
    nb = (1 << 14) - 1
    codes, scales, tail = src.kv8_views()
    for u in (0, 23):
        codes[u].view(torch.int32).random_(generator=torch.Generator("cuda").manual_seed(u))
    scales.uniform_()
    tail.zero_()
    src.evict_logit.normal_()
    src.ck.normal_()
    src.blk_evict.normal_()
    src.seq_len.fill_((1 << 20) - 5)
    src.gamma_n.fill_(0)
    w = (torch.rand(24, nb + 1, device="cuda") * 1000).floor()
    src.weights.copy_(w)
    keep = 8191
    kept = src.evict(dst, keep, 4, 4)
    torch.cuda.synchronize()
    for u in (0, 23):
        ids = P.keep_blocks(w[u].cpu().numpy(), nb, keep, 4, 4)
        assert kept[u].tolist() == ids + [nb]
        at = torch.tensor(ids, device="cuda")
        assert torch.equal(dst.kv8_views()[0][u, :keep], codes[u, at])
        assert torch.equal(dst.kv8_views()[1][u, :keep], scales[u, at])
        assert torch.equal(dst.ck.view(24, -1, 512)[u, :keep], src.ck.view(24, -1, 512)[u, at])


@pytest.mark.parametrize("fmt", FMTS)
def test_prompt_weigh_evict_decode(fmt):
    # as they are used together: a prompt, tokens that weigh its blocks, the heavy ones into a small
    # store, and decoding there over a block border, against the plain form over the kept tokens
    L, keep = 64 * 20 + 61, 5
    t = H.Tokens(2, 8, 2, L + 8, seed=33)
    big = H.layer(t, 64 * 22, fmt, k_q=2, k_e=2, weights=True)
    small = H.layer(t, 64 * 8, fmt, k_q=2, k_e=2, weights=True)
    t.prefill(big, L - 4)
    out = torch.empty((2, 8, 128), dtype=torch.int16, device="cuda")
    for i in range(4):
        t.append(big, np.full(4, L - 4 + i))
        big.dense_decode_weights(H.dev16(t.q()), out)
    kept = big.evict(small, keep, 1, 1).cpu().numpy()
    stale = t.k, t.v, t.e
    rows = [np.concatenate([np.arange(64 * b, min(64 * b + 64, L)) for b in kept[u]] + [np.arange(L, L + 8)])
            for u in range(4)]
    n0 = keep * 64 + 61
    t2 = H.Tokens(2, 8, 2, 1, seed=34)
    t2.k, t2.v, t2.e = (np.stack([x[u, rows[u]] for u in range(4)]) for x in stale)
    for i in range(8):
        q = t.q()
        small.decode_step(*t2.new(np.full(4, n0 + i)), H.dev16(q), out)
        units = [t2.unit(u, n0 + i + 1, fmt) for u in range(4)]
        H.check_out(t2, out, q, units, H.sels(small))
        small.dense_decode(H.dev16(q), out)
        H.check_out(t2, out, q, units, [range(r.local + 1) for r in units])
    if fmt != "bf16":
        H.check_store(small, t2, units, fmt)
    assert small.read_error() == 0


def test_evict_captured_and_refused():
    t = H.Tokens(1, 4, 2, 64 * 12, seed=35)
    src, dst = (H.layer(t, n, "bf16", k_q=2, k_e=2, weights=True) for n in (64 * 13, 64 * 6))
    t.prefill(src, 64 * 12)
    kept = torch.empty((2, 6), dtype=torch.int32, device="cuda")
    args = (src.cfg, src.state, src.weights, 5, 0, 0, dst.cfg, dst.state, dst.weights, kept)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        nosa.nosa_evict(*args)
    for seed in range(3):
        src.weights.uniform_(generator=torch.Generator("cuda").manual_seed(seed))
        g.replay()
        torch.cuda.synchronize()
        for u in range(2):
            assert kept[u].tolist() == P.keep_blocks(src.weights[u].cpu().numpy(), 11, 5, 0, 0) + [11]
    for bad in (dict(dst=src), dict(w=dst.weights)):
        with pytest.raises(nosa.NosaError) as ei:  # the same state, the same weights
            if "dst" in bad:
                src.evict(src, 5)
            else:
                nosa.nosa_evict(src.cfg, src.state, dst.weights, 5, 0, 0, dst.cfg, dst.state, dst.weights, kept)
        assert ei.value.code == nosa.ERR_ARG
    with pytest.raises(ValueError):
        H.layer(t, 640, "bf16").dense_decode_weights(None, None)
    with pytest.raises(nosa.NosaError) as ei:
        src.evict(dst, 6)
    assert ei.value.code == nosa.ERR_CAPACITY
    with pytest.raises(nosa.NosaError) as ei:
        nosa.nosa_evict(src.cfg, src.state, src.weights.cpu(), 5, 0, 0, dst.cfg, dst.state, dst.weights, kept)
    assert ei.value.code == nosa.ERR_PTR


def test_evict_on_another_stream():
    # the list of kept blocks is the given stream's memory: nothing queued on the current one holds it
    t = H.Tokens(2, 4, 2, 64 * 12, seed=36)
    src, dst = (H.layer(t, n, "int8", k_q=2, k_e=2, weights=True) for n in (64 * 13, 64 * 6))
    t.prefill(src, 64 * 12)
    src.weights.uniform_(generator=torch.Generator("cuda").manual_seed(3))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        busy = torch.full((4, 6), 77, dtype=torch.int32, device="cuda")  # freed while it may still be written
        del busy
        kept = src.evict(dst, 5, stream=s)
        s.synchronize()
        with torch.cuda.stream(s):
            got = kept.cpu()
        for u in range(4):
            assert got[u].tolist() == P.keep_blocks(src.weights[u].cpu().numpy(), 11, 5, 0, 0) + [11]
