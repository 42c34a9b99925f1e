"""The 8-bit KV store on the GPU: what the appends store, bit for bit, and the attention over it."""
import numpy as np
import pytest
import torch

import block_sparse_offloadable_b200 as nosa
from tests import kv8_harness as H
from tests import plain64 as P

pytestmark = pytest.mark.gpu
FMTS = ["int8", "e4m3"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,lens", [(1, None), (2, None), (63, None), (64, None), (65, None), (129, None), (200, [200, 1]),
                                    (192, [0, 192]), (320, [129, 320])])
def test_prefill_stores_the_formula(fmt, T, lens):
    t = H.Tokens(2, 8, 2, T, seed=T)
    lay = H.layer(t, (T + 63) // 64 * 64 + 64, fmt)
    t.prefill(lay, T, lens)
    n = np.repeat(lens or [T, T], 2)
    H.check_store(lay, t, [t.unit(u, n[u], fmt) for u in range(t.units)], fmt)
    assert lay.read_error() == 0 and lay.seq_len.cpu().tolist() == n.tolist()


@pytest.mark.parametrize("ck_bf16", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
def test_the_rest_of_the_state_is_the_bf16_stores(fmt, ck_bf16):
    # pooled keys, eviction scores, Gamma_e: bit-equal to a bf16 layer's after a ragged prefill
    t = H.Tokens(3, 8, 2, 64 * 40, seed=5)
    lens = [64 * 40, 64 * 17 + 5, 100]
    a, b = (H.layer(t, 64 * 41, f, ck_bf16=ck_bf16) for f in ("bf16", fmt))
    for lay in (a, b):
        t.prefill(lay, 64 * 40, lens)
    for u, n in enumerate(np.repeat(lens, 2)):
        ck = [x.ck.view(t.units, -1, 128)[u, :n // 16] for x in (a, b)]
        assert torch.equal(*ck)
        assert torch.equal(*[x.blk_evict.view(t.units, -1)[u, :n // 64] for x in (a, b)])
        assert torch.equal(*[x.evict_logit.view(t.units, -1)[u, :n] for x in (a, b)])
        g = int(a.gamma_n[u])
        assert g == int(b.gamma_n[u])
        assert torch.equal(*[x.gamma_e.view(t.units, -1)[u, :g] for x in (a, b)])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offload", [False, True])
@pytest.mark.parametrize("how", ["append", "append_select", "step"])
def test_decode_from_empty_over_block_borders(fmt, offload, how):
    # every step: the selection is the bf16 layer's, the attention is the plain form's over it
    n = 64 * 3 + 5
    t = H.Tokens(2, 6, 2, n, seed=3)
    lay, ref = (H.layer(t, 64 * 5, f, k_q=1, k_e=1, offload=offload) for f in (fmt, "bf16"))
    out, rout = (torch.empty((2, 6, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    for i in range(n):
        q = t.q()
        for x, o in ((lay, out), (ref, rout)):
            new = t.new(np.full(t.units, i))
            if how == "step":
                x.decode_step(*new, H.dev16(q), o)
                continue
            if how == "append":
                x.append(*new, 1)
                x.select(H.dev16(q))
            else:
                x.append_select(*new, H.dev16(q))
            if offload:
                x.cache_sync()
            x.sparse_decode(H.dev16(q), o)
        assert torch.equal(lay.sel, ref.sel) and torch.equal(lay.nsel, ref.nsel), i
        assert torch.equal(lay.gq, ref.gq)
        if offload:
            assert torch.equal(lay.n_fetched, ref.n_fetched)
        if i % 16 in (0, 15) or i in (1, 64, 65):
            H.check_out(t, out, q, [t.unit(u, i + 1, fmt) for u in range(t.units)], H.sels(lay))
    units = [t.unit(u, n, fmt) for u in range(t.units)]
    if not offload:
        H.check_store(lay, t, units, fmt)
    else:  # the resident blocks hold the codes; so does host memory
        torch.cuda.synchronize()
        codes = lay.kv8_views()[0].cpu()
        host = lay.kv_store.view(codes.dtype).view(t.units, -1, nosa.RECORD_BYTES)[:, :, :16384].unflatten(2, (2, 64, 128))
        bt = lay.block_table.cpu().numpy()
        for u, s in enumerate(H.sels(lay)):
            for j, b in enumerate(s):
                if b != units[u].local:
                    assert np.array_equal(codes[u, bt[u, j]].float().numpy(), units[u].codes[b])
            for b in units[u].codes:
                assert np.array_equal(host[u, b].float().numpy(), units[u].codes[b]), (u, b)
    assert lay.read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,Hq,Hkv,lens", [
    (1, 1, 1, [1]), (1, 8, 1, [64]), (1, 3, 1, [65]), (2, 10, 2, [128, 129]), (3, 7, 1, [0, 1000, 63]),
    (1, 16, 2, [64 * 70 + 1]), (24, 8, 2, [64 * 60 - 100 * i for i in range(24)]), (5, 16, 16, [200, 64, 65, 0, 511]), (40, 16, 4, [65 + 7 * i for i in range(40)]),
    (2048, 2, 1, [1 + i % 130 for i in range(2048)])])  # as many units as a call takes
def test_dense(fmt, B, Hq, Hkv, lens):
    T = max(lens)
    t = H.Tokens(B, Hq, Hkv, T, seed=B + T)
    lay = H.layer(t, (T + 63) // 64 * 64 + 64, fmt)
    t.prefill(lay, T, lens if T > 1 else None)
    q = t.q()
    out = torch.full((B, Hq, 128), 0x4242, dtype=torch.int16, device="cuda")
    units = [t.unit(u, lens[u // Hkv], fmt) for u in range(t.units)]
    for _ in range(2):  # the workspace is left as it was
        lay.dense_decode(H.dev16(q), out)
        H.check_out(t, out, q, units, [range(r.local + 1) for r in units])
    assert lay.read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offload", [False, True])
@pytest.mark.parametrize("B,Hkv,k_q,k_e,L", [(1, 1, 32, 96, 64 * 200 + 9), (2, 2, 0, 5, 64 * 9), (50, 4, 3, 4, 64 * 12 + 1),
                                             (3, 2, 5, 0, 64 * 20 + 33)])
def test_sparse_geometries(fmt, offload, B, Hkv, k_q, k_e, L):
    # many pieces per unit, units split over CTAs, more units than SMs; also the split decode
    t = H.Tokens(B, 4 * Hkv, Hkv, L + 2, seed=L)
    lay = H.layer(t, (L + 66) // 64 * 64 + 64, fmt, k_q=k_q, k_e=k_e, offload=offload)
    t.prefill(lay, L)
    out, out2 = (torch.empty((B, 4 * Hkv, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    for i in range(2):
        q = t.q()
        lay.append(*t.new(np.full(t.units, L + i)), 1)
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        lay.decode_resident(H.dev16(q), side)
        lay.select(H.dev16(q))
        if offload:
            lay.cache_sync()
        cur.wait_stream(side)
        lay.decode_rest(H.dev16(q), out2)
        lay.sparse_decode(H.dev16(q), out)
        some = range(0, t.units, max(1, t.units // 12))
        units, s = {u: t.unit(u, L + i + 1, fmt) for u in some}, H.sels(lay)
        for o in (out, out2):
            got, qq = H.out_of(o).reshape(t.units, -1, 128), P.bf16(q).reshape(t.units, -1, 128)
            for u, ref in units.items():
                want, tol = ref.attend(qq[u], s[u])[:2]
                assert (np.abs(got[u] - want) <= tol).all(), (i, u)
    assert lay.read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_masked_logits(fmt):
    # -inf on tokens, on whole blocks, on everything but one token, on everything; the lowest finite value
    L = 64 * 4 + 10
    t = H.Tokens(7, 4, 1, L, seed=9)
    t.e[6] = np.finfo(np.float32).min  # every token: their mean
    t.e[0, 5:150:3] = -np.inf
    t.e[1, :192] = -np.inf
    t.e[2] = -np.inf
    t.e[2, 77] = 0.25
    t.e[3] = -np.inf
    t.e[4, 64:128] = np.finfo(np.float32).min
    t.e[5, 200:] = 80.0  # one stretch far above the others
    t.e[5, :64] = -80.0
    lay = H.layer(t, 64 * 6, fmt)
    t.prefill(lay, L)
    q = t.q()
    out = torch.empty((7, 4, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode(H.dev16(q), out)
    units = [t.unit(u, L, fmt) for u in range(7)]
    H.check_out(t, out, q, units, [range(5)] * 7)
    assert not out[3].any()  # nothing seen: zeros


@pytest.mark.parametrize("fmt", FMTS)
def test_values_that_are_not_finite_stay_visible(fmt):
    # a block with one such key or value gives NaN to whoever attends it, and to no one else
    L = 64 * 3 + 4
    t = H.Tokens(6, 2, 1, L, seed=10)
    t.k[0, 70, 3] = 0x7F80  # +inf
    t.k[1, 10, 0] = 0x7FC0  # NaN
    t.v[2, 130, 127] = 0xFF80  # -inf
    t.v[3, 5, 5] = 0x7FC1
    t.v[4, L - 1, 7] = 0x7FC0  # in the tail: that dim alone
    lay = H.layer(t, 64 * 5, fmt)
    t.prefill(lay, L)
    scales = lay.kv8_views()[1].cpu()
    assert torch.isnan(scales[0, 1, 0]) and torch.isnan(scales[1, 0, 0]) and torch.isnan(scales[2, 2, 1])
    assert int(torch.isnan(scales[:, :3]).sum()) == 4
    q = t.q()
    out = torch.empty((6, 2, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode(H.dev16(q), out)
    got = H.out_of(out)
    assert np.isnan(got[:4]).all()
    assert np.isnan(got[4, :, 7]).all() and not np.isnan(np.delete(got[4], 7, 1)).any()
    H.check_out(t, out, q, [t.unit(u, L, fmt) for u in range(6)], [range(4)] * 6)
    # a selection that leaves the block out is not touched by it
    lay.sel.copy_(torch.tensor([[0, 2, 3] + [-1] * 14], dtype=torch.int32).repeat(6, 1))
    lay.nsel.fill_(3)
    lay.sparse_decode(H.dev16(q), out)
    assert not np.isnan(H.out_of(out)[0]).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ks,vs,qs", [(1e-3, 1e-4, 1e3), (30.0, 1e4, 0.02), (2.0 ** -60, 2.0 ** 40, 2.0 ** 60),
                                      (2.0 ** 70, 2.0 ** -90, 2.0 ** -71), (1.0, 2.0 ** -101, 1.0), (2.0 ** -104, 1.0, 1.0)])
def test_magnitudes(fmt, ks, vs, qs):
    L = 64 * 3 + 7
    t = H.Tokens(2, 4, 2, L, seed=11, k_scale=ks, v_scale=vs)
    t.v[1, 64:128] = 0  # a block of zero values
    lay = H.layer(t, 64 * 5, fmt)
    t.prefill(lay, L)
    units = [t.unit(u, L, fmt) for u in range(t.units)]
    H.check_store(lay, t, units, fmt)
    q = t.q(qs)
    out = torch.empty((2, 4, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode(H.dev16(q), out)
    H.check_out(t, out, q, units, [range(4)] * t.units)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_query_row_with_a_wide_range(fmt):
    # one entry of a head 2^20 above the others, a head of zeros, a head of subnormals
    L = 64 * 2 + 7
    t = H.Tokens(1, 4, 1, L, seed=12)
    t.k[0, :, 9] = 0  # the large entry meets zeros: the others decide
    lay = H.layer(t, 64 * 4, fmt)
    t.prefill(lay, L)
    q = P.to_bf16_bits(t.r.standard_normal((1, 4, 128)))
    q[0, 0, 9] = P.to_bf16_bits(np.array([2.0 ** 20]))[0]
    q[0, 1] = 0
    q[0, 2] = 0x0003
    out = torch.empty((1, 4, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode(H.dev16(q), out)
    H.check_out(t, out, q, [t.unit(0, L, fmt)], [range(3)])


@pytest.mark.parametrize("fmt", FMTS)
def test_many_small_weights_under_one_large(fmt):
    # 4095 tokens 2^-26 below one: together 2^-14 of it.  In f16 without the raised range they would all be lost.
    L = 4096
    t = H.Tokens(1, 1, 1, L, seed=13)
    t.k[:] = 0
    t.e[0] = -26 * np.log(2)
    t.e[0, 100] = 0
    t.v[0] = P.to_bf16_bits(np.full((L, 128), 64.0))
    t.v[0, 64:128] = 0  # the block of the large one
    lay = H.layer(t, L + 64, fmt)
    t.prefill(lay, L)
    q = t.q()
    out = torch.empty((1, 1, 128), dtype=torch.int16, device="cuda")
    lay.dense_decode(H.dev16(q), out)
    ref = t.unit(0, L, fmt)
    H.check_out(t, out, q, [ref], [range(64)])
    assert (H.out_of(out) > 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_eviction_head_and_ragged_offload(fmt):
    import synth
    lens = [64 * 5 + 1, 70]
    t = H.Tokens(2, 4, 2, max(lens) + 130, seed=14)
    w1, w2 = (torch.from_numpy(x).cuda() for x in synth.head_weights(0, 0, 2))
    layers = [H.layer(t, 64 * 9, f, k_q=2, k_e=2, offload=True) for f in (fmt, "bf16")]
    T, ln = max(lens), torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = [torch.empty((2, 4, 128), dtype=torch.int16, device="cuda") for _ in layers]
    for lay in layers:
        lay.append_head(H.dev16(t.k[:, :T]), H.dev16(t.v[:, :T]), w1, w2, T, ln)
    for i in range(130):
        at, q = np.repeat(lens, 2) + i, t.q()
        for lay, out in zip(layers, outs):
            k, v, _ = t.new(at)
            lay.append_head(k, v, w1, w2, 1)
            lay.select(H.dev16(q))
            lay.cache_sync()
            lay.sparse_decode(H.dev16(q), out)
        assert torch.equal(layers[0].sel, layers[1].sel) and torch.equal(layers[0].n_fetched, layers[1].n_fetched)
    e, e_ref = (lay.evict_logit.view(4, -1).cpu().numpy() for lay in layers)
    for u in range(4):
        assert np.array_equal(e[u, :lens[u // 2] + 130], e_ref[u, :lens[u // 2] + 130])
        t.e[u, :lens[u // 2] + 130] = e[u, :lens[u // 2] + 130]
    H.check_out(t, outs[0], q, [t.unit(u, lens[u // 2] + 130, fmt) for u in range(4)], H.sels(layers[0]))
    assert layers[0].read_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offload", [False, True])
def test_fill_reading_and_bf16_pooled_keys(fmt, offload):
    L, steps = 64 * 14 + 40, 60
    t = H.Tokens(2, 8, 2, L + steps, seed=18)
    lay, ref = (H.layer(t, 64 * 18, f, k_q=3, k_e=4, offload=offload, fill=True, ck_bf16=True) for f in (fmt, "bf16"))
    out, rout = (torch.empty((2, 8, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    for x in (lay, ref):
        t.prefill(x, L)
    for i in range(steps):
        q = t.q()
        for x, o in ((lay, out), (ref, rout)):
            x.decode_step(*t.new(np.full(t.units, L + i)), H.dev16(q), o)
        assert torch.equal(lay.sel, ref.sel) and torch.equal(lay.pool_n, ref.pool_n) and torch.equal(lay.gq, ref.gq)
        assert not offload or torch.equal(lay.n_fetched, ref.n_fetched)
        if i % 13 == 0:
            H.check_out(t, out, q, [t.unit(u, L + i + 1, fmt) for u in range(t.units)], H.sels(lay))
    assert lay.read_error() == 0


@pytest.mark.parametrize("fmt,offload", [("int8", True), ("e4m3", False)])
def test_full_size_layer(fmt, offload):
    # one layer of the 128K offload workload (and of the 32K device one), as bench.py runs it: the
    # selection and the fetches of the bf16 store, the attention of the plain form
    import bench
    c = dict(bench.WORKLOADS["offload28-128k" if offload else "stack28-32k"], step=False)
    seen = {}
    for f in ("bf16", fmt):  # one after the other: workloads share their pinned host store
        wl = bench.Workload(dict(c, kv_format=f), 3, seed=4, layers=1)
        lay, seen[f] = wl.layers[0][0], []
        for i in range(3):
            wl.cur.copy_(wl.inputs[i])
            q, k, v, e = wl.views(wl.cur, 0)
            out = torch.empty_like(q)
            lay.decode_step(k, v, e, q, out)
            seen[f] += [lay.sel.clone()] + ([lay.n_fetched.clone()] if offload else [])
        assert lay.read_error() == 0
    assert all(torch.equal(x, y) for x, y in zip(seen["bf16"], seen[fmt]))
    import synth
    n = c["L"] + 3
    sel, got = lay.sel.cpu().numpy(), H.out_of(out).reshape(lay.units, -1, 128)
    qq = P.bf16(q.cpu().numpy()).reshape(lay.units, -1, 128)
    for u in (0, lay.units - 1):
        K, V = (P.bf16(synth.kv_rows(4, s, 0, u // 2, u % 2, 0, n)) for s in (synth.K_STREAM, synth.V_STREAM))
        ref = P.Unit(K, V, synth.e_rows(4, 0, u // 2, u % 2, 0, n).astype(np.float64), fmt, lay.G, 128 ** -0.5)
        want, tol = ref.attend(qq[u], [x for x in sel[u] if x >= 0])[:2]
        assert (np.abs(got[u] - want) <= tol).all(), u


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    # 32 units of 2^20 tokens: 8.6 GB of codes; the last unit's blocks lie past 2^32 bytes
    t = H.Tokens(16, 4, 2, 200, seed=15)
    lay = H.layer(t, 1 << 20, fmt)
    t.prefill(lay, 200)
    q = t.q()
    out = torch.empty((16, 4, 128), dtype=torch.int16, device="cuda")
    units = [t.unit(u, 200, fmt) for u in range(t.units)]
    lay.dense_decode(H.dev16(q), out)
    H.check_out(t, out, q, units, [range(4)] * t.units)
    H.check_store(lay, t, units, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_graph_and_streams(fmt):
    # one decode step captured and replayed on new inputs, and two layers at once on two streams
    L = 64 * 6 + 62
    t = H.Tokens(2, 8, 2, L + 5, seed=16)
    lay = H.layer(t, 64 * 9, fmt, k_q=2, k_e=2)
    other = H.layer(t, 64 * 9, fmt, k_q=2, k_e=2)
    t.prefill(lay, L)
    t.prefill(other, L)
    k, v, e = t.new(np.full(t.units, L))
    q = H.dev16(t.q())
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    g, s, s2 = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        lay.decode_step(k, v, e, q, out)
    for i in range(5):  # over the border at 64 * 7
        for dst, src in zip((k, v, e), t.new(np.full(t.units, L + i))):
            dst.copy_(src)
        qn = t.q()
        q.copy_(H.dev16(qn))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        other.decode_step(k, v, e, q, out2, s2)
        torch.cuda.synchronize()
        assert torch.equal(lay.sel, other.sel) and torch.equal(out, out2)
        H.check_out(t, out, qn, [t.unit(u, L + i + 1, fmt) for u in range(t.units)], H.sels(lay))
    assert lay.read_error() == 0 and other.read_error() == 0


def test_errors_on_the_device():
    # a full store drops the token; a prefill into filled units leaves them; a selection past the newest
    # block attends nothing there
    t = H.Tokens(1, 4, 2, 200, seed=17)
    lay = H.layer(t, 128, "int8")
    t.prefill(lay, 128)
    before = lay.kv_store.clone()
    lay.append(*t.new(np.full(2, 130)), 1)
    assert lay.read_error() == nosa.EFLAG_CAPACITY
    t.prefill(lay, 100)
    assert lay.read_error() == nosa.EFLAG_STATE
    assert torch.equal(before, lay.kv_store) and lay.seq_len.tolist() == [128, 128]
    lay = H.layer(t, 640, "int8")
    t.prefill(lay, 128)
    lay.sel.fill_(-1)
    lay.sel[:, :3] = torch.tensor([0, 1, 7])
    lay.nsel.fill_(3)
    q = t.q()
    out = torch.empty((1, 4, 128), dtype=torch.int16, device="cuda")
    lay.sparse_decode(H.dev16(q), out)
    assert lay.read_error() == 0
    H.check_out(t, out, q, [t.unit(u, 128, "int8") for u in range(2)], [[0, 1]] * 2)
    lay.sel[:, 2] = 10  # no such block
    lay.sparse_decode(H.dev16(q), out)
    assert lay.read_error() == nosa.EFLAG_STATE
