"""The 8-bit store, weights and eviction on the host: flags, sizes and refusals, nothing launched."""
import ctypes

import numpy as np
import pytest

import block_sparse_offloadable_b200 as nosa
from tests import plain64


def cfg(**kw):
    base = dict(batch=2, heads_q=16, heads_kv=2, k_q=16, k_e=48, max_ctx=8192)
    base.update(kw)
    return nosa.make_config(**base)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_flags(fmt):
    assert nosa.nosa_validate_config(cfg(kv_format=fmt)) == nosa.OK
    assert nosa.nosa_validate_config(cfg(kv_format=fmt, ck_bf16=True, fill=True, offload=True)) == nosa.OK
    both = cfg()
    both.flags = nosa.FLAG_KV_INT8 | nosa.FLAG_KV_E4M3
    assert nosa.nosa_validate_config(both) == nosa.ERR_ARG
    with pytest.raises(ValueError):
        cfg(kv_format="fp8")


@pytest.mark.parametrize("max_ctx", [64, 192, 8192])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_sizes(fmt, max_ctx):
    u, nblk, slots, rec = 4, max_ctx // 64, 16 + 48 + 2, 16768  # 16384 codes, 66 floats, padded to lines of 128
    dev, off = cfg(kv_format=fmt, max_ctx=max_ctx), cfg(kv_format=fmt, max_ctx=max_ctx, offload=True)
    whole = lambda n: (u * n * rec + 255) // 256 * 256 + u * 32768  # noqa: E731  records, then bf16 tails
    assert nosa.nosa_state_bytes(dev, nosa.BUF_KV_STORE) == whole(nblk)
    assert nosa.nosa_state_bytes(dev, nosa.BUF_CACHE) == 0
    assert nosa.nosa_state_bytes(off, nosa.BUF_KV_STORE) == u * nblk * rec
    assert nosa.nosa_state_bytes(off, nosa.BUF_CACHE) == whole(slots)
    for c in (dev, off):  # the pooled keys and the other state do not change
        assert nosa.nosa_state_bytes(c, nosa.BUF_CK) == u * (max_ctx // 16) * 128 * 4
    assert nosa.nosa_workspace_bytes(dev, nosa.WS_FUSED_STEP) == 0
    assert nosa.nosa_workspace_bytes(dev, nosa.WS_SPARSE_DECODE) == nosa.nosa_workspace_bytes(
        cfg(max_ctx=max_ctx), nosa.WS_SPARSE_DECODE)


def test_weights_workspaces():
    c = cfg()
    base = 256 + (148 * 2 * (2 * 8 + 8 * 128) * 4 + 255) // 256 * 256
    assert nosa.nosa_workspace_bytes(c, nosa.WS_SPARSE_WEIGHTS) == base + 4 * 65 * 32
    assert nosa.nosa_workspace_bytes(c, nosa.WS_DENSE_WEIGHTS) == base + 4 * 128 * 32
    assert nosa.nosa_workspace_bytes(cfg(offload=True), nosa.WS_DENSE_WEIGHTS) == 0


def test_refusals_before_any_launch():
    L, P, st = nosa.lib(), ctypes.c_void_p, nosa.State()
    a, c8 = cfg(), cfg(kv_format="int8")
    assert L.nosa_fused_step(ctypes.byref(c8), ctypes.byref(st), P(16), P(16), P(16), P(16), P(16), P(16), None, P(16),
                             None, 0, None) == nosa.ERR_UNSUPPORTED

    def sparse(c, weights):
        return L.nosa_sparse_decode_weights(ctypes.byref(c), ctypes.byref(st), P(16), P(16), P(16), None, P(16),
                                            weights, None, 0, None)

    def dense(c, weights):
        return L.nosa_dense_decode_weights(ctypes.byref(c), ctypes.byref(st), P(16), P(16), weights, None, 0, None)

    assert sparse(a, None) == nosa.ERR_PTR and dense(a, None) == nosa.ERR_PTR
    assert sparse(a, P(16)) == nosa.ERR_PTR  # the state's buffers are missing
    assert dense(cfg(offload=True), P(16)) == nosa.ERR_ARG

    def evict(c=a, dc=a, keep=8, sink=0, recent=0):
        return L.nosa_evict(ctypes.byref(c), ctypes.byref(st), P(16), keep, sink, recent, ctypes.byref(dc),
                            ctypes.byref(st), P(16), P(16), None)

    assert evict() == nosa.ERR_PTR
    assert evict(keep=-1) == evict(sink=-1) == evict(recent=-1) == evict(sink=5, recent=4) == nosa.ERR_ARG
    assert evict(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == nosa.ERR_ARG
    assert evict(keep=128) == evict(keep=2 ** 31 - 1) == nosa.ERR_CAPACITY  # 128 blocks: 127 and the local one
    assert evict(dc=cfg(max_ctx=512), keep=8) == nosa.ERR_CAPACITY
    assert evict(c=cfg(offload=True)) == evict(dc=cfg(offload=True)) == nosa.ERR_UNSUPPORTED
    for other in (dict(batch=4), dict(heads_q=8), dict(k_q=8), dict(k_e=8), dict(kv_format="int8"), dict(ck_bf16=True),
                  dict(fill=True)):
        assert evict(dc=cfg(**other)) == nosa.ERR_ARG, other
    bad = cfg()
    bad.max_ctx = 100
    assert evict(c=bad) == evict(dc=bad) == nosa.ERR_ARG


def test_plain_e4m3_against_every_code():
    # the plain form's rounding, against the 256 codes by brute force
    import torch
    vals = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    vals = np.unique(vals[np.isfinite(vals)])
    r = np.random.default_rng(0)
    x = np.concatenate([r.uniform(-448, 448, 2000), r.standard_normal(2000) * 0.02, (vals[1:] + vals[:-1]) / 2, vals])
    got = plain64.e4m3(np.where(x == 0, 1e-300, x))
    best = np.abs(x[:, None] - vals[None]).min(1)
    assert np.array_equal(np.abs(x - got), best)
    assert np.isin(got, vals).all()


def test_plain_keep_blocks():
    w = np.array([1, 5, 5, 0, np.nan, 9, 2], np.float32)
    assert plain64.keep_blocks(w, 7, 3, 0, 0) == [1, 4, 5]
    assert plain64.keep_blocks(w, 7, 3, 1, 1) == [0, 4, 6]
    assert plain64.keep_blocks(w, 7, 9, 0, 0) == list(range(7))
    assert plain64.keep_blocks(w, 7, 0, 0, 0) == []
