"""The 8-bit KV store, the attention over it, accumulated attention weights, and eviction by them.

Four kinds of pass, each in a plain form (elementary torch operations) and as calls of the library:

  append        a new batch's prompt into an 8-bit store: codes, scales, the bf16 tail of the newest block, pooled
                keys, eviction scores, Gamma_e
  decode        one token's attention over an 8-bit store, over a selection of blocks or over all of them
  weights       the same attention (8-bit or bf16 store), adding each block's attention weight to a running total
  evict         the blocks with the largest accumulated weight moved into a store of smaller capacity

A unit is one (sequence, kv head) pair; a block is 64 tokens of a unit; the local block holds the newest token.
"""
import math

import torch

own = False

D, BLOCK, SUB = 128, 64, 16
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100  # blocks whose largest value is below this are stored as zeros


# ---- cases --------------------------------------------------------------------------------------

def _case(name, kind, fmt, B, Hq, Hkv, L, k_q=16, k_e=48, ragged=False, dense=False, keep=0, ck_bf16=False):
    c = dict(kind=kind, fmt=fmt, B=B, Hq=Hq, Hkv=Hkv, L=L, k_q=k_q, k_e=k_e, ragged=ragged, dense=dense, keep=keep,
             ck_bf16=ck_bf16)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # two short prompts of different length: the smallest prefill, launch latency counts
        _case("append-int8-short", "append", "int8", 2, 8, 2, 200, 4, 12, ragged=True),
        # a batch of 8 prompts of 16K, grouped heads
        _case("append-e4m3-16k", "append", "e4m3", 8, 16, 2, 16384),
        # a batch of 32 prompts of up to 32K of different lengths, bf16 pooled keys: the largest prefill of a layer
        _case("append-int8-32k", "append", "int8", 32, 16, 2, 32768, ragged=True, ck_bf16=True),
        # one layer of a 32K serving step, 65 of 512 blocks attended
        _case("sparse-int8-32k", "decode", "int8", 32, 16, 2, 32768),
        # one sequence, one query head per kv head, 8K: the smallest serving step
        _case("sparse-e4m3-mha-8k", "decode", "e4m3", 1, 16, 16, 8192),
        # full attention of one sequence just past a block border: latency
        _case("dense-int8-4k", "decode", "int8", 1, 16, 2, 4097, dense=True),
        # full attention of a ragged batch of up to 32K
        _case("dense-e4m3-32k", "decode", "e4m3", 32, 16, 2, 32768, ragged=True, dense=True),
        # a 32K serving step that also keeps the blocks' weights, bf16 store
        _case("sparse-weights-bf16-32k", "weights", "bf16", 32, 16, 2, 32768),
        # full attention with the weights over 8-bit blocks, 16K
        _case("dense-weights-int8-16k", "weights", "int8", 8, 16, 2, 16384, ragged=True, dense=True),
        # full attention with the weights of one short sequence, heads in threes
        _case("dense-weights-bf16-1k", "weights", "bf16", 1, 12, 4, 1000, dense=True),
        # after a 32K prompt: an eighth of the blocks kept, bf16 store
        _case("evict-bf16-32k", "evict", "bf16", 8, 16, 2, 32768, keep=64),
        # a full store cut to half, 8-bit blocks, ragged
        _case("evict-int8-16k", "evict", "int8", 32, 16, 2, 16384, ragged=True, keep=128),
    ]


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "weights", "evict"])
    fmt = rng.choice(["int8", "e4m3"] if kind in ("append", "decode") else ["bf16", "int8", "e4m3"])
    Hq, Hkv = rng.choice([(16, 2), (16, 16), (8, 2), (8, 8), (12, 4), (7, 1), (6, 2), (5, 1), (4, 4)])
    B = round(math.exp(rng.uniform(0.0, math.log(32.0))))
    most = min(32768, 64 * 24576 // (B * Hkv))
    L = max(1, round(math.exp(rng.uniform(0.0, math.log(most)))) if rng.random() < 0.3 else
            round(math.exp(rng.uniform(math.log(200.0), math.log(most)))))
    k_q, k_e = rng.choice([(16, 48), (8, 24), (32, 96), (4, 12), (0, 16), (5, 0), (32, 32)])
    keep = rng.randint(2, max(2, L // BLOCK)) if kind == "evict" else 0
    return _case(None, kind, fmt, B, Hq, Hkv, L, k_q, k_e, ragged=rng.random() < 0.5,
                 dense=kind in ("decode", "weights") and rng.random() < 0.5, keep=keep, ck_bf16=rng.random() < 0.3)


def _geo(c):
    units = c["B"] * c["Hkv"]
    max_ctx = (c["L"] + BLOCK - 1) // BLOCK * BLOCK + BLOCK
    return units, max_ctx, max_ctx // BLOCK


def _sink_recent(keep):
    return min(1, keep), min(1, max(keep - 1, 0))


# ---- inputs --------------------------------------------------------------------------------------

def _lens(c, seed):
    """Tokens of each sequence."""
    if not c["ragged"]:
        return [c["L"]] * c["B"]
    g = torch.Generator().manual_seed(seed * 7 + 1)
    f = torch.rand(c["B"], generator=g).tolist()
    lens = [max(1, round(c["L"] * (0.5 + 0.5 * x))) for x in f]
    lens[0] = c["L"]
    return lens


def _inputs(c, seed):
    units, max_ctx, nblk = _geo(c)
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = c["L"]
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    # keys have a few channels well above the others, values do not
    chan = torch.where(torch.rand(units, 1, D, generator=g, device="cuda") < 0.04, 4.0, 1.0)
    k = torch.empty(units, T, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for u0 in range(0, units, 8):
        n = min(8, units - u0)
        k[u0:u0 + n] = (rand(n, T, D) * chan[u0:u0 + n]).bfloat16()
        v[u0:u0 + n] = rand(n, T, D).bfloat16()
    e = 0.5 * rand(units, T)
    q = rand(c["B"], c["Hq"], D).bfloat16()
    lens = _lens(c, seed)
    len_b = torch.tensor(lens, dtype=torch.int32, device="cuda")
    len_u = len_b.repeat_interleave(c["Hkv"])
    local = (len_u.long() - 1) // BLOCK
    w0 = torch.rand(units, nblk, generator=g, device="cuda") * (torch.arange(nblk, device="cuda") <= local[:, None])
    if c["kind"] == "evict":
        w0 = (w0 * 64).floor() / 8  # sums of few steps: equal weights happen
    # a selection as the select step leaves it: up to k candidates in ascending order, then the local block
    k_all = c["k_q"] + c["k_e"]
    pri = torch.rand(units, nblk, generator=g, device="cuda") + 2.0 * (torch.arange(nblk, device="cuda") >= local[:, None])
    take = torch.sort(pri, dim=1).indices[:, :k_all] if k_all < nblk else torch.sort(pri, dim=1).indices
    take = torch.where(take < local[:, None], take, nblk)
    take = torch.sort(torch.cat([take, local[:, None]], 1), dim=1).values
    sel = torch.full((units, k_all + 1), -1, dtype=torch.int32, device="cuda")
    m = min(k_all + 1, take.shape[1])
    sel[:, :m] = torch.where(take[:, :m] < nblk, take[:, :m], -1).int()
    return dict(k=k, v=v, e=e, q=q, lens=lens, len_b=len_b, len_u=len_u, local=local, w0=w0, sel=sel,
                nsel=(sel >= 0).sum(1).int())


def _layer(c, max_ctx, weights=False):
    import block_sparse_offloadable_b200 as nosa
    cfg = nosa.make_config(c["B"], c["Hq"], c["Hkv"], c["k_q"], c["k_e"], max_ctx, ck_bf16=c["ck_bf16"],
                           kv_format=c["fmt"])
    lay = nosa.NosaLayer(cfg, weights=weights)
    for t in (lay.kv_store, lay.evict_logit, lay.ck, lay.blk_evict, lay.gamma_e):  # parts no token reaches: zeros
        t.zero_()
    return lay


def prepare(case, seed):
    c = case
    units, max_ctx, nblk = _geo(c)
    x = _inputs(c, seed)
    s = dict(c=c, x=x)
    lens_arg = x["len_b"] if c["ragged"] else None
    if own:
        s["layer"] = lay = _layer(c, max_ctx, weights=c["kind"] in ("weights", "evict"))
        s["lens"] = lens_arg
        s["T"] = c["L"]
        if c["kind"] != "append":
            lay.append(x["k"].view(torch.int16), x["v"].view(torch.int16), x["e"], c["L"],
                       lens_arg if c["L"] > 1 else None)
            lay.sel.copy_(x["sel"])
            lay.nsel.copy_(x["nsel"])
            s["out"] = torch.empty(c["B"], c["Hq"], D, dtype=torch.int16, device="cuda")
            x["k"] = x["v"] = None
        if c["kind"] == "evict":
            lay.weights.copy_(x["w0"])
            s["dst"] = _layer(c, (c["keep"] + 1) * BLOCK, weights=True)
    elif c["kind"] != "append":
        s["store"] = _plain_append(c, x, max_ctx)
        x["k"] = x["v"] = None
    return s


# ---- plain forms -----------------------------------------------------------------------------------

def _plain_quantise(x, fmt):
    """x [..., 64, 128] bf16 -> (codes, scale [...])."""
    xf = x.float()
    amax = xf.abs().amax((-1, -2))
    top = CODE_MAX[fmt]
    finite = torch.isfinite(amax)
    zero = amax < TINY
    scale = torch.where(finite, torch.where(zero, 0.0, amax / top), math.nan)
    inv = torch.where(finite & ~zero, top / amax, 0.0)[..., None, None]
    xf = torch.where(finite[..., None, None], xf, 0.0)
    if fmt == "int8":  # the product of 8 and 24 bits is exact in 64 bits: one rounding, ties to even
        return (xf.double() * inv.double()).round().to(torch.int8), scale
    return (xf * inv).clamp(-top, top).to(torch.float8_e4m3fn), scale


def _plain_append(c, x, max_ctx):
    units, T, nblk = x["k"].shape[0], c["L"], max_ctx // BLOCK
    dev = x["k"].device
    pos = torch.arange(max_ctx, device=dev)
    valid = pos[None, :] < x["len_u"][:, None]
    kb = torch.zeros(units, max_ctx, D, dtype=torch.bfloat16, device=dev)
    vb = torch.zeros_like(kb)
    kb[:, :T], vb[:, :T] = x["k"], x["v"]
    kb = torch.where(valid[..., None], kb, 0.0).view(units, nblk, BLOCK, D)
    vb = torch.where(valid[..., None], vb, 0.0).view(units, nblk, BLOCK, D)
    e = torch.zeros(units, max_ctx, device=dev)
    e[:, :T] = x["e"]
    e = torch.where(valid, e, 0.0)
    blk = torch.arange(nblk, device=dev)
    cand = blk[None, :] < x["local"][:, None]
    st = dict(e=e, seq_len=x["len_u"].clone())
    if c["fmt"] == "bf16":
        st["kv"] = torch.stack([kb, vb], 2)
    else:
        codes, scales = _plain_quantise(torch.stack([kb, vb], 2), c["fmt"])
        st["codes"] = torch.where(cand[..., None, None, None], codes.view(torch.uint8), 0).view(codes.dtype)
        st["scales"] = torch.where(cand[..., None], scales, 0.0)
        u = torch.arange(units, device=dev)
        st["tail"] = torch.stack([kb[u, x["local"]], vb[u, x["local"]]], 1)
    # pooled keys of whole sub-blocks, eviction scores of whole blocks
    sub_end = (torch.arange(max_ctx // SUB, device=dev) + 1) * SUB
    whole_sub = sub_end[None, :] <= x["len_u"][:, None]
    ck = kb.view(units, -1, SUB, D).double().mean(2)
    ck = torch.where(whole_sub[..., None], ck, 0.0)
    st["ck"] = ck.to(torch.bfloat16) if c["ck_bf16"] else ck.float()
    E = e.double().view(units, nblk, BLOCK // SUB, SUB).mean(-1).amax(-1)
    whole = (blk + 1)[None, :] * BLOCK <= x["len_u"][:, None]
    st["E"] = torch.where(whole, E, 0.0)
    # Gamma_e: the k_e candidates with the largest score, ties to the lower block, ascending
    k_e = c["k_e"]
    key = torch.where(cand, E, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :max(k_e, 1)]
    n = torch.clamp(x["local"], max=k_e)
    got = torch.where(torch.arange(order.shape[1], device=dev)[None, :] < n[:, None], order, nblk)
    got = torch.sort(got, dim=1).values
    ge = torch.zeros(units, max(k_e, 1), dtype=torch.int32, device=dev)
    ge[:, :got.shape[1]] = torch.where(got < nblk, got, 0).int()
    st["gamma_e"], st["gamma_n"] = ge, n.int()
    return st


def _plain_blocks(c, st, ids, x):
    """Keys and values [u][n][64][128] in 32 bits of blocks `ids` [u][n] (any block for negative ids)."""
    u = torch.arange(ids.shape[0], device=ids.device)[:, None]
    at = ids.clamp(min=0)
    if c["fmt"] == "bf16":
        kv = st["kv"][u, at].float()
        return kv[:, :, 0], kv[:, :, 1]
    kv = st["codes"].view(torch.uint8)[u, at].view(st["codes"].dtype).float() * st["scales"][u, at][..., None, None]
    kv = torch.where((ids == x["local"][:, None])[..., None, None, None], st["tail"].float()[:, None], kv)
    return kv[:, :, 0], kv[:, :, 1]


def _plain_attention(c, st, x, ids):
    """(out [B][Hq][D] bf16, weight of each of the blocks `ids` [u][n])."""
    units, n = ids.shape
    G = c["Hq"] // c["Hkv"]
    k, v = _plain_blocks(c, st, ids, x)
    pos = ids.clamp(min=0)[..., None] * BLOCK + torch.arange(BLOCK, device=ids.device)
    seen = (ids >= 0)[..., None] & (pos < x["len_u"].long()[:, None, None])
    u = torch.arange(units, device=ids.device)[:, None, None]
    e = torch.where(seen, st["e"][u, pos], -math.inf).view(units, 1, n * BLOCK)
    q = x["q"].float().view(units, G, D)
    z = torch.matmul(q, k.reshape(units, n * BLOCK, D).transpose(1, 2)) * D ** -0.5 + e
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v.reshape(units, n * BLOCK, D)).view(c["B"], c["Hq"], D).bfloat16()
    return out, p.view(units, G, n, BLOCK).sum((1, 3))


def _plain_ids(c, x, nblk):
    if not c["dense"]:
        return x["sel"].long()
    blk = torch.arange(nblk, device=x["sel"].device)[None, :]
    return torch.where(blk <= x["local"][:, None], blk, -1)


def _plain_weights(c, st, x, nblk):
    ids = _plain_ids(c, x, nblk)
    out, w = _plain_attention(c, st, x, ids)
    total = x["w0"].clone()
    total.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, w, 0.0))
    return out, total


def _plain_evict(c, st, x):
    units, nblk = x["w0"].shape
    dev = x["w0"].device
    keep, (sink, recent) = c["keep"], _sink_recent(c["keep"])
    blk = torch.arange(nblk, device=dev)[None, :]
    nb = x["local"][:, None]
    # rank of each candidate: protected ones first, then by weight, ties to the lower block
    key = torch.where((blk < sink) | (blk >= nb - recent), math.inf, x["w0"])
    key = torch.where(blk < nb, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, blk.expand_as(order))
    stay = ((rank < keep) & (blk < nb)) | (blk == nb)
    dst = torch.cumsum(stay, 1) - 1
    kept = torch.full((units, keep + 1), -1, dtype=torch.int64, device=dev)
    uu, bb = stay.nonzero(as_tuple=True)
    kept[uu, dst[uu, bb]] = bb
    n_old = x["len_u"].long()
    seq_len = (kept >= 0).sum(1) * BLOCK - ((x["local"] + 1) * BLOCK - n_old)
    ok = kept >= 0
    at = kept.clamp(min=0)
    u = torch.arange(units, device=dev)[:, None]
    pick = lambda t: torch.where(ok.view(units, keep + 1, *[1] * (t.dim() - 2)), t[u, at], torch.zeros((), dtype=t.dtype, device=dev))  # noqa: E731
    r = dict(kept=kept.int(), seq_len=seq_len.int(), weights=pick(x["w0"]), E=pick(st["E"]),
             e=pick(st["e"].view(units, nblk, BLOCK)).view(units, -1),
             ck=pick(st["ck"].view(units, nblk, BLOCK // SUB, D)).view(units, -1, D))
    if c["fmt"] == "bf16":
        r["kv"] = pick(st["kv"])
    else:
        r["codes"] = pick(st["codes"].view(torch.uint8)).view(st["codes"].dtype)
        r["scales"], r["tail"] = pick(st["scales"]), st["tail"].clone()
    # Gamma_e: its members that stay, renumbered
    old = st["gamma_e"].long()
    member = (torch.arange(old.shape[1], device=dev)[None, :] < st["gamma_n"][:, None]) & stay[u, old]
    slot = torch.cumsum(member, 1) - 1
    ge = torch.zeros_like(st["gamma_e"])
    uu, jj = member.nonzero(as_tuple=True)
    ge[uu, slot[uu, jj]] = dst[uu, old[uu, jj]].int()
    r["gamma_e"], r["gamma_n"] = ge, member.sum(1).int()
    return r


# ---- one pass ---------------------------------------------------------------------------------------

def _state_of(lay, c, nblk):
    """The layer's own buffers, shaped."""
    units = c["B"] * c["Hkv"]
    r = dict(e=lay.evict_logit.view(units, nblk * BLOCK), seq_len=lay.seq_len,
             ck=(lay.ck.view(torch.bfloat16) if c["ck_bf16"] else lay.ck).view(units, -1, D),
             E=lay.blk_evict.view(units, nblk), gamma_e=lay.gamma_e.view(units, -1), gamma_n=lay.gamma_n)
    if c["fmt"] == "bf16":
        r["kv"] = lay.kv_store.view(torch.bfloat16).view(units, nblk, 2, BLOCK, D)
    else:
        r["codes"], r["scales"], r["tail"] = lay.kv8_views()
    return r


def run(state):
    c, x = state["c"], state["x"]
    units, max_ctx, nblk = _geo(c)
    if own:
        import block_sparse_offloadable_b200 as nosa
        lay = state["layer"]
        if c["kind"] == "append":
            nosa.nosa_state_init(lay.cfg, lay.state)
            lay.append(x["k"].view(torch.int16), x["v"].view(torch.int16), x["e"], state["T"],
                       state["lens"] if state["T"] > 1 else None)
            return _state_of(lay, c, nblk)
        if c["kind"] == "evict":
            kept = lay.evict(state["dst"], c["keep"], *_sink_recent(c["keep"]))
            return dict(_state_of(state["dst"], c, c["keep"] + 1), kept=kept, weights=state["dst"].weights)
        out = state["out"]
        if c["kind"] == "weights":
            lay.weights.copy_(x["w0"])
            (lay.dense_decode_weights if c["dense"] else lay.sparse_decode_weights)(x["q"].view(torch.int16), out)
            return out.view(torch.bfloat16), lay.weights
        (lay.dense_decode if c["dense"] else lay.sparse_decode)(x["q"].view(torch.int16), out)
        return out.view(torch.bfloat16)
    if c["kind"] == "append":
        return _plain_append(c, x, max_ctx)
    if c["kind"] == "evict":
        return _plain_evict(c, state["store"], x)
    if c["kind"] == "weights":
        return _plain_weights(c, state["store"], x, nblk)
    return _plain_attention(c, state["store"], x, _plain_ids(c, x, nblk))[0]


def work(case):
    c = case
    units, max_ctx, nblk = _geo(c)
    share = 0.75 if c["ragged"] else 1.0  # ragged lengths are spread over the upper half
    L = max(1.0, c["L"] * share)
    nb = math.ceil(L / BLOCK) - 1  # candidates
    tail = L - nb * BLOCK
    G = c["Hq"] // c["Hkv"]
    half = 1 if c["fmt"] != "bf16" else 2
    block = 2 * BLOCK * D * half + (8 if half == 1 else 0)
    ck_row = D * (2 if c["ck_bf16"] else 4)
    if c["kind"] == "append":
        b = L * (4 * D + 4) + nb * block + tail * 4 * D + 4 * L + L // SUB * ck_row + L // BLOCK * 8
        return dict(bytes=units * b, flops=units * L * 2 * D * 3)
    if c["kind"] == "evict":
        n = min(c["keep"], nb)
        b = 2 * (n * (block + BLOCK * 4 + 4 * ck_row + 12) + tail * (4 * D + 4)) + nb * 4
        return dict(bytes=units * b, flops=units * nb)
    n = nb if c["dense"] else min(nb, c["k_q"] + c["k_e"])
    b = n * (block + BLOCK * 4) + tail * (4 * D + 4) + G * D * 4
    if c["kind"] == "weights":
        b += 8 * (n + 1)
    return dict(bytes=units * b, flops=units * (n * BLOCK + tail) * G * D * 4)


# ---- 64 bits -----------------------------------------------------------------------------------------

def _exact_block(t, fmt):
    """The values that a whole block [64][128] stands for in the store, and its scale."""
    if fmt == "bf16":
        return t.double(), None
    top = CODE_MAX[fmt]
    big = t.abs().max().float()
    if not bool(torch.isfinite(big)):
        return torch.full_like(t, math.nan, dtype=torch.float64), big * math.nan
    if float(big) < TINY:
        return torch.zeros_like(t, dtype=torch.float64), big * 0
    s, r = big / top, top / big
    y = t.double() * r.double()
    if fmt == "int8":
        y = torch.round(y)
    else:
        y = y.float().double()
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(y.abs().clamp(min=1e-30))), min=-6.0) - 3.0)
        y = (torch.round(y / step) * step).clamp(-top, top)
    return y, s


def _exact_unit(c, x, u):
    """Codes' values and scales of unit u's candidates, for keys and for values: [2][nb][64][128], [2][nb]."""
    nb = int(x["local"][u])
    vals, scales = [], []
    for t in (x["k"][u], x["v"][u]):
        got = [_exact_block(t[b * BLOCK:(b + 1) * BLOCK], c["fmt"]) for b in range(nb)]
        vals.append([y for y, _ in got])
        scales.append([s for _, s in got])
    return nb, vals, scales


def exact(case, seed):
    c = case
    units, max_ctx, nblk = _geo(c)
    if c["kind"] == "evict":  # moves values, computes none
        return None
    x = _inputs(c, seed)
    if c["kind"] == "append":
        dev = x["k"].device
        z = dict(e=torch.zeros(units, max_ctx, dtype=torch.float64, device=dev),
                 ck=torch.zeros(units, max_ctx // SUB, D, dtype=torch.float64, device=dev),
                 E=torch.zeros(units, nblk, dtype=torch.float64, device=dev),
                 scales=torch.zeros(units, nblk, 2, dtype=torch.float64, device=dev),
                 tail=torch.zeros(units, 2, BLOCK, D, dtype=torch.float64, device=dev),
                 codes=None, gamma_e=None, gamma_n=None, seq_len=None)
        if c["fmt"] == "e4m3":
            z["codes"] = torch.zeros(units, nblk, 2, BLOCK, D, dtype=torch.float64, device=dev)
        for u in range(units):
            n = int(x["len_u"][u])
            nb, vals, scales = _exact_unit(c, x, u)
            z["e"][u, :n] = x["e"][u, :n].double()
            subs = n // SUB
            z["ck"][u, :subs] = x["k"][u, :subs * SUB].double().view(subs, SUB, D).sum(1) / SUB
            whole = n // BLOCK
            z["E"][u, :whole] = (x["e"][u, :whole * BLOCK].double().view(whole, BLOCK // SUB, SUB).sum(-1) / SUB).max(-1).values \
                if whole else z["E"][u, :0]
            for i, t in enumerate((x["k"], x["v"])):
                for b in range(nb):
                    z["scales"][u, b, i] = scales[i][b].double()
                    if z["codes"] is not None:
                        z["codes"][u, b, i] = vals[i][b]
                z["tail"][u, i, :n - nb * BLOCK] = t[u, nb * BLOCK:n].double()
        return z
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(units, G, D, dtype=torch.float64, device=x["q"].device)
    total = x["w0"].double()
    q = x["q"].double().view(units, G, D)
    for u in range(units):
        n = int(x["len_u"][u])
        nb = int(x["local"][u])
        ids = list(range(nb + 1)) if c["dense"] else [b for b in x["sel"][u].tolist() if b >= 0]
        k, v, e = [], [], []
        for b in ids:
            rows = slice(b * BLOCK, min((b + 1) * BLOCK, n))
            for t, to in ((x["k"], k), (x["v"], v)):
                y, s = (t[u, rows].double(), None) if b == nb else _exact_block(t[u, rows], c["fmt"])
                to.append(y if s is None else y * s.double())
            e.append(x["e"][u, rows].double())
        k, v, sizes = torch.cat(k), torch.cat(v), [len(t) for t in e]
        z = q[u] @ k.T / math.sqrt(D) + torch.cat(e)
        p = torch.softmax(z, dim=-1)
        out[u] = p @ v
        if c["kind"] == "weights":
            w = torch.stack([t.sum() for t in p.split(sizes, dim=1)])
            total[u, torch.tensor(ids, device=w.device)] += w
    out = out.view(c["B"], c["Hq"], D)
    return (out, total) if c["kind"] == "weights" else out
