"""The operators around a compact KV cache that are measured: their cases, their
plain forms in elementary torch operations, and the calls a user makes.

Four operators, used together when a prompt is taken in and then decoded:

* ``prefill``: attention of a prompt's queries under the cache's eviction rule
  (causal; a token is visible while it is in the recent window, afterwards only
  if it is kept), with the log of each row's softmax denominator.
* ``scores``: the attention weight every token collects over those queries,
  summed over the query heads of its kv head (the denominators are inputs).
* ``select``: keep bits from such scores: the recent window, and the highest
  scores before it up to a budget per (sequence, kv head).
* ``sparse``: single-token decode over the compact cache that reads only the
  store blocks whose key bounds promise the largest scores.

Shapes are those of this repository's workloads (4/2 heads of 64, 32/8 heads of
64 and 128, context 512 to 32768, windows 16 and 256, their keep rates).
"""
import math

import torch

own = False
DEV = "cuda:0"
BLOCK = 64          # slots of a store block


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest workload's whole prompt (512 tokens, 4/2 heads of 64): latency
        dict(name="prefill_tiny", op="prefill", B=1, T=512, ragged=0.0, nq=0, Hq=4, Hkv=2, D=64,
             W=16, lo=0.25, hi=0.25, keep=True),
        # a whole 8K prompt on 32/8 heads of 64 with learned keep bits
        dict(name="prefill_d64_8k_evict", op="prefill", B=1, T=8192, ragged=0.0, nq=0, Hq=32,
             Hkv=8, D=64, W=256, lo=0.05, hi=0.30, keep=True),
        # a whole 8K prompt on 32/8 heads of 128, nothing evicted yet: the largest
        dict(name="prefill_d128_8k_dense", op="prefill", B=1, T=8192, ragged=0.0, nq=0, Hq=32,
             Hkv=8, D=128, W=256, lo=1.0, hi=1.0, keep=False),
        # five draft tokens per sequence verified against ragged contexts (few rows, long keys)
        dict(name="prefill_d128_verify5", op="prefill", B=8, T=8197, ragged=0.5, nq=5, Hq=32,
             Hkv=8, D=128, W=256, lo=0.06, hi=0.20, keep=True),
        # weights collected over a whole 8K prompt, 32/8 heads of 64
        dict(name="scores_d64_8k_all", op="scores", B=1, T=8192, ragged=0.0, nq=0, Hq=32, Hkv=8,
             D=64, W=256, lo=1.0, hi=1.0, keep=False),
        # weights collected over the last 64 queries of eight ragged prompts, 32/8 heads of 128
        dict(name="scores_d128_last64", op="scores", B=8, T=8192, ragged=0.5, nq=64, Hq=32, Hkv=8,
             D=128, W=256, lo=1.0, hi=1.0, keep=False),
        # weights under keep bits on the smallest workload
        dict(name="scores_tiny_evict", op="scores", B=1, T=512, ragged=0.0, nq=0, Hq=4, Hkv=2,
             D=64, W=16, lo=0.25, hi=0.25, keep=True),
        # keep bits of the smallest workload: latency
        dict(name="select_tiny", op="select", B=1, T=512, ragged=0.0, Hkv=2, W=16, part=0.25),
        # keep bits of 32 ragged prompts of up to 32K tokens
        dict(name="select_b32_32k", op="select", B=32, T=32768, ragged=0.9, Hkv=8, W=256,
             part=0.14),
        # one sequence, 8K context, 32/8 heads of 64, bf16: 4 of about 22 blocks per head
        dict(name="sparse_d64_8k_b1", op="sparse", B=1, T=8192, ragged=0.0, Hq=32, Hkv=8, D=64,
             W=256, lo=0.05, hi=0.30, blocks=4, kv="bf16"),
        # eight ragged contexts of up to 32K, 32/8 heads of 128, E4M3 with a scale per block
        dict(name="sparse_d128_32k_fp8_block", op="sparse", B=8, T=32768, ragged=0.6, Hq=32,
             Hkv=8, D=128, W=256, lo=0.03, hi=0.25, blocks=16, kv="fp8_e4m3_block"),
        # eight 16K contexts with every slot kept, 32/8 heads of 128, bf16: 32 of 252 blocks
        dict(name="sparse_d128_16k_keepall", op="sparse", B=8, T=16384, ragged=0.2, Hq=32, Hkv=8,
             D=128, W=256, lo=1.0, hi=1.0, blocks=32, kv="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "scores", "select", "sparse"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    c = dict(op=op, B=rng.choice([1, 2, 3, 8]), ragged=rng.choice([0.0, 0.3, 0.9]), Hkv=hkv,
             W=rng.choice([0, 1, 16, 100, 256]))
    if op in ("prefill", "scores"):
        c.update(Hq=hkv * g, D=rng.choice([64, 128]), keep=rng.random() < 0.6)
        few = rng.random() < 0.5
        c["T"] = _log_uniform(rng, 2, 16384 if few else 8192)
        c["nq"] = min(c["T"], rng.choice([1, 2, 7, 33, 64, 200])) if few else 0
        # at most the largest listed case's pairs of query rows and keys
        while c["B"] * c["Hq"] * (c["nq"] or c["T"]) * c["T"] > 32 * 8192 * 8192:
            c["T"] = max(1, c["T"] * 2 // 3)
            c["nq"] = min(c["nq"], c["T"])
        c.update(lo=0.05, hi=0.30) if c["keep"] else c.update(lo=1.0, hi=1.0)
    elif op == "select":
        c.update(B=rng.choice([1, 2, 8, 32]), T=c["W"] + _log_uniform(rng, 64, 32512),
                 part=rng.choice([0.05, 0.14, 0.3, 0.6]))
    else:
        c.update(Hq=hkv * g, D=rng.choice([64, 128]), T=_log_uniform(rng, 1, 16384),
                 blocks=rng.choice([1, 2, 5, 16, 40]),
                 kv=rng.choice(["bf16", "fp8_e4m3", "fp8_e4m3_block"]))
        lo, hi = rng.choice([(0.05, 0.30), (1.0, 1.0)])
        c.update(lo=lo, hi=hi)
    return c


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Tokens of each sequence: the first has T, the others down to (1 - ragged) T."""
    B, T = case["B"], case["T"]
    return [max(1, round(T * (1.0 - case["ragged"] * b / B))) for b in range(B)]


def _query_counts(case):
    return [min(n, case["nq"]) if case["nq"] else n for n in _lengths(case)]


def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 16 + tag)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _keep_bits(case, seed):
    """uint8 [B][T][Hkv], a keep rate of its own for every (sequence, kv head)."""
    g = _gen(seed, 4)
    rate = torch.rand((case["B"], 1, case["Hkv"]), generator=g, device=DEV)
    rate = case["lo"] + (case["hi"] - case["lo"]) * rate
    u = torch.rand((case["B"], case["T"], case["Hkv"]), generator=g, device=DEV)
    return (u < rate).to(torch.uint8)


def _key_values(case, seed):
    """K and V bf16 [B][T][Hkv][D], N(0, 1) times a channel scale of U[0.5, 2]."""
    shape = (case["B"], case["T"], case["Hkv"], case["D"])
    out = []
    for tag in (1, 2):
        g = _gen(seed, tag)
        cs = torch.rand(shape[2:], generator=g, device=DEV) * 1.5 + 0.5
        out.append((_randn(shape, g) * cs).to(torch.bfloat16))
    return out


def prepare(case, seed):
    op, B, T = case["op"], case["B"], case["T"]
    n = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    st = {"case": case, "op": op, "n": n, "cache": None}
    if op == "select":
        st["scores"] = _randn((B, case["Hkv"], T), _gen(seed, 1)).exp_()
        # equal weights occur in earnest: a third of the tokens shares few values
        coarse = torch.round(st["scores"][:, :, ::3] * 4) / 4
        st["scores"][:, :, ::3] = coarse
        st["budget"] = torch.round(n.float()[:, None] * case["part"] *
                                   torch.linspace(0.5, 1.5, case["Hkv"], device=DEV)
                                   ).to(torch.int32).contiguous()
        st["keep"] = torch.zeros((B, T, case["Hkv"]), dtype=torch.uint8, device=DEV)
        if own:   # the handle whose window and shape the calls go by
            st["cache"] = _cache(case, case["Hkv"], 64, "bf16", 1)
        return st
    if op == "sparse":
        return _prepare_sparse(st, case, seed)
    st["k"], v = _key_values(case, seed)
    st["keep"] = _keep_bits(case, seed) if case["keep"] else None
    max_q = case["nq"] or T
    st["nq"] = torch.tensor(_query_counts(case), dtype=torch.int32, device=DEV)
    st["q"] = _randn((B, max_q, case["Hq"], case["D"]), _gen(seed, 3)).to(torch.bfloat16)
    if op == "prefill":
        st["v"] = v
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(st["q"].shape[:3], dtype=torch.float32, device=DEV)
    else:
        st["lse"] = _denominators(st)
        st["scores"] = torch.zeros((B, case["Hkv"], T), dtype=torch.float32, device=DEV)
    if own:   # the handle, and the workspace a program keeps for these calls
        import compressed_decode_attention_fdms_b200 as fd
        st["cache"] = _cache(case, case["Hq"], case["D"], "bf16", 1)
        st["ws"] = torch.empty(max(1, fd.fdms_prefill_workspace(st["cache"], B, T, max_q)),
                               dtype=torch.uint8, device=DEV)
    return st


def _cache(case, hq, d, kv, num_blocks):
    import compressed_decode_attention_fdms_b200 as fd
    return fd.fdms_cache_create(fd.make_config(1, case["B"], hq, case["Hkv"], d, case["W"], 1,
                                               case["T"], num_blocks, kv))


def _prepare_sparse(st, case, seed):
    """A cache that has taken in the prompt; for the plain form, what it holds."""
    B, T, H, D, W = case["B"], case["T"], case["Hkv"], case["D"], case["W"]
    k, v = _key_values(case, seed)
    keep = _keep_bits(case, seed)
    st["q"] = _randn((B, case["Hq"], D), _gen(seed, 3)).to(torch.bfloat16)
    st["out"] = torch.empty_like(st["q"])
    st["blocks"] = torch.empty((B, H, case["blocks"]), dtype=torch.int32, device=DEV)
    if own:
        return _fill(st, case, seed, k, v, keep)
    n = st["n"].long()[:, None, None]
    pos = torch.arange(T, device=DEV)[None, :, None]
    inside = pos < n
    # the call's maxima set an E4M3 cache's scales, over every token it brings
    live = inside[..., None]
    keys, vals = k.float() * live, v.float() * live
    recent = inside & (pos >= n - W)
    stored = inside & ~recent & (keep > 0)
    order = torch.argsort((~stored).to(torch.uint8), dim=1, stable=True)   # survivors first
    length = stored.sum(1)                                                 # [B][H]
    room = max(1, int(length.max()))
    pick = order[:, :room, :, None].expand(-1, -1, -1, D)
    on = torch.arange(room, device=DEV)[None, None, :] < length[:, :, None]
    st["length"] = length
    scaled = {}
    for name, x in (("k", keys), ("v", vals)):
        s = torch.gather(x, 1, pick).permute(0, 2, 1, 3) * on[..., None]   # [B][H][room][D]
        r = x * recent[..., None]
        r = r.permute(0, 2, 1, 3)
        if case["kv"] == "fp8_e4m3":
            sc = torch.clamp(x.abs().amax((1, 3)), min=2.0 ** -126) / 448.0   # [B][H]
            s = _e4m3(s, sc[:, :, None, None])
            r = _e4m3(r, sc[:, :, None, None])
        elif case["kv"] == "fp8_e4m3_block":
            full = (length // BLOCK * BLOCK)[:, :, None, None]
            pad = -room % BLOCK
            blocks = torch.nn.functional.pad(s, (0, 0, 0, pad)).unflatten(2, (-1, BLOCK))
            sc = torch.clamp(blocks.abs().amax((3, 4), keepdim=True), min=2.0 ** -126) / 448.0
            sealed = _e4m3(blocks, sc).flatten(2, 3)[:, :, :room]
            at = torch.arange(room, device=DEV)[None, None, :, None]
            s = torch.where(at < full, sealed, s)
        scaled[name] = s
        st["store_" + name] = s
        tail = max(1, min(W, T))
        # each sequence's last min(W, n) tokens, at its end
        at = torch.clamp(n[:, :, 0] - tail + torch.arange(tail, device=DEV)[None, :], min=0)
        st["ring_" + name] = torch.gather(r, 2, at[:, None, :, None].expand(-1, H, -1, D))
    tail = st["ring_k"].shape[2]
    place = n[:, :, 0] - tail + torch.arange(tail, device=DEV)[None, :]
    st["ring_on"] = (place >= 0) & (place >= n[:, :, 0] - W)                # [B][tail]
    # the bounds of the full blocks' keys, an index that the cache keeps beside them
    nb = room // BLOCK
    kb = scaled["k"][:, :, :nb * BLOCK].unflatten(2, (nb, BLOCK)) if nb else \
        scaled["k"][:, :, :0].reshape(B, H, 0, BLOCK, D)
    st["kmin"], st["kmax"] = kb.amin(3), kb.amax(3)
    return st


def _fill(st, case, seed, k, v, keep):
    """The calls' cache, with what the plain form's store holds.

    A division of a GPU tensor by a number is a product with the number's rounded
    reciprocal, so that the plain form's E4M3 scales are one unit off the cache's
    quotients for some maxima, and a code next to a border can be another one. The
    calls are measured on the plain form's values all the same: a cache with a scale
    per head is given the scales; to one with a scale per block the rows of its full
    blocks come as the values their codes stand for (in bf16, which is 2^-9 of the
    value at most: they round to the same codes again)."""
    global own
    import compressed_decode_attention_fdms_b200 as fd
    B, T, H, D = k.shape
    n, scale = st["n"].long()[:, None, None], None
    pos = torch.arange(T, device=DEV)[None, :, None]
    if case["kv"] == "fp8_e4m3":
        scale = torch.stack([torch.clamp((x.float() * (pos < n)[..., None]).abs().amax((1, 3)),
                                         min=2.0 ** -126) / 448.0 for x in (k, v)], -1)
    elif case["kv"] == "fp8_e4m3_block":
        own = False
        try:
            held = _prepare_sparse({"n": st["n"]}, case, seed)
        finally:
            own = True
        room = held["store_k"].shape[2]
        stored = (pos < n - case["W"]) & (keep > 0)
        order = torch.argsort((~stored).to(torch.uint8), dim=1, stable=True)
        pick = order[:, :room, :, None].expand(-1, -1, -1, D)
        full = torch.arange(room, device=DEV)[:, None] < (held["length"] // BLOCK * BLOCK)[:, None]
        both = []
        for x, name in ((k, "k"), (v, "v")):
            rows = held["store_" + name].permute(0, 2, 1, 3).to(torch.bfloat16)
            rows = torch.where(full[..., None], rows, torch.gather(x, 1, pick))
            both.append(x.scatter(1, pick, rows))
        k, v = both
    c = _cache(case, case["Hq"], D, case["kv"], 0)
    fd.fdms_append_evict(c, 0, B, st["n"], T, k, v, keep, kv_scale=scale)
    fd.fdms_bounds_create(c)
    st["cache"] = c
    return st


def _e4m3(x, scale):
    """The value an E4M3 code stands for: x / scale rounded to E4M3, times the scale (in 64 bits)."""
    code = torch.clamp(x / scale, -448.0, 448.0).to(torch.float8_e4m3fn)
    return code.double() * scale.double()


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _run_own(st)
    return {"prefill": _plain_prefill, "scores": _plain_scores, "select": _plain_select,
            "sparse": _plain_sparse}[st["op"]](st)


def _run_own(st):
    import compressed_decode_attention_fdms_b200 as fd
    c, case, op = st["cache"], st["case"], st["op"]
    B, T = case["B"], case["T"]
    if op == "prefill":
        fd.fdms_prefill_attn(c, B, st["n"], T, st["q"], st["k"], st["v"], st["out"],
                             keep=st["keep"], nq=st["nq"], lse=st["lse"], workspace=st["ws"])
        return st["out"], st["lse"]
    if op == "scores":
        fd.fdms_prefill_scores(c, B, st["n"], T, st["q"], st["k"], st["lse"], st["scores"],
                               keep=st["keep"], nq=st["nq"], workspace=st["ws"])
        return st["scores"]
    if op == "select":
        fd.fdms_select_keep(c, B, st["n"], T, st["scores"], st["budget"], st["keep"])
        return st["keep"]
    fd.fdms_decode_attn_sparse(c, 0, B, case["blocks"], st["q"], st["out"],
                               blocks=st["blocks"])
    return st["out"], st["blocks"]


def _positions(st):
    """Query positions [B][max_q] (n - nq + t) and which of them exist."""
    t = torch.arange(st["q"].shape[1], device=DEV)[None, :]
    i = (st["n"] - st["nq"])[:, None] + t
    return i, t < st["nq"][:, None]


def _logits(st):
    """Masked scores [B][Hkv][G][max_q][T] in 32 bits, -inf where a token is not seen."""
    q, k, W = st["q"], st["k"], st["case"]["W"]
    B, Q, Hq, D = q.shape
    H = k.shape[2]
    qg = q.float().unflatten(2, (H, Hq // H)).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qg.reshape(B, H, -1, D), k.float().permute(0, 2, 3, 1))
    s = s.reshape(B, H, Hq // H, Q, -1)
    i, real = _positions(st)
    j = torch.arange(k.shape[1], device=DEV)
    seen = (j <= i[..., None]) & real[..., None]                              # [B][Q][T]
    seen = seen[:, None]
    if st["keep"] is not None:
        kept = (st["keep"] > 0).permute(0, 2, 1)[:, :, None, :]               # [B][H][1][T]
        seen = seen & (kept | (j > i[:, None, :, None] - W))
    return s.mul_(1.0 / math.sqrt(D)).masked_fill_(~seen[:, :, None], -math.inf)


def _denominators(st):
    """log sum exp of each query row, float [B][max_q][Hq]."""
    lse = torch.logsumexp(_logits(st).flatten(1, 2), -1)
    return lse.permute(0, 2, 1).contiguous()


def _plain_prefill(st):
    s = _logits(st)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    B, H, G, Q, T = p.shape
    v = st["v"].float().permute(0, 2, 1, 3)                                   # [B][H][T][D]
    o = torch.matmul(p.reshape(B, H, G * Q, T), v).reshape(B, H, G, Q, -1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log())[..., 0]
    _, real = _positions(st)
    lse = lse.permute(0, 3, 1, 2).flatten(2).masked_fill(~real[..., None], 0.0)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16), lse


def _plain_scores(st):
    s = _logits(st)
    B, H, G, Q, T = s.shape
    lse = st["lse"].permute(0, 2, 1).reshape(B, H, G, Q, 1)
    # rows that see nothing (or do not exist) add nothing
    w = s.sub_(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)).exp_()
    return w.sum((2, 3))


def _plain_select(st):
    x, n, W = st["scores"], st["n"], st["case"]["W"]
    j = torch.arange(x.shape[2], device=DEV)[None, None, :]
    end = n[:, None, None]
    recent = (j >= end - W) & (j < end)
    ranked = torch.where(j < end - W, x, torch.full_like(x, -math.inf))
    order = torch.argsort(ranked, dim=2, descending=True, stable=True)
    chosen = torch.zeros_like(x, dtype=torch.bool)
    chosen.scatter_(2, order, j.expand_as(order) < st["budget"][:, :, None])
    keep = (chosen & (j < end - W)) | recent
    return keep.permute(0, 2, 1).to(torch.uint8).contiguous()


def _plain_sparse(st):
    case, q = st["case"], st["q"]
    B, Hq, D = q.shape
    H = case["Hkv"]
    G = Hq // H
    qd = q.double().reshape(B, H, G, 1, D)
    # a block's bound: no key of it can have a larger product with the query
    u = torch.maximum(qd * st["kmin"].double()[:, :, None], qd * st["kmax"].double()[:, :, None])
    u = u.sum(-1).amax(2)                                                     # [B][H][nb]
    nb = u.shape[2]
    full = (st["length"] // BLOCK)[:, :, None]
    at = torch.arange(nb, device=DEV)[None, None, :]
    order = torch.argsort(u.masked_fill(at >= full, -math.inf), dim=2, descending=True,
                          stable=True)
    chosen = torch.zeros_like(u, dtype=torch.bool)
    chosen.scatter_(2, order, at.expand_as(order) < case["blocks"])
    chosen &= at < full
    # the chosen blocks in order, -1 after them
    ids, _ = torch.where(chosen, at, nb).sort(2)
    ids = torch.nn.functional.pad(ids, (0, max(0, case["blocks"] - nb)), value=nb)
    ids = ids[:, :, :case["blocks"]]
    ids = torch.where(ids < nb, ids, -1).to(torch.int32)
    room = st["store_k"].shape[2]
    slot = torch.arange(room, device=DEV)[None, None, :]
    on = (slot >= full * BLOCK) & (slot < st["length"][:, :, None])           # the partly filled block
    on[:, :, :nb * BLOCK] |= chosen.repeat_interleave(BLOCK, 2)
    on = torch.cat([on, st["ring_on"][:, None, :].expand(-1, H, -1)], 2)
    k = torch.cat([st["store_k"], st["ring_k"]], 2).float()
    v = torch.cat([st["store_v"], st["ring_v"]], 2).float()
    s = torch.matmul(q.float().reshape(B, H, G, D), k.transpose(2, 3)) / math.sqrt(D)
    s = s.masked_fill(~on[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.reshape(B, Hq, D).to(torch.bfloat16), ids


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    keep_own, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep_own
    op = case["op"]
    if op == "select":
        return None                       # whole values: the plain form is exact
    if op == "sparse":
        return _exact_sparse(st)
    B, Q, Hq, D = st["q"].shape
    T, H, W = case["T"], case["Hkv"], case["W"]
    out = torch.zeros((B, Q, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Q, Hq), dtype=torch.float64, device=DEV)
    sums = torch.zeros((B, H, T), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // T)         # query rows at a time
    for b in range(B):
        n, nq = int(st["n"][b]), int(st["nq"][b])
        for h in range(Hq):
            kh = h // (Hq // H)
            keys = st["k"][b, :n, kh].double()
            for t0 in range(0, nq, step):
                t1 = min(nq, t0 + step)
                i = torch.arange(n - nq + t0, n - nq + t1, device=DEV)[:, None]
                j = torch.arange(n, device=DEV)[None, :]
                hidden = j > i
                if st["keep"] is not None:
                    hidden |= (j <= i - W) & (st["keep"][b, :n, kh] == 0)[None, :]
                s = (st["q"][b, t0:t1, h].double() @ keys.T) / D ** 0.5
                s[hidden] = -math.inf
                if op == "scores":
                    r = st["lse"][b, t0:t1, h].double()[:, None]
                    w = torch.exp(s - r)
                    w[hidden] = 0.0
                    sums[b, kh, :n] += w.sum(0)
                else:
                    z = torch.logsumexp(s, 1)
                    lse[b, t0:t1, h] = z
                    w = torch.exp(s - z[:, None])
                    w[hidden] = 0.0
                    out[b, t0:t1, h] = w @ st["v"][b, :n, kh].double()
    return sums if op == "scores" else (out, lse)


def _exact_sparse(st):
    case, q = st["case"], st["q"].double()
    B, Hq, D = q.shape
    H = case["Hkv"]
    G = Hq // H
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        ring = st["ring_on"][b]
        for h in range(H):
            L = int(st["length"][b, h])
            nb = L // BLOCK
            k, v = st["store_k"][b, h, :L].double(), st["store_v"][b, h, :L].double()
            qs = q[b, h * G:(h + 1) * G]
            kb = k[:nb * BLOCK].reshape(nb, BLOCK, D)
            best = torch.where(qs[:, None, :] > 0, kb.amax(1), kb.amin(1)) if nb else \
                k.new_zeros((G, 0, D))
            bound = (best * qs[:, None, :]).sum(-1).amax(0).tolist()
            take = sorted(sorted(range(nb), key=lambda x: (-bound[x], x))[:case["blocks"]])
            rows = [torch.arange(x * BLOCK, (x + 1) * BLOCK, device=DEV) for x in take]
            rows = torch.cat(rows + [torch.arange(nb * BLOCK, L, device=DEV)])
            kk = torch.cat([k[rows], st["ring_k"][b, h][ring].double()])
            vv = torch.cat([v[rows], st["ring_v"][b, h][ring].double()])
            if len(kk):
                out[b, h * G:(h + 1) * G] = torch.softmax(qs @ kk.T / D ** 0.5, 1) @ vv
    return out, None


# ------------------------------------------------------------------ the least work
def work(case):
    op, H = case["op"], case["Hkv"]
    lens = _lengths(case)
    if op == "select":
        return {"bytes": float(sum(lens) * H * (4 + 1) + case["B"] * H * 4), "flops": 0.0}
    rate, D, Hq, W = (case["lo"] + case["hi"]) / 2, case["D"], case["Hq"], case["W"]
    if op == "sparse":
        kb = 2 if case["kv"] == "bf16" else 1
        ring_b = 1 if case["kv"] == "fp8_e4m3" else 2
        total = flops = 0.0
        for n in lens:
            kept = rate * max(0, n - W)
            full = kept // BLOCK
            sel = min(full, case["blocks"])
            part, ring = kept - full * BLOCK, min(n, W)
            rows = sel * BLOCK + part + ring
            part_b = 2 if case["kv"] == "fp8_e4m3_block" else kb
            total += H * 2 * D * (sel * BLOCK * kb + part * part_b + ring * ring_b)
            if full > sel:
                total += H * full * 2 * D * 2        # the bounds, 16 bits each
                flops += Hq * full * 3 * D
            flops += Hq * rows * 4 * D
        total += case["B"] * (2 * Hq * D * 2 + H * case["blocks"] * 4)
        return {"bytes": total, "flops": flops}
    pairs = rows = 0.0
    for n, nq in zip(lens, _query_counts(case)):
        i = torch.arange(n - nq + 1, n + 1, dtype=torch.float64)     # tokens up to each query
        near = torch.clamp(i, max=float(W))
        pairs += float((near + rate * (i - near)).sum()) if case["keep"] else float(i.sum())
        rows += nq
    tokens = float(sum(lens))
    byt = rows * Hq * (D * 2 + 4) + tokens * H * D * 2 + (tokens * H if case["keep"] else 0)
    if op == "prefill":
        return {"bytes": byt + rows * Hq * D * 2 + tokens * H * D * 2, "flops": pairs * Hq * 4 * D}
    return {"bytes": byt + tokens * H * 4, "flops": pairs * Hq * 2 * D}
