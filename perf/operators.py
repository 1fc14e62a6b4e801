"""Cases of the 8-bit latent cache and of the eviction by attention weight.

Each case is one call of an operator of the framework (``own`` true) or the same
mathematics in elementary torch operations (``own`` false):

* ``append``      new tokens into an 8-bit cache (RMSNorm, RoPE, block exponents, e4m3 codes)
* ``quantize``    windows of a bf16 / f32 latent cache into 8 bits
* ``dequantize``  and back
* ``attend``      decode attention over the 8-bit cache (dense, causal verify, selected positions)
* ``weights``     accumulated attention weight of every cached key (bf16, f32 or 8-bit cache)
* ``evict``       choice of the tokens to keep and in-place compaction of the cache

An 8-bit cache holds the latent as e4m3 codes and one exponent byte ``e`` (value
``2^(e - 127)``) for each ``block`` consecutive buffer rows; the rope key stays in
the query's type.
"""
import math

import torch

own = False

DEV = "cuda"
RANK, ROPE = 512, 64
THETA, EPS = 10000.0, 1e-6
E_MIN, E_MAX = 64, 134
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode step
        dict(name="append one token", op="append", type="bf16", batch=1, t_max=4096, lo=4000, s_new=1, block=1),
        # a prompt chunk for every row of a batch, at lengths that end inside a block
        dict(name="append prompt chunk", op="append", type="bf16", batch=8, t_max=16384, lo=1, s_new=2048, block=64),
        # a prefilled bf16 cache of a ragged batch moved into 8 bits
        dict(name="quantize ragged batch", op="quantize", type="bf16", batch=32, t_max=8192, lo=1, block=16),
        # an 8-bit prefix handed back to the reconstructed prefill, exponent per token, odd length
        dict(name="dequantize prefix", op="dequantize", type="bf16", batch=3, t_max=8191, lo=8191, block=1),
        # one sequence, one token
        dict(name="attend one row", op="attend", type="bf16", batch=1, t_max=4096, lo=4096, s_q=1, heads=128, block=64,
             top_k=0),
        # a ragged serving batch, 1k to 32k tokens
        dict(name="attend ragged batch", op="attend", type="bf16", batch=32, t_max=32768, lo=1024, s_q=1, heads=128,
             block=16, top_k=0),
        # causal verify of four drafted tokens per row
        dict(name="attend verify", op="attend", type="bf16", batch=8, t_max=65536, lo=65536, s_q=4, heads=128, block=64,
             top_k=0),
        # 2048 selected positions of a long cache, exponent per token
        dict(name="attend selected", op="attend", type="bf16", batch=8, t_max=131072, lo=131072, s_q=1, heads=128,
             block=1, top_k=2048),
        # weights of a ragged batch over the bf16 cache
        dict(name="weights ragged batch", op="weights", type="bf16", batch=32, t_max=32768, lo=1024, s_q=1, heads=128,
             block=0),
        # weights of one long row over the 8-bit cache, 64 heads, two tokens
        dict(name="weights one 8-bit row", op="weights", type="bf16", batch=1, t_max=32001, lo=32001, s_q=2, heads=64,
             block=32),
        # one bf16 row halved
        dict(name="evict one row", op="evict", type="bf16", batch=1, t_max=8192, lo=8192, keep=4096, sink=4, recent=256,
             block=0),
        # a ragged 8-bit batch brought back to its budget (short rows keep all)
        dict(name="evict 8-bit batch", op="evict", type="bf16", batch=32, t_max=32768, lo=1024, keep=8000, sink=4,
             recent=1024, block=1),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "quantize", "dequantize", "attend", "attend", "weights", "weights", "evict"])
    block = rng.choice([1, 2, 4, 8, 16, 32, 64])
    batch = _spread(rng, 1, 48)
    if op == "append":
        s_new = _spread(rng, 1, 2048)
        t_max = min(32768, s_new + _spread(rng, 200, 16384))
        batch = max(1, min(batch, 250000 // t_max))
        return dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]), batch=batch, t_max=t_max, lo=0, s_new=s_new,
                    block=block)
    if op in ("quantize", "dequantize"):
        t_max = _spread(rng, 65, 8192)
        return dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]), batch=min(batch, 32), t_max=t_max,
                    lo=rng.choice([0, t_max]), block=block)
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    s_q = rng.choice([1, 1, 1, 2, 3, 4])
    if kind == "f32":   # the general-shape kernels: small heads and ranks
        heads, rank, rope = rng.randint(1, 8), rng.randint(17, 160), 2 * rng.randint(1, 20)
        t_max, batch = _spread(rng, 65, 2048), min(batch, 4)
    else:
        heads, rank, rope = rng.choice([64, 128]), RANK, ROPE
        t_max = _spread(rng, 65, 32768)
        batch = max(1, min(batch, 600000 // (t_max * s_q)))
    lo = rng.choice([0, t_max // 3, t_max])
    if op == "attend":
        top_k = rng.choice([0, 0, _spread(rng, 5, 2048)])
        return dict(op=op, type=kind, batch=batch, t_max=t_max, lo=max(lo, 8) if top_k else lo, s_q=s_q, heads=heads,
                    block=block, top_k=top_k, rank=rank, rope=rope)
    if op == "weights":
        return dict(op=op, type=kind, batch=batch, t_max=t_max, lo=lo, s_q=s_q, heads=heads,
                    block=rng.choice([0, block]), rank=rank, rope=rope)
    keep = _spread(rng, 33, max(34, t_max))
    return dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]), batch=max(1, min(batch, 600000 // t_max)), t_max=t_max,
                lo=lo, keep=keep, sink=rng.randint(0, 8), recent=rng.randint(0, keep // 2), block=rng.choice([0, 1]))


def _dims(c):
    return c.get("rank", RANK), c.get("rope", ROPE)


# ---------------------------------------------------------------- inputs

def _pow2(e):
    """2^(e - 127) of exponent bytes, exact."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest exponent byte e with amax <= 448 * 2^(e - 127), kept in [E_MIN, E_MAX]."""
    bits = amax.contiguous().view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return e.clamp(E_MIN, E_MAX)


def _rows_of(e, block, t):
    """Exponents of blocks as exponents of buffer rows."""
    return e.repeat_interleave(block, dim=1)[:, :t]


def _encode(v, e_rows):
    return (v * _pow2(254 - e_rows.to(torch.int32)).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _decode(codes, e_rows):
    return codes.float() * _pow2(e_rows).unsqueeze(-1)


def _block_max(tok_amax, block):
    b, t = tok_amax.shape
    pad = -t % block
    return torch.nn.functional.pad(tok_amax, (0, pad)).view(b, -1, block).amax(2)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _geometry(c, g):
    """Lengths in [lo, t_max - room], and left pads that are whole blocks where there is room for one."""
    b, t_max = c["batch"], c["t_max"]
    block = max(1, c["block"])
    hi = t_max - c.get("s_new", 0)
    lo = min(c["lo"], hi)
    lens = torch.randint(lo, hi + 1, (b,), generator=g, device=DEV, dtype=torch.int64)
    pads = torch.randint(0, 4, (b,), generator=g, device=DEV, dtype=torch.int64) * block
    starts = torch.where(lens + pads <= hi, pads, torch.zeros_like(pads))
    return starts.to(torch.int32), lens.to(torch.int32)


def _latent(c, g, tokens):
    """Normalised latents: unit root mean square times a norm weight; some tokens much smaller or larger."""
    rank, _ = _dims(c)
    x = _normal(g, c["batch"], tokens, rank)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    gain = torch.exp(0.5 * _normal(g, rank))
    token = torch.exp(0.3 * _normal(g, c["batch"], tokens, 1))
    return x * gain * token


def _cache8(c, g):
    t, block = c["t_max"], c["block"]
    lat = _latent(c, g, t)
    e = _exponent(_block_max(lat.abs().amax(-1), block)).to(torch.uint8)
    return _encode(lat, _rows_of(e, block, t)).view(torch.uint8), e


def _zeros(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rank, rope_dim = _dims(c)
    dt = TYPES[c["type"]]
    start, length = _geometry(c, g)
    b, t = c["batch"], c["t_max"]
    s = {"c": c, "start": start, "len": length, "status": _zeros(1)}
    op = c["op"]
    if op == "append":
        s["codes"], s["scales"] = _cache8(c, g)
        s["rope"] = _normal(g, b, t, rope_dim).to(dt)
        s["raw"] = (2.0 * _normal(g, b, c["s_new"], rank)).to(dt)
        s["raw_rope"] = _normal(g, b, c["s_new"], rope_dim).to(dt)
        s["gain"] = torch.exp(0.3 * _normal(g, rank)).to(dt)
        # the position of the first new token: rows that lost tokens before are past their lengths
        s["offset"] = length + torch.randint(0, 5000, (b,), generator=g, device=DEV, dtype=torch.int32)
        s["len_out"] = _zeros(b)
        power = (torch.arange(0, rope_dim, 2, device=DEV, dtype=torch.float64) / -rope_dim).float().double()
        s["inv"] = torch.pow(torch.full_like(power, THETA), power).float().double()
    elif op == "quantize":
        s["latent"] = _latent(c, g, t).to(dt)
        s["codes"] = _zeros((b, t, rank), torch.uint8)
        s["scales"] = _zeros((b, -(-t // c["block"])), torch.uint8) + 127
    elif op == "dequantize":
        s["codes"], s["scales"] = _cache8(c, g)
        s["latent"] = _zeros((b, t, rank), dt)
    elif op in ("attend", "weights"):
        if c["block"]:
            s["codes"], s["scales"] = _cache8(c, g)
        else:
            s["latent"] = _latent(c, g, t).to(dt)
        s["rope"] = _normal(g, b, t, rope_dim).to(dt)
        n_q = b * c["s_q"]
        q = _normal(g, n_q, c["heads"], rank + rope_dim)
        q[..., :rank] *= 0.5
        s["q"] = q.to(dt)
        s["scale"] = 1.0 / math.sqrt(128 + 64)
        if op == "attend":
            s["ctx"] = _zeros((n_q, c["heads"], rank), dt)
            k = c["top_k"]
            if k:
                limit = (length.long()[:, None] - c["s_q"] + 1 + torch.arange(c["s_q"], device=DEV)[None, :]).reshape(-1, 1)
                pick = torch.rand(n_q, k, generator=g, device=DEV, dtype=torch.float64)
                s["sel"] = (pick * limit.clamp(min=0)).long().to(torch.int32)
                count = torch.randint(max(1, k // 2), k + 1, (n_q,), generator=g, device=DEV, dtype=torch.int32)
                count = torch.where(count.eq(k - 1), torch.full_like(count, -1), count)   # some rows stay dense
                s["count"] = count
            s["workspace"] = _zeros(0, torch.uint8)
        else:
            scores, seen = _scores(s)
            m = scores.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
            m = m.masked_fill(m.isinf(), 0.0)
            total = ((scores - m).exp() * seen).sum(-1)
            s["lse"] = (m.squeeze(-1) + total.log()).reshape(n_q, c["heads"])
            s["weights"] = torch.exp(_normal(g, b, t))
    else:
        if c["block"]:
            codes, scales = _cache8(c, g)
            s["arrays"] = [codes, _normal(g, b, t, rope_dim).to(dt), scales.view(b, t, 1)]
        else:
            s["arrays"] = [_latent(c, g, t).to(dt), _normal(g, b, t, rope_dim).to(dt)]
        # heavy-tailed weights, many of them nothing at all
        w = torch.exp(2.0 * _normal(g, b, t)) - 0.5
        s["weights"] = w.clamp(min=0.0)
        s["kept"] = _zeros((b, c["keep"]))
        s["counts"] = _zeros(b)
        s["len_out"] = _zeros(b)
    return s


# ---------------------------------------------------------------- the operators

def run(state):
    return {"append": _append, "quantize": _quantize, "dequantize": _dequantize, "attend": _attend,
            "weights": _weights, "evict": _evict}[state["c"]["op"]](state)


def _windows(s):
    """[B, t_max] truth values: buffer rows inside their batch row's window."""
    r = torch.arange(s["c"]["t_max"], device=DEV)[None, :]
    lo = s["start"].long()[:, None]
    return (r >= lo) & (r < lo + s["len"].long()[:, None])


def _append(s):
    c = s["c"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        mla.append_compressed_q8(s["raw"], s["raw_rope"], s["gain"], EPS, THETA, s["codes"], s["scales"], c["block"],
                                 s["rope"], s["start"], s["len"], kv_len_out=s["len_out"], row_offsets=s["offset"],
                                 device_status=s["status"])
    else:
        b, n, t, block = c["batch"], c["s_new"], c["t_max"], c["block"]
        x = s["raw"].float()
        v = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["gain"].float()
        rows = (s["start"] + s["len"]).long()[:, None] + torch.arange(n, device=DEV)[None, :]
        bi = torch.arange(b, device=DEV)[:, None].expand(b, n)
        amax = torch.zeros(b, t, device=DEV)
        amax[bi, rows] = v.abs().amax(-1)
        new = torch.zeros(b, t, dtype=torch.bool, device=DEV)
        new[bi, rows] = True
        old = _windows(s)
        touched = _block_max(new.float(), block) > 0
        e_old = s["scales"].to(torch.int32)
        need = _exponent(_block_max(amax, block))
        e = torch.where(touched, torch.where(_block_max(old.float(), block) > 0, torch.maximum(need, e_old), need), e_old)
        e_rows, e_old_rows = _rows_of(e, block, t), _rows_of(e_old, block, t)
        codes = s["codes"].view(torch.float8_e4m3fn)
        moved = old & (e_rows != e_old_rows)
        again = _encode(_decode(codes, e_old_rows), e_rows)
        kept = torch.where(moved.unsqueeze(-1), again.view(torch.uint8), s["codes"])
        kept[bi, rows] = _encode(v, e_rows[bi, rows]).view(torch.uint8)
        s["codes"].copy_(kept)
        s["scales"].copy_(e.to(torch.uint8))
        s["rope"][bi, rows] = _rotate(s["raw_rope"].float(), s["offset"], s["inv"]).to(s["rope"].dtype)
        s["len_out"].copy_(s["len"] + n)
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"].view(torch.float8_e8m0fnu),
            "rope": s["rope"], "len": s["len_out"]}


def _rotate(x, offset, inv):
    """Pairs (2j, 2j + 1) rotated by f32(p * f32(theta^(-2j/d))), real parts first, imaginary parts after them."""
    n = x.shape[1]
    pos = (offset.long()[:, None] + torch.arange(n, device=DEV)[None, :]).double()
    angle = (pos[:, :, None] * inv).float().double()
    cos, sin = angle.cos().float(), angle.sin().float()
    re, im = x[..., 0::2], x[..., 1::2]
    return torch.cat([re * cos - im * sin, im * cos + re * sin], -1)


def _quantize(s):
    c = s["c"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        mla.quantize_cache(s["latent"], s["codes"], s["scales"], c["block"], s["start"], s["len"],
                           device_status=s["status"])
    else:
        lat, inside = s["latent"].float(), _windows(s)
        amax = lat.abs().amax(-1) * inside
        some = _block_max(inside.float(), c["block"]) > 0
        e = torch.where(some, _exponent(_block_max(amax, c["block"])), s["scales"].to(torch.int32))
        codes = _encode(lat, _rows_of(e, c["block"], c["t_max"])).view(torch.uint8)
        s["codes"].copy_(torch.where(inside.unsqueeze(-1), codes, s["codes"]))
        s["scales"].copy_(e.to(torch.uint8))
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _dequantize(s):
    c = s["c"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        mla.dequantize_cache(s["codes"], s["scales"], c["block"], s["latent"], s["start"], s["len"],
                             device_status=s["status"])
    else:
        v = _decode(s["codes"].view(torch.float8_e4m3fn), _rows_of(s["scales"], c["block"], c["t_max"]))
        s["latent"].copy_(torch.where(_windows(s).unsqueeze(-1), v.to(s["latent"].dtype), s["latent"]))
    return s["latent"]


def _cache32(s):
    c = s["c"]
    if c["block"]:
        return _decode(s["codes"].view(torch.float8_e4m3fn), _rows_of(s["scales"], c["block"], c["t_max"]))
    return s["latent"].float()


def _scores(s, lat=None):
    """Scaled scores [B, s_q * H, t_max] and which of them their token sees."""
    c = s["c"]
    lat = _cache32(s) if lat is None else lat
    keys = torch.cat([lat, s["rope"].float()], -1)
    q = s["q"].float().reshape(c["batch"], c["s_q"] * c["heads"], -1)
    scores = torch.bmm(q, keys.transpose(1, 2)) * s["scale"]
    r = torch.arange(c["t_max"], device=DEV)[None, None, :] - s["start"].long()[:, None, None]
    limit = s["len"].long()[:, None] - c["s_q"] + 1 + torch.arange(c["s_q"], device=DEV)[None, :]
    seen = (r >= 0) & (r < limit[:, :, None])
    return scores, seen.repeat_interleave(c["heads"], dim=1)


def _softmax(scores, seen):
    m = scores.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = (scores - m.masked_fill(m.isinf(), 0.0)).exp() * seen
    return p / p.sum(-1, keepdim=True).clamp(min=1e-37)


def _attend(s):
    c = s["c"]
    k = c["top_k"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        if not s["workspace"].numel():
            s["workspace"] = torch.empty(max(256, mla.decode_workspace_size(
                c["batch"], c["s_q"], c["heads"], *_dims(c), c["t_max"], k, k > 0, s["q"].dtype)),
                dtype=torch.uint8, device=DEV)
        return mla.decode_attend_q8(s["q"], s["codes"], s["scales"], c["block"], s["rope"], s["start"], s["len"],
                                    c["batch"], c["s_q"], s["scale"], s["ctx"], sel=s.get("sel"),
                                    sel_count=s.get("count"), workspace=s["workspace"], device_status=s["status"])
    lat = _cache32(s)
    if not k:
        ctx = torch.bmm(_softmax(*_scores(s, lat)), lat)
    else:
        # every key as often as it is listed (a row with count -1: every key that it sees, once)
        n_q, sel, count = c["batch"] * c["s_q"], s["sel"].long(), s["count"].long()
        scores, seen = _scores(s, lat)
        seen = seen.reshape(n_q, c["heads"], -1)
        bounded = (torch.arange(k, device=DEV)[None, :] < count[:, None]).float()
        start = s["start"].long().repeat_interleave(c["s_q"])[:, None]
        often = torch.zeros(n_q, c["t_max"], device=DEV).scatter_add_(1, sel + start, bounded)
        often = torch.where(count[:, None] == -1, seen[:, 0].float(), often)[:, None, :]
        scores = scores.reshape(n_q, c["heads"], -1)
        m = scores.masked_fill(~(often > 0), -math.inf).amax(-1, keepdim=True)
        p = (scores - m.masked_fill(m.isinf(), 0.0)).exp().masked_fill(~(often > 0), 0.0) * often
        p = (p / p.sum(-1, keepdim=True).clamp(min=1e-37)).reshape(c["batch"], c["s_q"] * c["heads"], -1)
        ctx = torch.bmm(p, lat)
    s["ctx"].copy_(ctx.reshape(s["ctx"].shape))
    return s["ctx"]


def _weights(s):
    c = s["c"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        if c["block"]:
            mla.key_weights_q8(s["q"], s["codes"], s["scales"], c["block"], s["rope"], s["lse"], s["start"], s["len"],
                               c["batch"], c["s_q"], s["scale"], s["weights"], decay=0.75, n_new=c["s_q"],
                               device_status=s["status"])
        else:
            mla.key_weights(s["q"], s["latent"], s["rope"], s["lse"], s["start"], s["len"], c["batch"], c["s_q"],
                            s["scale"], s["weights"], decay=0.75, n_new=c["s_q"], device_status=s["status"])
        return s["weights"]
    scores, seen = _scores(s)
    lse = s["lse"].reshape(c["batch"], -1, 1)
    add = (scores - lse.masked_fill(lse.isinf(), 0.0)).exp().masked_fill(~seen, 0.0).sum(1)
    r = torch.arange(c["t_max"], device=DEV)[None, :] - s["start"].long()[:, None]
    fresh = r >= s["len"].long()[:, None] - c["s_q"]
    w = torch.where(fresh, torch.zeros_like(s["weights"]), s["weights"]) * 0.75 + add
    s["weights"].copy_(torch.where(_windows(s), w, s["weights"]))
    return s["weights"]


def _evict(s):
    c = s["c"]
    arrays = s["arrays"] + [s["weights"].unsqueeze(-1)]
    if own:
        from mla_latent_kv_12_gb300 import mla
        mla.evict_plan(s["weights"], s["start"], s["len"], c["keep"], c["sink"], c["recent"], s["kept"], s["counts"],
                       kv_len_out=s["len_out"], device_status=s["status"])
        mla.cache_compact(arrays, s["start"], s["kept"], s["counts"], device_status=s["status"])
    else:
        b, t, keep = c["batch"], c["t_max"], c["keep"]
        lens, starts = s["len"].long()[:, None], s["start"].long()[:, None]
        over = lens > keep
        pos = torch.arange(t, device=DEV)[None, :].expand(b, t)
        rows = (starts + pos).clamp(max=t - 1)
        w = s["weights"].gather(1, rows)
        middle = (pos >= c["sink"]) & (pos < lens - c["recent"])
        order = torch.sort(w.masked_fill(~middle, -math.inf), dim=1, descending=True, stable=True).indices
        rank = torch.empty_like(order).scatter_(1, order, pos)
        chosen = (pos < lens) & (~middle | (rank < keep - c["sink"] - c["recent"]))
        place = torch.where(chosen & over, chosen.long().cumsum(1) - 1, torch.full_like(pos, keep))
        kept = torch.zeros(b, t + keep + 1, dtype=torch.int64, device=DEV).scatter_(1, place, pos)[:, :keep]
        s["kept"].copy_(torch.where(over, kept, s["kept"].long()))
        s["counts"].copy_(torch.where(over, torch.full_like(lens, keep), torch.full_like(lens, -1)).squeeze(1))
        s["len_out"].copy_(lens.clamp(max=keep).squeeze(1))
        source = (pos - starts).clamp(min=0)
        inside = over & (pos >= starts) & (pos < starts + keep)
        source = torch.where(inside, starts + kept.gather(1, source.clamp(max=keep - 1)), pos)
        [a.copy_(a.gather(1, source.unsqueeze(-1).expand(a.shape))) for a in arrays]
    return {"kept": s["kept"], "counts": s["counts"], "len": s["len_out"],
            "arrays": [a.view(torch.float8_e4m3fn) if a.shape[-1] > 1 and a.dtype == torch.uint8 else
                       a.view(torch.float8_e8m0fnu) if a.dtype == torch.uint8 else a for a in s["arrays"]],
            "weights": s["weights"]}


# ---------------------------------------------------------------- work

def work(case):
    c = case
    rank, rope = _dims(c)
    size = 4 if c["type"] == "f32" else 2
    b, t = c["batch"], c["t_max"]
    mean = (min(c["lo"], t) + t) / 2
    block = c["block"]
    held = rank + 1 / block if block else rank * size
    op = c["op"]
    if op == "append":
        n = b * c["s_new"]
        return {"bytes": n * ((rank + rope) * size + held + rope * size) + rank * size, "flops": 8 * n * rank}
    if op in ("quantize", "dequantize"):
        return {"bytes": b * mean * (rank * size + held), "flops": 3 * b * mean * rank}
    if op == "attend":
        n_q = b * c["s_q"]
        seen = min(0.75 * c["top_k"] if c["top_k"] else mean, mean)
        keys = seen * (n_q if c["top_k"] else b)
        return {"bytes": keys * (held + rope * size) + n_q * c["heads"] * (2 * rank + rope) * size,
                "flops": 2 * n_q * seen * c["heads"] * (2 * rank + rope)}
    if op == "weights":
        n_q = b * c["s_q"]
        return {"bytes": b * mean * (held + rope * size + 8) + n_q * c["heads"] * ((rank + rope) * size + 4),
                "flops": 2 * n_q * mean * c["heads"] * (rank + rope)}
    keep = min(c["keep"], t)
    if c["lo"] >= t:
        part = 1.0 if t > keep else 0.0
    else:
        part = max(0.0, t - max(keep, c["lo"])) / (t - c["lo"])
    moved = b * part * keep
    # a row within its budget is only looked up
    return {"bytes": 4 * b * part * (t + max(keep, c["lo"])) / 2 + 2 * moved * (held + rope * size + 4) + 4 * moved + 12 * b,
            "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def _values64(codes, scales, block, t):
    """e4m3 codes from their bits, times the exponents."""
    n = codes.to(torch.int64)
    mant, ex = n & 7, (n >> 3) & 15
    mag = torch.where(ex == 0, mant.double() * 2.0 ** -9, (8 + mant).double() * torch.pow(2.0, (ex - 10).double()))
    v = torch.where(n >= 128, -mag, mag)
    e = scales.to(torch.int64)[:, torch.arange(t, device=DEV) // block]
    return v * torch.pow(2.0, (e - 127).double())[..., None]


def _nearest8(x):
    """x rounded to the nearest e4m3 value, ties to the even one, in 64 bits."""
    a = x.abs().clamp(max=448.0)
    step = torch.pow(2.0, torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _need64(amax):
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)) + 127
    return e.clamp(E_MIN, E_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op, b, t = c["op"], c["batch"], c["t_max"]
    block = c["block"]
    starts, lens = s["start"].tolist(), s["len"].tolist()
    if op == "append":
        units = (s["codes"].view(torch.float8_e4m3fn)).double()
        e_all = s["scales"].double()
        rope = s["rope"].double()
        rot = _rotate64(s["raw_rope"].double(), s["offset"].tolist())
        for i in range(b):
            x = s["raw"][i].double()
            v = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * s["gain"].double()
            end, row = starts[i] + lens[i], 0
            rope[i, end:end + c["s_new"]] = rot[i]
            first, last = end // block, (end + c["s_new"] - 1) // block
            top = torch.zeros((last - first + 1) * block, dtype=torch.float64, device=DEV)
            top[end - first * block:end - first * block + c["s_new"]] = v.abs().amax(-1)
            need = _need64(top.view(-1, block).amax(1))
            if end > max(first * block, starts[i]):   # the first block holds tokens already
                row = max(first * block, starts[i])
                before = float(e_all[i, first])
                need[0] = max(float(need[0]), before)
                if float(need[0]) != before:
                    units[i, row:end] = _nearest8(units[i, row:end] * 2.0 ** (before - float(need[0])))
            e_all[i, first:last + 1] = need
            rows = need.repeat_interleave(block)[end - first * block:end - first * block + c["s_new"], None]
            units[i, end:end + c["s_new"]] = _nearest8(v * torch.pow(2.0, 127 - rows))
        return {"codes": units, "scales": torch.pow(2.0, e_all - 127), "rope": rope,
                "len": s["len"] + c["s_new"]}
    if op == "quantize":
        units = s["codes"].view(torch.float8_e4m3fn).double()
        e_all = s["scales"].double()
        for i in range(b):
            if not lens[i]:
                continue
            lo, hi = starts[i], starts[i] + lens[i]
            v = s["latent"][i, lo:hi].double()
            nb = -(-lens[i] // block)
            top = torch.zeros(nb * block, dtype=torch.float64, device=DEV)
            top[:lens[i]] = v.abs().amax(-1)
            need = _need64(top.view(nb, block).amax(1))
            e_all[i, lo // block:lo // block + nb] = need
            units[i, lo:hi] = _nearest8(v * torch.pow(2.0, 127 - need.repeat_interleave(block)[:lens[i], None]))
        return {"codes": units, "scales": torch.pow(2.0, e_all - 127)}
    if op == "dequantize":
        out = s["latent"].double()
        for i in range(b):
            lo, hi = starts[i], starts[i] + lens[i]
            out[i, lo:hi] = _values64(s["codes"][i:i + 1], s["scales"][i:i + 1], block, t)[0, lo:hi]
        return out
    if op in ("attend", "weights"):
        ctx = torch.zeros(b * c["s_q"], c["heads"], _dims(c)[0], dtype=torch.float64, device=DEV)
        weights = s["weights"].double() if op == "weights" else None
        for i in range(b):
            lo, n = starts[i], lens[i]
            if block:
                lat = _values64(s["codes"][i:i + 1], s["scales"][i:i + 1], block, t)[0, lo:lo + n]
            else:
                lat = s["latent"][i, lo:lo + n].double()
            keys = torch.cat([lat, s["rope"][i, lo:lo + n].double()], 1)
            if op == "weights":
                weights[i, lo:lo + max(0, n - c["s_q"])] *= 0.75
                weights[i, lo + max(0, n - c["s_q"]):lo + n] = 0.0
            for j in range(c["s_q"]):
                row, limit = i * c["s_q"] + j, n - c["s_q"] + 1 + j
                if limit <= 0:
                    continue
                at = torch.arange(limit, device=DEV)
                if op == "attend" and c["top_k"] and int(s["count"][row]) != -1:
                    at = s["sel"][row, :int(s["count"][row])].long()
                x = (s["q"][row].double() @ keys[at].t()) * s["scale"]
                if op == "attend":
                    ctx[row] = torch.softmax(x, -1) @ lat[at]
                else:
                    weights[i, lo:lo + limit] += torch.exp(x - s["lse"][row].double()[:, None]).sum(0)
        return ctx if op == "attend" else weights
    keep, sink, recent = c["keep"], c["sink"], c["recent"]
    kept, counts, out_len = s["kept"].clone(), s["counts"].clone(), s["len_out"].clone()
    arrays = [a.view(torch.float8_e4m3fn) if a.shape[-1] > 1 and a.dtype == torch.uint8 else
              a.view(torch.float8_e8m0fnu) if a.dtype == torch.uint8 else a for a in s["arrays"]]
    arrays = [a.double() for a in arrays + [s["weights"]]]
    for i in range(b):
        lo, n = starts[i], lens[i]
        out_len[i] = min(n, keep)
        counts[i] = -1 if n <= keep else keep
        if n <= keep:
            continue
        w = s["weights"][i, lo + sink:lo + n - recent].tolist()
        best = sorted(range(len(w)), key=lambda p: (-w[p], p))[:keep - sink - recent]
        at = list(range(sink)) + sorted(sink + p for p in best) + list(range(n - recent, n))
        kept[i] = torch.tensor(at, dtype=torch.int32, device=DEV)
        for a in arrays:
            a[i, lo:lo + keep] = a[i, lo + kept[i].long()]
    return {"kept": kept, "counts": counts, "len": out_len, "arrays": arrays[:-1], "weights": arrays[-1]}


def _rotate64(x, offsets):
    b, n, d = x.shape
    out = torch.empty_like(x)
    theta = torch.tensor(THETA, dtype=torch.float32).double()
    for j in range(d // 2):
        inv = torch.pow(theta, torch.tensor(-2.0 * j / d, dtype=torch.float32).double()).float().double().to(DEV)
        for i in range(b):
            # the operator's angles are rounded to 32 bits
            a = ((offsets[i] + torch.arange(n, device=DEV)).double() * inv).float().double()
            out[i, :, j] = x[i, :, 2 * j] * a.cos() - x[i, :, 2 * j + 1] * a.sin()
            out[i, :, d // 2 + j] = x[i, :, 2 * j + 1] * a.cos() + x[i, :, 2 * j] * a.sin()
    return out
