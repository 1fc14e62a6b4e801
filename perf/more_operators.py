"""Cases of the paged latent cache and of drafted token trees over it.

Each case is one call of an operator of the framework (``own`` true) or the same
mathematics in elementary torch operations (``own`` false):

* ``append``  new tokens into the pages of their sequences (RMSNorm of the latent, RoPE of the key)
* ``attend``  latent attention over pages: one token, a few drafted in a row, or a prompt chunk per sequence
* ``tree``    the same for a tree of drafted tokens: a node sees its sequence and its own ancestors
* ``plan``    a tree's positions and ancestor masks from its parent list
* ``commit``  the accepted path of each tree moved to the end of its sequence, in every layer's pages

A paged cache is a pool ``[pages, page rows, width]``; key ``t`` of sequence ``b`` is row ``t % page`` of page
``table[b, t // page]``.  The table's entries behind a sequence's last page are -1.
"""
import math

import torch

own = False

DEV = "cuda"
RANK, ROPE = 512, 64
THETA, EPS = 10000.0, 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode step
        dict(name="append one token", op="append", type="bf16", batch=1, t_max=4096, lo=4000, s_q=1, page=64,
             ragged=False, tree=False),
        # prompt chunks of a batch of sequences, each of another length, over small pages
        dict(name="append prompt chunks", op="append", type="bf16", batch=8, t_max=16384, lo=1, s_q=2048, page=16,
             ragged=True, tree=False),
        # one sequence, one token
        dict(name="attend one row", op="attend", type="bf16", batch=1, t_max=4096, lo=4096, s_q=1, heads=128, page=64,
             ragged=False),
        # a ragged serving batch, 1k to 32k tokens
        dict(name="attend ragged batch", op="attend", type="bf16", batch=32, t_max=32768, lo=1024, s_q=1, heads=128,
             page=64, ragged=False),
        # four drafted tokens in a row per sequence, small pages
        dict(name="attend verify", op="attend", type="bf16", batch=8, t_max=65536, lo=65536, s_q=4, heads=128, page=16,
             ragged=False),
        # prompt chunks behind a cached prefix, 64 heads, one chunk shorter than the other
        dict(name="attend prompt chunk", op="attend", type="bf16", batch=2, t_max=8191, lo=5000, s_q=512, heads=64,
             page=64, ragged=True),
        # a small tree of one sequence
        dict(name="tree of one row", op="tree", type="bf16", batch=1, t_max=4096, lo=4000, s_q=16, heads=128, page=64,
             ragged=False),
        # full trees of a batch
        dict(name="trees of a batch", op="tree", type="bf16", batch=8, t_max=16384, lo=8000, s_q=64, heads=128,
             page=32, ragged=False),
        # one tree
        dict(name="plan one tree", op="plan", type="bf16", batch=1, t_max=4096, s_q=16, ragged=False),
        # large trees of a large batch, of different sizes
        dict(name="plan large trees", op="plan", type="bf16", batch=64, t_max=32768, s_q=256, ragged=True),
        # the accepted path of one tree, one layer
        dict(name="commit one row", op="commit", type="bf16", batch=1, t_max=4096, s_q=16, page=64, depth=5, layers=1),
        # accepted paths of a batch, every layer in one call
        dict(name="commit all layers", op="commit", type="bf16", batch=32, t_max=4096, s_q=64, page=16, depth=10,
             layers=24),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "tree", "tree", "tree", "plan", "commit"])
    page = rng.choice([1, 7, 16, 16, 32, 48, 64, 64, 64, 128, 256])
    batch = _spread(rng, 1, 48)
    ragged = rng.random() < 0.4
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        s_q = _spread(rng, 1, 2048)
        t_max = min(32768, s_q + _spread(rng, 100, 16384))
        return dict(op=op, type=kind, batch=max(1, min(batch, 250000 // t_max)), t_max=t_max, lo=0, s_q=s_q, page=page,
                    ragged=ragged, tree=s_q <= 64 and rng.random() < 0.4)
    if op == "plan":
        return dict(op=op, type="bf16", batch=batch, t_max=_spread(rng, 300, 32768), s_q=_spread(rng, 1, 256),
                    ragged=ragged)
    if op == "commit":
        s_q, t_max = _spread(rng, 2, 64), _spread(rng, 200, 8192)
        layers = _spread(rng, 1, 24)
        return dict(op=op, type=kind, batch=max(1, min(batch, 3000000 // (t_max * layers))), t_max=t_max, s_q=s_q,
                    page=page, depth=_spread(rng, 1, min(s_q, 16)), layers=layers)
    s_q = _spread(rng, 2, 64) if op == "tree" else rng.choice([1, 1, 1, 2, 3, 4, 5, 8, _spread(rng, 9, 512)])
    if kind == "f32":   # the general-shape kernels: small heads and ranks
        heads, rank, rope = rng.randint(1, 8), rng.randint(17, 160), 2 * rng.randint(1, 20)
        t_max, batch, s_q = _spread(rng, 100, 2048), min(batch, 4), min(s_q, 32)
    else:
        heads, rank, rope = rng.choice([64, 128]), RANK, ROPE
        t_max = _spread(rng, 100, 32768)
    t_max = max(t_max, s_q + 1)
    batch = max(1, min(batch, 600000 // t_max, 4000000 // (t_max * s_q)))
    lo = max(rng.choice([0, t_max // 3, t_max]), s_q if op == "tree" else 0)
    return dict(op=op, type=kind, batch=batch, t_max=t_max, lo=lo, s_q=s_q, heads=heads, page=page, ragged=ragged,
                rank=rank, rope=rope)


def _dims(c):
    return c.get("rank", RANK), c.get("rope", ROPE)


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _integers(g, lo, hi, *shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int64)


def _latent(g, *shape):
    """Normalised latents: unit root mean square times a norm weight; some tokens smaller or larger."""
    x = _normal(g, *shape)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * torch.exp(0.5 * _normal(g, shape[-1])) * torch.exp(0.3 * _normal(g, *shape[:-1], 1))


def _table(g, c, lens):
    """Pages of every sequence, spread over a pool that holds some more; -1 behind a sequence's last page."""
    b, page = c["batch"], c["page"]
    width = -(-c["t_max"] // page)
    pages = b * width + 3
    order = torch.randperm(pages, generator=g, device=DEV)[:b * width].view(b, width)
    used = (lens[:, None] + page - 1) // page
    return torch.where(torch.arange(width, device=DEV)[None, :] < used, order, -1).to(torch.int32), pages


def _parents(g, b, n):
    """Trees in the order in which a drafter grows them: each node below an earlier one, or a root (-1)."""
    back = (torch.rand(b, n, generator=g, device=DEV) ** 1.5 * 12).long() + 1
    j = torch.arange(n, device=DEV)[None, :]
    return torch.clamp(j - back, min=-1).to(torch.int32)


def _ancestors(parents):
    """[b, n, n] truth values: node j is i or one of its ancestors."""
    b, n = parents.shape
    eye = torch.eye(n, device=DEV).expand(b, n, n)
    up = torch.zeros(b, n, n + 1, device=DEV).scatter_(2, parents.long()[:, :, None] % (n + 1), 1.0)[:, :, :n]
    reach = eye + up
    for _ in range(max(1, (n - 1).bit_length())):   # paths of twice the length
        reach = (torch.bmm(reach, reach) > 0).float()
    return reach > 0


def _words(anc):
    """Truth values over nodes as 64-bit words, the first node the lowest bit."""
    b, n, _ = anc.shape
    words = -(-n // 64)
    bits = torch.nn.functional.pad(anc.long(), (0, words * 64 - n)).view(b * n, words, 64)
    return (bits << torch.arange(64, device=DEV)).sum(2)


def _inverse_frequencies(d):
    power = (torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / -d).float().double()
    return torch.pow(torch.full_like(power, THETA), power).float().double()


def _zeros(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rank, rope_dim = _dims(c)
    dt = TYPES[c["type"]]
    b, t, n, op = c["batch"], c["t_max"], c["s_q"], c["op"]
    s = {"c": c, "status": _zeros(1)}
    counts = _integers(g, 0, n, b).to(torch.int32) if c.get("ragged") else None
    s["counts"] = counts
    if op in ("append", "commit"):
        # lengths before the new tokens, whose pages are there already
        s["len"] = _integers(g, min(c.get("lo", 0), t - n), t - n, b).to(torch.int32)
        s["table"], pages = _table(g, c, s["len"].long() + n)
        s["len_out"] = _zeros(b)
    if op == "append":
        s["latent"] = _latent(g, pages, c["page"], rank).to(dt)
        s["rope"] = _normal(g, pages, c["page"], rope_dim).to(dt)
        s["raw"] = (2.0 * _normal(g, b, n, rank)).to(dt)
        s["raw_rope"] = _normal(g, b, n, rope_dim).to(dt)
        s["gain"] = torch.exp(0.3 * _normal(g, rank)).to(dt)
        s["inv"] = _inverse_frequencies(rope_dim)
        s["positions"] = None
        if c["tree"]:
            depth = _ancestors(_parents(g, b, n)).sum(2) - 1
            s["positions"] = (s["len"].long()[:, None] + depth).to(torch.int32)
    elif op in ("attend", "tree"):
        s["len"] = _integers(g, min(c["lo"], t), t, b).to(torch.int32)
        s["table"], pages = _table(g, c, s["len"].long())
        s["latent"] = _latent(g, pages, c["page"], rank).to(dt)
        s["rope"] = _normal(g, pages, c["page"], rope_dim).to(dt)
        q = _normal(g, b * n, c["heads"], rank + rope_dim)
        q[..., :rank] *= 0.5
        s["q"] = q.to(dt)
        s["scale"] = 1.0 / math.sqrt(128 + 64)
        s["ctx"] = _zeros((b * n, c["heads"], rank), dt)
        s["mask"] = None
        if op == "tree":
            s["parents"] = _parents(g, b, n)
            s["mask"] = _words(_ancestors(s["parents"]))
        s["workspace"] = _zeros(0, torch.uint8)
    elif op == "plan":
        s["parents"] = _parents(g, b, n)
        s["len"] = _integers(g, 0, t, b).to(torch.int32)
        s["positions"] = _zeros((b, n))
        s["mask"] = _zeros((b * n, -(-n // 64)), torch.int64)
    else:
        s["arrays"] = []
        for _ in range(c["layers"]):
            s["arrays"] += [_normal(g, pages, c["page"], rank).to(dt), _normal(g, pages, c["page"], rope_dim).to(dt)]
        # a path goes down the tree: ascending nodes, some rows with nothing accepted
        depth = min(c["depth"], n)
        order = torch.rand(b, n, generator=g, device=DEV).argsort(1)[:, :depth].sort(1).values
        s["path"] = order.to(torch.int32)
        s["accepted"] = _integers(g, 0, depth, b).to(torch.int32)
    return s


# ---------------------------------------------------------------- the operators

def run(state):
    return {"append": _append, "attend": _attend, "tree": _attend, "plan": _plan,
            "commit": _commit}[state["c"]["op"]](state)


def _place(s, rows):
    """Page and row in it of keys ``rows`` [b, n] of every sequence."""
    page = s["c"]["page"]
    return s["table"].long().gather(1, rows // page), rows % page


def _counts(s):
    c = s["c"]
    full = torch.full((c["batch"],), c["s_q"], dtype=torch.int64, device=DEV)
    return full if s["counts"] is None else s["counts"].long()


def _append(s):
    c = s["c"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        mla.append_paged(s["raw"], s["raw_rope"], s["gain"], EPS, THETA, s["latent"], s["rope"], s["table"], s["len"],
                         kv_len_out=s["len_out"], positions=s["positions"], counts=s["counts"],
                         device_status=s["status"])
    else:
        step = torch.arange(c["s_q"], device=DEV)[None, :]
        rows = s["len"].long()[:, None] + step
        page, row = _place(s, rows)
        new = step < _counts(s)[:, None]
        x = s["raw"].float()
        v = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["gain"].float()
        s["latent"][page[new], row[new]] = v[new].to(s["latent"].dtype)
        # pairs (2j, 2j + 1) rotated by f32(p * f32(theta^(-2j/d))), real parts first, imaginary parts after them
        pos = (rows if s["positions"] is None else s["positions"]).double()
        angle = (pos[:, :, None] * s["inv"]).float().double()
        cos, sin = angle.cos().float(), angle.sin().float()
        re, im = s["raw_rope"].float()[..., 0::2], s["raw_rope"].float()[..., 1::2]
        turned = torch.cat([re * cos - im * sin, im * cos + re * sin], -1)
        s["rope"][page[new], row[new]] = turned[new].to(s["rope"].dtype)
        s["len_out"].copy_(s["len"].long() + _counts(s))
    return {"latent": s["latent"], "rope": s["rope"], "len": s["len_out"]}


def _attend(s):
    c = s["c"]
    b, n, t, heads = c["batch"], c["s_q"], c["t_max"], c["heads"]
    rank, rope_dim = _dims(c)
    if own:
        from mla_latent_kv_12_gb300 import mla
        if not s["workspace"].numel():
            s["workspace"] = torch.empty(max(256, mla.decode_workspace_size(
                b, n, heads, rank, rope_dim, s["table"].shape[1] * c["page"], dtype=s["q"].dtype)),
                dtype=torch.uint8, device=DEV)
        return mla.decode_attend_paged(s["q"], s["latent"], s["rope"], s["table"], s["len"], b, n, s["scale"], s["ctx"],
                                       counts=s["counts"], tree_mask=s["mask"], workspace=s["workspace"],
                                       device_status=s["status"])
    rows = torch.arange(t, device=DEV)[None, :].expand(b, t)
    page, row = _place(s, rows)
    lat = s["latent"][page.clamp(min=0), row].float()
    keys = torch.cat([lat, s["rope"][page.clamp(min=0), row].float()], -1)
    scores = torch.bmm(s["q"].float().view(b, n * heads, -1), keys.transpose(1, 2)) * s["scale"]
    counts = _counts(s)
    first = (s["len"].long() - counts)[:, None, None]        # keys before the new tokens
    token, key = torch.arange(n, device=DEV)[None, :, None], rows[:, None, :]
    if s["mask"] is None:
        seen = key <= first + token
    else:
        node = key - first
        words = s["mask"].view(b, n, -1)
        at = node.clamp(0, n - 1).expand(b, n, t)
        seen = (node < 0) | ((words.gather(2, at // 64) >> (at % 64)) & 1).bool()
    seen = seen & (key < s["len"].long()[:, None, None]) & (token < counts[:, None, None])
    scores = scores.view(b, n, heads, t).masked_fill_(~seen[:, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top.masked_fill(top.isinf(), 0.0)).exp()
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-37)).view(b, n * heads, t)
    s["ctx"].copy_(torch.bmm(p, lat).view(s["ctx"].shape))
    return s["ctx"]


def _plan(s):
    c = s["c"]
    if own:
        from mla_latent_kv_12_gb300 import mla
        mla.tree_plan(s["parents"], s["len"], s["positions"], s["mask"], counts=s["counts"], device_status=s["status"])
    else:
        # nodes behind a tree's last have no ancestors and the position of its roots
        there = torch.arange(c["s_q"], device=DEV)[None, :, None] < _counts(s)[:, None, None]
        anc = _ancestors(s["parents"]) & there
        s["mask"].copy_(_words(anc))
        s["positions"].copy_(s["len"].long()[:, None] + (anc.sum(2) - 1).clamp(min=0))
    return {"positions": s["positions"], "mask": s["mask"]}


def _commit(s):
    if own:
        from mla_latent_kv_12_gb300 import mla
        if "pools" not in s:
            s["pools"] = mla.PagedArrays(s["arrays"])
        mla.commit_paged(s["pools"], s["table"], s["len"], s["path"], s["accepted"], kv_len_out=s["len_out"],
                         device_status=s["status"])
    else:
        step = torch.arange(s["path"].shape[1], device=DEV)[None, :]
        kept = step < s["accepted"].long()[:, None]
        to = _place(s, s["len"].long()[:, None] + step)
        of = _place(s, s["len"].long()[:, None] + s["path"].long())
        for a in s["arrays"]:
            a[to[0][kept], to[1][kept]] = a[of[0][kept], of[1][kept]]
        s["len_out"].copy_(s["len"] + s["accepted"])
    return {"arrays": s["arrays"], "len": s["len_out"]}


# ---------------------------------------------------------------- work

def work(case):
    c = case
    rank, rope = _dims(c)
    size = 4 if c["type"] == "f32" else 2
    b, n, op = c["batch"], c["s_q"], c["op"]
    tokens = b * n * (0.5 if c.get("ragged") else 1.0)
    if op == "append":
        return {"bytes": tokens * (rank + rope) * 2 * size + rank * size + 12 * b, "flops": 8 * tokens * rank}
    if op == "plan":
        return {"bytes": 4 * tokens + b * n * (4 + 8 * -(-n // 64)) + 4 * b, "flops": 0}
    if op == "commit":
        moved = b * min(c["depth"], n) / 2
        return {"bytes": 2 * moved * c["layers"] * (rank + rope) * size + 4 * moved + 12 * b, "flops": 0}
    mean = (min(c["lo"], c["t_max"]) + c["t_max"]) / 2
    # tokens of a row see, in the middle, half of one another; of a tree, few
    seen = max(1.0, mean - n * (0.25 if c.get("ragged") else 0.5))
    return {"bytes": b * mean * (rank + rope) * size + tokens * c["heads"] * (rank + rope) * size +
                     b * n * c["heads"] * rank * size,
            "flops": 2 * tokens * seen * c["heads"] * (2 * rank + rope)}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op, b, n, page = c["op"], c["batch"], c["s_q"], c.get("page", 0)
    lens = s["len"].tolist()
    counts = [n] * b if s["counts"] is None else s["counts"].tolist()
    if op == "append":
        latent, rope = s["latent"].double(), s["rope"].double()
        table, d = s["table"].cpu(), s["rope"].shape[-1]
        theta = torch.tensor(THETA, dtype=torch.float32).double()
        inv = torch.stack([torch.pow(theta, torch.tensor(-2.0 * j / d, dtype=torch.float32).double())
                           for j in range(d // 2)]).float().double().to(DEV)
        for i in range(b):
            m = counts[i]
            x = s["raw"][i, :m].double()
            v = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * s["gain"].double()
            pos = lens[i] + torch.arange(m) if s["positions"] is None else s["positions"][i, :m].cpu()
            # the operator's angles are rounded to 32 bits
            a = (pos.double().to(DEV)[:, None] * inv).float().double()
            re, im = s["raw_rope"][i, :m, 0::2].double(), s["raw_rope"][i, :m, 1::2].double()
            r = torch.cat([re * a.cos() - im * a.sin(), im * a.cos() + re * a.sin()], 1)
            at = torch.tensor([int(table[i, k // page]) * page + k % page for k in range(lens[i], lens[i] + m)],
                              dtype=torch.int64, device=DEV)
            latent.view(-1, latent.shape[-1])[at] = v
            rope.view(-1, d)[at] = r
        return {"latent": latent, "rope": rope, "len": s["len"] + torch.tensor(counts, dtype=torch.int32, device=DEV)}
    if op in ("attend", "tree"):
        ctx = torch.zeros(s["ctx"].shape, dtype=torch.float64, device=DEV)
        for i in range(b):
            ids = s["table"][i, :-(-lens[i] // page)].long()
            lat = s["latent"][ids].double().flatten(0, 1)[:lens[i]]
            keys = torch.cat([lat, s["rope"][ids].double().flatten(0, 1)[:lens[i]]], 1)
            first = lens[i] - counts[i]
            parents = s["parents"][i].tolist() if op == "tree" else None
            for j in range(counts[i]):
                if op == "tree":
                    path, node = [], j
                    while node >= 0:
                        path.append(first + node)
                        node = parents[node]
                    at = torch.tensor(list(range(first)) + path[::-1], dtype=torch.int64, device=DEV)
                    k, v = keys[at], lat[at]
                else:
                    k, v = keys[:max(0, first + j + 1)], lat[:max(0, first + j + 1)]
                if k.shape[0]:
                    x = (s["q"][i * n + j].double() @ k.t()) * s["scale"]
                    ctx[i * n + j] = torch.softmax(x, -1) @ v
        return ctx
    if op == "plan":
        words = -(-n // 64)
        positions, mask = [], []
        for parents, start, m in zip(s["parents"].tolist(), lens, counts):
            rows = []
            for j, p in enumerate(parents):
                rows.append(((rows[p] if p >= 0 else 0) | 1 << j) if j < m else 0)
                positions.append(start + max(0, bin(rows[-1]).count("1") - 1))
                for w in range(words):
                    bits = rows[-1] >> 64 * w & (1 << 64) - 1
                    mask.append(bits - (1 << 64) if bits >> 63 else bits)
        return {"positions": torch.tensor(positions, dtype=torch.int32, device=DEV).view(b, n),
                "mask": torch.tensor(mask, dtype=torch.int64, device=DEV).view(b * n, words)}
    arrays = [a.double() for a in s["arrays"]]
    table, accepted, path = s["table"].tolist(), s["accepted"].tolist(), s["path"].tolist()
    of, to = [], []
    for i in range(b):
        for j in range(accepted[i]):
            for rows, k in ((to, lens[i] + j), (of, lens[i] + path[i][j])):
                rows.append(table[i][k // page] * page + k % page)
    for a in arrays:
        flat = a.view(-1, a.shape[-1])
        flat[torch.tensor(to, dtype=torch.int64, device=DEV)] = flat[torch.tensor(of, dtype=torch.int64, device=DEV)]
    return {"arrays": arrays, "len": s["len"] + s["accepted"]}
