"""The paged cache on the GPU: append, attention of rows and trees of drafted tokens, plan, commit, and their run
together, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import helpers as H
from tests import paged_reference as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS, THETA = 1e-6, 10000.0
SCALE = 192 ** -0.5
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def page_table(seed, lengths, size, spare=2):
    """Pages in a random order; entries behind the last page would fault if they were read as pages."""
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-n // size) for n in lengths)) + 1
    need = [-(-n // size) for n in lengths]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lengths), width), 0x7FFFFFF0, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return torch.from_numpy(table).to(DEV), len(order)


def dirty_pool(pages, size, width, dtype):
    return torch.full((pages, size, width), float("nan"), dtype=dtype, device=DEV)


def fill(pool, table, lengths, values):
    """values [B, T, F] into the keys of every sequence (everything else stays)."""
    size = pool.shape[1]
    for b, n in enumerate(lengths):
        t = torch.arange(n, device=DEV)
        pool[table[b].long()[t // size], t % size] = values[b, :n].to(pool.dtype)


# ---------------------------------------------------------------- append

def check_append(raw, raw_rope, gain, before, after, table, lens, counts, positions):
    """Every element of both pools: new tokens against 64 bits, the rest bit for bit."""
    size, dtype = before[0].shape[1], before[0].dtype
    half = torch.finfo(dtype).eps / 2
    masks = []
    for pool, kind in ((0, "latent"), (1, "rope")):
        want, bound = P.as64(before[pool]), None
        bound = np.zeros_like(want)
        for b, n in enumerate(lens):
            c = counts[b]
            if c == 0:
                continue
            t = np.arange(n, n + c)
            at = table[b].cpu().numpy()[t // size], t % size
            if kind == "latent":
                v = P.rms_norm64(P.as64(raw[b, :c]), P.as64(gain), EPS)
                # up to 37 additions a lane and its tree, halved by the root; four more operations
                want[at], bound[at] = v, np.abs(v) * (half + 2.0 ** -18) + 1e-38
            else:
                x = P.as64(raw_rope[b, :c])
                pos = np.arange(n, n + c) if positions is None else positions[b, :c].cpu().numpy()
                v = P.rotate64(x, pos, THETA)
                # sine, cosine (2 ulp), two products and a sum, then the rounding to the pool's type
                pair = np.abs(x[:, 0::2]) + np.abs(x[:, 1::2])
                want[at] = v
                bound[at] = np.abs(v) * half + np.concatenate([pair, pair], 1) * 2.0 ** -21
        got = P.as64(after[pool])
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan), kind
        assert (np.abs(got[~nan] - want[~nan]) <= bound[~nan]).all(), kind
        masks.append(nan)


@pytest.mark.parametrize("in_type,type", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("rank,rope,size,s_new,lens,counts,tree", [
    (512, 64, 64, 1, [0, 63, 64, 1000], None, False),
    (512, 64, 16, 37, [0, 5, 16, 300], [37, 0, 1, 36], False),
    (512, 64, 1, 5, [3, 0], None, True),
    (256, 128, 7, 20, [0, 6, 7], [20, 13, 0], True),
    (1024, 256, 32, 3, [31, 90], None, False),
    (37, 6, 3, 9, [2, 0, 50], [9, 9, 4], True),
    (1, 2, 64, 2, [0, 200], None, False),
    (96, 0, 8, 4, [7], None, False),
])
def test_append(mla, in_type, type, rank, rope, size, s_new, lens, counts, tree):
    g = gen(rank + s_new)
    B = len(lens)
    table, pages = page_table(rank, [n + s_new for n in lens], size)
    pools = dirty_pool(pages, size, rank, type), dirty_pool(pages, size, rope, type)
    for p in pools:
        fill(p, table, lens, normal(g, B, max(lens) + 1, p.shape[2]))
    before = [p.clone() for p in pools]
    raw, raw_rope = (3 * normal(g, B, s_new, rank)).to(in_type), normal(g, B, s_new, rope).to(in_type)
    gain = torch.exp(0.3 * normal(g, rank)).to(in_type)
    positions = torch.randint(0, 200000, (B, s_new), generator=g, device=DEV, dtype=torch.int32) if tree else None
    out, st = i32([7] * B), status()
    mla.append_paged(raw, raw_rope, gain, EPS, THETA, *pools, table, i32(lens), kv_len_out=out, positions=positions,
                     counts=None if counts is None else i32(counts), device_status=st)
    counts = counts or [s_new] * B
    assert int(st) == 0 and out.tolist() == [n + c for n, c in zip(lens, counts)]
    check_append(raw, raw_rope, gain, before, pools, table, lens, counts, positions)


def test_append_views_and_lengths_in_place(mla):
    # one pool of latent || rope in wider rows, interleaved with another layer's; raw values of one projection
    g = gen(3)
    lens, s_new, size = [5, 0, 40], 30, 16
    table, pages = page_table(4, [n + s_new for n in lens], size)
    both = normal(g, pages, 2, size, 592).bfloat16()
    pool = both[:, 1]
    latent, rope = pool[..., 8:520], pool[..., 520:584]
    around = both.clone()
    before = [latent.clone(), rope.clone()]
    kv_a = normal(g, 3, s_new + 2, 600).bfloat16()[:, 1:-1, 8:584]
    gain = torch.ones(512, device=DEV).bfloat16()
    n = i32(lens)
    mla.append_paged(kv_a[..., :512], kv_a[..., 512:], gain, EPS, THETA, latent, rope, table, n, kv_len_out=n)
    assert n.tolist() == [k + s_new for k in lens]
    check_append(kv_a[..., :512], kv_a[..., 512:], gain, before, (latent, rope), table, lens, [s_new] * 3, None)
    pool[..., 8:584] = 0
    around[:, 1, :, 8:584] = 0
    assert torch.equal(both, around)


@pytest.mark.parametrize("s_new", [1, 3, 40])
def test_append_bad_rows_and_pages(mla, s_new):
    g = gen(5)
    size, width = 4, 20
    gain = torch.ones(64, device=DEV)
    for lens, counts, entry, left_out in [([81 - s_new, 2], None, None, s_new), ([-1, 2], None, None, s_new),
                                          ([0, 2], [-1, s_new], None, s_new), ([0, 2], [s_new + 1, s_new], None, s_new),
                                          ([0, 2], None, 40, min(s_new, 4)), ([0, 2], None, -1, min(s_new, 4))]:
        table = torch.arange(40, device=DEV, dtype=torch.int32).view(2, width)
        if entry is not None:
            table[0, 0] = entry
        latent, rope = normal(g, 40, size, 64), normal(g, 40, size, 8)
        l0, r0 = latent.clone(), rope.clone()
        raw = normal(g, 2, s_new, 64)
        st, out = status(), i32([9, 9])
        mla.append_paged(raw, normal(g, 2, s_new, 8), gain, EPS, THETA, latent, rope, table, i32(lens), kv_len_out=out,
                         counts=None if counts is None else i32(counts), device_status=st)
        assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE
        assert out.tolist() == [lens[0] if entry is None else s_new, 2 + s_new]
        changed = (latent != l0).flatten(0, 1).any(1)
        assert torch.equal(changed, (rope != r0).flatten(0, 1).any(1))
        assert int(changed[:80].sum()) == s_new - left_out and int(changed[80:].sum()) == s_new
    # a negative position: that token alone is left out
    latent, rope = normal(g, 40, size, 64), normal(g, 40, size, 8)
    l0 = latent.clone()
    position = torch.zeros(2, s_new, dtype=torch.int32, device=DEV)
    position[1, 0] = -5
    st = status()
    mla.append_paged(normal(g, 2, s_new, 64), normal(g, 2, s_new, 8), gain, EPS, THETA, latent, rope,
                     torch.arange(40, device=DEV, dtype=torch.int32).view(2, width), i32([0, 0]), positions=position,
                     device_status=st)
    assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE
    assert int((latent != l0).flatten(0, 1).any(1).sum()) == 2 * s_new - 1


# ---------------------------------------------------------------- attention

class Case:
    """Sequences of given lengths in pools that hold NaN everywhere else."""

    def __init__(self, seed, lens, s_q, heads, size, rank=512, rope=64, dtype=BF16, counts=None, tree=False, spare=2):
        g = gen(seed)
        self.lens, self.s_q, self.heads, self.dtype, self.rank = lens, s_q, heads, dtype, rank
        self.B = B = len(lens)
        self.counts = counts or [s_q] * B
        self.counts_d = None if counts is None else i32(counts)
        self.table, pages = page_table(seed, lens, size, spare)
        self.latent, self.rope = dirty_pool(pages, size, rank, dtype), dirty_pool(pages, size, rope, dtype)
        fill(self.latent, self.table, lens, normal(g, B, max(max(lens), 1), rank))
        fill(self.rope, self.table, lens, normal(g, B, max(max(lens), 1), rope))
        q = normal(g, B * s_q, heads, rank + rope)
        q[..., :rank] *= 0.1
        self.q = q.to(dtype)
        self.nodes = self.mask = None
        if tree:
            rng = np.random.default_rng(seed)
            lists = []
            for _ in range(B):
                lists += P.ancestors([int(rng.integers(max(-1, j - 9), j)) for j in range(s_q)])
            self.set_nodes(lists)

    def set_nodes(self, lists):
        self.nodes = lists
        self.mask = torch.from_numpy(P.mask_words(lists, self.s_q)).to(DEV)

    def run(self, mla, out_dtype=None, fillers=7.0, **kw):
        n_q = self.B * self.s_q
        ctx = torch.full((n_q, self.heads, self.rank), fillers, dtype=out_dtype or self.dtype, device=DEV)
        lse, st = torch.full((n_q, self.heads), fillers, device=DEV), status()
        mla.decode_attend_paged(self.q, self.latent, self.rope, self.table, i32(self.lens), self.B, self.s_q, SCALE, ctx,
                                lse, counts=self.counts_d, tree_mask=self.mask, device_status=st, **kw)
        return ctx, lse, int(st) & ~mla.DEVICE_SCORE_RANGE

    def check(self, ctx, lse, rows=None, lists=None):
        kind = "bf16" if self.dtype == BF16 else "f32"
        held = {}
        got, want = [], []
        for n in range(self.B * self.s_q) if rows is None else rows:
            b, i = n // self.s_q, n % self.s_q
            if b not in held:
                held[b] = [P.keys64(p, self.table[b], max(0, self.lens[b])) for p in (self.latent, self.rope)]
            at = P.seen(self.lens[b], self.counts[b], i, self.nodes[n] if self.nodes else None)
            if lists is not None and lists[n] is not None and i < self.counts[b]:
                at = lists[n]
            want.append(P.attend64(P.as64(self.q[n]), held[b][0][at], held[b][1][at], SCALE))
            got.append((P.as64(ctx[n]), P.as64(lse[n])))
        got_c, got_l = map(np.stack, zip(*got))
        want_c, want_l = map(np.stack, zip(*want))
        empty = np.isinf(want_l)
        assert np.array_equal(np.isinf(got_l), empty) and (got_c[empty] == 0).all()
        H.assert_close(got_c, want_c, kind, "ctx")
        # bf16: both score halves are exchanged in fp16 (the bound of the bf16 decode); f32: rounding of 576 products
        assert np.abs(got_l[~empty] - want_l[~empty]).max(initial=0) <= (2e-2 if kind == "bf16" else 1e-4)


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("size,s_q,lens,counts", [
    (64, 1, [1], None),
    (64, 1, [700, 0, 1, 63, 64, 65, 129], None),
    (16, 1, [4999, 33, 16, 17], None),
    (32, 1, [1000, 31], [1, 0]),
    (48, 1, [500, 47, 49], None),
    (128, 1, [129, 128, 3000], None),
    (1, 1, [200, 1], None),
    (7, 1, [701, 6, 7, 8], None),
    (8, 3, [600, 2, 0, 3, 130], None),              # rows shorter than their tokens
    (64, 4, [1500, 1, 777], None),
    (16, 4, [300, 300, 300, 300], [4, 3, 0, 1]),
    (64, 9, [300, 5], None),
    (32, 40, [333, 64, 40], [40, 33, 17]),
    (5, 12, [90, 400], [12, 5]),
])
def test_attend(mla, heads, size, s_q, lens, counts):
    c = Case(heads + size + s_q, lens, s_q, heads, size, counts=counts)
    ctx, lse, st = c.run(mla)
    assert st == 0
    c.check(ctx, lse)


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("size,s_q,lens,counts", [
    (64, 1, [1, 400], None),
    (64, 7, [7, 640, 71], None),                    # a tree without a prefix
    (16, 16, [500, 16, 129], [16, 9, 0]),
    (64, 33, [1000, 64], None),
    (32, 64, [700, 127, 128], [64, 64, 50]),
    (16, 65, [65, 300], None),                      # masks of two words
    (7, 20, [200, 25], None),                       # rows one by one
    (1, 3, [70], None),
    (64, 150, [400], [140]),
])
def test_tree(mla, heads, size, s_q, lens, counts):
    c = Case(heads + size + s_q, lens, s_q, heads, size, counts=counts, tree=True)
    ctx, lse, st = c.run(mla)
    assert st == 0
    c.check(ctx, lse)


@pytest.mark.parametrize("size", [64, 16, 5])
def test_keys_that_are_not_seen_may_hold_anything(mla, size):
    """Siblings that are NaN or infinite leave every node that does not see them alone; a mask need not be a tree,
    may be empty, and may hide a whole tile."""
    s_q = 70
    lens = [s_q, 30 + s_q, 64 + s_q]
    c = Case(11, lens, s_q, 128, size)
    rng = np.random.default_rng(2)
    lists = []
    for n in range(c.B * s_q):
        b, i = n // s_q, n % s_q
        keep = [j for j in range(s_q) if rng.random() < 0.3 and j not in (3, 40, 66)]
        lists.append([] if i == 5 else [69] if i == 6 else [3, 40] if i == 7 else keep)
    c.set_nodes(lists)
    clean = c.run(mla)
    assert clean[2] == 0
    c.check(*clean[:2])
    for b, n in enumerate(lens):
        for node, value in ((3, float("nan")), (40, float("inf")), (66, -float("inf"))):
            t = n - s_q + node
            page = int(c.table[b, t // size])
            c.latent[page, t % size] = value
            c.rope[page, t % size] = value
    ctx, lse, _ = c.run(mla)
    others = torch.tensor([n for n in range(c.B * s_q) if n % s_q != 7], device=DEV)
    assert torch.equal(ctx[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
    assert torch.isnan(ctx[7]).any()


@pytest.mark.parametrize("size", [64, 24, 5])
def test_a_key_that_is_not_finite_is_seen_by_some(mla, size):
    """One element of a key, in either half of the latents or of the rope dims: every token that sees the key gets NaN
    in its whole result, every other one what it got before, also where two tokens of 64 heads share a tile."""
    s_q = 9
    lens = [s_q, 60 + s_q, 64 * 3 + s_q]
    chain = [list(range(i + 1)) for i in range(s_q)]
    star = [[0, i] if i else [0] for i in range(s_q)]
    for heads in (64, 128):
        for lists in (None, star):
            c = Case(13, lens, s_q, heads, size, tree=lists is not None)
            if lists is not None:
                c.set_nodes(lists * c.B)
            clean = c.run(mla)
            assert clean[2] == 0
            c.check(*clean[:2])
            for node, dim, value in ((5, 3, "nan"), (4, 300, "nan"), (8, 515, "nan"), (3, 570, "nan"), (1, 511, "inf")):
                pool, at = (c.latent, dim) if dim < 512 else (c.rope, dim - 512)
                held = []
                for b, n in enumerate(lens):
                    t = n - s_q + node
                    where = int(c.table[b, t // size]), t % size, at
                    held.append((where, pool[where].clone()))
                    pool[where] = float(value)
                ctx, lse, _ = c.run(mla)
                for where, was in held:
                    pool[where] = was
                hit = [node in (lists or chain)[i] for i in range(s_q)] * c.B
                for n, seen in enumerate(hit):
                    if not seen:
                        assert torch.equal(ctx[n], clean[0][n]) and torch.equal(lse[n], clean[1][n]), (heads, node, n)
                    elif value == "nan":
                        assert torch.isnan(ctx[n]).all() and torch.isnan(lse[n]).all(), (heads, node, n)
                    else:
                        assert not torch.isfinite(ctx[n, :, at]).any(), (heads, node, n)


@pytest.mark.parametrize("size", [64, 16, 5])
def test_two_tokens_whose_masks_hide_what_is_not_finite(mla, size):
    """64 heads: siblings that are NaN or infinite, masks that are no tree, an empty one beside a full one."""
    s_q = 71
    lens = [s_q, 30 + s_q, 64 + s_q]
    c = Case(17, lens, s_q, 64, size, counts=[71, 70, 69])
    rng = np.random.default_rng(4)
    lists = []
    for n in range(c.B * s_q):
        i = n % s_q
        keep = [j for j in range(s_q) if rng.random() < 0.3 and j not in (3, 40, 66)]
        lists.append([] if i in (5, 20, 21) else [68] if i == 6 else [3, 40] if i == 7 else keep)
    c.set_nodes(lists)
    clean = c.run(mla)
    assert clean[2] == 0
    c.check(*clean[:2])
    for b, n in enumerate(lens):
        for node, value in ((3, float("nan")), (40, float("inf")), (66, -float("inf"))):
            t = n - c.counts[b] + node
            page = int(c.table[b, t // size])
            c.latent[page, t % size] = value
            c.rope[page, t % size] = value
    ctx, lse, _ = c.run(mla)
    others = torch.tensor([n for n in range(c.B * s_q) if n % s_q != 7], device=DEV)
    assert torch.equal(ctx[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
    assert torch.isnan(ctx[7::s_q]).all()


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("size,s_q,lens,counts,tree", [
    (8, 3, [700, 3, 65], None, False),
    (24, 5, [500, 100], [5, 4], True),
    (40, 2, [1000, 41, 2], None, False),
    (192, 7, [193, 1000], None, True),
    (16, 300, [900, 310], [300, 257], True),
    (64, 1024, [1500], None, True),
])
def test_f32_results_odd_pages_and_large_trees(mla, heads, size, s_q, lens, counts, tree):
    c = Case(heads + size, lens, s_q, heads, size, counts=counts, tree=tree)
    ctx, lse, st = c.run(mla, out_dtype=F32)
    assert st == 0
    c.check(ctx, lse, rows=sorted({i * (c.B * s_q - 1) // 24 for i in range(25)}))


@pytest.mark.parametrize("heads", [64, 128])
def test_many_short_rows(mla, heads):
    """Segments of one tile, hundreds of them to a cluster's stream, with rows of nothing between."""
    rng = np.random.default_rng(6)
    lens = [int(n) for n in rng.integers(0, 130, 700)]
    c = Case(81, lens, 2, heads, 16, counts=[min(n, int(k)) for n, k in zip(lens, rng.integers(0, 3, 700))])
    ctx, lse, st = c.run(mla)
    assert st == 0
    c.check(ctx, lse, rows=range(0, 1400, 9))


def test_calls_at_once_on_two_streams(mla):
    """Two attentions and an append into other pages at once, each call with a workspace of its own from the stream that
    it runs on."""
    cases = [Case(91, [5000, 900], 3, 128, 16), Case(92, [3000, 64, 1], 8, 64, 64, tree=True)]
    want = [c.run(mla) for c in cases]
    lens = [i32(c.lens) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for _ in range(20):
        for c, n, side in zip(cases, lens, streams):
            with torch.cuda.stream(side):
                ctx = torch.empty(c.B * c.s_q, c.heads, 512, dtype=BF16, device=DEV)
                mla.decode_attend_paged(c.q, c.latent, c.rope, c.table, n, c.B, c.s_q, SCALE, ctx, tree_mask=c.mask)
                outs.append(ctx)
    torch.cuda.synchronize()
    for k, ctx in enumerate(outs):
        assert torch.equal(ctx, want[k % 2][0])


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("gain", [1, 4, 64, 512])
def test_scores_at_and_past_the_exchange_range(mla, heads, gain):
    """Halves of a score up to the documented range meet the bf16 bounds; a larger one sets the flag and no other bit."""
    c = Case(15, [900, 40, 333], 2, heads, 64)
    c.q = (c.q.float() * gain).bfloat16()
    ctx, lse, st = torch.zeros(6, heads, 512, dtype=BF16, device=DEV), torch.zeros(6, heads, device=DEV), status()
    mla.decode_attend_paged(c.q, c.latent, c.rope, c.table, i32(c.lens), 3, 2, SCALE, ctx, lse, device_status=st)
    most = 0.0
    for n in range(6):
        lat, rope = (P.keys64(p, c.table[n // 2], c.lens[n // 2] - 1 + n % 2) for p in (c.latent, c.rope))
        q = P.as64(c.q[n])
        for r in (0, 1):
            half = q[:, 256 * r:256 * r + 256] @ lat[:, 256 * r:256 * r + 256].T
            most = max(most, np.abs(half + q[:, 512 + 32 * r:544 + 32 * r] @ rope[:, 32 * r:32 * r + 32].T).max())
    assert int(st) == (mla.DEVICE_SCORE_RANGE if most > mla.FP16_SCORE_LIMIT else 0)
    if most <= mla.FP16_SCORE_LIMIT:
        c.check(ctx, lse)
    assert torch.isfinite(ctx).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("size", [64, 8])
def test_halves_past_fp16_are_clamped(mla, heads, size):
    """One feature of each half decides, with products that fp16 holds exactly or that pass 65504: keys whose clamped
    halves tie for the largest sum share a row's weight, all others have none."""
    c = Case(16, [700, 65], 2, heads, size)
    rng = np.random.default_rng(4)
    for pool_dim in (0, 256):
        fill(c.latent[..., pool_dim:pool_dim + 1], c.table, c.lens,
             torch.from_numpy(rng.integers(-8, 9, (2, 700, 1)).astype(np.float32)).to(DEV))
    c.q.zero_()
    c.q[..., 0], c.q[..., 256] = 2.0 ** 14, 2.0 ** 13
    c.q[:, 1::2] *= -1
    ctx, lse, st = torch.zeros(4, heads, 512, dtype=BF16, device=DEV), torch.zeros(4, heads, device=DEV), status()
    mla.decode_attend_paged(c.q, c.latent, c.rope, c.table, i32(c.lens), 2, 2, SCALE, ctx, lse, device_status=st)
    assert int(st) == mla.DEVICE_SCORE_RANGE
    for n in range(4):
        lat = P.keys64(c.latent, c.table[n // 2], c.lens[n // 2] - 1 + n % 2)
        for h in (0, 1, heads - 1):
            sign = 1 - 2 * (h % 2)
            score = sum(np.clip(sign * g * lat[:, d], -65504, 65504) for g, d in ((2.0 ** 14, 0), (2.0 ** 13, 256)))
            tied = lat[score == score.max()]
            want = tied.mean(0)
            # the result's rounding; against it the weights of ties are rounded alike, a piece's context to fp16
            bound = np.abs(want) * 2.0 ** -8 + np.abs(tied).mean(0) * 2.0 ** -9
            assert (np.abs(P.as64(ctx[n, h]) - want) <= bound).all()
            # four roundings of a value near it
            top = score.max() * SCALE + np.log(len(tied))
            assert abs(float(lse[n, h]) - top) <= top * 2.0 ** -21


@pytest.mark.parametrize("size", [64, 16, 3])
def test_attend_selected(mla, size):
    s_q, k_max = 2, 200
    lens, counts = [3000, 2000, 40, 2500, 900], [2, 2, 2, 2, 1]
    c = Case(40 + size, lens, s_q, 128, size, counts=counts)
    rng = np.random.default_rng(9)
    n_q = c.B * s_q
    sel, cnt, lists = np.zeros((n_q, k_max), np.int32), [], []
    for n in range(n_q):
        b, i = n // s_q, n % s_q
        limit = lens[b] - counts[b] + i + 1
        count = [200, 65, 1, -1, 100][b]
        sel[n] = rng.integers(0, limit, k_max)                       # a multiset, any order
        lists.append(None if count == -1 else sel[n, :count].astype(np.int64))
        cnt.append(count)
    cnt[9] = 999                                                      # of a token that is not there: not read
    sel_d, cnt_d = torch.from_numpy(sel).to(DEV), i32(cnt)
    ctx, lse, st = c.run(mla, sel=sel_d, sel_count=cnt_d)
    assert st == 0
    c.check(ctx, lse, lists=lists)
    # bad positions are skipped and flagged, a bad count empties its row
    sel_d[0, 3], sel_d[0, 7] = -1, lens[0]
    cnt_d[2] = 0
    ctx, lse, st = c.run(mla, sel=sel_d, sel_count=cnt_d)
    assert st == mla.DEVICE_INDEX_OUT_OF_RANGE | mla.DEVICE_BAD_SELECTION_COUNT
    lists[0] = np.delete(lists[0], [3, 7])
    c.check(ctx, lse, rows=[0, 1, 3, 6], lists=lists)
    assert (ctx[2] == 0).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("heads,rank,rope,size,s_q,lens,counts,tree", [
    (4, 32, 8, 16, 1, [64, 1, 0, 1500], None, False),
    (3, 37, 6, 5, 2, [130, 1, 20], [2, 1, 0], False),
    (2, 512, 64, 64, 9, [900, 40], None, True),
    (1, 1, 2, 3, 70, [70, 95], [70, 60], True),
    (5, 100, 0, 7, 4, [33], None, True),
])
def test_attend_f32(mla, heads, rank, rope, size, s_q, lens, counts, tree, out_dtype):
    c = Case(rank, lens, s_q, heads, size, rank, rope, F32, counts, tree)
    ctx, lse, st = c.run(mla)
    assert st == 0
    c.check(ctx, lse)
    if out_dtype == BF16:
        assert torch.equal(c.run(mla, out_dtype=BF16)[0], ctx.bfloat16())


def test_attend_f32_selected_and_special(mla):
    c = Case(90, [300, 200, 50], 1, 3, 16, 40, 8, F32)
    sel = torch.randint(0, 50, (3, 20), generator=gen(1), device=DEV, dtype=torch.int32)
    lists = [P.as64(sel[0]).astype(np.int64), P.as64(sel[1, :7]).astype(np.int64), None]
    ctx, lse, st = c.run(mla, sel=sel, sel_count=i32([20, 7, -1]))
    assert st == 0
    c.check(ctx, lse, lists=lists)
    # NaN among a row's keys is NaN; a bad page is flagged, the other rows stay
    c.latent[int(c.table[0, 2]), 3] = float("nan")
    c.table[1, 1] = -1
    ctx, lse, st = c.run(mla)
    assert st == mla.DEVICE_INDEX_OUT_OF_RANGE and torch.isnan(ctx[0]).all()
    c.check(ctx, lse, rows=[2])


def test_views_and_shared_pages(mla):
    """Rows inside wider pools, pages between another layer's, a f32 context in wider rows; two sequences that share
    the pages of their prefix."""
    for size, step in ((16, 1), (64, 2), (10, 2)):
        c = Case(21, [400, 400, 130], 2, 128, size)
        pages = c.latent.shape[0]
        wide = torch.full((pages, step, size, 704), float("nan"), dtype=BF16, device=DEV)
        wide[:, 0, :, 32:544], wide[:, 0, :, 600:664] = c.latent, c.rope
        latent, rope = wide[:, 0, :, 32:544], wide[:, 0, :, 600:664]
        shared = 300 // size
        c.table[1, :shared] = c.table[0, :shared]
        qs = torch.zeros(6, 128, 640, dtype=BF16, device=DEV)
        qs[..., 64:] = c.q
        ctxs = torch.zeros(6, 128, 520, device=DEV)
        lse, st = torch.zeros(6, 128, device=DEV), status()
        wide_table = torch.full((3, c.table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
        wide_table[:, 2:2 + c.table.shape[1]] = c.table
        mla.decode_attend_paged(qs[..., 64:], latent, rope, wide_table[:, 2:-3], i32(c.lens), 3, 2, SCALE, ctxs[..., 4:516],
                                lse, device_status=st)
        assert int(st) & ~mla.DEVICE_SCORE_RANGE == 0
        c.check(ctxs[..., 4:516], lse)
        assert (ctxs[..., :4] == 0).all() and (ctxs[..., 516:] == 0).all()


@pytest.mark.parametrize("size", [64, 16, 7])
def test_bad_rows_and_pages(mla, size):
    for lens, counts, entry in [([-1, 100], None, None), ([10 ** 6, 100], None, None), ([100, 100], [2, 1], None),
                                ([100, 100], [-1, 1], None), ([100, 100], None, -1), ([100, 100], None, 10 ** 6)]:
        c = Case(31, [100, 100], 1, 64, size, counts=counts)
        c.lens = lens
        if entry is not None:
            c.table[0, 0] = entry
        ctx, lse, st = c.run(mla)
        assert st == mla.DEVICE_INDEX_OUT_OF_RANGE
        if entry is None:
            assert (ctx[0] == 0).all() and torch.isneginf(lse[0]).all()
        c.check(ctx, lse, rows=[1])


@pytest.mark.parametrize("tree", [False, True])
def test_many_rows_take_the_planner(mla, tree):
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 500, 90)]
    counts = [min(n, int(k)) for n, k in zip(lens, rng.integers(0, 4, 90))]
    c = Case(51, lens, 3, 64, 32, counts=counts, tree=tree)
    ctx, lse, st = c.run(mla)
    assert st == 0
    c.check(ctx, lse, rows=range(0, 270, 4))


@pytest.mark.parametrize("size,tree", [(64, False), (16, True), (6, True)])
def test_long_rows_in_many_pieces(mla, size, tree):
    c = Case(61, [20011, 40, 9000], 5, 128, size, tree=tree)
    ctx, lse, st = c.run(mla)
    assert st == 0
    c.check(ctx, lse, rows=[0, 4, 5, 9, 12, 14])


def test_pools_past_32_bits(mla):
    """Pages that lie past 2^32 bytes (and 2^31 elements) of the pool."""
    for size in (64, 20):
        pages = 3 * 2 ** 21 // size                                   # 6.4 GB of latents
        c = Case(71, [300, 70], 4, 128, size, tree=True)
        latent = torch.empty(pages, size, 512, dtype=BF16, device=DEV)
        rope = torch.empty(pages, size, 64, dtype=BF16, device=DEV)
        n = c.latent.shape[0]
        latent[-n:], rope[-n:] = c.latent, c.rope
        small = c.table.clone()
        c.table += pages - n
        c.latent, c.rope = latent, rope
        ctx, lse, st = c.run(mla)
        assert st == 0
        c.check(ctx, lse)
        kv = i32(c.lens)
        raw, raw_rope = normal(gen(1), 2, 1, 512).bfloat16(), normal(gen(2), 2, 1, 64).bfloat16()
        gain = torch.ones(512, device=DEV).bfloat16()
        kv -= 1
        mla.append_paged(raw, raw_rope, gain, EPS, THETA, latent, rope, c.table, kv)
        l2, r2 = latent[-n:].clone(), rope[-n:].clone()
        mla.append_paged(raw, raw_rope, gain, EPS, THETA, l2, r2, small, kv)
        assert torch.equal(torch.nan_to_num(l2), torch.nan_to_num(latent[-n:]))
        mla.commit_paged([latent, rope], c.table, i32([200, 10]), i32([[1, 5], [0, 9]]), i32([2, 2]))
        mla.commit_paged([l2, r2], small, i32([200, 10]), i32([[1, 5], [0, 9]]), i32([2, 2]))
        assert torch.equal(torch.nan_to_num(l2), torch.nan_to_num(latent[-n:]))
        assert torch.equal(torch.nan_to_num(r2), torch.nan_to_num(rope[-n:]))
        del latent, rope, c


# ---------------------------------------------------------------- trees

def random_parents(rng, n):
    return [int(rng.integers(-1, j)) if rng.random() < 0.5 else max(-1, j - int(rng.integers(1, 4))) for j in range(n)]


@pytest.mark.parametrize("n,counts", [(1, None), (5, [5, 0, 3]), (64, None), (65, [65, 64, 1]), (200, None),
                                      (1024, [1024, 700, 1023])])
def test_plan(mla, n, counts):
    rng = np.random.default_rng(n)
    B = 3
    parents = [random_parents(rng, n) for _ in range(B)]
    parents[1] = list(range(-1, n - 1))                               # one chain
    if n > 2:
        parents[2] = [-1] * n                                         # roots only
    lens = [0, 77, 31000]
    wide = torch.full((B, n + 3), 99, dtype=torch.int32, device=DEV)
    wide[:, 1:n + 1] = i32(parents)
    pos = torch.full((B, n), -9, dtype=torch.int32, device=DEV)
    mask = torch.full((B * n, -(-n // 64)), -9, dtype=torch.int64, device=DEV)
    st = status()
    mla.tree_plan(wide[:, 1:n + 1], i32(lens), pos, mask, counts=None if counts is None else i32(counts), device_status=st)
    assert int(st) == 0
    counts = counts or [n] * B
    for b in range(B):
        lists = [a if j < counts[b] else [] for j, a in enumerate(P.ancestors(parents[b]))]
        assert np.array_equal(mask[b * n:(b + 1) * n].cpu().numpy(), P.mask_words(lists, n))
        assert pos[b].tolist() == [lens[b] + max(0, len(a) - 1) for a in lists]


def test_plan_bad_parents_and_counts(mla):
    pos = torch.zeros(4, 4, dtype=torch.int32, device=DEV)
    mask = torch.zeros(16, 1, dtype=torch.int64, device=DEV)
    st = status()
    parents = i32([[-1, 1, 0, 2], [-2, 0, 5, 1], [-1, 0, 1, 2], [-1, 0, 9, 9]])   # below itself, -2, behind, of no node
    mla.tree_plan(parents, None, pos, mask, counts=i32([4, 4, 5, 2]), device_status=st)
    assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE
    assert mask.view(4, 4).tolist() == [[1, 2, 5, 13], [1, 3, 4, 11], [0, 0, 0, 0], [1, 3, 0, 0]]
    assert pos.tolist() == [[0, 0, 1, 2], [0, 1, 0, 2], [0, 0, 0, 0], [0, 1, 0, 0]]
    st = status()
    mla.tree_plan(parents, None, pos, mask, counts=i32([1, 0, 4, 2]), device_status=st)
    assert int(st) == 0


# ---------------------------------------------------------------- commit

@pytest.mark.parametrize("size,width", [(64, 5), (16, 12), (1, 6), (7, 40), (3, 200)])
def test_commit(mla, size, width):
    g, rng = gen(size), np.random.default_rng(size)
    n_nodes = 3 * width
    lens = [0, 50, size, 200, 33]
    B = len(lens)
    table, pages = page_table(size, [n + n_nodes for n in lens], size)
    path = np.stack([np.sort(rng.permutation(n_nodes)[:width]) for _ in range(B)]).astype(np.int32)
    path[1] = np.arange(width)                                        # already in place
    counts = [width, width, 0, width // 2, 1]
    wide = torch.randint(0, 200, (pages, size, 72), generator=g, device=DEV, dtype=torch.uint8)
    arrays = [normal(g, pages, size, 512).bfloat16(), normal(g, pages, 2, size, 64).bfloat16()[:, 1],
              normal(g, pages, size, 8)[..., 2:8], torch.randint(0, 9, (pages, size, 3), generator=g, device=DEV).short(),
              wide[..., 1:38], normal(g, pages, size, 130)[..., :130]]
    before = [a.clone() for a in arrays]
    around = wide.clone()
    n, out, st = i32(lens), i32([3] * B), status()
    mla.commit_paged(arrays, table, n, torch.from_numpy(path).to(DEV), i32(counts), kv_len_out=out, device_status=st)
    assert int(st) == 0 and out.tolist() == [k + c for k, c in zip(lens, counts)] and n.tolist() == lens
    for a, was in zip(arrays, before):
        want = was.clone()
        for b in range(B):
            to = torch.arange(counts[b], device=DEV) + lens[b]
            of = torch.from_numpy(path[b, :counts[b]]).to(DEV).long() + lens[b]
            row = table[b].long()
            want[row[to // size], to % size] = was[row[of // size], of % size]
        assert torch.equal(a, want)
    done = [a.clone() for a in arrays]
    wide[..., 1:38] = 0
    around[..., 1:38] = 0
    assert torch.equal(wide, around)
    # the same with a handle, lengths in place
    pools = mla.PagedArrays(before)
    mla.commit_paged(pools, table, n, torch.from_numpy(path).to(DEV), i32(counts), kv_len_out=n)
    assert n.tolist() == out.tolist() and all(torch.equal(a, b) for a, b in zip(done, before))


def test_commit_bad_entries(mla):
    g = gen(9)
    table = torch.arange(40, device=DEV, dtype=torch.int32).view(4, 10)      # 40 rows of 4 each
    a = normal(g, 40, 4, 64)
    was = a.clone()
    path = i32([[2, 1, 5, 37], [3, 3, 4, 6], [0, 2, 3, 9], [1, 2, 3, 4]])
    out, st = i32([0] * 4), status()
    mla.commit_paged([a], table, i32([4, 0, 36, -1]), path, i32([4, 4, 4, 2]), kv_len_out=out, device_status=st)
    assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE and out.tolist() == [8, 4, 40, -1]
    want = was.clone().view(4, 40, 64)
    old = was.view(4, 40, 64)
    want[0, 4], want[0, 6] = old[0, 6], old[0, 9]                     # 1 is not above 2; 37 is behind the table
    want[1, 0], want[1, 2], want[1, 3] = old[1, 3], old[1, 4], old[1, 6]
    want[2, 37], want[2, 38] = old[2, 38], old[2, 39]
    assert torch.equal(a.view(4, 40, 64), want)
    for counts in ([5, 0, 0, 0], [-1, 0, 0, 0]):
        a, st = was.clone(), status()
        mla.commit_paged([a], table, i32([4, 0, 0, 0]), path, i32(counts), kv_len_out=out, device_status=st)
        assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE and out.tolist() == [4, 0, 0, 0] and torch.equal(a, was)
    table[0, 1] = 40
    a, st = was.clone(), status()
    mla.commit_paged([a], table, i32([0, 0, 0, 0]), i32([[1, 6, 9, 10]] * 4), i32([3, 0, 0, 0]), device_status=st)
    assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE
    want = was.clone()
    want[0, 0], want[0, 2] = was[0, 1], was[2, 1]
    assert torch.equal(a, want)


# ---------------------------------------------------------------- together

def serve(mla, s, stream=None):
    """One verification round: plan, append, query rotation, attention, commit."""
    mla.tree_plan(s["parents"], s["len"], s["pos"], s["mask"], counts=s["counts"], device_status=s["status"], stream=stream)
    mla.append_paged(s["raw"], s["raw_rope"], s["gain"], EPS, THETA, s["latent"], s["rope"], s["table"], s["len"],
                     kv_len_out=s["after"], positions=s["pos"], counts=s["counts"], device_status=s["status"],
                     stream=stream)
    B, n = s["parents"].shape
    x = s["q_raw"].view(B * n, 1, 128, 576)[..., 512:]
    mla.rope_partial_interleaved(x, s["q"].view(B * n, 1, 128, 576)[..., 512:], 64, THETA,
                                 row_offsets=s["pos"].view(-1), stream=stream)
    mla.decode_attend_paged(s["q"], s["latent"], s["rope"], s["table"], s["after"], B, n, SCALE, s["ctx"], s["lse"],
                            counts=s["counts"], tree_mask=s["mask"], workspace=s["ws"], device_status=s["status"],
                            stream=stream)
    mla.commit_paged([s["latent"], s["rope"]], s["table"], s["len"], s["path"], s["accepted"], kv_len_out=s["len"],
                     device_status=s["status"], stream=stream)


def serve_state(mla, seed, lens, n=12, size=16, heads=128):
    g, rng = gen(seed), np.random.default_rng(seed)
    B = len(lens)
    table, pages = page_table(seed, [k + 6 * n for k in lens], size)
    parents = [random_parents(rng, n) for _ in range(B)]
    paths = [max(P.ancestors(p), key=len) for p in parents]
    depth = max(map(len, paths))
    s = dict(table=table, latent=dirty_pool(pages, size, 512, BF16), rope=dirty_pool(pages, size, 64, BF16), len=i32(lens),
             after=i32(lens), parents=i32(parents), pos=torch.zeros(B, n, dtype=torch.int32, device=DEV),
             mask=torch.zeros(B * n, 1, dtype=torch.int64, device=DEV), counts=i32([n] * (B - 1) + [n - 2]),
             raw=normal(g, B, n, 512).bfloat16(), raw_rope=normal(g, B, n, 64).bfloat16(),
             gain=torch.ones(512, device=DEV).bfloat16(), q_raw=normal(g, B * n, heads, 576).bfloat16() * 0.1,
             ctx=torch.zeros(B * n, heads, 512, dtype=BF16, device=DEV), lse=torch.zeros(B * n, heads, device=DEV),
             ws=torch.empty(mla.decode_workspace_size(B, n, heads, 512, 64, table.shape[1] * size), dtype=torch.uint8,
                            device=DEV), status=status(),
             path=i32([p + [0] * (depth - len(p)) for p in paths]),
             accepted=i32([len([j for j in p if j < (n if b < B - 1 else n - 2)]) for b, p in enumerate(paths)]))
    s["q"] = s["q_raw"].clone()
    fill(s["latent"], table, lens, normal(g, B, max(lens), 512))
    fill(s["rope"], table, lens, normal(g, B, max(lens), 64))
    s["lists"] = [P.ancestors(p) for p in parents]
    return s


def check_round(s, lens):
    """The round's attention against 64 bits, from the pools as they were before the commit (``s['held']``)."""
    n = s["parents"].shape[1]
    counts = s["counts"].tolist()
    got, want = [], []
    for b, k in enumerate(lens):
        lat, rope = (P.keys64(p, s["table"][b], k + counts[b]) for p in s["held"])
        for i in range(n):
            at = P.seen(k + counts[b], counts[b], i, s["lists"][b][i])
            want.append(P.attend64(P.as64(s["q"][b * n + i]), lat[at], rope[at], SCALE)[0])
            got.append(P.as64(s["ctx"][b * n + i]))
    H.assert_close(np.stack(got), np.stack(want), "bf16", "ctx")


def test_rounds_together_on_another_stream(mla):
    """Two rounds step by step on a side stream; the accepted tokens are then a plain sequence: appending them in a
    row gives the same pages."""
    lens = [100, 0, 700]
    s = serve_state(mla, 5, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plain = [s["latent"].clone(), s["rope"].clone()]
    n0 = list(lens)
    for _ in range(2):
        kept = s["latent"].clone(), s["rope"].clone(), s["len"].clone()
        torch.cuda.synchronize()
        serve(mla, s, side)
        side.synchronize()
        # the pools before the commit: the same append again
        mla.append_paged(s["raw"], s["raw_rope"], s["gain"], EPS, THETA, kept[0], kept[1], s["table"], kept[2],
                         positions=s["pos"], counts=s["counts"])
        s["held"] = kept[:2]
        check_round(s, kept[2].tolist())
        accepted = s["accepted"].tolist()
        rows = [s["path"][b, :accepted[b]].long() for b in range(3)]
        most = max(max(accepted), 1)
        raw, raw_rope = torch.zeros(3, most, 512, dtype=BF16, device=DEV), torch.zeros(3, most, 64, dtype=BF16, device=DEV)
        for b in range(3):
            raw[b, :accepted[b]], raw_rope[b, :accepted[b]] = s["raw"][b, rows[b]], s["raw_rope"][b, rows[b]]
        mla.append_paged(raw, raw_rope, s["gain"], EPS, THETA, *plain, s["table"], i32(n0), counts=i32(accepted))
        n0 = [k + a for k, a in zip(n0, accepted)]
        assert s["len"].tolist() == n0
        for b in range(3):
            for pool, want in zip((s["latent"], s["rope"]), plain):
                assert np.array_equal(P.keys64(pool, s["table"][b], n0[b]), P.keys64(want, s["table"][b], n0[b]))
        s["raw"].copy_(normal(gen(n0[0]), *s["raw"].shape))
    assert int(s["status"]) & ~mla.DEVICE_SCORE_RANGE == 0


def test_two_graphs_replayed(mla):
    """Rounds of two batches captured into two graphs with their own workspaces, replayed in turn and at once."""
    a, b = serve_state(mla, 6, [90, 300]), serve_state(mla, 7, [0, 1200, 64, 17], n=9, size=64)
    graphs, starts = [], []
    for s in (a, b):
        starts.append({k: v.clone() for k, v in s.items() if torch.is_tensor(v)})
        serve(mla, s)
        torch.cuda.synchronize()
        s["want"] = s["ctx"].clone(), s["lse"].clone(), s["latent"].clone(), s["len"].clone()
        for k, v in starts[-1].items():
            s[k].copy_(v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            serve(mla, s)
        graphs.append(graph)
    for s, graph in zip((a, b), graphs):
        graph.replay()
    torch.cuda.synchronize()
    for s in (a, b):
        for got, want in zip((s["ctx"], s["lse"], s["latent"], s["len"]), s["want"]):
            assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))
    streams = [torch.cuda.Stream() for _ in graphs]
    for s, start in zip((a, b), starts):
        for k, v in start.items():
            s[k].copy_(v)
    torch.cuda.synchronize()
    for graph, stream in zip(graphs, streams):
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for s in (a, b):
        for got, want in zip((s["ctx"], s["lse"], s["latent"], s["len"]), s["want"]):
            assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))


def test_pages_and_windows_give_the_same(mla):
    """A cache in contiguous windows seen as pages of one row after another (the kernels add in different orders: the
    bf16 bounds, twice over), and a chain as a tree against tokens in a row (the same bits)."""
    g = gen(8)
    B, T, heads = 3, 640, 128
    latent, rope = normal(g, B, T, 512).bfloat16(), normal(g, B, T, 64).bfloat16()
    lens = i32([640, 77, 1])
    for s_q in (1, 3):
        q = normal(g, B * s_q, heads, 576).bfloat16() * 0.1
        want, got, tree = (torch.zeros(B * s_q, heads, 512, dtype=BF16, device=DEV) for _ in range(3))
        mla.decode_attend(q, latent, rope, None, lens, B, s_q, SCALE, want)
        table = torch.arange(B * 10, device=DEV, dtype=torch.int32).view(B, 10)
        pools = latent.view(-1, 64, 512), rope.view(-1, 64, 64)
        mla.decode_attend_paged(q, *pools, table, lens, B, s_q, SCALE, got)
        assert (got.float() - want.float()).abs().max() <= 4e-2
        assert (got.float() - want.float()).norm() <= 1e-2 * want.float().norm()
        parents = torch.arange(-1, s_q - 1, device=DEV, dtype=torch.int32).expand(B, s_q)
        pos = torch.zeros(B, s_q, dtype=torch.int32, device=DEV)
        mask = torch.zeros(B * s_q, 1, dtype=torch.int64, device=DEV)
        mla.tree_plan(parents, None, pos, mask)
        mla.decode_attend_paged(q, *pools, table, lens, B, s_q, SCALE, tree, tree_mask=mask)
        assert torch.equal(tree, got)
