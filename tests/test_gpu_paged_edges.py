"""The paged attention's flags and edges on the GPU: what no token sees raises no flag, selections beside freed pages and
bad positions, pages of one row inside wider rows, workspaces of the size asked for, repeated calls."""
import numpy as np
import pytest
import torch

from tests import paged_reference as P
from tests.test_gpu_paged import DEV, F32, SCALE, Case, fill, i32, normal, gen, status

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


def attend(mla, c, **kw):
    """Case.run with every bit of the status."""
    n_q = c.B * c.s_q
    ctx = torch.full((n_q, c.heads, c.rank), 7.0, dtype=c.dtype, device=DEV)
    lse, st = torch.full((n_q, c.heads), 7.0, device=DEV), status()
    mla.decode_attend_paged(c.q, c.latent, c.rope, c.table, i32(c.lens), c.B, c.s_q, SCALE, ctx, lse, counts=c.counts_d,
                            tree_mask=c.mask, device_status=st, **kw)
    return ctx, lse, int(st)


# ---------------------------------------------------------------- the score range

@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("size", [64, 16, 7])
@pytest.mark.parametrize("tree", [False, True])
def test_tokens_that_are_not_there_set_no_flag(mla, heads, size, tree):
    """A padded batch: the query memory of tokens at and past a row's count holds anything."""
    lens, counts = [700, 64, 300, 130, 1], [3, 1, 0, 5, 1]
    c = Case(heads + size, lens, 5, heads, size, counts=counts, tree=tree)
    clean = attend(mla, c)
    assert clean[2] == 0
    c.check(*clean[:2])
    there = torch.tensor([i < counts[b] for b in range(5) for i in range(5)], device=DEV)
    for value in (3000.0, 1e30, float("inf"), float("nan")):
        c.q[~there] = value
        ctx, lse, st = attend(mla, c)
        assert st == 0, value
        assert torch.equal(ctx, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("size", [64, 8, 7])
def test_large_keys_that_a_token_does_not_see_set_no_flag(mla, heads, size):
    """A sibling that only one token sees, whose query is 0: its large finite key is nobody's large score.  Seen by a
    token with a query, it is."""
    s_q, big = 6, 5
    lens = [s_q, 61 + s_q, 500]
    star = [[0, i] if i else [0] for i in range(s_q)]
    chain = [list(range(i + 1)) for i in range(s_q)]
    for lists in (star, chain):
        c = Case(23, lens, s_q, heads, size, tree=True)
        c.set_nodes(lists * 3)
        c.q.view(3, s_q, heads, 576)[:, big] = 0
        clean = attend(mla, c)
        assert clean[2] == 0
        c.check(*clean[:2])
        for b, n in enumerate(lens):
            t = n - s_q + big
            c.latent[int(c.table[b, t // size]), t % size] = 3000.0
        ctx, lse, st = attend(mla, c)
        assert st == 0
        others = torch.tensor([n for n in range(3 * s_q) if n % s_q != big], device=DEV)
        assert torch.equal(ctx[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
        # one head of that token in one row, on one feature of either half
        for dim in (1, 300):
            c.q[s_q + big, heads - 1, dim] = 1.0
            assert attend(mla, c)[2] == mla.DEVICE_SCORE_RANGE
            c.q[s_q + big, heads - 1, dim] = 0
        assert attend(mla, c)[2] == 0


@pytest.mark.parametrize("heads", [64, 128])
def test_a_large_score_in_any_tile_sets_the_flag(mla, heads):
    """One key of a row, one token and head: in a whole tile, in the last one, in a row behind padding."""
    lens, counts, s_q = [400, 200, 131], [3, 0, 1], 3
    for b, t, i in ((0, 3, 0), (0, 397, 0), (0, 399, 2), (2, 5, 0), (2, 130, 0)):
        c = Case(29, lens, s_q, heads, 16, counts=counts)
        c.q[..., 7] = 0
        page = int(c.table[b, t // 16])
        c.latent[page, t % 16, 7] = 1000.0
        assert attend(mla, c)[2] == 0
        c.q[b * s_q + i, 11, 7] = 1.0
        assert attend(mla, c)[2] == mla.DEVICE_SCORE_RANGE, (b, t, i)


def test_calls_repeat_bit_for_bit(mla):
    for case in (Case(41, [4096], 1, 128, 64), Case(42, [9000, 300, 5000], 4, 128, 16), Case(43, [3000, 700], 90, 64, 64),
                 Case(44, [4000], 16, 128, 64, tree=True), Case(45, [2000, 900], 64, 128, 32, tree=True),
                 Case(46, [900, 80], 5, 64, 7)):
        first = attend(mla, case)
        for _ in range(5):
            again = attend(mla, case)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1]) and again[2] == first[2]


# ---------------------------------------------------------------- selections

def selection(c, rng, lows, counts, k_max):
    """Positions of each row from ``lows`` on, a multiset in any order."""
    sel = np.stack([rng.integers(low, n, k_max) for low, n in zip(lows, c.lens)]).astype(np.int32)
    lists = [None if k == -1 else sel[b, :k].astype(np.int64) for b, k in enumerate(counts)]
    return torch.from_numpy(sel).to(DEV), i32(counts), lists


@pytest.mark.parametrize("heads,dtype", [(64, BF16), (128, BF16), (3, F32)])
@pytest.mark.parametrize("size", [64, 16, 3])
def test_selections_that_need_no_first_page(mla, heads, dtype, size):
    """The pages of a row's first keys are freed; its selection names none of their keys, in numbers that fill a tile,
    end inside one, or are one."""
    shape = {} if dtype == BF16 else dict(rank=40, rope=8, dtype=F32)
    counts = [200, 64, 1, 130, 65]
    c = Case(50 + size, [1000, 500, 400, 900, 300], 1, heads, size, **shape)
    sel, cnt, lists = selection(c, np.random.default_rng(1), [64] * 5, counts, 200)
    for b in range(5):
        c.table[b, :64 // size] = -1 if b % 2 else 10 ** 6
    n = c.B * c.s_q
    ctx, lse, st = attend(mla, c, sel=sel, sel_count=cnt)
    assert st == 0
    whole = c.table.clone()
    c.table[:, :64 // size] = 0                       # (the reference reads the row's pages whole)
    c.check(ctx, lse, rows=range(n), lists=lists)
    # the page of a key that is named is still needed
    c.table.copy_(whole)
    sel[1, 5] = 0
    assert attend(mla, c, sel=sel, sel_count=cnt)[2] == mla.DEVICE_INDEX_OUT_OF_RANGE


@pytest.mark.parametrize("heads,dtype", [(64, BF16), (128, BF16), (3, F32)])
@pytest.mark.parametrize("size", [64, 16, 3])
def test_bad_positions_meet_no_key(mla, heads, dtype, size):
    """Positions out of range in any place of a selection: flagged and left out, whatever the row's first key and the
    pool's first row hold."""
    shape = {} if dtype == BF16 else dict(rank=40, rope=8, dtype=F32)
    counts = [200, 64, 2, 70]
    c = Case(60 + size, [1000, 500, 400, 90], 1, heads, size, **shape)
    sel, cnt, lists = selection(c, np.random.default_rng(2), [1] * 4, counts, 200)
    for value in (float("nan"), float("inf"), 3e4):
        for b in range(4):
            c.latent[int(c.table[b, 0]), 0] = value
            c.rope[int(c.table[b, 0]), 0] = value
        pool_row = c.latent[0, 0].clone()
        owner = [(b, int(k)) for b in range(4) for k in (c.table[b] == 0).nonzero().flatten()[:1]]
        if not any(k * size in lists[b] for b, k in owner):
            c.latent[0, 0] = value
        assert attend(mla, c, sel=sel, sel_count=cnt)[2] == 0
        held = sel.clone()
        sel[0, [0, 63, 64, 199]] = i32([-1, 1000, 2 ** 31 - 1, -2 ** 31])
        sel[1, 7], sel[2, 1], sel[3, 64:70] = 500, 400, -7
        left = [np.delete(lists[0], [0, 63, 64, 199]), np.delete(lists[1], 7), lists[2][:1], lists[3][:64]]
        ctx, lse, st = attend(mla, c, sel=sel, sel_count=cnt)
        assert st == mla.DEVICE_INDEX_OUT_OF_RANGE
        c.check(ctx, lse, lists=left)
        sel.copy_(held)
        c.latent[0, 0] = pool_row
    # nothing but bad positions: no key at all
    sel[2, :2] = -1
    ctx, lse, st = attend(mla, c, sel=sel, sel_count=cnt)
    assert st == mla.DEVICE_INDEX_OUT_OF_RANGE
    assert (ctx[2] == 0).all() and torch.isneginf(lse[2]).all()


# ---------------------------------------------------------------- pages of one row

@pytest.mark.parametrize("heads", [64, 128])
def test_pages_of_one_row_inside_wider_rows(mla, heads):
    """A pool [pages, width] seen as pages of one row: the stride of the page axis alone says where a row lies."""
    lens, s_q = [300, 64, 5], 3
    for tree in (False, True):
        c = Case(70, lens, s_q, heads, 1, tree=tree)
        clean = attend(mla, c)
        assert clean[2] == 0
        c.check(*clean[:2])
        wide = torch.full((c.latent.shape[0], 712), float("nan"), dtype=BF16, device=DEV)
        wide[:, 32:544], wide[:, 600:664] = c.latent[:, 0], c.rope[:, 0]
        held = c.latent, c.rope
        c.latent, c.rope = wide[:, 32:544].unsqueeze(1), wide[:, 600:664].unsqueeze(1)
        assert c.latent.stride() == (712, 512, 1) and c.rope.stride() == (712, 64, 1)
        ctx, lse, st = attend(mla, c)
        assert st == 0 and torch.equal(ctx, clean[0]) and torch.equal(lse, clean[1])
    sel = torch.arange(3 * s_q * 70, device=DEV, dtype=torch.int32).view(3 * s_q, 70).remainder(5).clamp(max=2)
    cnt = i32([70, 65, 1] * 3)
    got = attend(mla, c_without_tree(c), sel=sel, sel_count=cnt)
    c.latent, c.rope = held
    want = attend(mla, c, sel=sel, sel_count=cnt)
    assert got[2] == want[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # append and commit over the same views
    g = gen(3)
    raw, raw_rope = normal(g, 3, 2, 512).bfloat16(), normal(g, 3, 2, 64).bfloat16()
    gain = torch.ones(512, device=DEV).bfloat16()
    for latent, rope in (held, (wide[:, 32:544].unsqueeze(1), wide[:, 600:664].unsqueeze(1))):
        mla.append_paged(raw, raw_rope, gain, 1e-6, 1e4, latent, rope, c.table, i32([n - 2 for n in lens]))
        mla.commit_paged([latent, rope], c.table, i32([n - 3 for n in lens]), i32([[1]] * 3), i32([1, 0, 1]))
    assert torch.equal(torch.nan_to_num(wide[:, 32:544]), torch.nan_to_num(held[0][:, 0]))
    assert torch.equal(torch.nan_to_num(wide[:, 600:664]), torch.nan_to_num(held[1][:, 0]))
    assert torch.isnan(wide[:, :32]).all() and torch.isnan(wide[:, 544:600]).all() and torch.isnan(wide[:, 664:]).all()


def c_without_tree(c):
    c.nodes = c.mask = None
    return c


# ---------------------------------------------------------------- workspaces

@pytest.mark.parametrize("lens,s_q,heads,size,tree", [
    ([4096], 1, 128, 64, False),                           # one row in many pieces
    ([9000, 300, 5000], 4, 128, 16, False),
    ([2500, 1900, 77], 300, 64, 64, False),                # pairs, many more units than groups of clusters
    ([2500, 700], 150, 128, 32, False),
    ([3000, 900], 90, 64, 16, True),
    ([int(n) for n in np.random.default_rng(6).integers(0, 700, 500)], 1, 128, 16, False),
    ([2500, 300], 40, 128, 7, False),                      # row by row: a unit a token
    ([1500] * 80, 1, 64, 5, False),
    ([20000] * 19, 4, 128, 64, False),                     # as many units as groups, one more, two
    ([20000] * 19 + [9000], 4, 128, 64, False),
    ([4000] * 77, 1, 128, 64, False),
])
def test_the_workspace_asked_for_is_enough(mla, lens, s_q, heads, size, tree):
    """Of that size to the byte, between bytes that must stay, filled with NaN before the call; a larger one gives the
    same bits."""
    c = Case(80, lens, s_q, heads, size, counts=[min(n, s_q) for n in lens], tree=tree)
    need = mla.decode_paged_workspace_size(c.B, s_q, heads, 512, 64, c.table.shape[1] * size)
    guard = 1 << 16
    room = torch.full((need + 2 * guard,), 0xFF, dtype=torch.uint8, device=DEV)
    ctx, lse, st = attend(mla, c, workspace=room[guard:guard + need])
    assert st == 0
    assert (room[:guard] == 0xFF).all() and (room[guard + need:] == 0xFF).all()
    c.check(ctx, lse, rows=sorted({k * (c.B * s_q - 1) // 12 for k in range(13)}))
    large = torch.full((mla.decode_workspace_size(c.B, s_q, heads, 512, 64, c.table.shape[1] * size) + 4096,), 0xFF,
                       dtype=torch.uint8, device=DEV)
    again = attend(mla, c, workspace=large)
    assert torch.equal(again[0], ctx) and torch.equal(again[1], lse)
    with pytest.raises(mla.MLAError):
        attend(mla, c, workspace=room[guard:guard + need - 256])


# ---------------------------------------------------------------- threads and graphs

def test_calls_from_two_threads(mla):
    """Each thread on its own stream; a call leaves the interpreter to the other thread while it launches."""
    import threading

    cases = [Case(91, [3000, 900], 3, 128, 16), Case(92, [2000, 64, 1], 8, 64, 64, tree=True)]
    want = [attend(mla, c) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(c, ref):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(50):
                    got = attend(mla, c)
                    if not (torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and got[2] == ref[2]):
                        raise AssertionError("another result")
                    with pytest.raises(AssertionError):
                        mla.tree_plan(c.table.long(), None, c.table, c.table)
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("heads,size,s_q,tree", [(128, 64, 1, False), (64, 16, 5, False), (128, 7, 3, False), (64, 32, 40, True)])
def test_a_graph_follows_its_inputs(mla, heads, size, s_q, tree):
    """Lengths, counts, pages, masks and queries change between replays: each gives what a call then gives."""
    lens = [900, 300, 64]
    c = Case(95, lens, s_q, heads, size, counts=[s_q] * 3, tree=tree)
    n_q = 3 * s_q
    length, st = i32(lens), status()
    ctx, lse = torch.zeros(n_q, heads, 512, dtype=BF16, device=DEV), torch.zeros(n_q, heads, device=DEV)
    ws = torch.empty(mla.decode_paged_workspace_size(3, s_q, heads, 512, 64, c.table.shape[1] * size), dtype=torch.uint8,
                     device=DEV)

    def call():
        mla.decode_attend_paged(c.q, c.latent, c.rope, c.table, length, 3, s_q, SCALE, ctx, lse, counts=c.counts_d,
                                tree_mask=c.mask, workspace=ws, device_status=st)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    zeros = [0] * 3
    for cut, counts in ((zeros, [s_q, s_q, 1]), ([899, 300, 1], [1, 0, s_q]), ([5, 64, 7], [0, 0, 0]), (zeros, [s_q] * 3)):
        c.table.copy_(c.table.roll(1, 0))                # a row's pages go along with its length
        lens = lens[-1:] + lens[:-1]
        length.copy_(i32([max(0, n - k) for n, k in zip(lens, cut)]))
        c.counts_d.copy_(i32(counts))
        c.q.copy_(c.q.roll(1, 0))
        if tree:
            c.mask.copy_(c.mask.roll(1, 0) | 1)
        graph.replay()
        got = ctx.clone(), lse.clone()
        ctx.fill_(7), lse.fill_(7)
        call()
        assert torch.equal(ctx, got[0]) and torch.equal(lse, got[1])
        there = torch.tensor([i < counts[b] and int(length[b]) > 0 for b in range(3) for i in range(s_q)], device=DEV)
        assert (got[0][~there] == 0).all() and torch.isneginf(got[1][~there]).all()
        assert torch.isfinite(got[0]).all()
    assert int(st) == 0
