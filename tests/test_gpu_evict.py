"""Attention weight per key, eviction plan and in-place compaction on the GPU, against plain 64-bit forms, and the
whole cycle append -> attend -> weights -> evict over an 8-bit cache."""
import numpy as np
import pytest
import torch

from tests import q8_reference as R
from tests.test_gpu_q8 import (DEV, EPS, SCALE, THETA, attend_case, check_append, check_attend, gen, i32, normal,
                               random_cache, status)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


# ---------------------------------------------------------------- attention weights

def rows64(q, lat, rope, start, length, s_q):
    """Per batch row: its queries [s_q, H, D] and its window's latents and rope keys, in 64 bits."""
    for b in range(len(length)):
        lo, n = int(start[b]), int(length[b])
        yield b, lo, n, R.as64(q[b * s_q:(b + 1) * s_q]), lat[b][lo:lo + n], R.as64(rope[b, lo:lo + n])


def make_lse(q, lat, rope, start, length, s_q):
    lse = np.full((q.shape[0], q.shape[1]), -np.inf)
    for b, _, n, qb, l, r in rows64(q, lat, rope, start, length, s_q):
        for i in range(s_q):
            limit = max(0, min(n, n - s_q + 1 + i))
            lse[b * s_q + i] = R.attend64(qb[i], l[:limit], r[:limit], SCALE)[1]
    return torch.from_numpy(lse).float().to(DEV)


def check_weights(got, before, q, lat, rope, lse, start, length, s_q, decay, n_new):
    """A probability is exp(s - lse) with s an f32 sum of D products: the exponent is off by about
    sqrt(D) 2^-24 |q||k| scale plus 2^-23 of (s, lse) -- below 5e-5 here -- and the sums round by 2^-24
    per addition of non-negative terms: 1e-4 relative holds, with the smallest f32 normal below it."""
    got, before, lse = R.as64(got), R.as64(before), R.as64(lse).reshape(q.shape[0], q.shape[1])
    for b, lo, n, qb, l, r in rows64(q, lat, rope, start, length, s_q):
        want = before[b].copy()
        want[lo:lo + n] = R.key_weights64(qb, l, r, lse[b * s_q:(b + 1) * s_q], before[b, lo:lo + n], SCALE, decay, n_new)
        inside = np.zeros(len(want), dtype=bool)
        inside[lo:lo + n] = True
        assert np.array_equal(got[b][~inside], before[b][~inside], equal_nan=True)
        assert (np.abs(got[b][inside] - want[inside]) <= 1e-4 * want[inside] + 1e-37).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("s_q,block,T,lengths,starts,decay,n_new", [
    (1, 1, 64, [1], [0], 1.0, 1),
    (1, 16, 900, [900, 0, 63, 64, 65, 1, 500], [0, 0, 16, 32, 48, 0, 16], 0.5, 1),
    (1, 64, 20000, [20000, 19000], [0, 64], 1.0, 0),
    (2, 8, 300, [300, 1, 2, 0, 131], [0, 8, 0, 0, 16], 0.0, 2),
    (4, 32, 1400, [1400, 700, 3], [0, 64, 0], 0.9, 4),
    (11, 4, 200, [200, 9], [0, 4], 1.0, 300),
])
def test_key_weights(mla, q8, heads, s_q, block, T, lengths, starts, decay, n_new):
    g = gen(T + heads + s_q)
    B = len(lengths)
    q, codes, scales, rope, start, length = attend_case(g, B, s_q, heads, T, block, lengths, starts)
    if q8:
        lat = [R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), block) for b in range(B)]
    else:
        latent = normal(g, B, T, 512).bfloat16()
        lat = [R.as64(latent[b]) for b in range(B)]
    # what lies outside the windows is never read: NaN
    for b in range(B):
        lo, n = starts[b], lengths[b]
        for r in (slice(0, lo), slice(lo + n, T)):
            rope[b, r] = float("nan")
            codes[b, r] = 0x7F
            if not q8:
                latent[b, r] = float("nan")
    lse = make_lse(q, lat, rope, start, length, s_q)
    w = torch.exp(normal(g, B, T))
    if decay == 0.0:
        w.fill_(float("nan"))           # not read
    before, st = w.clone(), status()

    def call(weights):
        if q8:
            mla.key_weights_q8(q, codes, scales, block, rope, lse, start, length, B, s_q, SCALE, weights, decay=decay,
                               n_new=n_new, device_status=st)
        else:
            mla.key_weights(q, latent, rope, lse, start, length, B, s_q, SCALE, weights, decay=decay, n_new=n_new,
                            device_status=st)
    call(w)
    assert int(st) == 0
    check_weights(w, before, q, lat, rope, lse, start, length, s_q, decay, n_new)
    again = before.clone()
    call(again)
    assert torch.equal(w.view(torch.int32), again.view(torch.int32))     # the same bits


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("heads,rank,rope_dim,s_q,block,T", [(4, 32, 8, 1, 1, 64), (3, 37, 6, 3, 4, 130), (1, 1, 2, 1, 64, 70),
                                                            (2, 1024, 256, 2, 16, 90)])
def test_key_weights_f32(mla, q8, heads, rank, rope_dim, s_q, block, T):
    g = gen(rank + 1)
    q, codes, scales, rope, start, length = attend_case(g, 3, s_q, heads, T, block, [T, 1, 0], [0, block, 0], rank, rope_dim,
                                                        torch.float32)
    q *= 0.3
    latent = normal(g, 3, T, rank)
    lat = [R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), block) if q8 else R.as64(latent[b]) for b in range(3)]
    lse = make_lse(q, lat, rope, start, length, s_q)
    w = torch.exp(normal(g, 3, T))
    before, st = w.clone(), status()
    if q8:
        mla.key_weights_q8(q, codes, scales, block, rope, lse, start, length, 3, s_q, SCALE, w, decay=0.5, n_new=1, device_status=st)
    else:
        mla.key_weights(q, latent, rope, lse, start, length, 3, s_q, SCALE, w, decay=0.5, n_new=1, device_status=st)
    assert int(st) == 0
    check_weights(w, before, q, lat, rope, lse, start, length, s_q, 0.5, 1)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_key_weights_bad_windows(mla, q8, dtype):
    g = gen(90)
    for start, length, bit in [([8, 0], [64, 100], mla.DEVICE_BAD_BLOCK_START), ([16, 0], [300, 100], mla.DEVICE_INDEX_OUT_OF_RANGE),
                               ([-16, 0], [64, 100], mla.DEVICE_INDEX_OUT_OF_RANGE)]:
        q, codes, scales, rope, s, n = attend_case(g, 2, 1, 64, 300, 16, length, start, dtype=dtype)
        latent = normal(g, 2, 300, 512).to(dtype)
        w = torch.ones(2, 300, device=DEV)
        lse, st = torch.zeros(2, 64, device=DEV) + 9.0, status()
        if q8:
            mla.key_weights_q8(q, codes, scales, 16, rope, lse, s, n, 2, 1, SCALE, w, device_status=st)
        else:
            if bit == mla.DEVICE_BAD_BLOCK_START:
                continue
            mla.key_weights(q, latent, rope, lse, s, n, 2, 1, SCALE, w, device_status=st)
        assert int(st) == bit and (w[0] == 1).all() and (w[1, :100] > 1).all() and (w[1, 100:] == 1).all()


def test_key_weights_many_rows(mla):
    """More rows than one scan step holds, most of them empty, packed in one buffer."""
    g = gen(91)
    B = 100
    lengths = [(37 * b) % 150 if b % 3 == 0 else 0 for b in range(B)]
    starts = np.concatenate([[0], np.cumsum(lengths)])[:-1].tolist()
    T = sum(lengths)
    latent, rope = normal(g, 1, T, 512).bfloat16(), normal(g, 1, T, 64).bfloat16()
    q = normal(g, B, 128, 576).bfloat16() * 0.2
    one = R.as64(latent[0])
    lat = [one] * B
    ropes = rope.expand(B, T, 64)
    lse = make_lse(q, lat, ropes, starts, lengths, 1)
    w = torch.rand(1, T, generator=g, device=DEV)
    before = w.clone()
    mla.key_weights(q, latent, rope, lse, i32(starts), i32(lengths), B, 1, SCALE, w)
    got, base = R.as64(w[0]), R.as64(before[0])
    for b, lo, n, qb, l, r in rows64(q, lat, ropes, starts, lengths, 1):
        want = R.key_weights64(qb, l, r, R.as64(lse[b:b + 1]), base[lo:lo + n], SCALE, 1.0, 0)
        assert (np.abs(got[lo:lo + n] - want) <= 1e-4 * want).all()


# ---------------------------------------------------------------- eviction

def run_plan(mla, w, start, length, keep, sink, recent):
    B = w.shape[0]
    kept = torch.full((B, keep), -7, dtype=torch.int32, device=DEV)
    counts, out, st = i32([5] * B), i32([5] * B), status()
    mla.evict_plan(w, start, length, keep, sink, recent, kept, counts, kv_len_out=out, device_status=st)
    return kept, counts, out, int(st)


WEIGHTS = {
    "heavy tails": lambda g, b, t: torch.exp(2 * normal(g, b, t)),
    "many ties": lambda g, b, t: torch.randint(0, 3, (b, t), generator=g, device=DEV).float(),
    "all equal": lambda g, b, t: torch.full((b, t), 0.25, device=DEV),
    "signs, infinities and NaN": lambda g, b, t: torch.where(
        torch.rand(b, t, generator=g, device=DEV) < 0.2,
        torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0, 0.0], device=DEV)[torch.randint(0, 5, (b, t), generator=g, device=DEV)],
        normal(g, b, t)),
}


@pytest.mark.parametrize("kind", list(WEIGHTS))
@pytest.mark.parametrize("T,lengths,starts,keep,sink,recent", [
    (64, [64, 1, 0, 33, 32, 31], [0, 0, 5, 31, 1, 0], 32, 4, 8),
    (5000, [5000, 4000, 1000], [0, 999, 7], 1001, 0, 0),
    (5000, [5000, 4097, 300], [0, 3, 0], 300, 100, 200),          # sinks and recent tokens alone
    (40000, [40000, 39999], [0, 1], 39998, 3, 1000),              # two evicted
    (40000, [40000, 20000], [0, 0], 1, 0, 1),
    (40000, [40000, 20000], [0, 0], 1, 0, 0),
    (9, [9], [0], 2, 1, 1),
])
def test_evict_plan(mla, kind, T, lengths, starts, keep, sink, recent):
    g = gen(T + keep)
    w = WEIGHTS[kind](g, len(lengths), T)
    kept, counts, out, st = run_plan(mla, w, i32(starts), i32(lengths), keep, sink, recent)
    assert st == 0
    for b, n in enumerate(lengths):
        want = R.evict64(w[b, starts[b]:starts[b] + n].cpu().numpy(), n, keep, sink, recent)
        assert int(out[b]) == min(n, keep)
        if want is None:
            assert int(counts[b]) == -1 and (kept[b] == -7).all()
        else:
            assert int(counts[b]) == keep and np.array_equal(kept[b].cpu().numpy(), want)


def test_evict_plan_long_rows_read_from_memory(mla):
    """Slices too long for shared memory (one CTA per row: the rows alone fill the GPU)."""
    g = gen(3)
    B, T, keep = 200, 50000, 20000
    w = torch.exp(normal(g, B, T))
    length = i32([T - b for b in range(B)])
    kept, counts, out, st = run_plan(mla, w, None, length, keep, 4, 100)
    assert st == 0
    for b in (0, 77, 199):
        n = T - b
        assert np.array_equal(kept[b].cpu().numpy(), R.evict64(w[b, :n].cpu().numpy(), n, keep, 4, 100))


def test_evict_plan_bad_windows_and_aliased_lengths(mla):
    w = torch.rand(3, 100, device=DEV)
    length = i32([101, 80, -2])
    kept, counts, st = torch.zeros(3, 10, dtype=torch.int32, device=DEV), i32([0, 0, 0]), status()
    mla.evict_plan(w, None, length, 10, 1, 1, kept, counts, kv_len_out=length, device_status=st)
    assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE
    assert counts.tolist() == [-1, 10, -1] and length.tolist() == [101, 10, -2]
    assert np.array_equal(kept[1].cpu().numpy(), R.evict64(w[1, :80].cpu().numpy(), 80, 10, 1, 1))


def random_arrays(g, b, t):
    """State arrays of every vector width: 16, 8, 4, 2 and 1 bytes, and views inside wider rows."""
    byte = lambda n: torch.randint(0, 256, (b, t, n), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)  # noqa: E731
    wide = normal(g, b, t + 2, 576).bfloat16()
    return [byte(512), normal(g, b, t, 64).bfloat16(), normal(g, b, t, 1), byte(1), byte(24), wide[:, 1:-1, 64:],
            normal(g, b, t, 33).bfloat16(), byte(71)]


@pytest.mark.parametrize("T,keep,counts,starts", [
    (40, 16, [16, 0, -1, 7], [0, 3, 9, 1]),
    (3000, 2990, [2990, 1500, 1], [0, 10, 20]),
    (9001, 4000, [4000], [1]),                       # one row: clusters share each chunk
    (700, 300, [300, 299] * 40, [0, 5] * 40),
])
def test_compact(mla, T, keep, counts, starts):
    g = gen(T)
    B = len(counts)
    arrays = random_arrays(g, B, T)
    want = [a.clone() for a in arrays]
    kept = torch.zeros(B, keep, dtype=torch.int32)
    rng = np.random.default_rng(T)
    for b, n in enumerate(counts):
        if n > 0:
            at = np.sort(rng.choice(T - starts[b], n, replace=False))
            if b % 2:
                at[:n // 2] = np.arange(n // 2)      # a prefix that stays in place
                at = np.unique(np.concatenate([at[:n // 2], np.sort(rng.choice(np.arange(n // 2, T - starts[b]), n - n // 2, replace=False))]))
            kept[b, :n] = torch.from_numpy(at.astype(np.int32))
            for w, a in zip(want, arrays):
                w[b, starts[b]:starts[b] + n] = a[b, starts[b] + torch.from_numpy(at).to(DEV)]
    st = status()
    mla.cache_compact(arrays, i32(starts), kept.to(DEV), i32(counts), device_status=st)
    assert int(st) == 0
    for w, a in zip(want, arrays):
        assert torch.equal(w.contiguous().view(torch.uint8), a.contiguous().view(torch.uint8))


def test_compact_bad_counts_and_positions(mla):
    base = torch.arange(20, device=DEV, dtype=torch.int32).float().view(1, 20, 1).expand(2, 20, 1).contiguous()
    good = [0, 5, 6, 19]
    for count, kept, start, bit in [(5, good, 0, mla.DEVICE_BAD_SELECTION_COUNT), (-2, good, 0, mla.DEVICE_BAD_SELECTION_COUNT),
                                    (4, good, 18, mla.DEVICE_INDEX_OUT_OF_RANGE),      # the front does not fit
                                    (4, good, -1, mla.DEVICE_INDEX_OUT_OF_RANGE)]:
        a, st = base.clone(), status()
        mla.cache_compact([a], i32([start, 0]), i32([kept, good]), i32([count, 4]), device_status=st)
        assert int(st) == bit and torch.equal(a[0], base[0]) and a[1, :4, 0].tolist() == good
    # positions that fall, repeat, lie below their place or outside the buffer are not moved
    for kept, want in [([0, 6, 5, 7], [0, 6, 2, 7]), ([3, 3, 4, 5], [3, 1, 4, 5]), ([0, 1, 2, 20], [0, 1, 2, 3]),
                       ([0, 2, 1, 9], [0, 2, 2, 9]), ([-1, 4, 5, 6], [0, 4, 5, 6])]:
        a, st = base.clone(), status()
        mla.cache_compact([a], i32([0, 0]), i32([kept, good]), i32([4, 4]), device_status=st)
        assert int(st) == mla.DEVICE_INDEX_OUT_OF_RANGE
        assert a[0, :4, 0].tolist() == want and a[0, 4:, 0].tolist() == list(range(4, 20)) and a[1, :4, 0].tolist() == good


# ---------------------------------------------------------------- the whole cycle

def test_append_attend_weights_evict(mla):
    """A serving loop over an 8-bit cache with a budget: every step appends, attends and adds weights, and evicts
    when a row passes its budget; each step is checked from the state before it."""
    g = gen(1234)
    B, T, heads, keep, sink, recent = 3, 256, 128, 96, 2, 16
    codes = torch.zeros(B, T, 512, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(B, T, dtype=torch.uint8, device=DEV)
    rope = torch.zeros(B, T, 64, dtype=torch.bfloat16, device=DEV)
    weights = torch.full((B, T), float("nan"), device=DEV)     # new keys start from zero whatever was there
    start, length, offset = i32([0, 7, 40]), i32([0, 0, 0]), i32([0, 0, 0])
    gain = torch.exp(0.2 * normal(g, 512)).bfloat16()
    kept = torch.zeros(B, keep, dtype=torch.int32, device=DEV)
    counts, st = i32([0, 0, 0]), status()
    evicted = 0
    for step, s_new in enumerate([90, 1, 4, 40, 1, 2, 60]):
        s_q = min(s_new, 4)
        raw, raw_rope = normal(g, B, s_new, 512).bfloat16(), normal(g, B, s_new, 64).bfloat16()
        n0, off0 = length.tolist(), offset.tolist()
        before = codes.cpu().numpy().copy(), scales.cpu().numpy().copy(), R.as64(rope)
        mla.append_compressed_q8(raw, raw_rope, gain, EPS, THETA, codes, scales, 1, rope, start, length, kv_len_out=length,
                                 row_offsets=offset, device_status=st)
        check_append(raw, raw_rope, gain, before, (codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)), 1,
                     start.tolist(), n0, off0, s_new, torch.bfloat16)
        offset += s_new
        q = normal(g, B * s_q, heads, 576).bfloat16() * 0.2
        ctx = torch.empty(B * s_q, heads, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(B * s_q, heads, device=DEV)
        mla.decode_attend_q8(q, codes, scales, 1, rope, start, length, B, s_q, SCALE, ctx, lse, device_status=st)
        check_attend(ctx, lse, (q, codes, scales, rope, start, length), 1, s_q)
        w0 = weights.clone()
        mla.key_weights_q8(q, codes, scales, 1, rope, lse, start, length, B, s_q, SCALE, weights, decay=0.9, n_new=s_new,
                           device_status=st)
        lat = [R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), 1) for b in range(B)]
        check_weights(weights, w0, q, lat, rope, lse, start, length, s_q, 0.9, s_new)
        n1 = length.tolist()
        arrays = [codes, rope, scales.unsqueeze(-1), weights.unsqueeze(-1)]
        old = [a.clone() for a in arrays]
        mla.evict_plan(weights, start, length, keep, sink, recent, kept, counts, kv_len_out=length, device_status=st)
        mla.cache_compact(arrays, start, kept, counts, device_status=st)
        for b in range(B):
            lo = int(start[b])
            at = R.evict64(old[3][b, lo:lo + n1[b], 0].cpu().numpy(), n1[b], keep, sink, recent)
            assert int(length[b]) == min(n1[b], keep)
            if at is None:
                at = np.arange(n1[b])
            else:
                evicted += 1
            for a, o in zip(arrays, old):
                assert torch.equal(a[b, lo:lo + len(at)].contiguous().view(torch.uint8),
                                   o[b, lo + torch.from_numpy(at).to(DEV)].contiguous().view(torch.uint8))
    assert evicted >= 6 and int(st) & ~mla.DEVICE_SCORE_RANGE == 0


def test_key_weights_fp16_operand_range(mla):
    """As the attention over an 8-bit cache: small units and large query values are flagged, and rounded as documented."""
    g = gen(92)
    B, T = 2, 200
    q, codes, scales, rope, start, length = attend_case(g, B, 1, 128, T, 1, [T] * B, [0] * B)
    scales[0], scales[1] = 112, 105

    def run(n, w):
        st = status()
        mla.key_weights_q8(q, codes, scales, 1, rope, lse, start, n, B, 1, SCALE, w, decay=0.0, device_status=st)
        return int(st)
    lat = [np.round(R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), 1) * 2.0 ** 24) * 2.0 ** -24 for b in range(B)]
    lse = make_lse(q, lat, rope, start, length, 1)
    w = torch.zeros(B, T, device=DEV)
    assert run(i32([T, 0]), w) == 0 and run(i32([T, T]), w) == mla.DEVICE_VALUE_RANGE
    check_weights(w, torch.zeros_like(w), q, lat, rope, lse, start, length, 1, 0.0, 0)
    scales.fill_(120)
    codes[..., 3] = 0
    want, got = torch.zeros_like(w), torch.zeros_like(w)
    assert run(length, want) == 0
    q[1, 5, 3] = 65536.0
    assert run(length, got) == mla.DEVICE_VALUE_RANGE and torch.equal(got, want)


def cycle(mla, s, stream=None):
    """One serving step over state ``s``: append, attend, weights, eviction."""
    mla.append_compressed_q8(s["raw"], s["raw_rope"], s["gain"], EPS, THETA, s["codes"], s["scales"], 1, s["rope"], None,
                             s["length"], kv_len_out=s["length"], row_offsets=s["offset"], stream=stream)
    mla.decode_attend_q8(s["q"], s["codes"], s["scales"], 1, s["rope"], None, s["length"], 2, 1, SCALE, s["ctx"], s["lse"],
                         workspace=s["ws"], stream=stream)
    mla.key_weights_q8(s["q"], s["codes"], s["scales"], 1, s["rope"], s["lse"], None, s["length"], 2, 1, SCALE, s["weights"],
                       n_new=1, stream=stream)
    mla.evict_plan(s["weights"], None, s["length"], 300, 4, 32, s["kept"], s["counts"], kv_len_out=s["length"], stream=stream)
    mla.cache_compact([s["codes"], s["rope"], s["scales"].unsqueeze(-1), s["weights"].unsqueeze(-1)], None, s["kept"],
                      s["counts"], stream=stream)


def cycle_state(mla, seed):
    g = gen(seed)
    codes, scales = random_cache(g, 2, 400, 512, 1)
    return dict(codes=codes, scales=scales, rope=normal(g, 2, 400, 64).bfloat16(), weights=torch.rand(2, 400, generator=g, device=DEV),
                raw=normal(g, 2, 1, 512).bfloat16(), raw_rope=normal(g, 2, 1, 64).bfloat16(), gain=torch.ones(512, device=DEV).bfloat16(),
                q=normal(g, 2, 128, 576).bfloat16() * 0.2, length=i32([299, 250]), offset=i32([900, 250]),
                ctx=torch.empty(2, 128, 512, dtype=torch.bfloat16, device=DEV), lse=torch.empty(2, 128, device=DEV),
                kept=torch.zeros(2, 300, dtype=torch.int32, device=DEV), counts=i32([0, 0]),
                ws=torch.empty(mla.decode_workspace_size(2, 1, 128, 512, 64, 400), dtype=torch.uint8, device=DEV))


def same_state(a, b):
    return all(torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8)) for k in a if k != "ws")


def test_cycles_on_two_streams_and_in_two_graphs(mla):
    """Two caches stepped at once on two streams, and by two captured graphs replayed in turn, against one after the
    other: the same bits."""
    steps = 5
    want = [cycle_state(mla, k) for k in (1, 2)]
    for s in want:
        for _ in range(steps):
            cycle(mla, s)
    assert want[0]["length"].tolist() == [300, 255] and want[0]["counts"].tolist() == [300, -1]
    got = [cycle_state(mla, k) for k in (1, 2)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(steps):
        for s, side in zip(got, sides):
            cycle(mla, s, side)
    torch.cuda.synchronize()
    assert all(same_state(a, b) for a, b in zip(got, want))
    got = [cycle_state(mla, k) for k in (1, 2)]
    graphs = []
    for s in got:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cycle(mla, s)
        graphs.append(graph)
    for _ in range(steps):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(same_state(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("layout", ["broadcast rows", "heads first", "wide heads"])
def test_key_weights_query_layouts(mla, q8, layout):
    g = gen(93)
    B, s_q, T, block = 3, 2, 200, 8
    q, codes, scales, rope, start, length = attend_case(g, B, s_q, 128, T, block, [200, 5, 131], [0, 8, 16])
    if layout == "broadcast rows":
        q = q[:1].expand(B * s_q, 128, 576)
    elif layout == "heads first":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    else:
        wide = torch.full((B * s_q, 128, 592), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[..., 8:584] = q
        q = wide[..., 8:584]
    latent = normal(g, B, T, 512).bfloat16()
    lat = [R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), block) if q8 else R.as64(latent[b]) for b in range(B)]
    lse = make_lse(q, lat, rope, start, length, s_q)
    w = torch.exp(normal(g, B, T))
    before, st = w.clone(), status()
    if q8:
        mla.key_weights_q8(q, codes, scales, block, rope, lse, start, length, B, s_q, SCALE, w, n_new=1, device_status=st)
    else:
        mla.key_weights(q, latent, rope, lse, start, length, B, s_q, SCALE, w, n_new=1, device_status=st)
    assert int(st) == 0
    check_weights(w, before, q, lat, rope, lse, start, length, s_q, 1.0, 1)
    if q8:
        ctx, lse2 = torch.empty(B * s_q, 128, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B * s_q, 128, device=DEV)
        mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, s_q, SCALE, ctx, lse2)
        check_attend(ctx, lse2, (q, codes, scales, rope, start, length), block, s_q)


def test_every_row_empty(mla):
    """No key anywhere: nothing is written but empty results, and nothing is flagged."""
    g = gen(94)
    B, T, block = 3, 128, 16
    q, codes, scales, rope, start, length = attend_case(g, B, 1, 128, T, block, [0, 0, 0], [0, 16, 32])
    latent = normal(g, B, T, 512).bfloat16()
    ctx, lse, st = torch.ones(B, 128, 512, dtype=torch.bfloat16, device=DEV), torch.ones(B, 128, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, 1, SCALE, ctx, lse, device_status=st)
    assert (ctx == 0).all() and torch.isneginf(lse).all()
    w = torch.rand(B, T, generator=g, device=DEV)
    w0, c0, e0, l0 = w.clone(), codes.clone(), scales.clone(), latent.clone()
    mla.key_weights_q8(q, codes, scales, block, rope, lse, start, length, B, 1, SCALE, w, n_new=1, device_status=st)
    mla.key_weights(q, latent, rope, lse, start, length, B, 1, SCALE, w, n_new=1, device_status=st)
    mla.quantize_cache(latent, codes, scales, block, start, length, device_status=st)
    mla.dequantize_cache(codes, scales, block, latent, start, length, device_status=st)
    kept, counts, out, plan_status = run_plan(mla, w, start, length, 4, 1, 1)
    mla.cache_compact([codes, rope], start, kept, counts, device_status=st)
    assert int(st) == 0 and plan_status == 0 and counts.tolist() == [-1] * 3 and out.tolist() == [0] * 3
    for a, b in ((w, w0), (codes, c0), (scales, e0), (latent, l0)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shared", ["rope", "codes", "both"])
def test_rows_that_share_a_buffer(mla, shared):
    """Batch rows over one codes or rope buffer (a batch stride of zero), at different windows."""
    g = gen(95)
    B, T, block = 3, 300, 4
    q, codes, scales, rope, start, length = attend_case(g, B, 1, 128, T, block, [300, 70, 129], [0, 8, 12])
    if shared != "rope":
        codes, scales = codes[:1].expand(B, T, 512), scales[:1].expand(B, -1)
    if shared != "codes":
        rope = rope[:1].expand(B, T, 64)
    ctx, lse, st = torch.empty(B, 128, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B, 128, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, 1, SCALE, ctx, lse, device_status=st)
    check_attend(ctx, lse, (q, codes, scales, rope, start, length), block, 1)
    lat = [R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), block) for b in range(B)]
    exact = make_lse(q, lat, rope, start, length, 1)
    w = torch.exp(normal(g, B, T))
    before = w.clone()
    mla.key_weights_q8(q, codes, scales, block, rope, exact, start, length, B, 1, SCALE, w, n_new=1, device_status=st)
    check_weights(w, before, q, lat, rope, exact, start, length, 1, 1.0, 1)
    assert int(st) & ~mla.DEVICE_SCORE_RANGE == 0
