"""The 8-bit cache on the GPU: append, quantise, dequantise and decode attention, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import helpers as H
from tests import q8_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS, THETA = 1e-6, 10000.0


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


def random_cache(g, b, t, rank, block):
    """Codes of latents whose tokens differ in size, with exponents per block (no NaN codes)."""
    x = normal(g, b, t, rank) * torch.exp(0.5 * normal(g, b, t, 1))
    nb = -(-t // block)
    e = torch.randint(115, 125, (b, nb), generator=g, device=DEV, dtype=torch.int32)
    rows = e.repeat_interleave(block, 1)[:, :t]
    codes = (x * torch.exp2((127 - rows).float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, e.to(torch.uint8)


# ---------------------------------------------------------------- conversions

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_and_exponent_dequantises_exactly(mla, dtype):
    # 256 codes x every exponent byte (those outside [64, 134] read as the nearer end)
    codes = torch.arange(256, device=DEV).to(torch.uint8).view(1, 1, 256).expand(1, 256, 256).contiguous()
    scales = torch.arange(256, device=DEV).to(torch.uint8).view(1, 256)
    out = torch.empty(1, 256, 256, dtype=dtype, device=DEV)
    mla.dequantize_cache(codes, scales, 1, out, None, i32([256]))
    want = R.held64(codes[0].cpu().numpy(), scales[0].cpu().numpy(), 1)
    assert np.array_equal(R.as64(out[0]), want, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rank,block,t", [(512, 1, 130), (512, 64, 200), (96, 4, 77), (1024, 16, 65), (37, 8, 50), (1, 2, 3)])
def test_quantise_and_back(mla, dtype, rank, block, t):
    g = gen(rank + block)
    lat = (normal(g, 3, t, rank) * torch.exp(2 * normal(g, 3, t, 1))).to(dtype)
    lat[0, 1] = 0.0
    start, length = i32([0, block, 0]), i32([t, t - block - 1 if t > block + 1 else 0, 0])
    codes = torch.full((3, t, rank), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((3, -(-t // block)), 7, dtype=torch.uint8, device=DEV)
    st = status()
    mla.quantize_cache(lat, codes, scales, block, start, length, device_status=st)
    assert int(st) == 0
    x, c, e = R.as64(lat), codes.cpu().numpy(), scales.cpu().numpy()
    for b in range(3):
        lo, hi = int(start[b]), int(start[b]) + int(length[b])
        assert (c[b, :lo] == 0x55).all() and (c[b, hi:] == 0x55).all()          # rows outside stay
        for k in range(e.shape[1]):
            r0, r1 = max(lo, k * block), min(hi, (k + 1) * block)
            if r0 >= r1:
                assert e[b, k] == 7
                continue
            assert e[b, k] == R.exponent64(np.abs(x[b, r0:r1]).max())            # amax is exact: no rounding before it
            assert np.array_equal(R.codes64(c[b, r0:r1]), R.nearest_e4m3(x[b, r0:r1] * 2.0 ** (127.0 - e[b, k])))
    back = torch.full((3, t, rank), 5.0, dtype=dtype, device=DEV)
    mla.dequantize_cache(codes, scales, block, back, start, length)
    y = R.as64(back)
    for b in range(3):
        lo, hi = int(start[b]), int(start[b]) + int(length[b])
        assert np.array_equal(y[b, lo:hi], R.held64(c[b], e[b], block)[lo:hi])
        assert (y[b, :lo] == 5.0).all() and (y[b, hi:] == 5.0).all()


def test_quantise_special_values(mla):
    lat = torch.zeros(1, 4, 64, device=DEV)
    lat[0, 0, 3] = float("nan")
    lat[0, 0, 4] = 1.0
    lat[0, 1, 5] = float("inf")
    lat[0, 2, 6] = -1e6                      # beyond the largest unit
    lat[0, 3, 7] = 57344.0                   # the largest value held
    codes = torch.zeros(1, 4, 64, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(1, 4, dtype=torch.uint8, device=DEV)
    st = status()
    mla.quantize_cache(lat, codes, scales, 1, None, i32([4]), device_status=st)
    assert int(st) == mla.DEVICE_VALUE_RANGE
    held = R.held64(codes[0].cpu().numpy(), scales[0].cpu().numpy(), 1)
    assert np.isnan(held[0, 3]) and held[0, 4] == 1.0 and held[1, 5] == 57344.0 and held[2, 6] == -57344.0
    assert held[3, 7] == 57344.0
    assert scales[0].tolist() == [R.exponent64(1.0), 134, 134, 134]


def test_bad_windows_are_flagged_and_skipped(mla):
    codes = torch.full((4, 32, 64), 0x11, dtype=torch.uint8, device=DEV)
    scales = torch.full((4, 4), 120, dtype=torch.uint8, device=DEV)
    lat = torch.ones(4, 32, 64, device=DEV)
    for start, length, bit in [([4, 0, 0, 0], [8, 8, 0, 0], mla.DEVICE_BAD_BLOCK_START),
                               ([0, 8, 0, 0], [33, 8, 0, 0], mla.DEVICE_INDEX_OUT_OF_RANGE),
                               ([-8, 8, 0, 0], [8, 24, 0, 0], mla.DEVICE_INDEX_OUT_OF_RANGE),
                               ([8, 8, 0, 0], [-1, 24, 0, 0], mla.DEVICE_INDEX_OUT_OF_RANGE)]:
        st = status()
        c, e, out = codes.clone(), scales.clone(), lat.clone()
        mla.quantize_cache(lat, c, e, 8, i32(start), i32(length), device_status=st)
        assert int(st) == bit
        assert torch.equal(c[0], codes[0]) and torch.equal(e[0], scales[0])       # skipped
        assert not torch.equal(c[1], codes[1])                                    # the good row is done
        st = status()
        mla.dequantize_cache(codes, scales, 8, out, i32(start), i32(length), device_status=st)
        assert int(st) == bit and torch.equal(out[0], lat[0]) and not torch.equal(out[1], lat[1])


# ---------------------------------------------------------------- append

def check_append(raw, raw_rope, gain, before, after, block, start, length, offset, s_new, rope_dtype):
    """Codes, exponents and rope keys after an append, from the state before it.

    The f32 normalised value differs from the 64-bit one by at most a few
    2^-24 per operation (products, a sum of rank squares, a square root): slack
    1e-5 relative.  A code must be a nearest e4m3 value of a number within
    that slack, and an exponent the one of such a largest magnitude."""
    slack = 1e-5
    x = R.rms_norm64(R.as64(raw), R.as64(gain), EPS)
    codes0, scales0, rope0 = before
    codes1, scales1, rope1 = after
    B, T = codes0.shape[:2]
    for b in range(B):
        lo = start[b] + length[b]
        hi = lo + s_new
        v = np.full((T, x.shape[-1]), np.nan)
        v[lo:hi] = x[b]
        same = np.ones(T, dtype=bool)
        same[lo:hi] = False
        for k in range(lo // block, (hi - 1) // block + 1):
            r0, r1 = max(lo, k * block), min(hi, (k + 1) * block)
            old0 = max(k * block, start[b])
            amax = np.abs(v[r0:r1]).max()
            allowed = {R.exponent64(amax * (1 - slack)), R.exponent64(amax * (1 + slack))}
            if old0 < lo:
                e_old = min(max(int(scales0[b, k]), R.E_MIN), R.E_MAX)
                allowed = {max(a, e_old) for a in allowed}
            e = int(scales1[b, k])
            assert e in allowed
            want = v[r0:r1] * 2.0 ** (127.0 - e)
            got = R.codes64(codes1[b, r0:r1])
            d = np.abs(got - want)
            best = np.abs(R.nearest_e4m3(want) - want)
            assert (d <= best + 2 * slack * np.abs(want)).all()
            if old0 < lo:
                units = R.codes64(codes0[b, old0:lo]) * 2.0 ** (e_old - e)
                assert np.array_equal(R.codes64(codes1[b, old0:lo]), R.nearest_e4m3(units))
                same[old0:lo] = False
        assert np.array_equal(codes1[b, same], codes0[b, same])
        touched = range(lo // block, (hi - 1) // block + 1)
        rest = [k for k in range(scales0.shape[1]) if k not in touched]
        assert np.array_equal(scales1[b, rest], scales0[b, rest])
        # rope keys: f32 angles as the operator defines them; sincosf and two
        # products round to ~2^-22 of |a| + |b|, then the storage type rounds
        rr = R.as64(raw_rope)[b]
        d = rr.shape[-1]
        inv = np.float32(np.power(np.float64(np.float32(THETA)), np.float64(np.float32(-2.0 * np.arange(d // 2) / d))))
        pos = (offset[b] if offset is not None else length[b]) + np.arange(s_new)
        ang = (pos[:, None] * inv.astype(np.float64)).astype(np.float32).astype(np.float64)
        a, bb = rr[:, 0::2], rr[:, 1::2]
        want = np.concatenate([a * np.cos(ang) - bb * np.sin(ang), bb * np.cos(ang) + a * np.sin(ang)], 1)
        size = np.concatenate([np.abs(a) + np.abs(bb)] * 2, 1)
        half = 2.0 ** -9 if rope_dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(rope1[b, lo:hi] - want) <= 2 * half * np.abs(want) + 4e-7 * size).all()
        keep = np.r_[0:lo, hi:T]
        assert np.array_equal(rope1[b, keep], rope0[b, keep])


@pytest.mark.parametrize("dtype,rope_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                              (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("block", [1, 2, 16, 64])
@pytest.mark.parametrize("rank,rope_dim,s_new", [(512, 64, 1), (512, 64, 5), (512, 64, 200), (40, 8, 33), (33, 6, 17),
                                                (1024, 256, 3)])
def test_append(mla, dtype, rope_dtype, block, rank, rope_dim, s_new):
    g = gen(block * 1000 + rank + s_new)
    B, T = 4, 420
    codes, scales = random_cache(g, B, T, rank, block)
    rope = normal(g, B, T, rope_dim).to(rope_dtype)
    raw = (normal(g, B, s_new, rank) * torch.tensor([1.0, 100.0, 1e-3, 1.0], device=DEV).view(4, 1, 1)).to(dtype)
    raw[3, 0] = 0.0
    raw_rope = normal(g, B, s_new, rope_dim).to(dtype)
    # norm weights that make some new tokens larger and some smaller than what the blocks hold
    gain = torch.exp(1.5 * normal(g, rank)).to(dtype)
    start = i32([0, block, 2 * block, 0])
    length = i32([0, 37, 64, T - s_new])
    offset = i32([0, 5, 100000, 7])
    before = codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)
    out, st = torch.full_like(length, -9), status()
    mla.append_compressed_q8(raw, raw_rope, gain, EPS, THETA, codes, scales, block, rope, start, length,
                             kv_len_out=out, row_offsets=offset, device_status=st)
    assert int(st) == 0 and out.tolist() == [int(n) + s_new for n in length]
    check_append(raw, raw_rope, gain, before, (codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)), block,
                 start.tolist(), length.tolist(), offset.tolist(), s_new, rope_dtype)


def test_append_strided_views_and_aliased_lengths(mla):
    # codes and rope keys inside wider rows, raw latent and rope of one projection, offsets from the lengths
    g = gen(5)
    B, T, s_new, block = 3, 100, 40, 8
    wide = torch.zeros(B, T, 704, dtype=torch.uint8, device=DEV)
    codes = wide[..., 16:528]
    c0, scales = random_cache(g, B, T, 512, block)
    codes.copy_(c0)
    ropes = normal(g, B, T + 3, 72).bfloat16()
    rope = ropes[:, 3:, 8:]
    kv_a = normal(g, B, s_new, 576).bfloat16()
    gain = torch.ones(512, device=DEV).bfloat16()
    length = i32([0, 13, 60])
    n0 = length.tolist()
    around = wide.clone()
    before = codes.cpu().numpy().copy(), scales.cpu().numpy(), R.as64(rope)
    mla.append_compressed_q8(kv_a[..., :512], kv_a[..., 512:], gain, EPS, THETA, codes, scales, block, rope, None,
                             length, kv_len_out=length)
    assert length.tolist() == [n + s_new for n in n0]
    check_append(kv_a[..., :512], kv_a[..., 512:], gain, before, (codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)),
                 block, [0] * B, n0, None, s_new, torch.bfloat16)
    wide[..., 16:528] = 0
    around[..., 16:528] = 0
    assert torch.equal(wide, around)


def test_append_rows_that_do_not_fit(mla):
    g = gen(6)
    for start, length, offset, bit in [([0, 0], [97, 3], [0, 0], mla.DEVICE_INDEX_OUT_OF_RANGE),
                                       ([3, 0], [8, 3], [0, 0], mla.DEVICE_BAD_BLOCK_START),
                                       ([0, 0], [-1, 3], [0, 0], mla.DEVICE_INDEX_OUT_OF_RANGE),
                                       ([0, 0], [5, 3], [-2, 0], mla.DEVICE_INDEX_OUT_OF_RANGE)]:
        for s_new in (4, 60):
            codes, scales = random_cache(g, 2, 100, 512, 2)
            c0, e0 = codes.clone(), scales.clone()
            rope = normal(g, 2, 100, 64).bfloat16()
            r0 = rope.clone()
            n = i32(length)
            out, st = i32([0, 0]), status()
            mla.append_compressed_q8(normal(g, 2, s_new, 512).bfloat16(), normal(g, 2, s_new, 64).bfloat16(),
                                     torch.ones(512, device=DEV).bfloat16(), EPS, THETA, codes, scales, 2, rope,
                                     i32(start), n, kv_len_out=out, row_offsets=i32(offset), device_status=st)
            assert int(st) == bit and out.tolist() == [length[0], length[1] + s_new]
            assert torch.equal(codes[0], c0[0]) and torch.equal(scales[0], e0[0]) and torch.equal(rope[0], r0[0])
            assert not torch.equal(codes[1], c0[1])


def test_append_grows_a_block_token_by_token(mla):
    """64 tokens of growing size into one block: the unit only grows, and each held token is its value rounded
    at most once per growth (half a step each: 2^-4 relative, or half the smallest step of the unit)."""
    g = gen(7)
    codes = torch.zeros(1, 64, 512, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(1, 1, dtype=torch.uint8, device=DEV)
    rope = torch.zeros(1, 64, 64, dtype=torch.bfloat16, device=DEV)
    n = i32([0])
    raws, units = [], []
    for t in range(64):
        raw = normal(g, 1, 1, 512)
        gain = torch.full((512,), 2.0 ** (t / 8), device=DEV)
        raws.append(R.rms_norm64(R.as64(raw), R.as64(gain), EPS)[0, 0])
        mla.append_compressed_q8(raw, torch.zeros(1, 1, 64, device=DEV), gain, EPS, THETA, codes, scales, 64, rope, None,
                                 n, kv_len_out=n)
        units.append(int(scales))
    assert int(n) == 64 and units == sorted(units) and units[-1] > units[0] + 5
    held = R.held64(codes[0].cpu().numpy(), scales[0].cpu().numpy(), 64)
    for t in range(64):
        growths = len(set(units[t:])) - 1
        smallest = 2.0 ** (units[-1] - 127 - 9)
        # the first rounding to 4 bits; a growth rounds again only below the unit's normal range
        bound = (2.0 ** -4 + 1e-5) * np.abs(raws[t]) + smallest * (0.5 + growths)
        assert (np.abs(held[t] - raws[t]) <= bound).all()


# ---------------------------------------------------------------- attention

def attend_case(g, B, s_q, heads, T, block, lengths, starts, rank=512, rope_dim=64, dtype=torch.bfloat16):
    codes, scales = random_cache(g, B, T, rank, block)
    rope = normal(g, B, T, rope_dim).to(dtype)
    q = normal(g, B * s_q, heads, rank + rope_dim)
    q[..., :rank] *= 0.1
    return q.to(dtype), codes, scales, rope, i32(starts), i32(lengths)


SCALE = 192 ** -0.5


def want_row(q, codes, scales, rope, block, start, length, s_q, n, at=None):
    b, i = n // s_q, n % s_q
    lo = int(start[b])
    limit = max(0, min(int(length[b]), int(length[b]) - s_q + 1 + i))
    lat = R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), block)[lo:lo + limit]
    return R.attend64(R.as64(q[n]), lat, R.as64(rope[b, lo:lo + limit]), SCALE, at)


def check_attend(ctx, lse, case, block, s_q, rows=None, lists=None):
    q, codes, scales, rope, start, length = case
    kind = "bf16" if q.dtype == torch.bfloat16 else "f32"
    rows = range(q.shape[0]) if rows is None else rows
    got_c, got_l, want_c, want_l = [], [], [], []
    for n in rows:
        c, l = want_row(q, codes, scales, rope, block, start, length, s_q, n, lists[n] if lists else None)
        got_c.append(R.as64(ctx[n])), got_l.append(R.as64(lse[n])), want_c.append(c), want_l.append(l)
    got_c, got_l, want_c, want_l = map(np.stack, (got_c, got_l, want_c, want_l))
    empty = np.isinf(want_l)
    assert np.array_equal(np.isinf(got_l), empty) and (got_c[empty] == 0).all()
    H.assert_close(got_c, want_c, kind, "ctx")
    # bf16: both score halves are exchanged in fp16 (the bound of the bf16 decode); f32: rounding of 576 products
    assert np.abs(got_l[~empty] - want_l[~empty]).max(initial=0) <= (2e-2 if kind == "bf16" else 1e-4)


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("s_q,block,T,lengths,starts", [
    (1, 1, 64, [1], [0]),
    (1, 64, 700, [700, 0, 1, 63, 64, 65, 129], [0, 0, 64, 128, 64, 0, 64]),
    (1, 2, 5000, [4999, 33], [0, 6]),
    (3, 16, 600, [600, 2, 0, 3, 130], [0, 16, 0, 32, 64]),        # rows shorter than the block of tokens
    (4, 4, 1500, [1500, 1, 777], [0, 4, 8]),
    (9, 32, 300, [300, 5], [0, 0]),                              # past the lockstep width
])
def test_attend(mla, heads, s_q, block, T, lengths, starts):
    g = gen(heads + T + s_q)
    B = len(lengths)
    case = attend_case(g, B, s_q, heads, T, block, lengths, starts)
    q, codes, scales, rope, start, length = case
    ctx = torch.full((B * s_q, heads, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse, st = torch.full((B * s_q, heads), 7.0, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, s_q, SCALE, ctx, lse, device_status=st)
    assert int(st) & ~mla.DEVICE_SCORE_RANGE == 0
    check_attend(ctx, lse, case, block, s_q)


@pytest.mark.parametrize("s_q", [1, 2])
def test_attend_selected(mla, s_q):
    g = gen(40 + s_q)
    B, T, heads, block, k_max = 4, 3000, 128, 8, 200
    case = attend_case(g, B, s_q, heads, T, block, [3000, 2000, 40, 2500], [0, 8, 16, 0])
    q, codes, scales, rope, start, length = case
    n_q = B * s_q
    sel = torch.zeros(n_q, k_max, dtype=torch.int32)
    counts, lists = [], []
    rng = np.random.default_rng(9)
    for n in range(n_q):
        b, i = n // s_q, n % s_q
        limit = int(length[b]) - s_q + 1 + i
        count = [200, 65, 1, -1][b]
        sel[n] = torch.from_numpy(rng.integers(0, limit, k_max).astype(np.int32))   # a multiset, any order
        lists.append(None if count == -1 else sel[n, :count].numpy().astype(np.int64))
        counts.append(count)
    sel_d, cnt = sel.to(DEV), i32(counts)
    ctx = torch.empty(n_q, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse, st = torch.empty(n_q, heads, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, s_q, SCALE, ctx, lse, sel=sel_d, sel_count=cnt,
                         device_status=st)
    assert int(st) & ~mla.DEVICE_SCORE_RANGE == 0
    check_attend(ctx, lse, case, block, s_q, lists=lists)
    # bad positions are skipped and flagged, a bad count empties its row
    bad = sel_d.clone()
    bad[0, 3], bad[0, 7] = -1, int(length[0])
    cnt2 = cnt.clone()
    cnt2[s_q] = 0
    st = status()
    mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, s_q, SCALE, ctx, lse, sel=bad, sel_count=cnt2,
                         device_status=st)
    assert int(st) & ~mla.DEVICE_SCORE_RANGE == mla.DEVICE_INDEX_OUT_OF_RANGE | mla.DEVICE_BAD_SELECTION_COUNT
    lists[0] = np.delete(lists[0], [3, 7])
    check_attend(ctx, lse, case, block, s_q, rows=[0, s_q - 1 + 2 * s_q], lists=lists)
    assert (ctx[s_q] == 0).all() and torch.isneginf(lse[s_q]).all()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,rank,rope_dim,s_q,block,T", [(4, 32, 8, 1, 1, 64), (3, 37, 6, 2, 4, 130), (1, 1, 2, 1, 64, 70),
                                                            (2, 512, 64, 3, 16, 900)])
def test_attend_f32(mla, heads, rank, rope_dim, s_q, block, T, out_dtype):
    g = gen(rank)
    case = attend_case(g, 3, s_q, heads, T, block, [T, 1, 0], [0, block, 0], rank, rope_dim, torch.float32)
    q, codes, scales, rope, start, length = case
    ctx = torch.empty(3 * s_q, heads, rank, dtype=out_dtype, device=DEV)
    lse, st = torch.empty(3 * s_q, heads, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, block, rope, start, length, 3, s_q, SCALE, ctx, lse, device_status=st)
    assert int(st) == 0
    if out_dtype == torch.float32:
        check_attend(ctx, lse, case, block, s_q)
    else:
        want = torch.empty(3 * s_q, heads, rank, device=DEV)
        mla.decode_attend_q8(q, codes, scales, block, rope, start, length, 3, s_q, SCALE, want, lse)
        assert torch.equal(ctx, want.bfloat16())


def test_attend_packed_rows_and_strides(mla):
    """Rows packed in one buffer, codes and rope keys inside wider rows, a f32 context, NaN behind every window."""
    g = gen(77)
    lengths, block = [70, 0, 513, 128], 16
    starts = [16, 96, 112, 640]
    T = 800
    wide = torch.full((1, T, 672), 0x7F, dtype=torch.uint8, device=DEV)      # NaN codes everywhere
    c0, scales = random_cache(g, 1, T, 512, block)
    ropes = torch.full((1, T, 80), float("nan"), dtype=torch.bfloat16, device=DEV)
    r0 = normal(g, 1, T, 64).bfloat16()
    codes, rope = wide[..., 32:544], ropes[..., 16:]
    for s, n in zip(starts, lengths):
        codes[:, s:s + n] = c0[:, s:s + n]
        rope[:, s:s + n] = r0[:, s:s + n]
    qs = normal(g, 4, 128, 640).bfloat16()
    q = qs[..., 64:]
    q[..., :512] *= 0.125
    ctxs = torch.zeros(4, 128, 520, device=DEV)
    ctx, lse, st = ctxs[..., 4:516], torch.empty(4, 128, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, block, rope, i32(starts), i32(lengths), 4, 1, SCALE, ctx, lse, device_status=st)
    assert int(st) == 0
    every = lambda t: t.expand(4, *t.shape[1:])  # noqa: E731
    check_attend(ctx, lse, (q, every(codes), every(scales), every(rope), i32(starts), i32(lengths)), block, 1)
    assert (ctxs[..., :4] == 0).all() and (ctxs[..., 516:] == 0).all()


def test_attend_bad_windows(mla):
    g = gen(78)
    for start, length, bit in [([8, 0], [64, 100], mla.DEVICE_BAD_BLOCK_START), ([16, 0], [300, 100], mla.DEVICE_INDEX_OUT_OF_RANGE),
                               ([-16, 0], [64, 100], mla.DEVICE_INDEX_OUT_OF_RANGE)]:
        for dtype, heads, rank, rope_dim in [(torch.bfloat16, 128, 512, 64), (torch.float32, 2, 48, 8)]:
            case = attend_case(g, 2, 1, heads, 300, 16, length, start, rank, rope_dim, dtype)
            q, codes, scales, rope, s, n = case
            ctx = torch.empty(2, heads, rank, dtype=dtype, device=DEV)
            lse, st = torch.empty(2, heads, device=DEV), status()
            mla.decode_attend_q8(q, codes, scales, 16, rope, s, n, 2, 1, SCALE, ctx, lse, device_status=st)
            assert int(st) & ~mla.DEVICE_SCORE_RANGE == bit
            assert (ctx[0] == 0).all() and torch.isneginf(lse[0]).all()
            check_attend(ctx, lse, case, 16, 1, rows=[1])


def test_attend_nan_inside_and_exponent_range(mla):
    g = gen(79)
    case = attend_case(g, 2, 1, 128, 200, 1, [200, 200], [0, 0])
    q, codes, scales, rope, start, length = case
    codes[0, 150, 300] = 0xFF                       # a NaN in row 0 only
    scales[1, :3] = torch.tensor([64, 134, 20], device=DEV, dtype=torch.uint8)   # both ends, and below
    codes[1, 1] &= 0x80                             # (the largest unit on zeros: scores stay in range)
    ctx = torch.empty(2, 128, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 128, device=DEV)
    mla.decode_attend_q8(q, codes, scales, 1, rope, start, length, 2, 1, SCALE, ctx, lse)
    assert torch.isnan(ctx[0]).all()
    check_attend(ctx, lse, case, 1, 1, rows=[1])


def test_attend_offsets_past_32_bits(mla):
    """A cache whose rows lie past 2^32 bytes."""
    T, block = 3 * 2 ** 20, 64
    g = gen(80)
    codes = torch.zeros(3, T, 512, dtype=torch.uint8, device=DEV)     # 4.8 GB
    scales = torch.full((3, T // block), 120, dtype=torch.uint8, device=DEV)
    rope = torch.zeros(3, T, 64, dtype=torch.bfloat16, device=DEV)
    n = 300
    start = i32([0, T - 512, T - 320])
    small, _ = random_cache(g, 3, n, 512, 1)
    for b in range(3):
        s = int(start[b])
        codes[b, s:s + n] = small[b]
        rope[b, s:s + n] = normal(g, n, 64).bfloat16()
    q = normal(g, 3, 128, 576).bfloat16() * 0.1
    ctx = torch.empty(3, 128, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, 128, device=DEV)
    mla.decode_attend_q8(q, codes, scales, block, rope, start, i32([n] * 3), 3, 1, SCALE, ctx, lse)
    view = torch.stack([codes[b, int(start[b]):int(start[b]) + n] for b in range(3)])
    ropes = torch.stack([rope[b, int(start[b]):int(start[b]) + n] for b in range(3)])
    check_attend(ctx, lse, (q, view, torch.full((3, 5), 120, dtype=torch.uint8, device=DEV), ropes, i32([0] * 3), i32([n] * 3)),
                 block, 1)


def test_attend_many_rows_takes_the_planner(mla):
    g = gen(81)
    B = 150
    lengths = torch.randint(0, 400, (B,), generator=torch.Generator().manual_seed(3)).tolist()
    case = attend_case(g, B, 1, 64, 400, 4, lengths, [0] * B)
    q, codes, scales, rope, start, length = case
    ctx = torch.empty(B, 64, 512, dtype=torch.bfloat16, device=DEV)
    lse, st = torch.empty(B, 64, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, 4, rope, start, length, B, 1, SCALE, ctx, lse, device_status=st)
    assert int(st) & ~mla.DEVICE_SCORE_RANGE == 0
    check_attend(ctx, lse, case, 4, 1, rows=range(0, B, 7))


def test_capture_replay_and_other_stream(mla):
    """append + attend captured on a side stream, replayed over new inputs."""
    g = gen(82)
    B, T, block = 2, 600, 16
    codes, scales = random_cache(g, B, T, 512, block)
    rope = normal(g, B, T, 64).bfloat16()
    raw, raw_rope = normal(g, B, 1, 512).bfloat16(), normal(g, B, 1, 64).bfloat16()
    gain = torch.ones(512, device=DEV).bfloat16()
    q = normal(g, B, 128, 576).bfloat16() * 0.1
    length, start = i32([500, 3]), i32([16, 0])
    ctx, lse = torch.empty(B, 128, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B, 128, device=DEV)
    ws = torch.empty(mla.decode_workspace_size(B, 1, 128, 512, 64, T), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        mla.append_compressed_q8(raw, raw_rope, gain, EPS, THETA, codes, scales, block, rope, start, length,
                                 kv_len_out=length, stream=stream)
        mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, 1, SCALE, ctx, lse, workspace=ws,
                             stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert length.tolist() == [501, 4]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert length.tolist() == [501, 4]
    for k in range(3):
        raw.copy_(normal(g, B, 1, 512))
        q.copy_(normal(g, B, 128, 576) * 0.1)
        graph.replay()
    torch.cuda.synchronize()
    assert length.tolist() == [504, 7]
    check_attend(ctx, lse, (q, codes, scales, rope, start, length), block, 1)


def test_append_lengths_over_the_offsets(mla):
    """New lengths written over the offsets tensor, rows of several tiles: every tile reads the old offsets."""
    g = gen(83)
    B, T, s_new, block = 3, 900, 700, 16
    codes, scales = random_cache(g, B, T, 512, block)
    rope = normal(g, B, T, 64).bfloat16()
    raw, raw_rope = normal(g, B, s_new, 512).bfloat16(), normal(g, B, s_new, 64).bfloat16()
    gain = torch.ones(512, device=DEV).bfloat16()
    length, offset = i32([0, 100, 33]), i32([7, 5000, 33])
    off0 = offset.tolist()
    before = codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)
    mla.append_compressed_q8(raw, raw_rope, gain, EPS, THETA, codes, scales, block, rope, None, length,
                             kv_len_out=offset, row_offsets=offset)
    assert offset.tolist() == [700, 800, 733] and length.tolist() == [0, 100, 33]
    check_append(raw, raw_rope, gain, before, (codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)), block,
                 [0] * B, [0, 100, 33], off0, s_new, torch.bfloat16)


def test_attend_fp16_operand_range(mla):
    """Held values of units below 2^-15 are rounded to multiples of 2^-24 and flagged; so is a query value beyond
    65504, which saturates.  Each row has few keys (one piece), its rope scores spread the probabilities."""
    g = gen(84)
    B, T = 3, 100
    q, codes, scales, rope, start, length = attend_case(g, B, 1, 128, T, 1, [T] * B, [0] * B)
    scales[0], scales[1], scales[2] = 112, 111, 105        # units 2^-15, 2^-16, 2^-22
    ctx, lse = torch.empty(B, 128, 512, device=DEV), torch.empty(B, 128, device=DEV)

    def run(n, **kw):
        st = status()
        mla.decode_attend_q8(q, codes, scales, 1, rope, start, n, B, 1, SCALE, ctx, lse, device_status=st, **kw)
        return int(st) & ~mla.DEVICE_SCORE_RANGE
    assert run(i32([T, 0, 0])) == 0
    assert run(i32([0, T, 0])) == mla.DEVICE_VALUE_RANGE and run(i32([0, 0, 1])) == mla.DEVICE_VALUE_RANGE
    assert run(i32([T, T, T])) == mla.DEVICE_VALUE_RANGE
    for b in range(B):
        lat = np.round(R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), 1) * 2.0 ** 24) * 2.0 ** -24
        c, l = R.attend64(R.as64(q[b]), lat, R.as64(rope[b]), SCALE)
        # p rounds to fp16 (2^-11), the exchanged scores to fp16 within the bf16 bound on the lse: 2e-2 of each weight
        assert np.abs(R.as64(ctx[b]) - c).max() <= (2e-2 + 2.0 ** -11) * np.abs(lat).max()
        assert np.abs(R.as64(lse[b]) - l).max() <= 2e-2
    # the query: feature 3 meets zero latents, so the scores are those of any finite value
    scales.fill_(120)
    codes[..., 3] = 0
    assert run(length) == 0
    want = ctx.clone()
    q[1, 5, 3] = 65280.0                                   # the largest bf16 that fp16 holds
    assert run(length) == 0 and torch.equal(ctx, want)
    for big in (65536.0, -1e30, float("inf")):
        q[1, 5, 3] = big
        assert run(length) == mla.DEVICE_VALUE_RANGE and torch.equal(ctx, want)
