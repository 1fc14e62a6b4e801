"""The 8-bit cache where it can go wrong: non-finite tokens, dominant keys, wide rope keys, far positions, and
weights from the attention's own lse."""
import math

import numpy as np
import pytest
import torch

from tests import q8_reference as R
from tests.test_gpu_q8 import (DEV, EPS, SCALE, THETA, attend_case, check_append, gen, i32, normal, random_cache,
                               status)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


# ---------------------------------------------------------------- append

# encode_kernel serves aligned ranks up to 512, encode_walk_kernel the others
SHAPES = [(512, torch.bfloat16), (512, torch.float32), (96, torch.bfloat16), (1024, torch.bfloat16), (33, torch.float32)]


def normalised(raw, gain, eps):
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        return R.rms_norm64(R.as64(raw), R.as64(gain), eps)


def append_into_partly_filled_blocks(mla, raw, gain, eps, block, slack=1e-5):
    """Appends raw [2, s_new, rank] behind 37 tokens of row 0 and at the front of row 1, and checks every code
    and exponent against 64 bits: a NaN value is held as NaN and sets no unit.  (The slack is that of the f32 norm,
    as for other appends.)  Returns the status."""
    B, s_new, rank = raw.shape
    T = 160
    codes, scales = random_cache(gen(block), B, T, rank, block)
    rope = torch.zeros(B, T, 8, dtype=raw.dtype, device=DEV)
    start, length = [block, 0], [37, 0]
    codes0, scales0 = codes.cpu().numpy(), scales.cpu().numpy()
    st = status()
    mla.append_compressed_q8(raw, torch.zeros(B, s_new, 8, dtype=raw.dtype, device=DEV), gain, eps, THETA, codes, scales,
                             block, rope, i32(start), i32(length), device_status=st)
    codes1, scales1 = codes.cpu().numpy(), scales.cpu().numpy()
    v = normalised(raw, gain, eps)
    for b in range(B):
        lo = start[b] + length[b]
        hi = lo + s_new
        same = np.r_[0:lo, hi:T]
        for k in range(lo // block, (hi - 1) // block + 1):
            r0, r1, old0 = max(lo, k * block), min(hi, (k + 1) * block), max(k * block, start[b])
            want = v[b, r0 - lo:r1 - lo]
            size = np.abs(want)
            amax = size[~np.isnan(size)].max(initial=0.0)
            allowed = {R.exponent64(amax * (1 - slack)), R.exponent64(amax * (1 + slack))}
            if old0 < lo:
                allowed = {max(a, int(scales0[b, k])) for a in allowed}
            e = int(scales1[b, k])
            assert e in allowed
            units = want * 2.0 ** (127.0 - e)
            got = R.codes64(codes1[b, r0:r1])
            assert np.array_equal(np.isnan(got), np.isnan(units))
            fine = np.isfinite(units)
            assert (np.abs(got - units)[fine] <= (np.abs(R.nearest_e4m3(units) - units) + 2 * slack * np.abs(units))[fine]).all()
            assert np.array_equal(got[np.isinf(units)], np.copysign(448.0, units[np.isinf(units)]))
            if old0 < lo:
                held = R.codes64(codes0[b, old0:lo]) * 2.0 ** (float(scales0[b, k]) - e)
                assert np.array_equal(R.codes64(codes1[b, old0:lo]), R.nearest_e4m3(held))
                same = np.setdiff1d(same, np.arange(old0, lo))
        assert np.array_equal(codes1[b, same], codes0[b, same])
    return int(st)


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf", "zero, eps 0"])
@pytest.mark.parametrize("block", [1, 4, 8, 64])
@pytest.mark.parametrize("rank,dtype", SHAPES)
def test_append_of_a_token_without_a_norm(mla, rank, dtype, block, bad):
    """One new token that is NaN after its norm leaves the unit, the tokens beside it and those held before alone."""
    g = gen(rank + block)
    raw = normal(g, 2, 6, rank).to(dtype)
    gain = torch.exp(0.3 * normal(g, rank)).to(dtype)
    eps = EPS
    if bad == "zero, eps 0":
        raw[0, 1], raw[1, 0], eps = 0.0, 0.0, 0.0
    else:
        raw[0, 1, 5] = raw[1, 0, rank - 1] = float(bad)
    assert append_into_partly_filled_blocks(mla, raw, gain, eps, block) == 0


@pytest.mark.parametrize("block", [1, 8])
@pytest.mark.parametrize("rank,dtype", SHAPES)
def test_append_of_infinite_values(mla, rank, dtype, block):
    """An infinite norm weight: those values saturate at 57344 and are flagged."""
    g = gen(rank + block)
    gain = torch.ones(rank, device=DEV, dtype=dtype)
    gain[7] = float("inf")
    assert append_into_partly_filled_blocks(mla, normal(g, 2, 6, rank).to(dtype), gain, EPS, block) == mla.DEVICE_VALUE_RANGE


@pytest.mark.parametrize("block", [1, 8])
@pytest.mark.parametrize("rank,dtype", SHAPES)
def test_append_of_tiny_tokens_under_zero_weights(mla, rank, dtype, block):
    """Tokens of 1e-21 at eps = 0 have an inverse norm of 1e21: times a weight of 0 they are 0, not NaN."""
    raw = torch.full((2, 6, rank), 1e-21, device=DEV, dtype=dtype)
    assert append_into_partly_filled_blocks(mla, raw, torch.zeros(rank, device=DEV, dtype=dtype), 0.0, block) == 0


def test_append_after_a_rollback(mla):
    """A block that keeps tokens keeps its unit, one that keeps none takes that of its next tokens."""
    g = gen(12)
    codes, scales = torch.zeros(2, 32, 512, dtype=torch.uint8, device=DEV), torch.zeros(2, 4, dtype=torch.uint8, device=DEV)
    rope, n = torch.zeros(2, 32, 8, device=DEV), i32([0, 0])

    def append(s_new, size):
        mla.append_compressed_q8(normal(g, 2, s_new, 512), torch.zeros(2, s_new, 8, device=DEV),
                                 torch.full((512,), size, device=DEV), EPS, THETA, codes, scales, 8, rope, None, n, kv_len_out=n)
    append(8, 1.0)
    before = n.clone()
    append(8, 100.0)
    large = scales[:, 1].tolist()
    mla.rollback_lengths(before, i32([0, 3]), n)
    assert n.tolist() == [8, 11]
    append(2, 1.0)
    assert n.tolist() == [10, 13]
    # unit 2^k holds rms 1 (a largest magnitude of 2.5 to 7 among 512 values), 2^(k + 6) or more rms 100
    assert int(scales[0, 1]) <= large[0] - 5 and int(scales[1, 1]) == large[1]


@pytest.mark.parametrize("dtype,rope_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("rank,rope_dim,s_new,block", [(512, 128, 7, 1), (256, 256, 70, 16), (512, 66, 7, 64), (512, 64, 130, 8),
                                                      (33, 6, 7, 4), (1024, 256, 20, 16)])
def test_append_wide_rope_keys_and_far_positions(mla, dtype, rope_dtype, rank, rope_dim, s_new, block):
    """Rope keys of more than 64 values beside a latent held in registers; positions across 2^24, from where an f32
    no longer holds them, and across 2^31."""
    g = gen(rank + rope_dim)
    B, T = 4, 420
    codes, scales = random_cache(g, B, T, rank, block)
    rope = normal(g, B, T, rope_dim).to(rope_dtype)
    raw, raw_rope = normal(g, B, s_new, rank).to(dtype), normal(g, B, s_new, rope_dim).to(dtype)
    gain = torch.exp(0.3 * normal(g, rank)).to(dtype)
    start, length, offset = [0, block, 0, 2 * block], [5, 37, 0, 64], [2 ** 24 - 3, 2 ** 31 - 4, 65530, 2 ** 24 + 1]
    before = codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)
    st = status()
    mla.append_compressed_q8(raw, raw_rope, gain, EPS, THETA, codes, scales, block, rope, i32(start), i32(length),
                             row_offsets=i32(offset), device_status=st)
    assert int(st) == 0
    check_append(raw, raw_rope, gain, before, (codes.cpu().numpy(), scales.cpu().numpy(), R.as64(rope)), block, start, length,
                 offset, s_new, rope_dtype)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("gap", [21.625, 23.375, 26.625])
def test_attend_light_keys_behind_a_heavy_one(mla, gap):
    """One key 2^gap times heavier than 16384 equal ones, its latent zero: the context is that of the light keys.
    80 rows over one buffer, so that a piece holds thousands of keys.

    Scores are exact (one rope feature, log2 units).  p rounds to 2^-11 of itself, or to half of 2^-31 of the heavy
    key's weight; a piece's context to fp16 (2^-11, 2^-25 below its normal range); sums of positive f32 values,
    accumulated 16 keys a step, to 2^-23 per step and 2^-24 per tile."""
    g = gen(int(8 * gap))
    B, T, heads = 80, 16385, 64
    codes, scales = random_cache(g, 1, T, 512, 1)
    codes = codes & 0x7F                                  # positive latents: no cancellation
    codes[0, 0] = 0
    rope = torch.zeros(1, T, 64, dtype=torch.bfloat16, device=DEV)
    rope[0, 0, 0] = gap
    q = torch.zeros(B, heads, 576, dtype=torch.bfloat16, device=DEV)
    q[..., 512] = 1.0
    ctx, lse, st = torch.empty(B, heads, 512, device=DEV), torch.empty(B, heads, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, 1, rope, None, i32([T] * B), B, 1, math.log(2.0), ctx, lse, device_status=st)
    assert int(st) == 0
    lat = R.held64(codes[0].cpu().numpy(), scales[0].cpu().numpy(), 1)
    total = 2.0 ** gap + T - 1
    want = lat.sum(0) / total
    bound = max(2.0 ** -11, 2.0 ** (gap - 32)) + 2.0 ** -11 + T / 16 * 2.0 ** -23 + T / 64 * 2.0 ** -24 + 1e-5
    got = R.as64(ctx)
    assert (np.abs(got - want) <= bound * want + 2.0 ** -25).all()
    # The sum takes one f32 addition per tile of 64 keys, each off by up to 2^-24 of it, always the same way here
    # (the light keys add the same small number to a sum of 2^7): T / 64 * 2^-24 = 1.53e-5 in the logarithm.  Then
    # three f32 operations on values up to 32 round to half of 2^-19 (m less 7 and log2 l added, the logarithm itself, the
    # product with ln 2): 3 * 2^-20 = 2.9e-6.
    assert np.abs(R.as64(lse) - math.log(total)).max() <= T / 64 * 2.0 ** -24 + 3 * 2.0 ** -20


@pytest.mark.parametrize("q8", [True, False])
def test_own_workspace_outlives_a_call_on_another_stream(mla, q8, monkeypatch):
    """A call on a side stream that is still busy: its workspace is not handed to the current stream meanwhile."""
    g = gen(3)
    B, T, heads = 2, 3000, 128
    codes, scales = random_cache(g, B, T, 512, 16)
    latent, rope = normal(g, B, T, 512).bfloat16(), normal(g, B, T, 64).bfloat16()
    q = normal(g, B, heads, 576).bfloat16() * 0.1
    ctx, lse, length = torch.empty(B, heads, 512, device=DEV), torch.empty(B, heads, device=DEV), i32([T, 5])
    taken, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        taken.append((t.data_ptr(), t.numel()))
        return t

    def call(stream):
        if q8:
            mla.decode_attend_q8(q, codes, scales, 16, rope, None, length, B, 1, 0.07, ctx, lse, stream=stream)
        else:
            mla.decode_attend(q, latent, rope, None, length, B, 1, 0.07, ctx, lse, stream=stream)
    call(None)                              # (a kernel's first launch loads its code, which waits for the device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)      # 0.2 s
    monkeypatch.setattr(torch, "empty", spy)
    call(side)
    monkeypatch.undo()
    (ptr, size), = taken
    others = [empty(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert not side.query() and all(t.data_ptr() != ptr for t in others)
    side.synchronize()
    assert torch.isfinite(ctx).all()


@pytest.mark.parametrize("q8", [True, False])
def test_weights_from_the_attentions_own_lse(mla, q8):
    """attend, then weights from its lse: that is off by up to 2e-2 (the bound of its tests), the weights by the
    exponential of that, and by 1e-4 of their own (as with an exact lse)."""
    g = gen(96)
    B, T, heads, block = 2, 1500, 128, 8
    q, codes, scales, rope, start, length = attend_case(g, B, 1, heads, T, block, [1500, 700], [0, 8])
    latent, ctx = normal(g, B, T, 512).bfloat16(), torch.empty(B, heads, 512, device=DEV)
    lse, w = torch.empty(B, heads, device=DEV), torch.zeros(B, T, device=DEV)
    if q8:
        mla.decode_attend_q8(q, codes, scales, block, rope, start, length, B, 1, SCALE, ctx, lse)
        mla.key_weights_q8(q, codes, scales, block, rope, lse, start, length, B, 1, SCALE, w)
    else:
        mla.decode_attend(q, latent, rope, start, length, B, 1, SCALE, ctx, lse)
        mla.key_weights(q, latent, rope, lse, start, length, B, 1, SCALE, w)
    got, bound = R.as64(w), math.expm1(2e-2) + 1e-4
    for b in range(B):
        lo, n = int(start[b]), int(length[b])
        lat = R.held64(codes[b].cpu().numpy(), scales[b].cpu().numpy(), block)[lo:lo + n] if q8 else R.as64(latent[b, lo:lo + n])
        keys = R.as64(rope[b, lo:lo + n])
        exact = R.attend64(R.as64(q[b]), lat, keys, SCALE)[1]
        want = R.key_weights64(R.as64(q[b:b + 1]), lat, keys, exact[None], np.zeros(n), SCALE, 0.0, 0)
        assert (np.abs(got[b, lo:lo + n] - want) <= bound * want).all()
        assert abs(got[b].sum() - heads) <= bound * heads


@pytest.mark.parametrize("order", ["rising", "falling", "heavy last"])
def test_attend_moves_its_reference(mla, order):
    """Scores that rise by a quarter (log2 units) from tile to tile, fall so, or jump by 60 at the last key: the reference
    moves and the context is rescaled, or most keys are far lighter than it.

    Exact scores; roundings as for light keys behind a heavy one, 2^-32 of the heaviest weight per key for those below
    fp16's normal range, and 2^-21 for each of at most 9 rescales."""
    g = gen(len(order))
    B, T, heads = 80, 16385, 64
    codes, scales = random_cache(g, 1, T, 512, 1)
    codes = codes & 0x7F
    score = torch.arange(T, device=DEV) // 64 * 0.25                  # up to 64: 8 bits
    if order == "falling":
        score = score.flip(0)
    elif order == "heavy last":
        score = torch.where(torch.arange(T, device=DEV) == T - 1, 60.0, 0.0)
    rope = torch.zeros(1, T, 64, dtype=torch.bfloat16, device=DEV)
    rope[0, :, 0] = score
    q = torch.zeros(B, heads, 576, dtype=torch.bfloat16, device=DEV)
    q[..., 512] = 1.0
    ctx, lse, st = torch.empty(B, heads, 512, device=DEV), torch.empty(B, heads, device=DEV), status()
    mla.decode_attend_q8(q, codes, scales, 1, rope, None, i32([T] * B), B, 1, math.log(2.0), ctx, lse, device_status=st)
    assert int(st) == 0
    lat = R.held64(codes[0].cpu().numpy(), scales[0].cpu().numpy(), 1)
    p = np.exp2(R.as64(rope[0, :, 0]) - R.as64(score).max())
    want = p @ lat / p.sum()
    bound = 2 * 2.0 ** -11 + T / 16 * 2.0 ** -23 + T / 64 * 2.0 ** -24 + 9 * 2.0 ** -21 + 1e-5
    assert (np.abs(R.as64(ctx) - want) <= bound * want + lat.sum(0) * 2.0 ** -32 / p.sum() + 2.0 ** -25).all()
    # the lse: additions and three f32 operations on values up to 64 (2^-19 each, and as much for the rescales)
    exact = (R.as64(score).max() + math.log2(p.sum())) * math.log(2.0)
    assert np.abs(R.as64(lse) - exact).max() <= T / 64 * 2.0 ** -24 + 4 * 2.0 ** -18
