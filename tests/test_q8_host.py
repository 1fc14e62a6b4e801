"""Refusals of the 8-bit cache, attention-weight and eviction entry points (host checks: nothing is
launched, the pointers are not device memory), and the plain 64-bit forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from tests import q8_reference as R


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


def _call(mla, fn, names, base, changes, arrays=None):
    args = dict(base)
    args.update(changes)
    st = getattr(mla.lib, fn)(*[args[n] for n in names])
    return st, mla.lib.mla_last_error_detail().decode()


APPEND = dict(raw=16, raw_rs=512, raw_ts=512, rr=16, rr_rs=64, rr_ts=64, dtype=1, w=16, eps=1e-6, theta=1e4, off=None,
              codes=16, c_rs=512, c_bs=0, scales=16, s_bs=0, block=16, rope=16, r_rs=64, r_bs=0, rope_dtype=1,
              start=None, length=16, out=None, batch=1, s_new=1, rank=512, rope_dim=64, t_max=64, status=None,
              stream=None)


@pytest.mark.parametrize("change,needle", [
    (dict(raw=None), "NULL"), (dict(w=None), "NULL"), (dict(length=None), "NULL"), (dict(rope=None), "NULL"),
    (dict(codes=None), "NULL"), (dict(scales=None), "NULL"),
    (dict(dtype=2), "dtype"), (dict(rope_dtype=-1), "dtype"),
    (dict(batch=0), "positive"), (dict(batch=65536), "65535"), (dict(s_new=0), "positive"), (dict(t_max=0), "positive"),
    (dict(t_max=1 << 31), "int32"), (dict(rank=1025, raw_ts=2000, c_rs=2000), "rank"), (dict(rope_dim=63), "rope_dim"),
    (dict(eps=-1.0), "epsilon"), (dict(theta=0.0), "theta"), (dict(raw_ts=500), "strides"), (dict(c_rs=511), "strides"),
    (dict(r_rs=10), "strides"), (dict(s_bs=-1), "strides"),
    (dict(block=0), "scale_block"), (dict(block=3), "scale_block"), (dict(block=128), "scale_block"),
    (dict(block=-16), "scale_block"),
])
def test_append_q8_refusals(mla, change, needle):
    st, why = _call(mla, "mla_append_compressed_q8", list(APPEND), APPEND, change)
    assert st == 1 and needle in why, why


CONVERT = dict(lat=16, l_rs=512, l_bs=0, dtype=1, codes=16, c_rs=512, c_bs=0, scales=16, s_bs=0, block=1, start=None,
               length=16, batch=1, rank=512, t_max=64, status=None, stream=None)
BACK = ["codes", "c_rs", "c_bs", "scales", "s_bs", "block", "lat", "l_rs", "l_bs", "dtype", "start", "length", "batch",
        "rank", "t_max", "status", "stream"]


@pytest.mark.parametrize("fn,names", [("mla_quantize_cache", list(CONVERT)), ("mla_dequantize_cache", BACK)])
@pytest.mark.parametrize("change,needle", [
    (dict(lat=None), "NULL"), (dict(codes=None), "NULL"), (dict(scales=None), "NULL"), (dict(length=None), "NULL"),
    (dict(dtype=7), "dtype"), (dict(batch=-1), "positive"), (dict(rank=0), "positive"), (dict(l_rs=100), "strides"),
    (dict(c_rs=100), "strides"), (dict(block=12), "scale_block"), (dict(batch=70000), "65535"),
])
def test_convert_refusals(mla, fn, names, change, needle):
    st, why = _call(mla, fn, names, CONVERT, change)
    assert st == 1 and needle in why, why


ATTEND = dict(q=16, q_rs=576 * 128, q_hs=576, codes=16, c_rs=512, c_bs=0, scales=16, s_bs=0, block=16, rope=16,
              r_rs=64, r_bs=0, dtype=1, start=None, length=16, batch=1, s_q=1, heads=128, rank=512, rope_dim=64,
              t_max=4096, sel=None, count=None, k_max=0, scale=0.07, ctx=16, x_rs=65536, x_hs=512, out_dtype=1,
              lse=None, ws=256, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(q=None), 1, "NULL"), (dict(codes=None), 1, "NULL"), (dict(scales=None), 1, "NULL"),
    (dict(block=48), 1, "scale_block"), (dict(scale=0.0), 1, "softmax_scale"), (dict(sel=16), 1, "selection"),
    (dict(c_rs=500), 1, "strides"), (dict(ws_bytes=8), 1, "workspace"), (dict(ws=16), 1, "aligned"),
    (dict(codes=24), 1, "16-byte"), (dict(c_rs=520), 1, "multiples"), (dict(rope=24), 1, "16-byte"),
    (dict(r_rs=68), 1, "multiples"), (dict(c_bs=8), 1, "multiples"), (dict(out_dtype=3), 1, "out_dtype"),
    (dict(heads=32), 2, "served"), (dict(rank=256), 2, "served"), (dict(rope_dim=32), 2, "served"),
    (dict(dtype=0, batch=65536), 1, "65535"),
])
def test_attend_q8_refusals(mla, change, status, needle):
    st, why = _call(mla, "mla_decode_attend_q8", list(ATTEND), ATTEND, change)
    assert st == status and needle in why, why


W8 = dict(q=16, q_rs=576 * 128, q_hs=576, codes=16, c_rs=512, c_bs=0, scales=16, s_bs=0, block=16, rope=16, r_rs=64,
          r_bs=0, dtype=1, start=None, length=16, batch=1, s_q=1, heads=128, rank=512, rope_dim=64, t_max=4096, lse=16,
          scale=0.07, decay=1.0, n_new=0, weights=16, w_bs=0, status=None, stream=None)
W16 = [n for n in W8 if n not in ("scales", "s_bs", "block")]


@pytest.mark.parametrize("fn,names", [("mla_key_weights_q8", list(W8)), ("mla_key_weights", W16)])
@pytest.mark.parametrize("change,status,needle", [
    (dict(q=None), 1, "NULL"), (dict(lse=None), 1, "NULL"), (dict(weights=None), 1, "NULL"),
    (dict(codes=None), 1, "NULL"), (dict(decay=-0.1), 1, "decay"), (dict(decay=1.5), 1, "decay"),
    (dict(decay=float("nan")), 1, "decay"), (dict(n_new=-1), 1, "n_new"), (dict(scale=float("inf")), 1, "softmax_scale"),
    (dict(q_hs=500), 1, "strides"), (dict(batch=65536), 1, "65535"), (dict(heads=96), 2, "served"),
    (dict(rank=384), 2, "served"), (dict(codes=18), 1, "16-byte"), (dict(c_rs=514), 1, "multiples"),
    (dict(w_bs=-5), 1, "weights_batch_stride"),
])
def test_key_weights_refusals(mla, fn, names, change, status, needle):
    st, why = _call(mla, fn, names, W8, change)
    assert st == status and needle in why, why


def test_key_weights_needs_equal_layouts(mla):
    st, why = _call(mla, "mla_key_weights", W16, W8, dict(c_bs=4096 * 512, r_bs=0))
    assert st == 1 and "packed" in why


PLAN = dict(weights=16, w_bs=64, start=None, length=16, batch=2, t_max=64, keep=32, sink=4, recent=8, kept=16, k_rs=32,
            counts=16, out=None, status=None, stream=None)


@pytest.mark.parametrize("change,needle", [
    (dict(weights=None), "NULL"), (dict(length=None), "NULL"), (dict(kept=None), "NULL"), (dict(counts=None), "NULL"),
    (dict(batch=0), "positive"), (dict(keep=0), "positive"), (dict(t_max=0), "positive"), (dict(batch=65536), "65535"),
    (dict(sink=-1), "n_sink"), (dict(recent=-1), "n_recent"), (dict(sink=20, recent=13), "n_keep"),
    (dict(sink=2**31 - 1, recent=2**31 - 1), "n_keep"), (dict(k_rs=31), "strides"), (dict(w_bs=-1), "strides"),
])
def test_evict_plan_refusals(mla, change, needle):
    st, why = _call(mla, "mla_evict_plan", list(PLAN), PLAN, change)
    assert st == 1 and needle in why, why


COMPACT = dict(arrays=None, n=1, start=None, kept=16, k_rs=32, counts=16, keep=32, batch=2, t_max=64, status=None,
               stream=None)


def _arrays(mla, *rows):
    return (mla.StateArray * len(rows))(*[mla.StateArray(*r) for r in rows])


GOOD = (4096, 1024, 65536, 1024)


@pytest.mark.parametrize("rows,change,needle", [
    ([GOOD], dict(kept=None), "NULL"), ([GOOD], dict(counts=None), "NULL"), ([GOOD], dict(arrays=None), "NULL"),
    ([GOOD], dict(n=0), "arrays"), ([GOOD] * 9, dict(n=9), "arrays"), ([(0, 1024, 0, 1024)], dict(), "NULL"),
    ([(4096, 1000, 0, 1024)], dict(), "strides"), ([(4096, 1024, 0, 0)], dict(), "strides"),
    ([GOOD], dict(batch=0), "positive"), ([GOOD], dict(keep=-1), "positive"), ([GOOD], dict(k_rs=8), "kept_row_stride"),
])
def test_cache_compact_refusals(mla, rows, change, needle):
    arr = _arrays(mla, *rows)
    args = dict(COMPACT, arrays=arr)
    args.update(change)
    st = mla.lib.mla_cache_compact(*[args[n] for n in COMPACT])
    assert st == 1 and needle in mla.lib.mla_last_error_detail().decode()


def test_wrappers_check_their_tensors(mla):
    codes, scales = torch.zeros(1, 8, 32, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.uint8)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(AssertionError):   # too few exponents
        mla.dequantize_cache(codes, scales, 2, torch.zeros(1, 8, 32), None, lens)
    with pytest.raises(AssertionError):   # lengths of another type
        mla.dequantize_cache(codes, scales, 4, torch.zeros(1, 8, 32), None, lens.long())
    with pytest.raises(AssertionError):   # codes of another type
        mla.quantize_cache(torch.zeros(1, 8, 32), codes.int(), scales, 4, None, lens)


# ---------------------------------------------------------------- the plain forms themselves

def test_codes_are_torchs_e4m3():
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = every.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.codes64(every.numpy()), want, equal_nan=True)


def test_nearest_e4m3_is_torchs_rounding():
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(3)) * s for s in (1e-3, 0.1, 1, 100)])
    x = x.clamp(-448, 448)
    # midpoints of neighbouring values (ties), and the values themselves
    v = np.unique(R.codes64(np.arange(127)))
    x = torch.cat([x, torch.from_numpy((v[1:] + v[:-1]) / 2).float(), torch.from_numpy(v).float()])
    assert np.array_equal(R.nearest_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_exponents():
    for k in (-20, -3, 0, 5):
        assert R.exponent64(1.75 * 2.0 ** k) == 127 + k - 8          # just fits
        assert R.exponent64(np.nextafter(1.75 * 2.0 ** k, 1e9)) == 127 + k - 7
        assert R.near_exponent_border(1.75 * 2.0 ** k, 1e-6) and not R.near_exponent_border(1.5 * 2.0 ** k, 1e-6)
    assert R.exponent64(0.0) == 64 and R.exponent64(1e30) == 134


def test_evict_keeps_sinks_recent_and_heaviest():
    w = np.array([0, 9, 1, 5, 5, 5, 2, 0, 0, 0], dtype=np.float32)
    assert R.evict64(w, 10, 10, 1, 1) is None
    assert R.evict64(w, 10, 5, 1, 1).tolist() == [0, 1, 3, 4, 9]     # ties: the lower positions
    assert R.evict64(w, 10, 3, 1, 2).tolist() == [0, 8, 9]


def test_weights_of_one_token_sum_to_the_heads():
    g = np.random.default_rng(0)
    q, lat, rope = g.normal(size=(1, 6, 20)), g.normal(size=(30, 16)), g.normal(size=(30, 4))
    _, lse = R.attend64(q[0], lat, rope, 0.3)
    w = R.key_weights64(q, lat, rope, lse[None], np.full(30, np.nan), 0.3, 0.0, 0)
    assert np.isclose(w.sum(), 6.0)
