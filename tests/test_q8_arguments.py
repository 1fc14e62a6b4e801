"""Tensors too small for what the kernels read or write are refused by the bindings of the 8-bit cache, the attention
weights and the eviction, before any launch (CPU tensors)."""
import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


B, T, RANK, ROPE, HEADS = 3, 16, 32, 8, 2


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


def tensors():
    return dict(
        start=i32(B), length=i32(B), out=i32(B), offset=i32(B), counts=i32(B), status=i32(1),
        raw=torch.zeros(B, 1, RANK), raw_rope=torch.zeros(B, 1, ROPE), gain=torch.zeros(RANK),
        codes=torch.zeros(B, T, RANK, dtype=torch.uint8), scales=torch.zeros(B, T, dtype=torch.uint8),
        rope=torch.zeros(B, T, ROPE), latent=torch.zeros(B, T, RANK), q=torch.zeros(B, HEADS, RANK + ROPE),
        ctx=torch.zeros(B, HEADS, RANK), lse=torch.zeros(B, HEADS), weights=torch.zeros(B, T),
        sel=torch.zeros(B, 4, dtype=torch.int32), sel_count=i32(B), kept=torch.zeros(B, 4, dtype=torch.int32))


CALLS = {
    "append": (lambda m, s: m.append_compressed_q8(
        s["raw"], s["raw_rope"], s["gain"], 1e-6, 1e4, s["codes"], s["scales"], 1, s["rope"], s["start"], s["length"],
        kv_len_out=s["out"], row_offsets=s["offset"], device_status=s["status"]),
        ["start", "length", "out", "offset", "status"]),
    "quantize": (lambda m, s: m.quantize_cache(s["latent"], s["codes"], s["scales"], 1, s["start"], s["length"],
                                               device_status=s["status"]), ["start", "status"]),
    "dequantize": (lambda m, s: m.dequantize_cache(s["codes"], s["scales"], 1, s["latent"], s["start"], s["length"],
                                                   device_status=s["status"]), ["start", "status"]),
    "attend": (lambda m, s: m.decode_attend_q8(
        s["q"], s["codes"], s["scales"], 1, s["rope"], s["start"], s["length"], B, 1, 0.1, s["ctx"], s["lse"], s["sel"],
        s["sel_count"], device_status=s["status"]), ["start", "length", "lse", "sel_count", "status"]),
    "weights": (lambda m, s: m.key_weights(s["q"], s["latent"], s["rope"], s["lse"], s["start"], s["length"], B, 1, 0.1,
                                           s["weights"], device_status=s["status"]), ["start", "length", "lse", "status"]),
    "weights q8": (lambda m, s: m.key_weights_q8(s["q"], s["codes"], s["scales"], 1, s["rope"], s["lse"], s["start"],
                                                 s["length"], B, 1, 0.1, s["weights"], device_status=s["status"]),
                   ["start", "length", "lse", "status"]),
    "plan": (lambda m, s: m.evict_plan(s["weights"], s["start"], s["length"], 4, 1, 1, s["kept"], s["counts"],
                                       kv_len_out=s["out"], device_status=s["status"]), ["start", "counts", "out", "status"]),
    "compact": (lambda m, s: m.cache_compact([s["codes"]], s["start"], s["kept"], s["counts"], device_status=s["status"]),
                ["start", "counts", "status"]),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in CALLS.items() for n in names])
def test_short_tensors_are_refused(mla, call, name):
    s = tensors()
    s[name] = s[name].reshape(-1)[:-1]
    with pytest.raises(AssertionError):
        CALLS[call][0](mla, s)


@pytest.mark.parametrize("call", list(CALLS))
def test_full_tensors_pass_the_checks(mla, call, monkeypatch):
    """The same calls with whole tensors get as far as the launch."""
    def reached(*_):
        raise KeyError("the launch")
    monkeypatch.setattr(mla, "_launch_stream", reached)
    with pytest.raises(KeyError, match="the launch"):
        CALLS[call][0](mla, tensors())
