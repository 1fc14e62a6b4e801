"""The paged cache on the host: which keys a token sees, refusals of the C ABI, and checks of the bindings, none of
which reaches a launch."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tests import paged_reference as P

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mla_latent_kv_12_gb300", "csrc")


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


def test_keys_seen_against_brute_force(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "paged_keys_test"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "paged_keys_test.cpp"), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_reference_masks():
    lists = P.ancestors([-1, 0, 0, 2, -1])
    assert lists == [[0], [0, 1], [0, 2], [0, 2, 3], [4]]
    assert P.mask_words(lists, 5)[:, 0].tolist() == [1, 3, 5, 13, 16]
    assert P.mask_words([[0, 63, 64]], 65).tolist() == [[-2 ** 63 + 1, 1]]
    assert P.seen(10, 3, 1).tolist() == list(range(9))
    assert P.seen(10, 5, 3, lists[3]).tolist() == [0, 1, 2, 3, 4, 5, 7, 8]
    assert P.seen(10, 3, 3).tolist() == [] and P.seen(2, 4, 1).tolist() == []


# ------------------------------------------------ the C ABI (the pointers are no device memory: nothing may launch)

MB = 1 << 20
# raw, strides, rope raw, strides, dtype, weight, eps, theta, positions, latent, strides, rope, strides, cache dtype,
# table, stride, width, page size, pages, kv_len, counts, out, batch, s_new, rank, rope dim, status, stream
APPEND = [MB, 512, 512, MB, 64, 64, 1, MB, 1e-6, 1e4, None, MB, 512, 512 * 16, MB, 64, 64 * 16, 1, MB, 8, 8, 16, 100, MB,
          None, None, 4, 1, 512, 64, None, None]


@pytest.mark.parametrize("changes,needle", [
    ({0: None}, "NULL"), ({3: None}, "NULL"), ({7: None}, "NULL"), ({11: None}, "NULL"), ({18: None}, "page_table"),
    ({23: None}, "NULL"), ({6: 4}, "dtype"), ({17: 3}, "dtype"), ({8: -1.0}, "epsilon"), ({8: float("nan")}, "epsilon"),
    ({9: 0.0}, "theta"), ({9: float("inf")}, "theta"), ({2: 511}, "strides"), ({12: 511}, "strides"), ({13: -1}, "strides"),
    ({5: 63}, "strides"), ({15: 63}, "strides"), ({26: 0}, "positive"), ({27: 0}, "positive"), ({28: 0}, "positive"),
    ({20: 0}, "positive"), ({21: 0}, "positive"), ({22: 0}, "positive"), ({19: 7}, "page_table_stride"),
    ({20: 1 << 20, 19: 1 << 20, 21: 1 << 12}, "int32"), ({28: 1025, 2: 2048, 12: 2048}, "rank"), ({29: 63}, "even"),
    ({29: 258, 5: 300, 15: 300}, "even"), ({25: MB + 4}, "apart"), ({24: 2 * MB, 25: 2 * MB}, "apart"),
])
def test_append_refusals(mla, changes, needle):
    args = list(APPEND)
    for i, v in changes.items():
        args[i] = v
    assert mla.lib.mla_append_paged(*args) == 1
    assert needle in mla.lib.mla_last_error_detail().decode()


# q, strides, latent, strides, rope, strides, dtype, table, stride, width, page size, pages, kv_len, counts, tree, batch,
# s_q, heads, rank, rope dim, sel, counts, k_max, scale, ctx, strides, out dtype, lse, workspace, bytes, status, stream
ATTEND = [MB, 128 * 576, 576, MB, 512, 512 * 16, MB, 64, 64 * 16, 1, MB, 8, 8, 16, 100, MB, None, None, 4, 1, 128, 512, 64,
          None, None, 0, 0.07, MB, 128 * 512, 512, 1, None, MB, 1 << 40, None, None]


@pytest.mark.parametrize("changes,status,needle", [
    ({0: None}, 1, "NULL"), ({3: None}, 1, "NULL"), ({6: None}, 1, "NULL"), ({10: None}, 1, "page_table"),
    ({15: None}, 1, "NULL"), ({27: None}, 1, "NULL"), ({9: 2}, 1, "dtype"), ({30: 2}, 1, "dtype"), ({2: 575}, 1, "strides"),
    ({4: 511}, 1, "strides"), ({5: -16}, 1, "non-negative"), ({5: 0}, 1, "positive"), ({11: 7}, 1, "page_table_stride"),
    ({12: 0}, 1, "positive"), ({13: 0}, 1, "positive"), ({14: 0}, 1, "positive"), ({18: 0}, 1, "positive"),
    ({19: 0}, 1, "positive"), ({26: 0.0}, 1, "scale"), ({26: float("nan")}, 1, "scale"), ({23: MB}, 1, "counts"),
    ({33: 100}, 1, "workspace"), ({32: MB + 8}, 1, "256-byte"), ({0: MB + 2}, 1, "aligned"), ({3: MB + 8}, 1, "aligned"),
    ({4: 516}, 1, "multiples"), ({8: 1028}, 1, "multiples"), ({28: 65540}, 1, "multiples"),
    ({17: MB, 19: 1025, 33: 1 << 60}, 1, "nodes"), ({17: MB + 4}, 1, "8-byte"),
    ({20: 16}, 2, "bf16 is served"), ({21: 256}, 2, "bf16 is served"), ({22: 32}, 2, "bf16 is served"),
    ({17: MB, 23: MB, 24: MB, 25: 4}, 2, "tree_mask"),
    ({1: 0}, 1, "q_row_stride"), ({18: 1 << 20, 19: 2, 33: 1 << 60}, 1, "2^20"),
    # rows one by one: page strides of whole rows, fewer than 2^31 rows
    ({13: 15, 5: 512 * 16 + 8}, 2, "whole rows"), ({23: MB, 24: MB, 25: 4, 8: 64 * 16 + 8}, 2, "whole rows"),
    ({13: 1, 14: 2 ** 31 - 1, 5: 1024}, 2, "2^31"),
    # f32: at most 65535 query rows
    ({9: 0, 18: 1 << 14, 19: 4, 33: 1 << 60}, 2, "65535"),
])
def test_attend_refusals(mla, changes, status, needle):
    args = list(ATTEND)
    for i, v in changes.items():
        args[i] = v
    assert mla.lib.mla_decode_attend_paged(*args) == status
    assert needle in mla.lib.mla_last_error_detail().decode()


@pytest.mark.parametrize("changes,needle", [
    ({11: 1 << 24, 12: (1 << 24) + 1, 13: 64}, "page_table_stride"),
    ({11: 1 << 25, 12: (1 << 24) + 1, 13: 64}, "2^30"),                             # keys of a row: by boxes, row by row, f32
    ({11: 1 << 31, 12: (1 << 30) + 1, 13: 1}, "2^30"),
    ({11: 1 << 25, 12: (1 << 24) + 1, 13: 64, 9: 0, 33: 1 << 60}, "2^30"),
    ({11: 1 << 21, 12: 1 << 21, 13: 64, 18: 1024, 33: 1 << 60}, "plan"),            # 2^37 keys of all query rows
    ({11: 1 << 21, 12: 1 << 21, 13: 64, 18: 512, 19: 8, 33: 1 << 60}, "plan"),      # four tokens share a unit
    ({11: 1 << 21, 12: 1 << 21, 13: 63, 18: 256, 19: 8, 33: 1 << 60}, "plan"),
])
def test_attend_refuses_more_keys_than_its_indexes_hold(mla, changes, needle):
    args = list(ATTEND)
    for i, v in changes.items():
        args[i] = v
    assert mla.lib.mla_decode_attend_paged(*args) == (1 if needle == "page_table_stride" else 2)
    assert needle in mla.lib.mla_last_error_detail().decode()


# parents, stride, kv_len, counts, batch, nodes, positions, mask, status, stream
PLAN = [MB, 16, MB, None, 4, 16, MB, MB, None, None]


@pytest.mark.parametrize("i,v", [(0, None), (6, None), (7, None), (4, 0), (4, 65536), (5, 0), (5, 1025), (1, -1), (7, MB + 4)])
def test_plan_refusals(mla, i, v):
    args = list(PLAN)
    args[i] = v
    assert mla.lib.mla_tree_plan(*args) == 1


def test_commit_refusals(mla):
    def call(changes, n_arrays=2, **array):
        states = (mla.StateArray * 300)()
        for s in states:
            s.data, s.token_stride_bytes, s.batch_stride_bytes, s.row_bytes = MB, 1024, 16384, 1024
        for k, v in array.items():
            setattr(states[1], k, v)
        # table, stride, width, page size, pages, kv_len, path, stride, path width, counts, out, batch, status, stream
        args = [MB, 8, 8, 16, 100, MB, MB, 16, 16, MB, None, 4, None, None]
        for i, v in changes.items():
            args[i] = v
        return mla.lib.mla_commit_paged(states, n_arrays, *args)

    for changes in ({0: None}, {1: 7}, {2: 0}, {3: 0}, {4: 0}, {5: None}, {6: None}, {7: -1}, {8: 0}, {8: 1025},
                    {9: None}, {11: 0}, {11: 65536}, {10: MB + 4}, {9: 2 * MB, 10: 2 * MB + 8}):
        assert call(changes) == 1, changes
    assert call({}, n_arrays=0) == 1 and call({}, n_arrays=257) == 1
    assert call({}, data=None) == 1 and call({}, row_bytes=0) == 1 and call({}, row_bytes=2048) == 1
    assert call({}, batch_stride_bytes=-1) == 1


# ------------------------------------------------ the bindings

B, S, PAGES, SIZE, RANK, ROPE, HEADS = 3, 2, 5, 4, 32, 8, 2


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def tensors():
    return dict(raw=torch.zeros(B, S, RANK), raw_rope=torch.zeros(B, S, ROPE), gain=torch.zeros(RANK),
                latent=torch.zeros(PAGES, SIZE, RANK), rope=torch.zeros(PAGES, SIZE, ROPE), table=i32(B, 2), len=i32(B),
                out=i32(B), positions=i32(B, S), counts=i32(B), status=i32(1), q=torch.zeros(B * S, HEADS, RANK + ROPE),
                ctx=torch.zeros(B * S, HEADS, RANK), lse=torch.zeros(B * S, HEADS), sel=i32(B * S, 4), sel_count=i32(B * S),
                mask=torch.zeros(B * S, 1, dtype=torch.int64), parents=i32(B, S), path=i32(B, S))


CALLS = {
    "append": (lambda m, s: m.append_paged(s["raw"], s["raw_rope"], s["gain"], 1e-6, 1e4, s["latent"], s["rope"],
                                           s["table"], s["len"], kv_len_out=s["out"], positions=s["positions"],
                                           counts=s["counts"], device_status=s["status"]),
               ["gain", "len", "out", "positions", "counts", "status"]),
    "attend": (lambda m, s: m.decode_attend_paged(s["q"], s["latent"], s["rope"], s["table"], s["len"], B, S, 0.1,
                                                  s["ctx"], s["lse"], counts=s["counts"], sel=s["sel"],
                                                  sel_count=s["sel_count"], device_status=s["status"]),
               ["len", "lse", "counts", "sel_count", "status"]),
    "tree": (lambda m, s: m.decode_attend_paged(s["q"], s["latent"], s["rope"], s["table"], s["len"], B, S, 0.1, s["ctx"],
                                                s["lse"], tree_mask=s["mask"], device_status=s["status"]),
             ["len", "lse", "mask", "status"]),
    "plan": (lambda m, s: m.tree_plan(s["parents"], s["len"], s["positions"], s["mask"], counts=s["counts"],
                                      device_status=s["status"]), ["len", "positions", "mask", "counts", "status"]),
    "commit": (lambda m, s: m.commit_paged([s["latent"], s["rope"]], s["table"], s["len"], s["path"], s["counts"],
                                           kv_len_out=s["out"], device_status=s["status"]),
               ["len", "counts", "out", "status"]),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in CALLS.items() for n in names])
def test_short_tensors_are_refused(mla, call, name):
    s = tensors()
    s[name] = s[name].reshape(-1)[:-1]
    with pytest.raises(AssertionError):
        CALLS[call][0](mla, s)


@pytest.mark.parametrize("call,name,value", [
    ("append", "table", i32(B - 1, 2)), ("attend", "table", i32(B - 1, 2)), ("commit", "table", i32(B - 1, 2)),
    ("append", "table", torch.zeros(B, 2, dtype=torch.int64)), ("append", "rope", torch.zeros(PAGES, SIZE + 1, ROPE)),
    ("append", "rope", torch.zeros(PAGES - 1, SIZE, ROPE)), ("attend", "rope", torch.zeros(PAGES - 1, SIZE, ROPE)),
    ("append", "latent", torch.zeros(PAGES, RANK, SIZE).transpose(1, 2)), ("append", "gain", torch.zeros(RANK).double()),
    ("attend", "latent", torch.zeros(PAGES, SIZE, RANK, dtype=torch.bfloat16)), ("tree", "mask", i32(B * S, 1)),
    ("attend", "ctx", torch.zeros(B * S, HEADS, RANK + 1)), ("plan", "parents", torch.zeros(B, S, dtype=torch.int64)),
    ("commit", "path", torch.zeros(B, S, dtype=torch.int64)), ("commit", "rope", torch.zeros(PAGES, SIZE + 1, ROPE)),
])
def test_wrong_tensors_are_refused(mla, call, name, value):
    s = tensors()
    s[name] = value
    with pytest.raises(AssertionError):
        CALLS[call][0](mla, s)


@pytest.mark.parametrize("call", list(CALLS))
def test_full_tensors_pass_the_checks(mla, call):
    """The same calls with whole tensors get as far as the device: there is none, or these are not on it."""
    with pytest.raises((RuntimeError, ValueError), match="NVIDIA|CUDA"):
        CALLS[call][0](mla, tensors())


@pytest.mark.parametrize("call", list(CALLS))
def test_what_is_no_tensor_is_refused(mla, call):
    s = tensors()
    s["len"] = [1, 2, 3]
    with pytest.raises(TypeError):
        CALLS[call][0](mla, s)


def test_pools_of_a_handle(mla):
    pools = mla.PagedArrays([torch.zeros(PAGES, SIZE, RANK), torch.zeros(PAGES, SIZE, ROPE, dtype=torch.bfloat16)])
    assert [(s.token_stride_bytes, s.batch_stride_bytes, s.row_bytes) for s in pools.states] == [
        (4 * RANK, 4 * RANK * SIZE, 4 * RANK), (2 * ROPE, 2 * ROPE * SIZE, 2 * ROPE)]
    assert np.array_equal([s.data for s in pools.states], [t.data_ptr() for t in pools.tensors])
