"""The workspace of the paged attention on the host: its size, and where the pieces of split rows lie in it."""
import os
import shutil
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mla_latent_kv_12_gb300", "csrc")


@pytest.fixture(scope="module")
def mla():
    from mla_latent_kv_12_gb300 import mla
    return mla


def test_every_piece_has_a_place_of_its_own(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "paged_pieces_test"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "paged_pieces_test.cpp"), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_size_does_not_grow_with_the_rows(mla):
    """Prompt chunks of thousands of tokens: a few bytes each beside a fixed part."""
    size = mla.decode_paged_workspace_size
    fixed = size(1, 4096, 128, 512, 64, 1 << 20)
    for batch, s_q in ((8, 2048), (1, 1 << 20), (1 << 20, 1), (300, 7)):
        for heads in (64, 128):
            assert size(batch, s_q, heads, 512, 64, 1 << 15) <= fixed + 16 * batch * s_q
    assert fixed < 32 << 20


def test_a_window_decodes_workspace_is_enough(mla):
    for dtype, heads, rank, rope in ((torch.bfloat16, 128, 512, 64), (torch.bfloat16, 64, 512, 64), (torch.float32, 3, 40, 8)):
        for batch, s_q in ((1, 1), (1, 7), (3, 25), (19, 4), (77, 1), (2, 500), (5, 301)):
            sizes = [f(batch, s_q, heads, rank, rope, 5000, dtype=dtype)
                     for f in (mla.decode_paged_workspace_size, mla.decode_workspace_size)]
            assert 0 <= sizes[0] <= sizes[1], (dtype, batch, s_q)
    # what is refused has no size
    assert mla.decode_paged_workspace_size(1 << 20, 2, 128, 512, 64, 4096) == 0
    assert mla.decode_paged_workspace_size(1, 1, 16, 512, 64, 4096) == 0
    assert mla.decode_paged_workspace_size(0, 1, 128, 512, 64, 4096) == 0
