"""Pointers that a kernel could not read are refused on the host, one at a time; calls
without a device end with ATLAS_ERR_CUDA (4) once everything is accepted.  Made-up addresses:
only on machines without a GPU, where a call that slipped through cannot reach one."""
import ctypes
import os

import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build

pytestmark = pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/nvidiactl"),
                                reason="calls with made-up addresses: only where no GPU can get them")
FAR = 1 << 32


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def build(kind, names, **fixed):
    x = kind()
    for k, name in enumerate(names):
        setattr(x, name, (k + 16) * FAR)
    for name, value in fixed.items():
        setattr(x, name, value)
    return x


def attention(lib, name, moved, by):
    L = build(atlas._Launch, ("out", "lse", "workspace", "status_word", "sinks", "q_lens"), batch=2,
              max_pages_per_seq=8, num_pages=16, q_len=1, q_dtype=1, kv_dtype=1, out_dtype=1,
              workspace_bytes=1 << 30)
    args = {n: (k + 1) * FAR for k, n in enumerate(("q", "k_pages", "v_pages", "page_table", "seq_lens"))}
    return run(getattr(lib, f"atlas_attn_{name}"), args, L, moved, by, 8, 2, 128, 16, 0.1)


def weights(lib, moved, by):
    W = build(atlas._Weights, ("weights", "workspace", "status_word", "q_lens"), batch=2, max_pages_per_seq=8,
              num_pages=16, q_len=4, dtype=1, row_tokens=128, accumulate=1, workspace_bytes=1 << 30)
    args = {n: (k + 1) * FAR for k, n in enumerate(("q", "k_pages", "page_table", "seq_lens", "lse"))}
    return run(lib.atlas_kv_weights, args, W, moved, by, 8, 2, 128, 16, 0.1)


def rope(lib, moved, by):
    R = build(atlas._Rope, ("q", "q_out", "positions", "status_word"), batch=2, max_pages_per_seq=4, num_pages=8,
              max_new=3, kv_dtype=1, n_q_heads=8, n_axes=1, rot_dim=128, theta=1e4)
    args = {n: (k + 1) * FAR for k, n in enumerate(("k_new", "v_new", "k_pages", "v_pages", "page_table",
                                                    "seq_lens", "n_new"))}
    return run(lib.atlas_kv_append_rope, args, R, moved, by, 2, 128, 16)


def run(fn, args, x, moved, by, *rest):
    if moved in args:
        args[moved] += by
    elif moved:
        setattr(x, moved, getattr(x, moved) + by)
    return fn(*args.values(), *rest, ctypes.byref(x))


@pytest.mark.parametrize("name", ["decode", "suffix", "cross"])
def test_attention(lib, name):
    assert attention(lib, name, None, 0) == 4
    for p in ("page_table", "seq_lens", "lse", "status_word", "sinks", "q_lens"):
        for by in (1, 2):
            assert attention(lib, name, p, by) == 1, p
        assert attention(lib, name, p, 4) == 4, p
    for p in ("q", "k_pages", "v_pages", "out", "workspace"):
        assert attention(lib, name, p, 8) == 1, p


def test_weights(lib):
    assert weights(lib, None, 0) == 4
    for p in ("page_table", "seq_lens", "lse", "weights", "status_word", "q_lens"):
        assert weights(lib, p, 2) == 1 and weights(lib, p, 4) == 4, p
    for p in ("q", "k_pages", "workspace"):
        assert weights(lib, p, 8) == 1, p


def test_rotary_append(lib):
    assert rope(lib, None, 0) == 4
    for p in ("page_table", "seq_lens", "n_new", "positions", "status_word"):
        assert rope(lib, p, 2) == 1 and rope(lib, p, 4) == 4, p
    for p in ("k_new", "v_new", "k_pages", "v_pages", "q", "q_out"):
        assert rope(lib, p, 8) == 1, p
