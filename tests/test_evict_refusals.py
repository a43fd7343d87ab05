"""What atlas_kv_select and atlas_kv_compact refuse on the host, one field away from a call
they accept.

Every pointer of the accepted call has an address of its own, far from the others', so
that a refusal can only come from the field that was changed.  The addresses are no
memory: where a GPU is visible, a call that the library failed to refuse would reach it
with them, so these tests run on machines without one, where an accepted call ends with
ATLAS_ERR_CUDA (4), the launch having no device."""
import ctypes
import os

import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build

pytestmark = pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/nvidiactl"),
                                reason="calls with made-up addresses: only where no GPU can get them")

INVALID, UNSUPPORTED, NO_DEVICE = 1, 2, 4
FAR = 1 << 32  # between any two addresses: more than any range here


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def at(k, offset=0):
    return (k + 1) * FAR + offset


# ------------------------------------------------------------------ selection
B, HKV, T, BUDGET = 2, 2, 100, 10
ROWS = 4 * B * HKV  # bytes of one float or int32 of every row
WEIGHTS, LENS, KEPT, NEW, KEPT_W = (at(k) for k in range(5))


def select(lib, w=WEIGHTS, lens=LENS, Hkv=HKV, **kw):
    S = atlas._Select()
    for k, v in {**dict(batch=B, row_tokens=T, budget=BUDGET, keep_first=1, keep_recent=2, kept=KEPT,
                        new_lens=NEW, kept_weights=KEPT_W), **kw}.items():
        setattr(S, k, v)
    return lib.atlas_kv_select(w, lens, Hkv, ctypes.byref(S))


def test_select_accepts_the_call_the_others_differ_from(lib):
    assert select(lib) == NO_DEVICE
    assert select(lib, kept_row_tokens=BUDGET) == NO_DEVICE
    assert select(lib, kept_row_tokens=T + 1) == NO_DEVICE
    assert select(lib, kept_weights=None) == NO_DEVICE
    assert select(lib, keep_first=8) == NO_DEVICE and select(lib, keep_recent=9) == NO_DEVICE


@pytest.mark.parametrize("kw", [
    dict(w=None), dict(lens=None), dict(kept=None), dict(new_lens=None),
    dict(w=WEIGHTS + 1), dict(kept=KEPT + 2), dict(kept_weights=KEPT_W + 3),
    dict(lens=LENS + 2), dict(new_lens=NEW + 1), dict(status_word=at(6, 2)),
    dict(batch=0), dict(batch=65536), dict(Hkv=0), dict(Hkv=65536), dict(row_tokens=0),
    dict(row_tokens=2 ** 31 - 1), dict(budget=0), dict(budget=2 ** 31 - 1), dict(keep_first=-1),
    dict(keep_recent=-1), dict(keep_first=9), dict(keep_first=2 ** 31 - 1, keep_recent=2 ** 31 - 1),
    dict(kept_row_tokens=-1), dict(kept_row_tokens=BUDGET - 1), dict(kept_row_tokens=2 ** 31 - 1)])
def test_select_refuses(lib, kw):
    assert select(lib, **kw) == INVALID


# Outputs over an input or another output: the same address, or the last or the first four
# bytes of a range alone; and next to it, which is fine.
@pytest.mark.parametrize("name,start,size,own", [
    ("new_lens", LENS, 4 * B, 4 * B),                  # lengths updated in place: other CTAs read them
    ("new_lens", WEIGHTS, ROWS * T, 4 * B), ("new_lens", KEPT, ROWS * BUDGET, 4 * B),
    ("new_lens", KEPT_W, ROWS * BUDGET, 4 * B),
    ("kept", LENS, 4 * B, ROWS * BUDGET), ("kept", WEIGHTS, ROWS * T, ROWS * BUDGET),
    ("kept", KEPT_W, ROWS * BUDGET, ROWS * BUDGET),
    ("kept_weights", LENS, 4 * B, ROWS * BUDGET), ("kept_weights", WEIGHTS, ROWS * T, ROWS * BUDGET)])
def test_select_refuses_outputs_over_anything_else(lib, name, start, size, own):
    for where in (start, start + size - 4, start - own + 4):
        assert select(lib, **{name: where}) == INVALID, hex(where)
    for where in (start + size, start - own):
        assert select(lib, **{name: where}) == NO_DEVICE, hex(where)


def test_select_counts_the_rows_of_kept_weights_as_wide_as_they_are(lib):
    wide = dict(kept_row_tokens=BUDGET + 3)
    for name, end in (("new_lens", KEPT_W + ROWS * (BUDGET + 3)), ("kept", KEPT_W + ROWS * (BUDGET + 3))):
        assert select(lib, **{name: end - 4}, **wide) == INVALID
        assert select(lib, **{name: end}, **wide) == NO_DEVICE


def test_the_row_length_took_no_new_place_in_the_struct():
    """It lies where the struct was padded: callers built before it was there pass 0."""
    assert atlas._Select.kept_row_tokens.offset == 20 and atlas._Select.kept.offset == 24
    assert ctypes.sizeof(atlas._Select) == 64


# ------------------------------------------------------------------ compaction
K, V, TABLE, INDEX, COUNT, FRESH = (at(k) for k in range(8, 14))
POOL = 8 * 2 * 16 * 128 * 2  # bytes: pages, kv heads, tokens, head_dim, bf16


def compact(lib, k=K, v=V, table=TABLE, kept=INDEX, lens=COUNT, Hkv=2, D=128, P=16, **kw):
    C = atlas._Compact()
    for key, value in {**dict(batch=2, max_pages_per_seq=4, num_pages=8, max_kept=10, kv_dtype=1),
                       **kw}.items():
        setattr(C, key, value)
    return lib.atlas_kv_compact(k, v, table, kept, lens, Hkv, D, P, ctypes.byref(C))


FRESH_PAGES = dict(new_page_table=FRESH, new_max_pages=1)


@pytest.mark.parametrize("kw", [{}, FRESH_PAGES])
def test_compact_accepts_the_call_the_others_differ_from(lib, kw):
    assert compact(lib, **kw) == NO_DEVICE
    assert compact(lib, Hkv=4095, **kw) == NO_DEVICE
    assert compact(lib, D=64, P=1, kv_dtype=0, **kw) == NO_DEVICE


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID),
    (dict(kept=None), INVALID), (dict(lens=None), INVALID), (dict(k=K + 8), INVALID),
    (dict(v=V + 4), INVALID), (dict(table=TABLE + 2), INVALID), (dict(kept=INDEX + 1), INVALID),
    (dict(lens=COUNT + 2), INVALID), (dict(status_word=at(6, 1)), INVALID), (dict(batch=0), INVALID), (dict(batch=65536), INVALID),
    (dict(max_pages_per_seq=0), INVALID), (dict(max_pages_per_seq=2 ** 30), INVALID),
    (dict(num_pages=0), INVALID), (dict(max_kept=0), INVALID), (dict(max_kept=2 ** 31 - 1), INVALID),
    (dict(Hkv=0), INVALID), (dict(Hkv=4096), INVALID), (dict(D=80), UNSUPPORTED),
    (dict(P=12), UNSUPPORTED), (dict(P=256), UNSUPPORTED), (dict(kv_dtype=3), UNSUPPORTED)])
@pytest.mark.parametrize("where", [{}, FRESH_PAGES])
def test_compact_refuses(lib, kw, status, where):
    assert compact(lib, **{**where, **kw}) == status


def test_compact_refuses_fresh_pages_without_a_row_length(lib):
    assert compact(lib, new_page_table=FRESH) == INVALID
    assert compact(lib, new_page_table=FRESH + 2, new_max_pages=1) == INVALID


def test_compact_in_place_refuses_overlapping_pools(lib):
    for v in (K, K + POOL - 16, K - POOL + 16):
        assert compact(lib, v=v) == INVALID
    for v in (K + POOL, K - POOL):
        assert compact(lib, v=v) == NO_DEVICE
