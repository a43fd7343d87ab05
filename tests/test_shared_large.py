"""Attention behind shared prefixes for batches of very many rows or wide tables: some of the
sequences against fp64 on the GPU.  Tolerances are those of tests/test_shared.py."""
import math

import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.gpu_helpers import BF16_ABS, F32_REL

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SPLIT, TC, WHOLE = atlas.DEBUG_SHARED_SPLIT, atlas.DEBUG_SHARED_TC, atlas.DEBUG_SHARED_WHOLE | atlas.DEBUG_SHARED_TC


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """B sequences of own lengths lens, groups from starts on behind prefixes of pre keys; tables as
    wide as asked, whose entries behind the last page are out of range."""

    def __init__(self, dtype, Hq, Hkv, D, P, q_len, starts, pre, lens, own_width=0, pre_width=0, ragged=None):
        g = torch.Generator(device="cuda").manual_seed(len(lens) + q_len)
        lens, pre = torch.tensor(lens), torch.tensor(pre)
        pages, shared = -(-lens // P), -(-pre // P)
        n = int(pages.sum() + shared.sum())

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda", dtype=DT[dtype])

        def table(count, first, width):
            width = max(width, int(count.max()), 1)
            at = first + torch.cumsum(count, 0)[:, None] - count[:, None] + torch.arange(width)
            at = torch.where(torch.arange(width) < count[:, None], ids[at.clamp(max=n - 1)], 10 ** 6)
            return at.int().cuda()

        ids = torch.randperm(n, generator=g, device="cuda").cpu()
        self.starts, self.pre, self.lens, self.ragged = list(starts), pre.tolist(), lens.tolist(), ragged
        self.q, self.k, self.v = normal(len(lens), Hq, q_len, D), normal(n, Hkv, P, D), normal(n, Hkv, P, D)
        self.prefix_table, self.table = table(shared, 0, pre_width), table(pages, int(shared.sum()), own_width)
        self.sizes = Hq, Hkv, D, P
        self.scale = D ** -0.5

    def __call__(self, starts=None, pre=None, lens=None, **kw):
        return atlas.shared(self.q, self.k, self.v, self.prefix_table, ints(pre or self.pre),
                            ints(starts or self.starts), self.table, ints(lens or self.lens), *self.sizes, self.scale,
                            q_lens=None if self.ragged is None else ints(self.ragged), **kw)

    def workspace(self, **kw):
        return atlas.shared_workspace_size(self.q.shape, *self.sizes, self.table.shape[1], len(self.pre),
                                           self.prefix_table.shape[1], self.k.shape[0], dtype=self.q.dtype, **kw)

    def keys(self, pages, row, length):
        Hkv, P, D = pages.shape[1:]
        return pages[row[: -(-length // P)].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :length].double()

    def exact(self, b):
        """out, lse of sequence b's rows, in fp64."""
        Hq, Hkv, D, _ = self.sizes
        rows, L = self.q.shape[2] if self.ragged is None else self.ragged[b], self.lens[b]
        parts = [(self.table[b], L)]
        for n, length in enumerate(self.pre):
            if self.starts[n] <= b < self.starts[n + 1]:
                parts.insert(0, (self.prefix_table[n], length))
        k, v = (torch.cat([self.keys(x, *p) for p in parts], 1).repeat_interleave(Hq // Hkv, 0) for x in (self.k, self.v))
        T = k.shape[1]
        seen = torch.arange(T, device="cuda") <= torch.arange(T - rows, T, device="cuda")[:, None]
        s = (self.q[b, :, :rows].double() @ k.transpose(1, 2) * self.scale).masked_fill(~seen, -math.inf)
        return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)

    def check(self, some, **kw):
        """Rows of the sequences `some`; padding stays as it is, and nothing is written behind the workspace."""
        f32 = self.q.dtype == torch.float32
        out = torch.full(self.q.shape, 99.0, device="cuda")
        lse, status = torch.full(self.q.shape[:3], 99.0, device="cuda"), ints([0])
        need = self.workspace(**{k: v for k, v in kw.items() if k in ("split_tokens", "debug_flags", "sm_count")})
        space = torch.full((need + 1024,), 77, dtype=torch.uint8, device="cuda")
        self(out=out, lse=lse, status=status, workspace=space[:need], **kw)
        assert int(status.item()) == 0 and bool((space[need:] == 77).all())
        for b in some:
            rows = self.q.shape[2] if self.ragged is None else self.ragged[b]
            want, want_lse = self.exact(b)
            tol = F32_REL * float(want.abs().max()) if f32 and rows else BF16_ABS
            assert bool(((out[b, :, :rows].double() - want).abs() <= tol).all()), b
            assert bool(((lse[b, :, :rows].double() - want_lse).abs() <= (2e-5 if f32 else 1e-4)).all()), b
            assert bool((out[b, :, rows:] == 99).all()) and bool((lse[b, :, rows:] == 99).all()), b
        assert bool(torch.isfinite(out).all())
        return out


@pytest.mark.parametrize("B,q_len,prefix", [(2049, 128, 100), (256, 1024, 300)])
def test_more_tiles_than_a_grid_of_splits_has(B, q_len, prefix):
    x = Batch("bf16", 32, 8, 64, 16, q_len, [0, B // 2, B], [prefix, 77], [q_len + b % 40 for b in range(B)], own_width=80)
    x.check([0, 1, B // 2 - 1, B // 2, B - 2, B - 1])


@pytest.mark.parametrize("B,q_len,starts,sms", [(256, 512, [0, 100, 256], 0), (40, 256, [0, 39, 40], 3)])
def test_tables_far_wider_than_the_lengths(B, q_len, starts, sms):
    x = Batch("bf16", 32, 8, 64, 16, q_len, starts, [300, 5000], [q_len + b % 40 for b in range(B)], own_width=8192,
              pre_width=8192)
    x.check([0, starts[1] - 1, starts[1], B - 1], sm_count=sms)


def test_whole_tiles_fill_whole_waves():
    """10240 tiles of 256 rows among three CTAs to an SM, not a few more: 22.5 tiles a share have room
    among a CTA's 38 pieces, so none counts for more blocks than it has."""
    B, n, prefix, sms = 256, 320, 300, 152
    x = Batch("bf16", 32, 8, 64, 16, n, [0, B], [prefix], [n] * B)
    space = torch.zeros(x.workspace(debug_flags=WHOLE, sm_count=sms), dtype=torch.uint8, device="cuda")
    x(workspace=space, debug_flags=WHOLE, sm_count=sms)
    # a CTA has 40 places for its pieces: unit, kv head, first row, rows, first block, blocks, state, keys,
    # own keys, group
    words = space[: space.numel() // 4 * 4].view(torch.int32)
    at = ((words[3:-6] == 4 * n) & (words[7:-2] == prefix) & (words[9:] == 0)).nonzero().flatten()
    ctas = torch.unique((at - at[0]) // 400).numel()
    assert 2 * sms < ctas <= 3 * sms


def test_shares_that_grow_save_a_wave_of_ctas():
    """Prompts of 275 rows, 4 tiles of 256 and a short one for each of 8 kv heads, of 11 blocks with what a
    tile takes besides: a head is 32 * 11 long.  167 of them: shares of 1548, in which tiles count as 12 blocks
    for their pieces, grow to 1688 and stay 304, two for each SM.  210: shares of 1946 and tiles of 15 blocks
    would have to grow by more than an eighth, and do not: 806400 / 1946 = 415 CTAs."""
    for B, ctas in ((167, 304), (210, 415)):
        x = Batch("bf16", 32, 8, 64, 16, 275, [0, B], [300], [275] * B)
        space = torch.zeros(x.workspace(debug_flags=WHOLE, sm_count=152), dtype=torch.uint8, device="cuda")
        x(workspace=space, debug_flags=WHOLE, sm_count=152)
        words = space[: space.numel() // 4 * 4].view(torch.int32)
        at = ((words[3:-6] == 1100) & (words[7:-2] == 300) & (words[9:] == 0)).nonzero().flatten()
        assert torch.unique((at - at[0]) // 400).numel() == ctas


PARTS = [
    # dtype, Hq, Hkv, q_len, path, ragged: few rows on each path, and tiles of many
    ("bf16", 16, 2, 1, SPLIT, False), ("bf16", 16, 2, 1, TC, False), ("bf16", 8, 2, 2, 0, True),
    ("bf16", 4, 2, 12, TC, True), ("f32", 16, 2, 1, SPLIT, False), ("f32", 16, 2, 1, TC, False),
    ("f32", 4, 1, 7, 0, True)]
STARTS, PRE = [0, 5, 30, 31, 31, 60], [700, 40, 0, 9, 129]   # (the last four sequences in no group)


def in_parts(dtype, Hq, Hkv, q_len, ragged):
    """64 sequences whose states of 64 keys each, of tables of 65536 keys, need more than one part."""
    return Batch(dtype, Hq, Hkv, 64, 128, q_len, STARTS, PRE, [q_len + 5 * b % 300 for b in range(64)], own_width=512,
                 pre_width=512, ragged=[b % (q_len + 1) for b in range(64)] if ragged else None)


@pytest.mark.parametrize("dtype,Hq,Hkv,q_len,path,ragged", PARTS)
def test_in_parts(dtype, Hq, Hkv, q_len, path, ragged):
    """Groups whose sequences are in several parts, none, or in no group at all."""
    x = in_parts(dtype, Hq, Hkv, q_len, ragged)
    rows = 64 * Hq * q_len
    whole = rows * 2 * 1024 * (64 * 4 + 8)   # states of the batch in one part
    assert x.workspace(split_tokens=64, debug_flags=path) <= 512 << 20 < whole
    x.check(range(64), split_tokens=64, debug_flags=path)


@pytest.mark.parametrize("dtype,Hq,Hkv,q_len,path,ragged", PARTS)
def test_in_parts_what_is_out_of_range_is_reported(dtype, Hq, Hkv, q_len, path, ragged):
    x = in_parts(dtype, Hq, Hkv, q_len, False)
    kw = dict(split_tokens=64, debug_flags=path, out_dtype=torch.float32)
    good = x(**kw)
    lens, pre = list(x.lens), list(x.pre)
    lens[40] = q_len - 1
    pre[0] = 512 * 128 + 1
    for change, nan in ((dict(lens=lens), {40}), (dict(pre=pre), set(range(5))),
                        (dict(starts=[0, 5, 30, 31, 31, 65]), set(range(64))),
                        (dict(starts=[0, 5, 4, 31, 31, 60]), set(range(64))),
                        (dict(starts=[-1, 5, 30, 31, 31, 60]), set(range(64)))):
        status = ints([0])
        out = x(status=status, **change, **kw)
        assert int(status.item()) == atlas.DEV_BAD_SEQLEN
        for b in range(64):
            if b in nan:
                assert bool(torch.isnan(out[b]).all())
            else:   # (twice the bound: tiles may be cut elsewhere when a sequence drops out)
                tol = 2 * (BF16_ABS if dtype == "bf16" else F32_REL * 8)
                assert float(good.abs().max()) <= 8 and float((out[b] - good[b]).abs().max()) <= tol


def test_in_parts_rows_of_padding_alone():
    """Parts in which no sequence has a query, before and behind parts that have."""
    for ragged in ([0] * 40 + [1] * 24, [1] * 20 + [0] * 44, [0] * 64):
        for path in (SPLIT, TC):
            x = in_parts("bf16", 16, 2, 1, False)
            x.ragged = ragged
            x.check(range(64), split_tokens=64, debug_flags=path)


@pytest.mark.parametrize("dtype,path,B,D", [("bf16", WHOLE, 5200, 128), ("f32", 0, 8200, 64), ("bf16", TC, 8200, 64)])
def test_many_sequences_in_parts(dtype, path, B, D):
    """More than 512 MB of cut tiles' places, and more than 65535 tiles of own keys."""
    x = Batch(dtype, 8, 8, D, 32, 17, [0, 3000, 3001, B - 1], [100, 33, 200], [17 + b % 40 for b in range(B)])
    some = sorted({*range(0, B, 97), 2999, 3000, 3001, B - 2, B - 1, *range(B // 2 - 3, B // 2 + 3)})
    x.check(some, debug_flags=path)


@pytest.mark.parametrize("dtype,path", [("bf16", SPLIT), ("bf16", TC), ("f32", 0)])
def test_in_parts_captured_and_replayed(dtype, path):
    x = in_parts(dtype, 16, 2, 1, False)
    space = torch.empty(x.workspace(split_tokens=64, debug_flags=path), dtype=torch.uint8, device="cuda")
    args = [ints(x.pre), ints(x.starts), ints(x.lens)]
    out = torch.empty(x.q.shape, device="cuda")

    def call():
        return atlas.shared(x.q, x.k, x.v, x.prefix_table, args[0], args[1], x.table, args[2], *x.sizes, x.scale,
                            out=out, workspace=space, split_tokens=64, debug_flags=path)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for pre, starts, lens in ((x.pre, x.starts, x.lens), ([3, 40, 0, 9, 100], [1, 1, 40, 50, 50, 64], x.lens[::-1])):
        lens = [min(a, b) for a, b in zip(lens, x.lens)]
        torch.cuda.synchronize()
        for t, v in zip(args, (pre, starts, lens)):
            t.copy_(torch.tensor(v, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(out).all())
        assert torch.equal(out, x(starts, pre, lens, split_tokens=64, debug_flags=path, out_dtype=torch.float32))


@pytest.mark.parametrize("dtype,path", [("bf16", SPLIT), ("bf16", TC), ("bf16", WHOLE), ("f32", SPLIT), ("f32", TC)])
def test_more_groups_than_the_plan_has_threads_in_parts_of_fewer_sequences(dtype, path):
    """700 sequences with a prefix each, in two parts (of states; whole tiles in one)."""
    x = Batch(dtype, 8, 2, 64, 128, 1, list(range(701)), [n % 300 for n in range(700)], [1 + b % 90 for b in range(700)],
              own_width=128, pre_width=128)
    x.check([*range(0, 700, 23), 349, 350, 351, 699], split_tokens=64, debug_flags=path)


@pytest.mark.parametrize("dtype,path", [("bf16", 0), ("bf16", SPLIT), ("bf16", TC), ("bf16", WHOLE), ("f32", SPLIT),
                                        ("f32", TC)])
def test_more_sequences_than_a_grid_has_in_z(dtype, path):
    B = 70000
    x = Batch(dtype, 2, 1, 64, 8, 1, [0, 30000, 35001, B - 1], [60, 300, 9], [1 + b % 20 for b in range(B)])
    x.check([*range(0, B, 997), 29999, 30000, 34999, 35000, 35001, B - 2, B - 1], debug_flags=path)


@pytest.mark.parametrize("dtype,path", [("bf16", SPLIT), ("bf16", TC), ("f32", 0)])
def test_in_parts_events_and_fewer_sms(dtype, path):
    x = in_parts(dtype, 16, 2, 1, False)
    timer = atlas.EventTimer()
    for sms in (1, 7, 300):
        x.check(range(0, 64, 5), split_tokens=64, debug_flags=path, sm_count=sms, events=timer.handles)
        torch.cuda.synchronize()
        assert timer.main_ms() > 0 and timer.merge_ms() > 0
