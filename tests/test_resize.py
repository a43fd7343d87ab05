"""Page tables and slots from the sequences' lengths (atlas_kv_resize) against a plain form that
takes one sequence after the other; everything is whole numbers and equal."""
import ctypes

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build
from tests.serving_refs import resize

gpu = pytest.mark.gpu


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def call(lib, ptrs=(0x1000, 0x2000, 0x3000, 0x4000, 0x5000), P=16, **kw):
    Z = atlas._Resize(batch=2, max_pages_per_seq=4, num_pages=8, max_new=3, slots=0x6000)
    for k, v in kw.items():
        setattr(Z, k, v)
    return lib.atlas_kv_resize(*ptrs, P, ctypes.byref(Z))


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(max_pages_per_seq=0), 1), (dict(num_pages=0), 1), (dict(max_new=-1), 1),
    (dict(slots=None), 1), (dict(P=0), 2), (dict(P=24), 2), (dict(P=256), 2), (dict(slots=0x6002), 1),
    (dict(n_new=0x7001), 1), (dict(status_word=0x7002), 1),
    (dict(batch=1 << 16, max_pages_per_seq=1 << 15), 1), (dict(batch=1 << 16, max_new=1 << 15), 1),
    (dict(num_pages=1 << 27, P=16), 1), (dict(batch=1, max_pages_per_seq=1 << 27), 1),
    # what is written overlaps: slots and the table, n_new and slots, the status word and the ring
    (dict(slots=0x101c), 1), (dict(slots=0x2004), 1), (dict(n_new=0x6014), 1), (dict(status_word=0x401c), 1)])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_refuses_null_misaligned_and_overlapping_arrays(lib):
    good = (0x1000, 0x2000, 0x3000, 0x4000, 0x5000)
    assert lib.atlas_kv_resize(*good, 16, None) == 1
    for i in range(5):
        for value in (None, good[i] + 2):
            assert call(lib, tuple(value if j == i else x for j, x in enumerate(good))) == 1
    for i in range(5):
        for j in range(i):
            # (i at the last word of j: table 8 words, n_pages and lens 2, ring 8, state 2)
            last = good[j] + 4 * ((8, 2, 2, 8, 2)[j] - 1)
            if not (i == 2 and j == 2):
                assert call(lib, tuple(last if k == i else x for k, x in enumerate(good))) == 1


def test_the_plain_form_on_a_case_worked_by_hand():
    table = np.array([[5, -1, -1], [6, 7, -1], [-1, -1, -1]])
    # 4 tokens a page; 0 grows from 1 page to 3, 1 shrinks from 2 to 1, 2 asks for one: 3 free
    out = resize(table, [1, 2, 0], [9, 4, 1], [9, 8, 0, 1, 2, 3, 4, 9, 9, 9], [2, 3], 4, [2, 0, 1], 3)
    assert out[0].tolist() == [[5, 0, 1], [6, -1, -1], [2, -1, -1]]
    assert out[1] == [3, 1, 1] and out[2] == [9, 8, 0, 1, 2, 7, 4, 9, 9, 9] and out[3] == [5, 1]
    assert out[4].tolist() == [[3, 4, -1], [-1] * 3, [8, -1, -1]] and out[5] == 0
    out = resize(table, [1, 2, 0], [9, 4, 1], [9, 8, 0, 1, 2, 3, 4, 9, 9, 9], [2, 2], 4, [2, 0, 1], 3)
    assert out[0].tolist() == [[5, 0, 1], [6, -1, -1], [-1, -1, -1]] and out[5] == 8


# ------------------------------------------------------------------ on the GPU
class Pages:
    """A batch's tables, ring and state on both sides."""

    def __init__(self, B, width, N, P, seed, free=None):
        self.r = np.random.default_rng(seed)
        self.P, self.N = P, N
        self.table = np.full((B, width), -1, np.int32)
        self.held = [0] * B
        ids = self.r.permutation(N).tolist()
        head = int(self.r.integers(N))
        self.ring = [ids[(i - head) % N] for i in range(N)]
        self.state = [head, N if free is None else free]

    def dev(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return [torch.from_numpy(self.table.copy()).cuda(), torch.tensor(self.held, **i32),
                torch.tensor(self.ring, **i32), torch.tensor(self.state, **i32)]

    def step(self, dev, lens, n_new=None, max_new=0):
        """One call on both sides; its status bits."""
        i32 = dict(dtype=torch.int32, device="cuda")
        status = torch.zeros(1, **i32)
        slots = torch.full((len(lens), max_new), 99, **i32) if max_new else None
        got = atlas.kv_resize(dev[0], dev[1], torch.tensor(lens, **i32), dev[2], dev[3], self.P,
                              n_new=None if n_new is None else torch.tensor(n_new, **i32), slots=slots,
                              status=status)
        assert got is slots
        want = resize(self.table, self.held, lens, self.ring, self.state, self.P, n_new, max_new)
        self.table, self.held, self.ring, self.state = want[:4]
        for t, x in zip(dev, want):
            assert np.array_equal(t.cpu().numpy(), np.array(x))
        if max_new:
            assert np.array_equal(slots.cpu().numpy(), want[4])
        assert int(status.item()) == want[5]
        return want[5]


SIZES = [
    # batch, max pages, pages, page tokens: a CTA, a cluster, more than a round of sequences, a
    # grid, a grid with more than a round
    (1, 1, 1, 16), (3, 5, 9, 1), (7, 60, 300, 8), (600, 9, 3000, 4), (40, 7000, 90000, 16), (1100, 300, 150000, 128)]


@gpu
@pytest.mark.parametrize("B,width,N,P", SIZES)
@pytest.mark.parametrize("max_new,some", [(0, False), (1, False), (5, True), (70, True), (3, False)])
def test_random_lengths_step_by_step(B, width, N, P, max_new, some):
    x = Pages(B, width, N, P, B + max_new)
    dev = x.dev()
    r = x.r
    seen = 0
    for k in range(6):
        # some requests end, some come, some go on; sometimes more than there are pages for
        top = max(1, min(width * P, int(N * P / B * (0.5, 1.0, 2.5)[k % 3])))
        lens = [int(v) for v in r.integers(0, top + 1, B)]
        new = [int(r.integers(0, min(n, max_new) + 1)) for n in lens] if some and max_new else None
        seen |= x.step(dev, lens, new, max_new)
        assert sorted([p for b in range(B) for p in x.table[b, : x.held[b]].tolist()] +
                      [x.ring[(x.state[0] + i) % N] for i in range(x.state[1])]) == list(range(N))
    assert x.step(dev, [0] * B) == 0 and x.state[1] == N
    assert seen in (0, 8)


@gpu
@pytest.mark.parametrize("B,width,N,P", SIZES[1:])
def test_the_rings_last_page_and_one_more(B, width, N, P):
    need = [min(width, -(-N // B)) for _ in range(B)]
    while sum(need) > N:
        need[int(np.argmax(need))] -= 1
    x = Pages(B, width, N, P, 5, free=sum(need))
    dev = x.dev()
    assert x.step(dev, [n * P for n in need]) == 0 and x.state[1] == 0
    lens = [n * P for n in x.held]
    k = next((b for b in range(B) if x.held[b] < width), None)
    if k is not None:
        lens[k] += 1
        assert x.step(dev, lens, max_new=2) == 8


@gpu
@pytest.mark.parametrize("B,width,N", [(4, 6, 40), (40, 7000, 90000)])
def test_what_is_out_of_range_is_reported_and_left(B, width, N):
    P = 16
    lens = [17 * (b % 5) for b in range(B)]
    for change, bits in ((("lens", -1), 2), (("lens", width * P + 1), 2), (("lens", -(2 ** 31)), 2),
                         (("lens", 2 ** 31 - 1), 2), (("held", -1), 2), (("held", width + 1), 2), (("new", -1), 2),
                         (("new", 4), 2), (("new", 3), 2), (("state", [-1, 3]), 1), (("state", [N, 3]), 1),
                         (("state", [0, -1]), 1), (("state", [0, N + 1]), 1), (("state", [0, N]), 1)):
        x = Pages(B, width, N, P, 6)
        x.step(x.dev(), lens)
        to = [n + 3 for n in lens]
        to[3] = 1                                    # gives pages back: more than a full ring holds
        new = [1] * B
        name, value = change
        if name == "lens":
            to[2] = value
        elif name == "held":
            x.held[2] = value
        elif name == "state":
            x.state = value
        else:
            new[2], to[2] = value, (2 if value == 3 else to[2])
        assert x.step(x.dev(), to, new, 3) == bits
    # ids that are none, taken and given back, are passed on; slots on them are -1
    x = Pages(B, width, N, P, 6)
    x.step(x.dev(), lens)
    x.table[3, 1] = N + 5
    x.ring[x.state[0]] = -9
    dev = x.dev()
    to = list(lens)
    to[0], to[3] = 5, 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = atlas.kv_resize(*dev[:2], torch.tensor(to, dtype=torch.int32, device="cuda"), *dev[2:], P, max_new=2,
                            status=status)
    assert int(status.item()) == 1 and int(dev[0][0, 0]) == -9 and slots[0].tolist() == [-1, -1]


@gpu
@pytest.mark.parametrize("B,width,N", [(4, 6, 40), (40, 7000, 90000)])
def test_captured_and_replayed(B, width, N):
    """A captured step goes on from the state that the one before it left."""
    x = Pages(B, width, N, 16, 9)
    dev = x.dev()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        atlas.kv_resize(*dev[:2], lens, *dev[2:], 16, slots=slots)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            atlas.kv_resize(*dev[:2], lens, *dev[2:], 16, slots=slots)
    for k in range(4):
        now = [(7 * b + 23 * k) % (width * 8) for b in range(B)]
        torch.cuda.synchronize()
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = resize(x.table, x.held, now, x.ring, x.state, 16, None, 2)
        x.table, x.held, x.ring, x.state = want[:4]
        for t, y in zip(dev + [slots], want):
            assert np.array_equal(t.cpu().numpy(), np.array(y))


def apart(t):
    return torch.stack([t, t], -1)[..., 0]


@gpu
@pytest.mark.parametrize("name,change", [
    *((n, f) for n in ("page_table", "n_pages", "seq_lens", "free_pages", "free_state", "n_new", "slots")
      for f in (apart, torch.Tensor.cpu, torch.Tensor.long)),
    ("page_table", lambda t: t[0]), ("page_table", lambda t: t[:2]), ("n_pages", lambda t: t[:2]),
    ("seq_lens", lambda t: t[:2]), ("free_state", lambda t: t[:1]), ("n_new", lambda t: t[:2]),
    ("slots", lambda t: t[:2]), ("slots", lambda t: t[0]), ("slots", lambda t: None), ("max_new", lambda t: 3)])
def test_one_wrong_tensor(name, change):
    i32 = dict(dtype=torch.int32, device="cuda")
    x = dict(page_table=torch.zeros((3, 4), **i32), n_pages=torch.zeros(3, **i32), seq_lens=torch.ones(3, **i32),
             free_pages=torch.arange(9, **i32), free_state=torch.tensor([0, 9], **i32), page_tokens=16,
             n_new=torch.ones(3, **i32), slots=torch.zeros((3, 2), **i32), max_new=None)
    x[name] = change(x[name])
    with pytest.raises(ValueError):
        atlas.kv_resize(**x)
    torch.cuda.synchronize()
    assert int(x["free_state"].reshape(-1)[0]) == 0


def test_tensors_on_the_host():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="page_table must be a CUDA tensor"):
        atlas.kv_resize(torch.zeros((3, 4), **i32), torch.zeros(3, **i32), torch.ones(3, **i32),
                        torch.arange(9, **i32), torch.tensor([0, 9], **i32), 16)


@gpu
def test_the_most_slots_there_may_be():
    """2^31 - 1 of them: places in the list, a step past its last among them, need more than 31 bits."""
    i32 = dict(dtype=torch.int32, device="cuda")
    n = 2 ** 31 - 1
    table, held = torch.full((1, 4), -1, **i32), torch.zeros(1, **i32)
    ring, state = torch.arange(5, 14, **i32).flip(0).contiguous() - 5, torch.tensor([7, 9], **i32)
    slots, status = torch.full((1, n), 7, **i32), torch.zeros(1, **i32)
    for new, first in (([3], 47), (None, 0)):
        new = None if new is None else torch.tensor(new, **i32)
        atlas.kv_resize(table, held, torch.tensor([50], **i32), ring, state, 16, n_new=new, slots=slots, status=status)
        torch.cuda.synchronize()
        assert table.tolist() == [[1, 0, 8, 7]] and held.tolist() == [4] and state.tolist() == [2, 5]
        pages = torch.tensor([1, 0, 8, 7], **i32)
        t = torch.arange(first, 50, **i32)
        assert torch.equal(slots[0, : 50 - first], pages[(t // 16).long()] * 16 + t % 16)
        assert bool((slots[0, 50 - first:] == -1).all()) and int(status.item()) == 0


@gpu
def test_the_most_moves_there_may_be():
    """Two sequences that take 2^31 - 2 pages of one token between them, and give them back."""
    i32 = dict(dtype=torch.int32, device="cuda")
    width = 2 ** 30 - 1
    table, held = torch.full((2, width), -1, **i32), torch.zeros(2, **i32)
    ring, state = torch.arange(2 * width, **i32), torch.tensor([0, 2 * width], **i32)
    status = torch.zeros(1, **i32)
    atlas.kv_resize(table, held, torch.tensor([width, width], **i32), ring, state, 1, status=status)
    torch.cuda.synchronize()
    assert held.tolist() == [width, width] and state.tolist() == [0, 0] and int(status.item()) == 0
    assert torch.equal(table.reshape(-1), ring)
    ring.fill_(-1)
    atlas.kv_resize(table, held, torch.tensor([0, 0], **i32), ring, state, 1, status=status)
    torch.cuda.synchronize()
    assert held.tolist() == [0, 0] and state.tolist() == [0, 2 * width] and int(status.item()) == 0
    assert bool((table == -1).all()) and torch.equal(ring, torch.arange(2 * width, **i32))
