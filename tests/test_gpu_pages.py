"""kv4_reserve, kv4_fork, kv4_truncate, kv4_compact against the rules one step
at a time, and what they do to the pages' contents."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as aorc
from quantized_moe_decode_route_amd import ops

from _attn import DEV, ints, rows, starts

pytestmark = pytest.mark.gpu


class Both:
    """A cache on the GPU and its page tables on the host, kept in step."""

    def __init__(self, n_pages, n_seqs, max_pages, page=32, layers=2, kv_heads=1, dim=64):
        self.cache = ops.KvCache.allocate(layers, n_pages, page, kv_heads, dim, n_seqs, max_pages, DEV)
        self.cache.data.random_(0, 256)
        self.host = aorc.Pages(n_pages, page, n_seqs, max_pages)

    def same(self):
        c, h = self.cache, self.host
        assert c.len.tolist() == h.len
        assert c.ref.tolist() == h.ref
        table = c.table.tolist()
        for s, pages in enumerate(h.table):
            assert table[s][:len(pages)] == pages

    def _data(self, before):
        want = before.clone()
        for a, b in self.host.copies:
            want[:, b] = before[:, a]
        assert torch.equal(self.cache.data, want)

    def reserve(self, new):
        before = self.cache.data.clone()
        assert ops.kv4_reserve(self.cache, ints(new)).tolist() == self.host.reserve(new)
        self.same()
        self._data(before)

    def fork(self, src, dst, n_tokens=None):
        got = ops.kv4_fork(self.cache, ints(src), ints(dst), None if n_tokens is None else ints(n_tokens))
        assert got.tolist() == self.host.fork(src, dst, n_tokens)
        self.same()

    def truncate(self, new_len):
        ops.kv4_truncate(self.cache, ints(new_len))
        self.host.truncate(new_len)
        self.same()

    def compact(self):
        before = self.cache.data.clone()
        remap, live = ops.kv4_compact(self.cache)
        want, n = self.host.compact()
        assert remap.tolist() == want and live.tolist() == [n]
        self.same()
        self._data(before)


def test_grow_from_empty():
    b = Both(40, 6, 8)
    b.reserve([1, 0, 31, 32, 33, 100])
    b.reserve([31, 5, 1, 1, 0, 28])
    b.reserve([0, -4, 0, 0, 0, 1])
    b.reserve([0] * 6)


def test_refusals_change_nothing():
    b = Both(5, 5, 4)
    b.reserve([33, 200, 10, 70, 1])       # 200 exceeds the table, 70 the pool, and so the later 1
    b.reserve([1, 1, 1, 1, 0])            # the pool still serves what needs little
    b.reserve([0, 128, 0, 0, 0])
    b.reserve([1, 0, 0, 0, 0])
    b.reserve([2 ** 31 - 1, 0, 0, 2 ** 31 - 1, 0])


def test_copy_on_write():
    b = Both(60, 10, 5)
    b.reserve([40, 32, 5] + [0] * 7)
    b.fork([0, 0, 0, 1, 2, 2], [3, 4, 5, 6, 7, 8])
    b.reserve([1, 1, 0, 1, 0, 1, 1, 0, 1, 3])        # some of the sharers grow: each of them copies
    b.reserve([1] * 10)                              # the last holder of a page keeps it
    b.reserve([1] * 10)


def test_all_sharers_grow_at_once():
    b = Both(30, 5, 4)
    b.reserve([7, 0, 0, 0, 0])
    b.fork([0, 0, 0, 0], [1, 2, 3, 4])
    b.reserve([1] * 5)
    assert sorted(b.cache.ref.tolist(), reverse=True)[:6] == [1, 1, 1, 1, 1, 0]


def test_refused_sharer_blocks_later_ones():
    """Sequence 0 gets its copy, sequence 1 no page: the last sharer must not
    write into the page that sequence 1 still holds."""
    b = Both(2, 3, 4)
    b.reserve([7, 0, 0])
    b.fork([0, 0], [1, 2])
    b.reserve([1, 1, 1])


def test_fork_refusals():
    b = Both(30, 8, 4)
    b.reserve([50, 20, 0, 0, 0, 0, 0, 3])
    b.fork([0, 1, 9, -1, 0, 2, 0], [2, 2, 3, 4, 7, 5, 8])   # a slot twice, bad indices, a full slot
    b.fork([0, 0, 1, 1], [3, 4, 5, 6], [33, 51, 0, -1])
    b.fork([], [])
    b.fork([6, 0], [4, 6])                                  # from a slot that fills in the same call: empty
    b.reserve([1] * 8)


def test_truncate_and_free():
    b = Both(40, 6, 8)
    b.reserve([100, 64, 33, 5, 0, 200])
    b.fork([0, 1], [4, 4])
    b.truncate([64, 64, 32, 0, 50, -1])
    b.truncate([63, 65, 0, 7, 0, 0])
    b.reserve([10] * 6)


@pytest.mark.parametrize("n_pages", [3, 17, 64, 2049, 17000, 40000])
def test_compact(n_pages):
    rng = np.random.default_rng(n_pages)
    b = Both(n_pages, 40, 64, layers=1 if n_pages > 5000 else 2)
    for _ in range(3):
        b.reserve([int(x) for x in rng.integers(0, 32 * 20, 40)])
        keep = [int(x) if rng.random() < 0.5 else -1 for x in rng.integers(0, 300, 40)]
        b.truncate(keep)
        b.fork([int(x) for x in rng.integers(0, 40, 8)], [int(x) for x in rng.integers(0, 40, 8)])
    b.compact()
    b.compact()                                      # nothing is left to move
    b.reserve([5] * 40)


def test_large_pool_lowest_first():
    """The free pages lie far apart and past the first step of the scan."""
    n = 50000
    b = Both(n, 4, 32, layers=1)
    free = [20, 16383, 16384, 16400, 33000, 49999]
    b.host.ref = [0 if p in free else 1 for p in range(n)]
    b.cache.ref.copy_(ints(b.host.ref))
    b.reserve([40, 0, 33, 32])
    b.reserve([32, 0, 0, 1])


def test_most_sequences():
    """1024 sequences, many sharing one page, and a pool that ends inside the call."""
    b = Both(1500, 1024, 4, layers=1)
    b.reserve([40] + [0] * 1023)
    b.fork([0] * 600, list(range(1, 601)))
    b.reserve([1] * 1024)
    b.reserve([20 if s % 3 else 0 for s in range(1024)])
    b.truncate([0 if s % 2 else -1 for s in range(1024)])
    b.compact()


@pytest.mark.parametrize("seed", range(4))
def test_random_walk(seed):
    rng = np.random.default_rng(seed)
    S = int(rng.integers(2, 30))
    b = Both(int(rng.integers(10, 150)), S, int(rng.integers(2, 12)), page=int(rng.choice([32, 64])))
    for _ in range(25):
        k = rng.integers(0, 5)
        if k < 2:
            b.reserve([int(x) for x in rng.integers(-1, 40, S) * (rng.random(S) < 0.6)])
        elif k == 2:
            n = int(rng.integers(0, S + 1))
            b.fork([int(x) for x in rng.integers(0, S, n)], [int(x) for x in rng.integers(0, S, n)])
        elif k == 3:
            b.truncate([int(x) if rng.random() < 0.4 else -1 for x in rng.integers(0, 120, S)])
        else:
            b.compact()


def test_branches_decode_on_their_own():
    """A forked sequence continues with other tokens: each branch attends to the
    shared prefix and to its own rows, before and after a compaction."""
    cache = ops.KvCache.allocate(1, 40, 32, 2, 64, 3, 8, DEV)
    rng = np.random.default_rng(1)
    old = rows(rng, 45, 2, 64, "f32"), rows(rng, 45, 2, 64, "f32")
    new = rows(rng, 12, 2, 64, "f32"), rows(rng, 12, 2, 64, "f32")
    g = ops.kv4_reserve(cache, ints([45, 0, 0]))
    ops.kv4_append(cache, 0, old[0].to(DEV), old[1].to(DEV), ints([0, 45, 45, 45]), g)
    ops.kv4_fork(cache, ints([0, 0]), ints([1, 2]))
    g = ops.kv4_reserve(cache, ints([4, 4, 4]))
    ops.kv4_append(cache, 0, new[0].to(DEV), new[1].to(DEV), ints([0, 4, 8, 12]), g)
    q = rows(rng, 3, 4, 64, "f32", strong=False)
    out = ops.kv4_attention(q.to(DEV), cache, 0, ints([0, 1, 2, 3]))
    for s in range(3):
        k, v = (aorc.cache_values(torch.cat((o, n[4 * s:4 * s + 4])).numpy()).astype(np.float64)
                for o, n in zip(old, new))
        o, _, mag, dots = aorc.attention(q[s:s + 1].double().numpy(), k, v, 48, 64 ** -0.5)
        err = np.abs(out[s:s + 1].double().cpu().numpy() - o)
        assert (err <= 2e-5 * (1 + np.abs(mag))).all()   # sizes of order one, fp32 throughout
    ops.kv4_truncate(cache, ints([0, -1, -1]))
    ops.kv4_compact(cache)
    again = ops.kv4_attention(q.to(DEV), cache, 0, ints([0, 0, 1, 2]), out=torch.empty_like(out))
    alone = ops.kv4_attention(q[1:].to(DEV), cache, 0, ints([0, 0, 1, 2]))
    assert torch.equal(alone, out[1:]) and torch.equal(again[:2].isnan(), torch.zeros_like(again[:2], dtype=torch.bool))


def test_captured_step():
    """Reserve, append and attend in one graph, replayed as the sequences grow."""
    def build():
        c = ops.KvCache.allocate(1, 30, 32, 2, 64, 3, 8, DEV)
        c.data.zero_()
        g0 = ops.kv4_reserve(c, ints([30, 5, 0]))
        k = torch.from_numpy(np.random.default_rng(0).standard_normal((35, 2, 64)).astype(np.float32)).to(DEV)
        ops.kv4_append(c, 0, k, k, ints([0, 30, 35, 35]), g0)
        return c

    def step(c, k, q, out):
        g = ops.kv4_reserve(c, one)
        ops.kv4_append(c, 0, k, k, start, g)
        ops.kv4_attention(q, c, 0, start, granted=g, out=out)

    one, start = ints([1, 1, 0]), ints([0, 1, 2, 2])
    a, b = build(), build()
    k, q = torch.randn((2, 2, 64), device=DEV), torch.randn((2, 4, 64), device=DEV)
    oa, ob = torch.empty((2, 4, 64), device=DEV), torch.empty((2, 4, 64), device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, k, q, oa)
    for _ in range(6):
        graph.replay()
        step(b, k, q, ob)
        torch.cuda.synchronize()
        assert torch.equal(oa, ob) and torch.equal(a.len, b.len) and torch.equal(a.data, b.data)
        k.mul_(0.9)
        q.add_(0.1)
    assert a.len.tolist() == [36, 11, 0]
