"""kv4_append and kv4_read: the 4-bit cache holds exactly what the row quantiser's
rule gives, and nothing else changes."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as aorc
from quantized_moe_decode_route_amd import ops

from _attn import DEV, DT, fill, ints, new_cache, rows, starts

pytestmark = pytest.mark.gpu


def _read(cache, lens, layer=0, dtype=torch.float32, first=None):
    n = len(lens)
    return ops.kv4_read(cache, layer, ints(first or [0] * n), ints(starts(lens)), sum(lens), dtype)


def _same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=123.0), torch.nan_to_num(b, nan=123.0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 32, 1), (128, 64, 3), (192, 32, 2), (256, 128, 1)])
def test_round_trip(dim, page, heads, dtype):
    lens = [1, 7, 8, 9, 0, 31, 32, 33, 100, 129]
    cache, rng = new_cache(lens, page, heads, dim), np.random.default_rng(dim)
    held = fill(cache, lens, rng, dtype)
    for out in ("f32", dtype):
        k, v = _read(cache, lens, dtype=DT[out])
        for i, got in enumerate((k, v)):
            want = torch.from_numpy(np.concatenate([h[i] for h in held])).to(DT[out])
            assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("step", [1, 3, 8, 13])
def test_grows_token_by_token(step):
    """Appends in parts give what one append gives, and leave earlier and
    neighbouring positions alone, codes and scales."""
    n, page = 70, 32
    lens = [n, 0, n - 9]
    rng = np.random.default_rng(step)
    whole, parts = new_cache(lens, page), new_cache(lens, page)
    parts.data.copy_(whole.data)
    k, v = (rows(rng, sum(lens), 2, 64, "f32").to(DEV) for _ in range(2))
    ops.kv4_append(whole, 0, k, v, ints(starts(lens)))
    parts.len.zero_()
    at = [0, 0, 0]
    while at != lens:
        new = [min(step, a - b) for a, b in zip(lens, at)]
        pick = [s0 + b + i for s0, b, m in zip(starts(lens), at, new) for i in range(m)]
        at = [b + m for b, m in zip(at, new)]
        parts.len.copy_(ints(at))
        idx = torch.tensor(pick, device=DEV)
        ops.kv4_append(parts, 0, k[idx], v[idx], ints(starts(new)))
    assert torch.equal(whole.data, parts.data)


def test_edge_rows():
    """Zeros, NaN, infinities, subnormal and underflowing rows, ties at half a code."""
    x = np.zeros((8, 1, 64), np.float32)
    x[1, 0, 5] = np.nan
    x[2, 0, 6], x[2, 0, 7] = np.inf, 1
    x[3, 0] = np.linspace(-1, 1, 64) * 1e-40
    x[4, 0, 0] = 1e-45                                # the scale underflows to zero
    x[5, 0] = np.tile(np.arange(-7, 9, dtype=np.float32) / 2, 4)
    x[5, 0, 0] = 7
    x[6, 0] = 3e38
    x[7, 0] = np.random.default_rng(0).standard_normal(64)
    cache = new_cache([8], 32, 1, 64)
    t = torch.from_numpy(x).to(DEV)
    ops.kv4_append(cache, 0, t, t, ints([0, 8]))
    k, v = _read(cache, [8])
    want = torch.from_numpy(aorc.cache_values(x))
    assert _same(k.cpu(), want) and _same(v.cpu(), want)


def test_layers_strides_and_other_bytes():
    """A fused projection's output as strided views; only the named layer changes."""
    lens, new = [40, 65, 20], [3, 1, 0]
    cache, rng = new_cache(lens, 32, 2, 64, layers=3), np.random.default_rng(4)
    fill(cache, lens, rng, layer=1)
    before = cache.data.clone()
    k0, v0 = _read(cache, lens, 1)
    wide = torch.from_numpy(rng.standard_normal((4, 5 * 64)).astype(np.float32)).to(DEV)
    k, v = wide[:, 64:192].unflatten(1, (2, 64)), wide[:, 192:].unflatten(1, (2, 64))
    ops.kv4_append(cache, 1, k, v, ints(starts(new)))
    assert torch.equal(cache.data[0], before[0]) and torch.equal(cache.data[2], before[2])
    k1, v1 = _read(cache, lens, 1)
    at = [37, 38, 39, 40 + 64]
    for got, old, x in ((k1, k0, k), (v1, v0, v)):
        want = old.clone()
        want[at] = torch.from_numpy(aorc.cache_values(x.cpu().numpy())).to(DEV)
        assert torch.equal(got, want)
    spare = [p for p in range(cache.n_pages) if cache.ref[p] == 0]
    assert torch.equal(cache.data[:, spare], before[:, spare])


def test_granted_limits_and_bad_pages():
    lens, new = [10, 33, 12, 5], [2, 2, 2, 2]
    cache, rng = new_cache(lens, 32), np.random.default_rng(5)
    fill(cache, lens, rng)
    before = cache.data.clone()
    k, v = (rows(rng, 8, 2, 64, "f32").to(DEV) for _ in range(2))
    cache.table[1, 1] = cache.n_pages                 # not a page: position 32 is not there
    cache.table[3, 0] = -1
    ops.kv4_append(cache, 0, k, v, ints(starts(new)), granted=ints([0, 2, 1, 2]))
    k1, _ = _read(cache, lens)
    want = torch.from_numpy(aorc.cache_values(k.cpu().numpy())).to(DEV)
    assert torch.equal(k1[10 + 31], want[2]) and (k1[10 + 32] == 0).all()
    assert torch.equal(k1[10 + 33 + 11], want[4])     # one granted row is the last position
    assert (k1[55:60] == 0).all()                     # a bad page reads as zeros
    page0 = int(cache.table[0, 0])
    assert torch.equal(cache.data[:, page0], before[:, page0])


def test_read_ranges():
    lens = [50, 10]
    cache, rng = new_cache(lens, 32), np.random.default_rng(6)
    held = fill(cache, lens, rng)
    k, v = _read(cache, [20, 6], first=[-3, 7])
    for i, got in enumerate((k, v)):
        want = np.zeros((26, 2, 64), np.float32)
        want[3:20] = held[0][i][:17]
        want[20:23] = held[1][i][7:10]                # positions past the length are zeros
        assert np.array_equal(got.cpu().numpy(), want)


def test_rows_of_no_sequence_are_left_alone():
    cache = new_cache([4, 6], 32)
    before = cache.data.clone()
    k = torch.randn((9, 2, 64), device=DEV)
    ops.kv4_append(cache, 0, k, k, ints([2, 2, 2]))
    assert torch.equal(cache.data, before)
    ops.kv4_append(cache, 0, k[:0], k[:0], ints([0, 0, 0]))
    assert torch.equal(cache.data, before)


@pytest.mark.parametrize("lead", [1, 9, 100])
def test_rows_before_the_first_sequence(lead):
    lens = [20, 0, 45]
    rng = np.random.default_rng(lead)
    a, b = new_cache(lens), new_cache(lens)
    b.data.copy_(a.data)
    k, v = (rows(rng, lead + sum(lens), 2, 64, "f32").to(DEV) for _ in range(2))
    ops.kv4_append(a, 0, k[lead:], v[lead:], ints(starts(lens)))
    ops.kv4_append(b, 0, k, v, ints([lead + n for n in starts(lens)]))
    assert torch.equal(a.data, b.data)
    got = ops.kv4_read(b, 0, ints([0, 0, 0]), ints([lead + n for n in starts(lens)]), lead + sum(lens))
    for x, y in zip(got, _read(a, lens)):
        assert torch.equal(x[lead:], y)


def test_many_sequences():
    """The 64-way search over sequences, with empty ones between."""
    rng = np.random.default_rng(11)
    lens = [int(n) for n in rng.integers(0, 4, 700)]
    lens[0] = lens[699] = 0
    cache = new_cache(lens, 32, 1, 64, max_pages=1)
    held = fill(cache, lens, rng)
    k, _ = _read(cache, lens)
    assert np.array_equal(k.cpu().numpy(), np.concatenate([h[0] for h in held]))
