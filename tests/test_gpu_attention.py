"""kv4_attention against float64 attention over the values the cache holds."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as aorc
from quantized_moe_decode_route_amd import ops

from _attn import DEV, DT, attention_bound, fill, ints, new_cache, rows, starts

pytestmark = pytest.mark.gpu


def _check(lens, news, *, heads=4, kv_heads=2, dim=64, page=32, dtype="f32", window=0, max_len=None, scale=None,
           seed=0, granted=None, kv_dtype="f32", q=None):
    rng = np.random.default_rng(seed)
    cache = new_cache(lens, page, kv_heads, dim, seed=seed)
    held = fill(cache, lens, rng, kv_dtype)
    T = sum(news)
    if q is None:
        q = rows(rng, T + 2, heads, dim, dtype, strong=False)
    out = torch.full((T + 2, heads, dim), 5.0, dtype=DT[dtype], device=DEV)
    lse = torch.full((T + 2, heads), 5.0, device=DEV)
    ops.kv4_attention(q.to(DEV), cache, 0, ints(starts(news)), window=window, max_len=max_len, out=out, lse=lse,
                      scale=scale, granted=None if granted is None else ints(granted))
    assert (out[T:] == 5).all() and (lse[T:] == 5).all()             # rows behind the last sequence
    got, glse, at = out.double().cpu().numpy(), lse.double().cpu().numpy(), 0
    for s, (n, m) in enumerate(zip(lens, news)):
        real = m if granted is None else min(m, granted[s])
        k, v = (x.astype(np.float64) for x in held[s])
        o, l, mag, dots = aorc.attention(q[at:at + real].double().numpy(), k, v, n - real,
                                         dim ** -0.5 if scale is None else scale, window)
        tol = attention_bound(mag, dots, o, n, dim, dtype)
        err = np.abs(got[at:at + real] - o)
        assert (err <= tol).all(), f"sequence {s}: worst error is {np.nanmax(err / tol):.2f} of its bound"
        fin = np.isfinite(l)
        assert np.array_equal(np.isfinite(glse[at:at + real]), fin)
        ltol = (np.abs(l) + 4 + dots * (dim + 16)) * 2.0 ** -21 + n * 2.0 ** -23
        assert (np.abs(glse[at:at + real][fin] - l[fin]) <= ltol[fin]).all()
        assert (got[at + real:at + m] == 0).all() and np.isneginf(glse[at + real:at + m]).all()
        at += m
    return cache, q, out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 64), (192, 128), (256, 32)])
def test_decode_lengths(dim, page, dtype):
    lens = [1, 2, 31, 32, 33, 0, 64, 127, 128, 129, 300, 1000]
    _check(lens, [min(n, 1) for n in lens], dim=dim, page=page, dtype=dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (8, 8), (6, 2), (16, 1), (20, 1), (48, 8), (40, 1)])
def test_head_layouts(heads, kv_heads):
    _check([5, 70, 200], [1, 3, 2], heads=heads, kv_heads=kv_heads, seed=heads)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (6, 1)])
@pytest.mark.parametrize("news", [[3, 0, 5], [40, 1, 17], [100, 64, 33], [16, 130, 8]])
def test_many_queries(news, heads, kv_heads, dtype):
    _check([130, 130, 90], news, heads=heads, kv_heads=kv_heads, dtype=dtype)
    _check([n if n else 3 for n in news], news, heads=heads, kv_heads=kv_heads, dtype=dtype)   # whole prompts


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_prompt_head_dims(dim, dtype):
    _check([150, 70], [140, 33], dim=dim, dtype=dtype, page=64)


@pytest.mark.parametrize("window", [1, 5, 32, 33, 100, 5000])
@pytest.mark.parametrize("news", [[1, 1], [9, 70]])
def test_window(window, news):
    _check([260, 90], news, window=window)


@pytest.mark.parametrize("max_len", [1, 600, 3000, None])
def test_splits(max_len):
    """However the keys are split, and whatever bound the caller gives."""
    _check([2900, 700, 1], [1, 2, 1], max_len=max_len, page=128)
    _check([2900, 700, 1], [1, 40, 1], max_len=max_len, page=128, dtype="bf16", window=900)


def test_long_and_peaked():
    """A score that towers over 5000 others, late and early: the running maximum moves."""
    rng = np.random.default_rng(3)
    q = rows(rng, 4, 4, 64, "f32", strong=False)
    _check([5000, 4000], [1, 1], scale=3.0, q=q, page=128, seed=4)
    _check([5000, 4000], [1, 1], scale=0.0, q=q, page=128, seed=4)
    _check([5000, 4000], [1, 1], scale=-2.0, q=q, page=128, seed=4)


def test_granted():
    _check([40, 33, 64], [3, 2, 20], granted=[0, 2, 7])


@pytest.mark.parametrize("lead", [1, 7, 40, 130])
@pytest.mark.parametrize("news", [[1, 1, 1], [0, 3, 30], [70, 0, 9]])
def test_rows_before_the_first_sequence(news, lead):
    """q_start[0] > 0: rows of no sequence in front stay as they were, the others do
    not notice them; one part and several, with and without heads that share.

    The rows in front may change how the call is cut, so both results are within
    their bound (_attn.attention_bound): with sum |q||k| / 8 below 32, values below
    32 and at most 2000 keys that is 32 * (2 * 32 * (82 * 2^-24 + 2^-22) + 2^-18)
    < 2^-6 each at the worst; rows mixed up would be off by their size."""
    for heads, lens in ((4, [80, 33, 45]), (2, [2000, 40, 1200])):
        rng = np.random.default_rng(lead)
        cache = new_cache(lens)
        fill(cache, lens, rng)
        q = rows(rng, sum(news) + lead, heads, 64, "f32", strong=False).to(DEV)
        st = starts(news)
        want = ops.kv4_attention(q[lead:], cache, 0, ints(st))
        out, lse = torch.full_like(q, 5.0), torch.full((q.shape[0], heads), 5.0, device=DEV)
        ops.kv4_attention(q, cache, 0, ints([lead + a for a in st]), out=out, lse=lse)
        assert (out[:lead] == 5).all() and (lse[:lead] == 5).all()
        assert (out[lead:] - want).abs().max() <= 2.0 ** -5


def test_positions_below_zero_are_empty():
    """More queries than tokens: the first ones see nothing."""
    _check([2, 5], [4, 5])


@pytest.mark.parametrize("news", [[1, 1], [20, 3]])
def test_masked_positions_hold_anything(news):
    """Stale codes with NaN and infinite scales behind a sequence's end, and keys
    after a query, never reach a result."""
    lens = [37, 9]
    rng = np.random.default_rng(8)
    cache = new_cache(lens, 32)
    held = fill(cache, lens, rng)
    q = rows(rng, sum(news), 4, 64, "f32", strong=False).to(DEV)
    want = ops.kv4_attention(q, cache, 0, ints(starts(news)))
    unit = 32 * (64 + 8)
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        for s, n in enumerate(lens):
            page = int(cache.table[s, n // 32])
            body = cache.data[0, page].view(2, unit)
            scales = body[:, 32 * 64:].reshape(2, 2, 32, 4).clone().view(torch.float32)
            scales[:, :, n % 32:] = value
            body[:, 32 * 64:] = scales.view(torch.uint8).reshape(2, -1)
        assert torch.equal(ops.kv4_attention(q, cache, 0, ints(starts(news))), want)
    assert torch.isfinite(want).all()


def test_nan_key_shows_in_its_rows_only():
    lens = [40, 20]
    cache, rng = new_cache(lens, 32), np.random.default_rng(2)
    fill(cache, lens, rng)
    k = torch.randn((1, 2, 64), device=DEV)
    v = torch.randn((1, 2, 64), device=DEV)
    k[0, 1, 3] = float("nan")                         # head 1 of the last token of sequence 0
    ops.kv4_append(cache, 0, k, v, ints([0, 1, 1]))
    q = torch.randn((3, 4, 64), device=DEV)
    out = ops.kv4_attention(q, cache, 0, ints([0, 2, 3]))
    assert torch.isnan(out[1, 2:]).all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :2]).all() and torch.isfinite(out[2]).all()


def test_all_keys_nan():
    cache = new_cache([3], 32)
    k = torch.full((3, 2, 64), float("nan"), device=DEV)
    ops.kv4_append(cache, 0, k, k, ints([0, 3]))
    assert torch.isnan(ops.kv4_attention(torch.randn((1, 4, 64), device=DEV), cache, 0, ints([0, 1]))).all()


def test_bad_pages_are_not_there():
    lens = [100, 64]
    cache, rng = new_cache(lens, 32), np.random.default_rng(12)
    held = fill(cache, lens, rng)
    cache.table[0, 1] = cache.n_pages + 5
    cache.table[1] = -1
    q = rows(rng, 2, 4, 64, "f32", strong=False)
    out = ops.kv4_attention(q.to(DEV), cache, 0, ints([0, 1, 2])).double().cpu().numpy()
    keep = list(range(32)) + list(range(64, 100))
    k, v = (x[keep].astype(np.float64) for x in held[0])
    o, _, mag, dots = aorc.attention(q[:1].double().numpy(), k, v, len(keep) - 1, 64 ** -0.5)
    assert (np.abs(out[:1] - o) <= attention_bound(mag, dots, o, 100, 64, "f32")).all()
    assert (out[1] == 0).all()


@pytest.mark.parametrize("size", [1e-30, 1e-4, 1e5, 1e30])
@pytest.mark.parametrize("news", [[1, 1], [30, 2]])
def test_value_and_query_ranges(size, news):
    """Value scales far outside fp16's range, queries of any size, and scales that
    grow along the sequence."""
    lens = [90, 300]
    rng = np.random.default_rng(13)
    cache = new_cache(lens, 32)
    T = sum(lens)
    k = rows(rng, T, 2, 64, "f32")
    v = rows(rng, T, 2, 64, "f32") * (size * np.float32(1.05) ** torch.arange(T))[:, None, None]
    v = v.float()
    ops.kv4_append(cache, 0, k.to(DEV), v.to(DEV), ints(starts(lens)))
    m = sum(news)
    q = (rows(rng, m, 4, 64, "f32", strong=False) / size).float()
    out = ops.kv4_attention(q.to(DEV), cache, 0, ints(starts(news)), scale=0.1 * size).double().cpu().numpy()
    at = row = 0
    for n, mm in zip(lens, news):
        kk, vv = (aorc.cache_values(x[at:at + n].numpy()).astype(np.float64) for x in (k, v))
        o, _, mag, dots = aorc.attention(q[row:row + mm].double().numpy(), kk, vv, n - mm, 0.1 * size)
        tol = attention_bound(mag, dots, o, n, 64, "f32")
        # the largest rows overflow fp32 (1e30 * 1.05^389 * 6 > 3.4e38): such a value row is NaN on both sides
        got = out[row:row + mm]
        assert np.array_equal(np.isnan(got), np.isnan(o))
        assert ((np.abs(got - o) <= tol) | np.isnan(o)).all()
        at, row = at + n, row + mm


def test_strided_queries_and_output():
    lens = [70, 12]
    cache, rng = new_cache(lens, 32), np.random.default_rng(14)
    fill(cache, lens, rng)
    wide = torch.randn((3, 8 * 64), device=DEV)
    q = wide[:, :256].unflatten(1, (4, 64))
    dst = torch.full((3, 320), 3.0, device=DEV)
    ops.kv4_attention(q, cache, 0, ints([0, 1, 3]), out=dst[:, 32:288].unflatten(1, (4, 64)))
    want = ops.kv4_attention(q.contiguous(), cache, 0, ints([0, 1, 3]))
    assert torch.equal(dst[:, 32:288].reshape(3, 4, 64), want)
    assert (dst[:, :32] == 3).all() and (dst[:, 288:] == 3).all()


@pytest.mark.parametrize("news", [[1, 1, 0], [50, 1, 3]])
def test_captured_and_replayed(news):
    """One graph serves a growing cache; replays match the eager call bit for bit."""
    lens = [600, 300, 3]
    cache, rng = new_cache(lens, 32, spare=60, max_pages=40), np.random.default_rng(15)
    fill(cache, lens, rng)
    q = torch.randn((sum(news), 4, 64), device=DEV)
    start, out = ints(starts(news)), torch.empty((sum(news), 4, 64), device=DEV)
    ops.kv4_attention(q, cache, 0, start, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.kv4_attention(q, cache, 0, start, out=out)
    for i in range(4):
        out.fill_(float(i))
        g.replay()
        assert torch.equal(out, ops.kv4_attention(q, cache, 0, start))
        torch.cuda.synchronize()
        cache.len.sub_(ints([100 * i, 1, 0]))
        q.add_(0.25)


def test_two_streams_at_once():
    lens, news = [900, 400], [1, 2]
    cache, rng = new_cache(lens, 32), np.random.default_rng(16)
    fill(cache, lens, rng)
    q, start = torch.randn((3, 4, 64), device=DEV), ints(starts(news))
    want = ops.kv4_attention(q, cache, 0, start)
    torch.cuda.synchronize()
    side, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(8):
        with torch.cuda.stream(side[i % 2]):
            got.append(ops.kv4_attention(q, cache, 0, start))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


def test_pool_past_32_bits():
    """Pages that lie beyond 4 GB of the pool, in its second layer."""
    dim, heads, page = 128, 8, 128
    unit = page * heads * (dim + 8)
    n_pages = (3 << 30) // unit + 1
    cache = ops.KvCache.allocate(2, n_pages, page, heads, dim, 2, 8, DEV)
    lens = [300, 129]
    cache.table[0, :3] = ints([n_pages - 1, 0, n_pages - 3])
    cache.table[1, :2] = ints([n_pages - 2, n_pages // 2])
    cache.len.copy_(ints(lens))
    rng = np.random.default_rng(17)
    held = fill(cache, lens, rng, layer=1)
    k, v = ops.kv4_read(cache, 1, ints([0, 0]), ints(starts(lens)), sum(lens))
    assert np.array_equal(k.cpu().numpy(), np.concatenate([h[0] for h in held]))
    assert np.array_equal(v.cpu().numpy(), np.concatenate([h[1] for h in held]))
    q = rows(rng, 2, 16, dim, "f32", strong=False)
    out = ops.kv4_attention(q.to(DEV), cache, 1, ints([0, 1, 2])).double().cpu().numpy()
    for s, n in enumerate(lens):
        kk, vv = (x.astype(np.float64) for x in held[s])
        o, _, mag, dots = aorc.attention(q[s:s + 1].double().numpy(), kk, vv, n - 1, dim ** -0.5)
        assert (np.abs(out[s:s + 1] - o) <= attention_bound(mag, dots, o, n, dim, "f32")).all()


def test_long_flat_cache():
    """200,000 keys of nearly equal weight in one sequence: the sums and the joins
    of many splits keep their digits."""
    n = 200_000
    cache = new_cache([n], 128, 1, 64)
    rng = np.random.default_rng(18)
    (k, v), = fill(cache, [n], rng)
    for dtype in ("f32", "bf16"):
        q = rows(rng, 1, 2, 64, dtype, strong=False)
        out = ops.kv4_attention(q.to(DEV), cache, 0, ints([0, 1]), scale=0.01).double().cpu().numpy()
        o, _, mag, dots = aorc.attention(q.double().numpy(), k.astype(np.float64), v.astype(np.float64), n - 1, 0.01)
        # the probabilities' roundings are independent: their part of the bound falls with
        # the root of the keys (six standard deviations), the sums' stays
        p = 2.0 ** -21 if dtype == "f32" else 2.0 ** -11
        loose = attention_bound(mag, dots, o, 64, 64, dtype) - mag * p
        assert (np.abs(out - o) <= loose + mag * (6 * p / np.sqrt(n) + 2.0 ** -17)).all()


def test_output_beside_and_over_queries():
    lens, news = [50, 20], [3, 1]
    cache = new_cache(lens)
    fill(cache, lens, np.random.default_rng(0))
    buf = torch.randn(4, 8, 64, device=DEV)
    want = ops.kv4_attention(buf[:, :4].contiguous(), cache, 0, ints(starts(news)))
    ops.kv4_attention(buf[:, :4], cache, 0, ints(starts(news)), out=buf[:, 4:])
    assert torch.equal(buf[:, 4:], want)
    for bad in (buf[:, :4], buf[:, 2:6]):
        with pytest.raises(ops.MoedecError):
            ops.kv4_attention(buf[:, :4], cache, 0, ints(starts(news)), out=bad)


def test_binding_refuses():
    cache = new_cache([4], 32)
    q, start = torch.zeros((1, 4, 64), device=DEV), ints([0, 1])
    for bad in (dict(window=-1), dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(max_len=0)):
        with pytest.raises((ValueError, ops.MoedecError)):
            ops.kv4_attention(q, cache, 0, start, **bad)
    for layer in (-1, 1, 1 << 32):
        with pytest.raises(ValueError):
            ops.kv4_attention(q, cache, layer, start)
    with pytest.raises(ValueError):
        ops.kv4_attention(q, cache, 0, start.long())
    with pytest.raises(ValueError):
        ops.kv4_attention(q[:, :, :32], cache, 0, start)
    with pytest.raises(ValueError):
        ops.kv4_attention(q.transpose(1, 2).contiguous().transpose(1, 2), cache, 0, start)
    with pytest.raises(ops.MoedecError):
        ops.kv4_attention(torch.zeros((1, 3, 64), device=DEV), cache, 0, start)    # 3 heads over 2
    with pytest.raises(ops.MoedecError):
        ops.kv4_attention(torch.zeros((2, 5 * 64 + 1), device=DEV)[:, 1:257].unflatten(1, (4, 64)), cache, 0, start)
