"""The attention half's C ABI and binding: exports, struct layout, and refusals
that return before anything reaches a device."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import attn_oracle as aorc
from quantized_moe_decode_route_amd import ops

FAKE = 1 << 20                       # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ops.LIB_PATH):
        from quantized_moe_decode_route_amd import build
        build.build()
    return ops.lib()


def test_exports_every_declared_function(lib):
    with open(os.path.join(ops.INCLUDE_DIR, "moedec_attn.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:dense|kv4)_\w+)\s*\(", text)))
    assert len(names) == 12
    for n in names:
        assert hasattr(lib, n) and n in ops._SIGS, n


def test_struct_layout():
    assert ctypes.sizeof(ops._KvCache) == 64 and ops._KvCache.data.offset == 32


def _cache(**kw):
    f = dict(layers=2, n_pages=10, page_tokens=32, kv_heads=2, head_dim=64, n_seqs=3, max_pages=4, data=FAKE,
             table=FAKE, len=FAKE, ref=FAKE)
    f.update(kw)
    return ops._KvCache(*f.values())


BAD_CACHE = [(dict(data=None), 1), (dict(table=None), 1), (dict(len=None), 1), (dict(ref=None), 1),
             (dict(data=FAKE + 8), 1), (dict(ref=FAKE + 4), 1), (dict(layers=0), 1), (dict(n_pages=0), 1),
             (dict(n_seqs=0), 1), (dict(max_pages=0), 1), (dict(kv_heads=0), 1), (dict(page_tokens=48), 2),
             (dict(page_tokens=16), 2), (dict(head_dim=80), 2), (dict(head_dim=512), 2), (dict(n_seqs=1025), 2),
             (dict(kv_heads=1025), 2), (dict(n_pages=(1 << 24) + 1), 2), (dict(max_pages=1 << 26), 2)]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches(lib, kw, want):
    c = ctypes.byref(_cache(**kw))
    assert lib.kv4_append(c, 0, FAKE, 128, FAKE, 128, 0, 1, FAKE, None, None) == want
    assert lib.kv4_read(c, 0, FAKE, FAKE, 1, FAKE, 128, FAKE, 128, 0, None) == want
    assert lib.kv4_attention(c, 0, FAKE, 256, 0, 1, 4, FAKE, None, 1.0, 0, 100, FAKE, 256, None, None, 0, None) == want
    assert lib.kv4_attention_workspace(c, 1, 4, 100) == -1
    assert lib.kv4_reserve(c, FAKE, FAKE, FAKE, None) == want
    assert lib.kv4_fork(c, 1, FAKE, FAKE, None, FAKE, None) == want
    assert lib.kv4_truncate(c, FAKE, None) == want
    assert lib.kv4_compact(c, FAKE, FAKE, FAKE, None) == want


def test_bad_rows(lib):
    c = ctypes.byref(_cache())
    good = dict(layer=0, k=FAKE, ldk=128, v=FAKE, ldv=128, dtype=0, rows=1, q=FAKE, g=None)
    for bad in (dict(layer=2), dict(layer=-1), dict(k=None), dict(v=None), dict(ldk=127), dict(ldk=130), dict(ldv=64),
                dict(dtype=3), dict(rows=-1), dict(q=None), dict(k=FAKE + 4), dict(q=FAKE + 1), dict(g=FAKE + 2)):
        f = {**good, **bad}
        assert lib.kv4_append(c, f["layer"], f["k"], f["ldk"], f["v"], f["ldv"], f["dtype"], f["rows"], f["q"], f["g"],
                              None) == 1, bad
    assert lib.kv4_append(c, 0, FAKE, 132, FAKE, 128, 2, 1, FAKE, None, None) == 1     # 264 bytes a row
    assert lib.kv4_append(c, 0, FAKE, 128, FAKE, 128, 0, 1 << 24, FAKE, None, None) == 2
    assert lib.kv4_append(c, 0, None, 128, None, 128, 0, 0, FAKE, None, None) == 0     # no rows: nothing to do
    assert lib.kv4_read(c, 0, None, FAKE, 1, FAKE, 128, FAKE, 128, 0, None) == 1


def test_bad_attention(lib):
    c = ctypes.byref(_cache())
    good = dict(layer=0, q=FAKE, ldq=256, dtype=0, rows=1, heads=4, start=FAKE, g=None, scale=1.0, window=0, max_len=64,
                out=FAKE, ldo=256, lse=None, ws=None, nb=0)

    def call(**kw):
        return lib.kv4_attention(c, *{**good, **kw}.values(), None)

    for bad in (dict(layer=2), dict(q=None), dict(ldq=255), dict(ldo=254), dict(dtype=7), dict(rows=-1),
                dict(heads=3), dict(heads=0), dict(start=None), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(window=-1), dict(max_len=0), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2)):
        assert call(**bad) == 1, bad
    assert call(heads=16386) == 2 and call(rows=1 << 24) == 2
    assert call(rows=0, q=None, out=None) == 0
    need = lib.kv4_attention_workspace(c, 1, 4, 100000)
    assert need > 0
    assert call(max_len=100000) == 1 and call(max_len=100000, ws=FAKE, nb=need - 1) == 1
    assert call(max_len=100000, ws=FAKE + 4, nb=need) == 1


def test_bad_page_calls(lib):
    c = ctypes.byref(_cache())
    for i in range(3):
        a = [FAKE] * 3
        a[i] = None
        assert lib.kv4_reserve(c, *a, None) == 1
        assert lib.kv4_compact(c, *a, None) == 1
    assert lib.kv4_fork(c, -1, FAKE, FAKE, None, FAKE, None) == 1
    assert lib.kv4_fork(c, 1, None, FAKE, None, FAKE, None) == 1
    assert lib.kv4_fork(c, 1025, FAKE, FAKE, None, FAKE, None) == 2
    assert lib.kv4_fork(c, 0, None, None, None, None, None) == 0
    assert lib.kv4_truncate(c, None, None) == 1


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_bad_linear(lib, bits):
    fn = getattr(lib, f"dense_linear_q{bits}")
    good = dict(x=FAKE, dtype=0, ldx=128, w=FAKE, scale=FAKE, bias=None, act=0, res=None, ldr=0, y=FAKE, ldy=8, T=1,
                K=128, N=8, ws=FAKE, nb=1 << 30)

    def call(**kw):
        return fn(*{**good, **kw}.values(), None)

    for bad in (dict(x=None), dict(w=None), dict(scale=None), dict(y=None), dict(dtype=3), dict(act=4), dict(act=-1),
                dict(ldx=127), dict(ldx=126), dict(ldy=7), dict(res=FAKE, ldr=7), dict(T=-1), dict(K=0), dict(N=0),
                dict(K=128 // bits + 4, ldx=128), dict(x=FAKE + 4), dict(w=FAKE + 8), dict(bias=FAKE + 2),
                dict(y=FAKE + 2)):
        assert call(**bad) == 1, bad
    assert call(K=1 << 17, ldx=1 << 17) == 2 and call(T=1 << 24) == 2 and call(N=1 << 24, ldy=1 << 24) == 2
    assert call(T=0, x=None, y=None) == 0
    need = lib.dense_linear_workspace(bits, 0, 300, 128, 8)
    assert need > 0 and call(T=300, nb=need - 1) == 1 and call(T=300, ws=None, nb=need) == 1
    for sizes in ((4, 5, 1, 128, 8), (4, 0, -1, 128, 8), (3, 0, 1, 128, 8), (4, 0, 1, 1 << 17, 8), (4, 0, 1, 128, 0)):
        assert lib.dense_linear_workspace(*sizes) == -1


def test_overlaps(lib):
    """Outputs over inputs are refused (that columns of one buffer are not, the GPU
    tests show)."""
    need = lib.dense_linear_workspace(4, 0, 300, 128, 64)

    def linear(y, ldy, res=None, ldr=0, ldx=128, nb=need - 1, T=300):
        return lib.dense_linear_q4(FAKE, 0, ldx, FAKE + (1 << 24), FAKE, None, 0, res, ldr, y, ldy, T, 128, 64, FAKE,
                                   nb, None)

    assert need > 0
    for y, ldy in ((FAKE, 64), (FAKE + 4 * 128 * 299, 64), (FAKE + 4 * 64, 128), (FAKE - 4 * 63, 256)):
        assert linear(y, ldy, nb=need, ldx=256 if ldy == 256 else 128) == 1, (y - FAKE, ldy)
    far = FAKE + (1 << 23)
    for res, ldr in ((far + 4, 64), (far - 4, 64), (far, 80)):
        assert linear(far, 64, res, ldr, nb=need) == 1, (res - far, ldr)
    c = ctypes.byref(_cache())

    def attend(out, rows=4, ldq=512, ldo=512, ws=None, nb=0):
        return lib.kv4_attention(c, 0, FAKE, ldq, 0, rows, 4, FAKE, None, 1.0, 0, 64, out, ldo, None, ws, nb, None)

    for out, ld in ((FAKE, 512), (FAKE + 4 * 252, 512), (FAKE - 4 * 252, 512), (FAKE + 4 * 256 * 3, 256)):
        assert attend(out, ldq=ld, ldo=ld) == 1, (out - FAKE, ld)


def test_binding_refuses(lib):
    x = torch.zeros((2, 128))
    lin = ops.Linear(torch.zeros((8, 64), dtype=torch.uint8), torch.zeros(8), 4)
    with pytest.raises(ValueError):
        ops.linear(x, lin)                            # not on a GPU
    with pytest.raises(ValueError):
        ops.linear(x, lin, act="tanh")
    with pytest.raises(TypeError):
        ops._rows([1], (1,), "x", torch.device("cpu"))
    cache = ops.KvCache.allocate(1, 4, 32, 2, 64, 3, 2, "cpu")
    assert cache.data.shape == (1, 4, 2 * 32 * 72) and (cache.ref == 0).all()
    with pytest.raises(ValueError):
        ops.kv4_truncate(cache, torch.zeros(3, dtype=torch.int32))


# ------------------------------------------------------- the oracle's own pins

def test_oracle_attention_closed_forms():
    """Equal scores average the values; one towering score picks its value; the
    window and the causal mask cut exactly where they should."""
    rng = np.random.default_rng(0)
    k, v = np.ones((6, 1, 4)), rng.standard_normal((6, 1, 4))
    q = rng.standard_normal((3, 2, 4))
    out, lse, _, _ = aorc.attention(q, k, v, 3, 0.5)
    for i in range(3):
        for h in range(2):
            assert np.allclose(out[i, h], v[:4 + i, 0].mean(0))
            assert np.isclose(lse[i, h], 0.5 * q[i, h].sum() + np.log(4 + i))
    out, _, _, _ = aorc.attention(q, k, v, 3, 0.5, window=2)
    assert np.allclose(out[1, 0], v[3:5, 0].mean(0))
    k[2] = 1000 * q[2, 0]
    assert np.allclose(aorc.attention(q, k, v, 3, 0.5)[0][2, 0], v[2, 0])
    assert (aorc.attention(q, k, v, -3, 0.5)[0] == 0).all()


def test_oracle_linear_closed_form():
    codes = np.eye(4, dtype=np.int8) * 3
    x = np.arange(8.0).reshape(2, 4)
    y = aorc.linear(x, codes, np.full(4, 0.5, np.float32), np.ones(4), "relu", -x)
    assert np.allclose(y, np.maximum(1.5 * x + 1, 0) - x)
    assert np.isclose(aorc.ACT["gelu"](np.array([1.0]))[0], 0.8413447460685429)


def test_oracle_pages():
    p = aorc.Pages(6, 4, 4, 3)
    assert p.reserve([5, 4, 0, 0]) == [5, 4, 0, 0] and p.table[:2] == [[0, 1], [2]]
    assert p.fork([0, 0], [2, 2]) == [1, 0] and p.ref == [2, 2, 1, 0, 0, 0]
    assert p.reserve([1, 0, 1, 0]) == [1, 0, 1, 0] and p.copies == [(1, 3)]
    assert p.table[0] == [0, 3] and p.table[2] == [0, 1] and p.ref == [2, 1, 1, 1, 0, 0]
    p.truncate([-1, 0, 0, -1])
    assert p.ref == [1, 0, 0, 1, 0, 0]
    assert p.compact() == ([0, -1, -1, 1, -1, -1], 2) and p.table[0] == [0, 1] and p.copies == [(3, 1)]
