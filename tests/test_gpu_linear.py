"""dense_linear_q*: product with a packed weight, bias, activation and residual
in its epilogue, against float64 over the dequantised weight."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as aorc
from quantized_moe_decode_route_amd import ops

from _attn import DEV, DT, EPS32, HALF

pytestmark = pytest.mark.gpu

RANGE = {8: 128, 4: 8, 2: 2}


def _case(T, K, N, bits, dtype, bias, residual, seed=0, xscale=1.0):
    rng = np.random.default_rng(seed)
    codes = rng.integers(-RANGE[bits], RANGE[bits], (N, K)).astype(np.int8)
    scale = rng.uniform(0.005, 0.02, N).astype(np.float32)
    x = torch.from_numpy((rng.standard_normal((T, K)) * xscale).astype(np.float32)).to(DT[dtype])
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    r = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).to(DT[dtype]) if residual else None
    return codes, scale, x, b, r


def _lin(codes, scale, bits, b):
    q = ops.pack(torch.from_numpy(codes).to(DEV), bits)
    return ops.Linear(q, torch.from_numpy(scale).to(DEV), bits, None if b is None else torch.from_numpy(b).to(DEV))


def _bound(codes, scale, x, b, r, act, dtype):
    """Oracle value and the error it allows: products exact (fp32 activations
    within 2^-22), a sum of K fp32 terms within K * 2^-24 of the terms' sizes
    (plus the 2^-39 of the row's largest element that fp16 pairs drop), scale,
    bias and activation a few roundings each (the activations' slopes are below
    1.13), the result rounded once."""
    xd = x.double().numpy()
    y = aorc.linear(xd, codes, scale, b, act, None if r is None else r.double().numpy())
    w = np.abs(codes.astype(np.float64)) * scale[:, None]
    size = np.abs(xd) @ w.T
    low = np.abs(xd).max(1, keepdims=True) * w.sum(1)[None] * 2.0 ** -38
    pre = size * ((x.shape[1] + 8) * EPS32 + (2.0 ** -22 if dtype == "f32" else 0)) + low
    if b is not None:
        pre = pre + 4 * EPS32 * (np.abs(b)[None] + size)
    res = 0 if r is None else np.abs(r.double().numpy())
    return y, 1.2 * pre + 16 * EPS32 * (np.abs(y) + res) + HALF[dtype] * np.abs(y) + 1e-30


def _check(y, want, tol):
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst error is {np.nanmax(err / tol):.2f} of its bound"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (1, 2048, 257), (2, 192, 1), (3, 640, 33), (5, 64, 130),
                                   (16, 320, 48), (17, 1088, 95), (33, 128, 300), (64, 2048, 129), (130, 192, 257),
                                   (257, 448, 64), (300, 704, 513)])
def test_shapes(T, K, N, bits, dtype):
    codes, scale, x, b, r = _case(T, K, N, bits, dtype, True, True, seed=T + K + N)
    y = ops.linear(x.to(DEV), _lin(codes, scale, bits, b), residual=r.to(DEV))
    _check(y, *_bound(codes, scale, x, b, r, "none", dtype))


@pytest.mark.parametrize("T", [1, 4, 20, 150])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_epilogue(act, bias, residual, T):
    codes, scale, x, b, r = _case(T, 256, 70, 4, "f32", bias, residual, seed=5, xscale=0.5)
    y = ops.linear(x.to(DEV), _lin(codes, scale, 4, b), act=act, residual=None if r is None else r.to(DEV))
    _check(y, *_bound(codes, scale, x, b, r, act, "f32"))


@pytest.mark.parametrize("K", [32, 96, 6144, 16384])
@pytest.mark.parametrize("T", [1, 19])
def test_inner_sizes(K, T):
    codes, scale, x, b, r = _case(T, K, 40, 4, "f32", False, False, seed=K)
    _check(ops.linear(x.to(DEV), _lin(codes, scale, 4, None)), *_bound(codes, scale, x, b, r, "none", "f32"))


@pytest.mark.parametrize("T", [2, 40, 200])
def test_rows_of_very_different_size(T):
    """Each row has its own power of two: a tiny row beside a huge one keeps its bits."""
    codes, scale, x, b, r = _case(T, 256, 64, 4, "f32", False, False, seed=9)
    x = x * torch.tensor([2.0 ** (-60 + 7 * (i % 18)) for i in range(T)])[:, None]
    x[1] = 0
    y = ops.linear(x.to(DEV), _lin(codes, scale, 4, None))
    _check(y, *_bound(codes, scale, x, b, r, "none", "f32"))
    assert (y[1] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 70])
def test_strides_and_in_place_residual(T, dtype):
    codes, scale, x, b, r = _case(T, 128, 45, 4, dtype, True, True, seed=3)
    wide = torch.full((T, 128 + 64), 7.0, dtype=DT[dtype], device=DEV)
    wide[:, 32:160] = x.to(DEV)
    out = torch.full((T, 61), 9.0, dtype=DT[dtype], device=DEV)
    out[:, 5:50] = r.to(DEV)
    view = out[:, 5:50]
    got = ops.linear(wide[:, 32:160], _lin(codes, scale, 4, b), act="silu", residual=view, out=view)
    assert got.data_ptr() == view.data_ptr()
    _check(view, *_bound(codes, scale, x, b, r, "silu", dtype))
    assert (out[:, :5] == 9).all() and (out[:, 50:] == 9).all()      # nothing beside the rows


@pytest.mark.parametrize("T", [4, 100])
def test_non_finite_row_stays_alone(T):
    codes, scale, x, b, r = _case(T, 128, 30, 8, "f32", False, False, seed=1)
    want, tol = _bound(codes, scale, x, b, r, "none", "f32")
    x = x.clone()
    x[1, 7], x[3, 100] = float("nan"), float("inf")
    y = ops.linear(x.to(DEV), _lin(codes, scale, 8, None))
    keep = [i for i in range(T) if i not in (1, 3)]
    _check(y[keep], want[keep], tol[keep])
    assert torch.isnan(y[1]).all()


def test_no_rows():
    codes, scale, x, b, r = _case(1, 128, 30, 4, "f32", False, False)
    assert ops.linear(torch.empty((0, 128), device=DEV), _lin(codes, scale, 4, None)).shape == (0, 30)


@pytest.mark.parametrize("T", [1, 6, 90])
def test_deterministic_and_captured(T):
    codes, scale, x, b, r = _case(T, 2048, 200, 4, "f32", True, True, seed=2)
    lin, xd, rd = _lin(codes, scale, 4, b), x.to(DEV), r.to(DEV)
    first = ops.linear(xd, lin, "gelu", rd)
    out = torch.empty_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ops.linear(xd, lin, "gelu", rd, out=out)
    for i in range(3):
        out.fill_(float(i))
        g.replay()
        assert torch.equal(out, ops.linear(xd, lin, "gelu", rd)) and torch.equal(out, first)
    xd.mul_(2.0)                                     # the same graph on new contents
    g.replay()
    assert torch.equal(out, ops.linear(xd, lin, "gelu", rd))


def test_two_streams_at_once():
    codes, scale, x, b, r = _case(60, 1024, 300, 4, "f32", False, False, seed=8)
    lin, xd = _lin(codes, scale, 4, None), x.to(DEV)
    want = ops.linear(xd, lin)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(8):
        with torch.cuda.stream(side[i % 2]):
            got.append(ops.linear(xd, lin))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("T", [5, 40, 300])
def test_fp32_sums_keep_their_bits(T, bits):
    """The error's rms, relative to the result's.  The pair drops 2^-22 of a
    product; 2048 columns are 64 additions of 32 products to a partial sum whose rms
    rises to the result's, each within a unit of its last place, 2^-23: at most
    64 * 2^-23 + 2^-22 < 2^-16.9 in all, were they all one way."""
    codes, scale, x, b, r = _case(T, 2048, 512, bits, "f32", False, False, seed=T + bits)
    y = ops.linear(x.to(DEV), _lin(codes, scale, bits, None)).double().cpu().numpy()
    want = aorc.linear(x.double().numpy(), codes, scale, None, "none", None)
    assert np.sqrt(((y - want) ** 2).mean()) <= 2.0 ** -16.9 * np.sqrt((want ** 2).mean())


@pytest.mark.parametrize("T", [1, 40])
def test_columns_of_one_buffer(T):
    """x, residual and out may be columns of one buffer; out over x is refused."""
    codes, scale, x, b, r = _case(T, 128, 64, 4, "f32", True, True, seed=T)
    lin, buf = _lin(codes, scale, 4, b), torch.zeros(T, 256, device=DEV)
    buf[:, :128], buf[:, 192:] = x.to(DEV), r.to(DEV)
    want = ops.linear(x.to(DEV), lin, residual=r.to(DEV))
    ops.linear(buf[:, :128], lin, residual=buf[:, 192:], out=buf[:, 128:192])
    assert torch.equal(buf[:, 128:192], want) and torch.equal(buf[:, :128].cpu(), x)
    for bad in (buf[:, 64:128], buf[:, 96:160]):
        with pytest.raises(ops.MoedecError):
            ops.linear(buf[:, :128], lin, out=bad)
    with pytest.raises(ops.MoedecError):
        ops.linear(x.to(DEV), lin, residual=buf[:, 4:68], out=buf[:, :64])
