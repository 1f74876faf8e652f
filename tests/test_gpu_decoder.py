"""Whole decoder layers: ops.stack_forward with attention over the 4-bit cache
(the projections, the cache, attention, the page calls and the experts together),
against the same stack in float64."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as aorc
from oracle import moe_oracle as orc
from quantized_moe_decode_route_amd import ops, synth

from _attn import DEV, ints, starts

pytestmark = pytest.mark.gpu

HEADS, KV, D, PAGE, SEQS = 4, 2, 64, 32, 4
CFG = synth.CONFIGS["tiny"]
MOE = dict(n_group=CFG.n_group, topk_group=CFG.topk_group, top_k=CFG.top_k, rsf=CFG.rsf)


def _weights(layers):
    rng = np.random.default_rng(3)
    H, out = CFG.hidden, []
    for _ in range(layers):
        ws = []
        for n, k in (((HEADS + 2 * KV) * D, H), (H, HEADS * D)):
            ws.append((rng.integers(-8, 8, (n, k)).astype(np.int8),
                       (rng.uniform(0.5, 1.5, n) / (4.6 * np.sqrt(k))).astype(np.float32),
                       (rng.standard_normal(n) * 0.1).astype(np.float32)))
        out.append(ws)
    return out


def _device(ws):
    lins = [ops.Linear(ops.pack(torch.from_numpy(c).to(DEV), 4), torch.from_numpy(s).to(DEV), 4,
                       torch.from_numpy(b).to(DEV)) for c, s, b in ws]
    return ops.Attention(lins[0], lins[1], HEADS)


class Stack:
    def __init__(self, n_layers, n_pages=40):
        self.n = n_layers
        self.weights = _weights(n_layers)
        self.attn = [_device(w) for w in self.weights]
        self.cache = ops.KvCache.allocate(n_layers, n_pages, PAGE, KV, D, SEQS, 8, DEV)
        self.layers = []
        for l in range(n_layers):
            lay = synth.layer_device(CFG, l, DEV)
            self.layers.append((lay["router_w"], lay["bias"],
                                ops.Experts.from_layer(lay, CFG.n_experts, CFG.n_shared, CFG.bits)))
        self.held = [[([], []) for _ in range(SEQS)] for _ in range(n_layers)]

    def buffers(self, T):
        return [ops.LayerBuffers.allocate(T, CFG.hidden, CFG.inter, CFG.n_experts, CFG.top_k, CFG.n_shared, DEV)
                for _ in range(self.n)]

    def step(self, x, counts, fused=None):
        """counts[s] new tokens of each sequence; returns the stack's output."""
        granted = ops.kv4_reserve(self.cache, ints(counts))
        y = x.clone()
        ops.stack_forward(y, self.layers, self.buffers(x.shape[0]), attn=self.attn, cache=self.cache,
                          q_start=ints(starts(counts)), granted=granted, fused=fused, **MOE)
        return y

    def oracle(self, x, counts):
        """The same in float64, one layer after the other on the values the cache
        holds.  The cache rounds to 4 bits, so a key that sits at a code's border
        may fall either way: callers compare with that in mind."""
        x = x.double().cpu().numpy()
        at = starts(counts)
        for l in range(self.n):
            (cq, sq, bq), (co, so, bo) = self.weights[l]
            qkv = aorc.linear(orc.rmsnorm(x), cq, sq, bq)
            q, k, v = np.split(qkv, [HEADS * D, (HEADS + KV) * D], axis=1)
            o = np.zeros((x.shape[0], HEADS * D))
            for s, m in enumerate(counts):
                if m == 0:
                    continue
                rows = slice(at[s], at[s] + m)
                ks, vs = self.held[l][s]
                ks.append(aorc.cache_values(k[rows].reshape(m, KV, D).astype(np.float32)))
                vs.append(aorc.cache_values(v[rows].reshape(m, KV, D).astype(np.float32)))
                kk, vv = np.concatenate(ks).astype(np.float64), np.concatenate(vs).astype(np.float64)
                o[rows] = aorc.attention(q[rows].reshape(m, HEADS, D), kk, vv, len(kk) - m, D ** -0.5)[0].reshape(m, -1)
            x = x + aorc.linear(o, co, so, bo)
            r = orc.moe_layer(orc.rmsnorm(x).astype(np.float32), synth.router_weight(CFG, l), synth.router_bias(CFG, l),
                              synth.expert_loader(CFG, l), n_shared=CFG.n_shared, bits=CFG.bits, **MOE)
            x = x + r.y
        return x


def _tokens(seed, T):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((T, CFG.hidden)).astype(np.float32)).to(DEV)


@pytest.mark.parametrize("fused", [None, False])
def test_one_layer(fused):
    """One layer: nothing upstream of the cache but the projection, so the only
    freedom is a key or value element that lies at a code's border (fp32 sums of
    256 terms move it by 2^-16 of its size, a step is 2^-3 of the row's largest):
    one such element changes a score by at most a step times |q|, far less than
    the bound, which is a hundredth of the output's size."""
    st = Stack(1)
    for i, counts in enumerate(([5, 0, 9, 1], [1, 1, 1, 0], [3, 2, 0, 1])):
        x = _tokens(10 + i, sum(counts))
        y = st.step(x, counts, fused).double().cpu().numpy()
        want = st.oracle(x, counts)
        assert np.abs(y - want).max() <= 1e-2 * np.abs(want).max()
    assert st.cache.len.tolist() == [9, 3, 10, 2]


def test_forms_agree():
    """The fused and the separate expert calls see the same attention half: the
    same routing, so outputs differ by fp32 rounding only (three layers)."""
    a, b = Stack(3), Stack(3)
    for i, counts in enumerate(([4, 7, 0, 2], [1, 1, 0, 1])):
        x = _tokens(20 + i, sum(counts))
        ya, yb = a.step(x, counts, True), b.step(x, counts, False)
        assert (ya - yb).abs().max() <= 2e-2 * ya.abs().max()


def test_prompt_in_parts_and_token_by_token():
    """A prompt at once, in chunks, and token by token leave the same cache but for
    codes at a border, and the same last output within the 4-bit cache's steps."""
    x = _tokens(30, 12)
    outs = []
    for cuts in ([12], [5, 7], [1] * 12):
        st, at = Stack(2), 0
        for m in cuts:
            y = st.step(x[at:at + m], [m, 0, 0, 0], False)
            at += m
        outs.append(y[-1])
        assert st.cache.len.tolist() == [12, 0, 0, 0]
    for y in outs[1:]:
        assert (y - outs[0]).abs().max() <= 2e-2 * outs[0].abs().max()


def test_padding_and_refused_sequences():
    """Rows behind the last sequence and rows of a sequence without room pass
    through the attention half unchanged but for the bias; others are not touched
    by them."""
    st, full = Stack(1), Stack(1, n_pages=3)
    counts = [3, 2, 0, 0]
    x = _tokens(40, 8)
    g = ops.kv4_reserve(st.cache, ints(counts))
    y = x.clone()
    ops.attention_block(y, st.attn[0], st.cache, 0, ints(starts(counts)), granted=g)
    bias = st.attn[0].out.bias
    assert torch.equal(y[5:], x[5:] + bias)
    alone = x[:5].clone()
    other = Stack(1)
    g = ops.kv4_reserve(other.cache, ints(counts))
    ops.attention_block(alone, other.attn[0], other.cache, 0, ints(starts(counts)), granted=g)
    assert (alone - y[:5]).abs().max() <= 1e-5 * alone.abs().max()
    full.step(_tokens(1, 64), [40, 24, 0, 0])                     # all three pages are taken
    y = _tokens(2, 2)
    keep = y.clone()
    g = ops.kv4_reserve(full.cache, ints([0, 0, 1, 1]))
    assert g.tolist() == [0, 0, 0, 0]
    ops.attention_block(y, full.attn[0], full.cache, 0, ints([0, 0, 0, 1, 2]), granted=g)
    assert torch.equal(y, keep + bias)


def test_verify_and_roll_back():
    """Three drafted tokens verified together, two rejected: the sequence goes on
    as if they had never been there."""
    x = _tokens(50, 10)
    a, b = Stack(2), Stack(2)
    for st in (a, b):
        st.step(x[:6], [6, 0, 0, 0], False)
    a.step(x[6:9], [3, 0, 0, 0], False)                           # x[7:9] turn out wrong
    ops.kv4_truncate(a.cache, ints([7, -1, -1, -1]))
    b.step(x[6:7], [1, 0, 0, 0], False)
    ya, yb = a.step(x[9:], [1, 0, 0, 0], False), b.step(x[9:], [1, 0, 0, 0], False)
    assert a.cache.len.tolist() == b.cache.len.tolist() == [8, 0, 0, 0]
    assert (ya - yb).abs().max() <= 2e-2 * ya.abs().max()


def test_captured_decode():
    """One graph of a whole decode step (pages, attention, experts), replayed as the
    sequences grow past a page, against the eager stack bit for bit."""
    a, b = Stack(2), Stack(2)
    for st in (a, b):
        st.cache.data.zero_()
        st.step(_tokens(60, 32), [30, 2, 0, 0], False)
    counts = [1, 1, 0, 0]
    new, start = ints(counts), ints(starts(counts))
    x, y = _tokens(61, 2), torch.empty((2, CFG.hidden), device=DEV)
    bufs, xn = a.buffers(2), torch.empty((2, CFG.hidden), device=DEV)

    def run():
        y.copy_(x)
        g = ops.kv4_reserve(a.cache, new)
        ops.stack_forward(y, a.layers, bufs, attn=a.attn, cache=a.cache, q_start=start, granted=g, xn=xn,
                          fused=False, check=False, max_len=256, **MOE)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(5):
        x.copy_(_tokens(70 + i, 2))
        graph.replay()
        g = ops.kv4_reserve(b.cache, new)
        want = x.clone()
        ops.stack_forward(want, b.layers, b.buffers(2), attn=b.attn, cache=b.cache, q_start=start, granted=g,
                          fused=False, max_len=256, **MOE)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(a.cache.len, b.cache.len) and torch.equal(a.cache.data, b.cache.data)
    assert a.cache.len.tolist() == [35, 7, 0, 0]


def test_refuses():
    st = Stack(1)
    with pytest.raises(ValueError):
        ops.stack_forward(_tokens(0, 1), st.layers, st.buffers(1), attn=st.attn, **MOE)
    with pytest.raises(ValueError):
        ops.stack_forward(_tokens(0, 1), st.layers, st.buffers(1), attn=st.attn * 2, cache=st.cache,
                          q_start=ints([0, 1, 1, 1, 1]), **MOE)
    with pytest.raises(ValueError):
        bad = ops.Attention(st.attn[0].out, st.attn[0].out, HEADS)
        ops.attention_block(_tokens(0, 1), bad, st.cache, 0, ints([0, 1, 1, 1, 1]))
