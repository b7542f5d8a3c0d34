"""The 8-bit operators in a run, as a decode step uses them (needs a B200).

A small decoder layer in front of an LM head, its projections in 8 bits on both
pathways: norm -> q, k, v -> attention over the 8-bit cache -> quantised rows -> o ->
residual and norm -> LM head -> drafts, verification -> the accepted rows into the
cache. Every operator is checked against float64 on the inputs it got in the run,
with the bounds of its own tests; the run repeats bit for bit, and as a captured graph.
"""

import pytest
import torch

import tests.test_gpu_block_attention as attention
import tests.test_gpu_dualpath_int8 as linear
import tests.test_gpu_row_quant as rows
from tests.eight_bit import kv_append, rms_norm, same_codes

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B, K, HID, HQ, HKV, D, V, R, PAGE = 3, 4, 320, 4, 2, 64, 1003, 32, 16
T = K + 1


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_decoding_b200 import api as A
    return A


def _projection(api, d_in, d_out, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def w(n, d, std):
        return (torch.randn(n, d, generator=g, device=DEV) * std).bfloat16()

    Wq, ws = api.quantize_rows(w(d_out, d_in, d_in ** -0.5))
    Aq, as_ = api.quantize_rows(w(R, d_in, d_in ** -0.5))
    return dict(Wq=Wq, w_scale=ws, Aq=Aq, a_scale=as_, Bm=w(d_out, R, 0.05), scale=2.0)


class Layer:
    def __init__(self, api):
        self.api = api
        names = {"q": (HID, HQ * D), "k": (HID, HKV * D), "v": (HID, HKV * D), "o": (HQ * D, HID),
                 "head": (HID, V)}
        self.p = {n: _projection(api, i, o, seed) for seed, (n, (i, o)) in enumerate(names.items())}
        g = torch.Generator(device=DEV).manual_seed(9)
        self.embed = (torch.randn(V, HID, generator=g, device=DEV)).bfloat16()
        self.w = [(1 + 0.1 * torch.randn(HID, generator=g, device=DEV)).bfloat16()
                  for _ in range(2)]
        # the first row of a block is on the AR weights alone
        self.gate = (torch.arange(B * T, device=DEV) % T != 0).to(torch.uint8)
        table = torch.randperm(B * 4, generator=torch.Generator().manual_seed(1))
        self.table = table.view(B, 4).int().to(DEV)

    def cache(self):
        return self.api.kv_cache(self.table, B * 4, HKV, PAGE, D)

    def forward(self, tokens, cache, lens):
        """Logits of both pathways, the new keys and values, and what each operator got."""
        api, seen = self.api, {}

        def lin(name, q, s):
            y = api.dualpath_linear_int8(q, s, gate=self.gate, **self.p[name])
            seen[name] = (q, s, y)
            return y[1]

        x = self.embed[tokens.long().flatten()]
        n = api.rms_norm(x, self.w[0], 1e-6)
        seen["norm0"] = (x, None, n)
        q, k, v = (lin(m, n.q, n.scale).view(B, T, -1, D) for m in "qkv")
        o = api.block_attention(q, k, v, cache, lens)
        seen["attention"] = (q, k, v, o)
        oq, os = api.quantize_rows(o.view(B * T, HQ * D))
        seen["quantize"] = (o, oq, os)
        n1 = api.rms_norm(lin("o", oq, os), self.w[1], 1e-6, residual=n.h)
        seen["norm1"] = (seen["o"][2][1], n.h, n1)
        lin("head", n1.q, n1.scale)
        return seen["head"][2], k, v, seen


def _check(layer, seen, cache, lens):
    for name in ("q", "k", "v", "o", "head"):
        xq, xs, (ya, yd) = seen[name]
        linear._check(ya, yd, dict(xq=xq, x_scale=xs, **layer.p[name]), torch.bfloat16, layer.gate)
    for name, w in (("norm0", layer.w[0]), ("norm1", layer.w[1])):
        x, res, got = seen[name]
        h, y, scale = rms_norm(x, w, 1e-6, res)
        assert torch.equal(got.h.cpu(), h)
        rows._check_q(got.q, got.scale, y, scale)
    o, oq, os = seen["quantize"]
    o = o.reshape(B * T, HQ * D).cpu().double()
    rows._check_q(oq, os, o, o.abs().amax(1) / 127)
    q, k, v, out = seen["attention"]
    attention._check(out, q, k, v, cache, lens.tolist())


def test_decode_steps(api):
    layer = Layer(api)

    def run(check):
        cache, lens = layer.cache(), torch.zeros(B, dtype=torch.int32, device=DEV)
        tokens = torch.arange(B * T, device=DEV).view(B, T) % V
        trace = []
        for step in range(6):
            (p, q), k, v, seen = layer.forward(tokens, cache, lens)
            if check:
                torch.cuda.synchronize()
                _check(layer, seen, cache, lens)
            # drafts of the block from its own draft rows, verified by its AR rows
            q = q.view(B, T, V)[:, :K].contiguous()
            drafts = api.sample_drafts(q, 5, step)
            res = api.verify_block(p.view(B, T, V), q, drafts, 5, step)
            count = res.accepted_len + 1
            before = [t.clone() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
            api.kv_append(cache, k, v, lens, count=count)
            if check:
                torch.cuda.synchronize()
                for c, s, new, (gc, gs) in ((before[0], before[1], k, (cache.k, cache.k_scale)),
                                            (before[2], before[3], v, (cache.v, cache.v_scale))):
                    wc, ws = kv_append(c, s, new, cache.page_table, lens, count)
                    assert torch.equal(gs.cpu(), ws) and same_codes(gc, wc)
            lens = lens + count
            tokens = torch.cat([res.out_tokens.gather(1, res.accepted_len[:, None].long()),
                                drafts], 1)
            trace.append((p, q, lens, tokens, cache.k.clone().view(torch.uint8), cache.v_scale.clone()))
        torch.cuda.synchronize()
        assert api.device_fault_flags() == 0
        return trace

    a, b = run(True), run(False)
    assert int(a[-1][2].min()) >= 6  # every step keeps at least its first token
    for x, y in zip(a, b):
        assert all(torch.equal(s, t) for s, t in zip(x, y))


def test_a_captured_step(api):
    """One step as a graph, replayed while lengths, tokens and cache move on."""
    layer = Layer(api)
    eager, graph = layer.cache(), layer.cache()
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    tokens = torch.arange(B * T, device=DEV).view(B, T) % V
    count = torch.tensor([1, 5, 3], dtype=torch.int32, device=DEV)

    def step(cache):
        (p, q), k, v, _ = layer.forward(tokens, cache, lens)
        api.kv_append(cache, k, v, lens, count=count)
        return p, q

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(layer.cache())
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(graph)
    for t in (graph.k, graph.v, graph.k_scale, graph.v_scale):
        t.zero_()
    for i in range(6):
        g.replay()
        want = step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        for n in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(eager, n).view(torch.uint8), getattr(graph, n).view(torch.uint8))
        lens += count
        tokens.copy_((tokens * 7 + i) % V)


def test_a_trees_accepted_path(api):
    """Nodes of the tree sampler attended by their parents, an accepted path appended by rows."""
    q = torch.randn(2, 3, 500, device=DEV)
    tree = api.tree_draft(q, top_k=2, budget=3)
    N = api.tree_nodes(3, 3)
    table = torch.arange(4, device=DEV).view(2, 2).int()
    cache = api.kv_cache(table, 4, HKV, PAGE, D)
    qs, k, v = attention._new(2, N, HQ, HKV, D, 3)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    api.kv_append(cache, k, v, lens, count=torch.full_like(lens, 7))
    lens = lens + 7
    out = api.block_attention(qs, k, v, cache, lens, parent=tree.node_parent, num_new=tree.n_nodes)
    torch.cuda.synchronize()
    nodes = tree.n_nodes.tolist()
    attention._check(out, qs, k, v, cache, [7, 7], tree.node_parent, nodes)
    # the chain from the last node up, root first
    par = tree.node_parent.cpu()
    paths = []
    for b in range(2):
        path, n = [], nodes[b] - 1
        while n >= 0:
            path.insert(0, n)
            n = int(par[b, n])
        paths.append(path + [0] * (N - len(path)))
    path = torch.tensor(paths, dtype=torch.int32)
    count = torch.tensor([p.index(nodes[b] - 1) + 1 for b, p in enumerate(paths)], dtype=torch.int32)
    want = kv_append(cache.k, cache.k_scale, k, table, lens, count, path)
    api.kv_append(cache, k, v, lens, count=count.to(DEV), rows=path.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(cache.k_scale.cpu(), want[1]) and same_codes(cache.k, want[0])
