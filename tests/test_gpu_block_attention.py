"""Attention of drafted blocks and trees over the paged 8-bit cache (needs a B200).

Against float64. With p the softmax weights, A_old and A_new the weighted sums of
|v| over cached and new tokens and n the tokens of a row, an output may be off by
- 2^-11 A_old + 2^-8 A_new: the weights' rounding to half and to bfloat16,
- n 2^-25 448 max(p v_scale): half's subnormal steps under the largest weight,
- 2 d (A_old + A_new), d the error of a score in nats: D + 8 float32 roundings
  relative to scale |q| . |k| and four of the score in log2 units, in numerator and
  denominator alike; over cached tokens also the queries' two e4m3 parts, which drop
  what is below half a subnormal step, 2^-10, with the row's largest element at
  128 or more, so at most 2^-17 max|q| of each element: 2^-17 scale max|q| sum|k|;
  the same d covers the float32 sums of n <= 2^17 terms by
  16 (tiles and shuffles chain fewer than 2^13 additions of positive terms,
  each rounding a part of the sum) steps of 2^-24 times 2^9,
- half a bfloat16 step of the output.
"""

import math

import pytest
import torch

from tests.eight_bit import FP8

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_decoding_b200 import api as A
    return A


def _cache(api, lens, width, H, page, D, seed, spread=0):
    """A cache for sequences of `lens` tokens; slots behind them hold NaN codes, unused
    table entries an id that is not in the pool."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    B = len(lens)
    N = B * width + 2
    table = torch.randperm(N, generator=g, device=DEV)[:B * width].view(B, width).int()
    c = api.kv_cache(table.contiguous(), N, H, page, D)
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes.copy_((torch.randn(codes.shape, generator=g, device=DEV) * 90).clamp(-448, 448))
        e = torch.randint(-spread, spread + 1, scale.shape, generator=g, device=DEV)
        scale.copy_(2.0 ** (e - 6.5))
    for b, n in enumerate(lens):
        for p in range(width):
            used = min(max(n - p * page, 0), page)
            pid = int(table[b, p])
            for codes in (c.k, c.v):
                codes[pid, :, used:] = math.nan
            if used == 0:
                c.page_table[b, p] = N + 5 if p % 2 else -3
    return c


def _new(B, T, Hq, Hkv, D, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(B, T, h, D, generator=g, device=DEV) * std).bfloat16()
            for h in (Hq, Hkv, Hkv)]


def _parents(B, T, seed):
    g = torch.Generator().manual_seed(seed)
    par = torch.full((B, T), -1, dtype=torch.int32)
    for t in range(1, T):
        lo = max(0, t - 20)
        par[:, t] = torch.randint(lo, t, (B,), generator=g).int()
    return par.to(DEV)


def _see(parent, b, T):
    if parent is None:
        return torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
    m, par = torch.zeros(T, T, dtype=torch.bool), parent[b].tolist()
    for i in range(T):
        j = i
        while j >= 0:
            m[i, j] = True
            j = par[j] if par[j] < j else -1
    return m.to(DEV)


def _check(out, q, k, v, c, lens, parent=None, num_new=None, scale=None):
    B, T, Hq, D = q.shape
    H, page = k.shape[2], c.k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        n = int(lens[b])
        nn = T if num_new is None else max(0, min(T, int(num_new[b])))
        pages = c.page_table[b, :-(-n // page)].long()
        see = _see(parent, b, T)
        for h in range(H):
            def old(codes, s):
                return (codes[pages, h].double() * s[pages, h].double()[:, None, None]
                        ).reshape(-1, D)[:n]

            vs = c.v_scale[pages, h].double().repeat_interleave(page)[:n]
            # rows that see a non-finite value come out non-finite, the others must not:
            # `see` picks the tokens before anything is multiplied
            kk, vv = torch.cat([old(c.k, c.k_scale), k[b, :, h].double()]), \
                torch.cat([old(c.v, c.v_scale), v[b, :, h].double()])
            for i in range(nn):
                on = torch.cat([torch.ones(n, dtype=torch.bool, device=DEV), see[i]])
                K, V, m = kk[on], vv[on], int(on.sum()) - n
                Q = q[b, i, h * (Hq // H):(h + 1) * (Hq // H)].double()
                z = Q @ K.t() * scale
                p = torch.softmax(z, 1)
                ref, got = p @ V, out[b, i, h * (Hq // H):(h + 1) * (Hq // H)].double()
                a_old, a_new = p[:, :n] @ V[:n].abs(), p[:, n:] @ V[n:].abs()
                mag = (Q.abs() @ K.abs().t()).amax(1, keepdim=True) * abs(scale)
                d = (D + 8) * 2.0 ** -24 * mag + 4 * 2.0 ** -24 * z.abs().amax(1, keepdim=True) \
                    + 2.0 ** -11 * 2.0 ** -1
                if n:
                    d = d + 2.0 ** -17 * abs(scale) * Q.abs().amax(1, keepdim=True) * \
                        K[:n].abs().sum(1).amax()
                top = torch.cat([p[:, :n] * vs, p[:, n:]], 1).amax(1, keepdim=True)
                tol = 2.0 ** -11 * a_old + 2.0 ** -8 * a_new + (n + m) * 2.0 ** -25 * 448 * top \
                    + 2 * d * (a_old + a_new) + 2.0 ** -8 * ref.abs() + 1e-38
                bad = ~((got - ref).abs() <= tol)
                assert not bad.any(), (b, h, i, float(((got - ref).abs() / tol).max()))


def _run(api, lens, T, Hq, H, D, page, seed, tree=False, nodes=None, spread=0, scale=None,
         q_std=1.0):
    B, width = len(lens), max(1, -(-max(lens) // page))
    c = _cache(api, lens, width, H, page, D, seed, spread)
    q, k, v = _new(B, T, Hq, H, D, seed + 1)
    q = q * q_std
    parent = _parents(B, T, seed) if tree else None
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    nn = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    got = api.block_attention(q, k, v, c, ln, parent=parent, num_new=nn, scale=scale, out=out)
    torch.cuda.synchronize()
    assert got is out and api.device_fault_flags() == 0
    _check(out, q, k, v, c, lens, parent, nodes, scale)
    if nodes is not None:
        for b, n in enumerate(nodes):
            assert torch.all(out[b, max(0, n):] == 7.0)
    return q, k, v, c, ln, out


LENS = [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 700, 1023]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 4), (2, 5), (5, 4), (17, 2), (9, 8)])
def test_blocks_of_a_ragged_batch(api, D, page, T, G):
    _run(api, LENS, T, 2 * G, 2, D, page, seed=T * G + page)


@pytest.mark.parametrize("T,G", [(1, 16), (1, 17), (8, 4), (3, 11), (16, 4), (17, 4), (20, 4),
                                 (21, 4), (33, 4), (70, 2), (1, 80), (1, 81), (1, 130)])
def test_row_tiles(api, T, G):
    _run(api, [130, 7, 64], T, 3 * G, 3, 128, 64, seed=T + G)
    _run(api, [65, 0], T, G, 1, 64, 16, seed=T + G)


@pytest.mark.parametrize("T,G,D", [(17, 4, 128), (65, 2, 64), (241, 4, 128), (300, 1, 128)])
def test_trees(api, T, G, D):
    _run(api, [200, 0, 77], T, 2 * G, 2, D, 32, seed=T, tree=True, nodes=[T, T // 2, 1])
    _run(api, [513], T, G, 1, D, 64, seed=T + 1, tree=True)


def test_rows_behind_the_last_are_left(api):
    _run(api, [100, 64, 3, 0], 9, 8, 2, 128, 16, seed=5, nodes=[9, 0, 1, 4])
    _run(api, [100, 64], 9, 8, 2, 128, 16, seed=5, nodes=[0, 0])


@pytest.mark.parametrize("lens,H,T", [([70000], 1, 1), ([70000], 2, 17), ([33000, 1, 40], 1, 9)])
def test_long_caches_split_over_many_ctas(api, lens, H, T):
    _run(api, lens, T, 4 * H, H, 128, 128, seed=7)


def test_many_short_sequences(api):
    _run(api, [(37 * i) % 200 for i in range(150)], 2, 4, 1, 64, 16, seed=8)


def test_more_sequences_than_a_cta_keeps_in_shared_memory(api):
    """Their sizes are then read from memory; most sequences here are empty or unused."""
    B = 1100
    lens = [0] * B
    nodes = [0] * B
    for b in (0, 31, 32, 511, 512, 513, 700, 1099):
        lens[b], nodes[b] = 20 + b % 37, 1 + b % 2
    _run(api, lens, 2, 4, 1, 64, 32, seed=40, nodes=nodes)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_non_finite_query_row_stays_alone(api, bad):
    lens = [200, 0]
    c = _cache(api, lens, 4, 2, 64, 128, seed=41)
    q, k, v = _new(2, 5, 8, 2, 128, 42)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean = api.block_attention(q, k, v, c, ln)
    q[0, 2, 3, 17] = q[1, 4, 6, 0] = bad
    out = api.block_attention(q, k, v, c, ln)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 2, 3]).all() and torch.isnan(out[1, 4, 6]).all()
    keep = torch.ones(2, 5, 8, dtype=torch.bool, device=DEV)
    keep[0, 2, 3] = keep[1, 4, 6] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("spread", [3, 20])
def test_value_scales_of_very_different_pages(api, spread):
    _run(api, [1000, 300], 3, 4, 2, 128, 16, seed=9, spread=min(spread, 3))
    # value scales alone over 40 binades
    lens = [1000, 300]
    c = _cache(api, lens, 63, 2, 16, 128, seed=10)
    g = torch.Generator(device=DEV).manual_seed(11)
    c.v_scale.copy_(2.0 ** torch.randint(-spread, spread + 1, c.v_scale.shape, generator=g,
                                         device=DEV))
    q, k, v = _new(2, 3, 4, 2, 128, 12)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v, c, ln)
    _check(out, q, k, v, c, lens)


@pytest.mark.parametrize("q_std,scale", [(0.0, None), (1e-30, None), (30.0, None), (1.0, 0.0),
                                         (1.0, -0.3), (1e4, 1e-5)])
def test_scores_of_every_size(api, q_std, scale):
    _run(api, [500, 3], 4, 8, 2, 128, 64, seed=13, q_std=q_std, scale=scale)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_new_tokens_reach_only_rows_that_see_them(api, bad, tree):
    B, T, H, G, D = 2, 24, 2, 4, 128
    lens = [70, 0]
    c = _cache(api, lens, 2, H, 64, D, seed=14)
    q, k, v = _new(B, T, H * G, H, D, 15)
    parent = _parents(B, T, 16) if tree else None
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean = api.block_attention(q, k, v, c, ln, parent=parent)
    v[0, 5, 1, 17] = bad
    k[1, 9, 0, 3] = math.nan
    out = api.block_attention(q, k, v, c, ln, parent=parent)
    torch.cuda.synchronize()
    for b, tok, h in ((0, 5, 1), (1, 9, 0)):
        sees = _see(parent, b, T)[:, tok]
        for i in range(T):
            rows = slice(h * G, (h + 1) * G)
            if not sees[i]:
                assert torch.isfinite(out[b, i, rows]).all()
            elif b == 0:
                x = out[b, i, rows, 17].float()
                assert torch.isnan(x).all() if math.isnan(bad) else torch.all(x == bad)
                keep = torch.arange(D, device=DEV) != 17
                assert torch.isfinite(out[b, i, rows][:, keep]).all()
            else:
                assert torch.isnan(out[b, i, rows]).all()
        other = slice(0, G) if h else slice(G, 2 * G)
        assert torch.equal(out[b, :, other], clean[b, :, other])


def test_bad_lengths_and_pages_make_their_sequences_nan(api):
    lens = [100, 100, 100, 100, 100, 20]
    c = _cache(api, lens, 8, 2, 16, 64, seed=17)
    q, k, v = _new(6, 3, 4, 2, 64, 18)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = api.block_attention(q, k, v, c, ln)
    ln[1], ln[2] = -1, 129
    c.page_table[3, 6], c.page_table[4, 0] = -1, c.k.shape[0]
    out = api.block_attention(q, k, v, c, ln)
    torch.cuda.synchronize()
    assert torch.isnan(out[1:5]).all()
    _check(out[:1], q[:1], k[:1], v[:1], c, lens[:1])
    assert torch.isfinite(out[5]).all() and torch.isfinite(want).all()


def test_an_empty_pool(api):
    table = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    c = api.kv_cache(table, 0, 2, 64, 128)
    q, k, v = _new(2, 5, 8, 2, 128, 19)
    ln = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v, c, ln)
    torch.cuda.synchronize()
    _check(out, q, k, v, c, [0, 0])
    ln[1] = 1
    out = api.block_attention(q, k, v, c, ln)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all()


def test_codes_behind_the_32_bit_offset(api):
    H, page, D = 8, 128, 128
    N = (1 << 31) // (H * page * D) + 3
    c = api.kv_cache(torch.tensor([[N - 1, N - 2]], dtype=torch.int32, device=DEV), N, H, page, D)
    small = api.kv_cache(torch.tensor([[2, 1]], dtype=torch.int32, device=DEV), 3, H, page, D)
    q, k, v = _new(1, 200, 16, H, D, 20)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for x in (c, small):
        api.kv_append(x, k, v, z)
        outs.append(api.block_attention(q[:, :2].contiguous(), k[:, :2].contiguous(),
                                        v[:, :2].contiguous(), x, z + 200))
    assert torch.equal(outs[0], outs[1])


def test_empty_calls_and_refusals(api):
    c = _cache(api, [20, 20], 2, 2, 16, 64, seed=21)
    q, k, v = _new(2, 3, 4, 2, 64, 22)
    ln = torch.tensor([20, 20], dtype=torch.int32, device=DEV)
    assert api.block_attention(q[:, :0], k[:, :0], v[:, :0], c, ln).shape == (2, 0, 4, 64)
    with pytest.raises(TypeError):
        api.block_attention(q.float(), k, v, c, ln)
    with pytest.raises(TypeError):
        api.block_attention(q, k, v, c, ln.long())
    with pytest.raises(ValueError):
        api.block_attention(q, k, v, c, ln[:1])
    with pytest.raises(ValueError):
        api.block_attention(q, k[:, :2], v[:, :2], c, ln)
    with pytest.raises(ValueError):
        api.block_attention(q, k, v, c, ln, parent=ln)
    with pytest.raises(ValueError):
        api.block_attention(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), c, ln)
    with pytest.raises(api.UnoError):
        api.block_attention(q[:, :, :3].contiguous(), k, v, c, ln)  # 3 heads over 2
    with pytest.raises(api.UnoError):
        api.block_attention(q, k, v, c, ln, scale=math.inf)
    with pytest.raises(api.UnoError):
        api.block_attention(q, k, v, c, ln, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_streams_and_captured_graphs(api):
    """Lengths are read on the device: a captured call follows them. Two streams, and two
    graphs replayed side by side, share nothing."""
    jobs = []
    for i, (T, page) in enumerate(((1, 16), (17, 64))):
        lens = [300, 41, 1000]
        c = _cache(api, lens, -(-1000 // page), 2, page, 128, seed=23 + i)
        q, k, v = _new(3, T, 8, 2, 128, 24 + i)
        jobs.append((q, k, v, c, torch.tensor(lens, dtype=torch.int32, device=DEV)))
    want = [api.block_attention(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(10):
        for i, j in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(api.block_attention(*j))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(w, g) for g in gs)
    graphs, outs = [], []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.block_attention(*j))
        graphs.append(g)
    for short in (False, True):
        if short:
            for j in jobs:
                j[4].copy_(torch.tensor([7, 0, 999], dtype=torch.int32))
        want = [api.block_attention(*j) for j in jobs]
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert torch.equal(w, o)


def test_append_then_attend_equals_attending_with_the_rows_as_new(api):
    """A block verified, its accepted rows appended, the next block verified: the run of a
    decode step, against float64 over the cache's own values."""
    B, T, H, G, D, page = 3, 6, 2, 4, 128, 16
    table = torch.randperm(3 * 6, device=DEV).view(3, 6).int()
    c = api.kv_cache(table, 18, H, page, D)
    lens = [0, 0, 0]
    accepted = [[6, 3, 1], [6, 6, 6], [2, 0, 5], [6, 1, 6]]
    for step, acc in enumerate(accepted):
        q, k, v = _new(B, T, H * G, H, D, 30 + step)
        ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
        out = api.block_attention(q, k, v, c, ln)
        torch.cuda.synchronize()
        _check(out, q, k, v, c, lens)
        api.kv_append(c, k, v, ln, count=torch.tensor(acc, dtype=torch.int32, device=DEV))
        lens = [n + a for n, a in zip(lens, acc)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 2), (1, 3), (3, 1), (1, 5), (1, 7), (2, 4), (1, 8), (3, 3),
                                 (1, 9), (5, 3), (4, 4), (2, 8), (1, 18)])
def test_few_rows(api, T, G, D):
    """Row counts around those at which the layout of a tile changes."""
    _run(api, [900, 1, 0, 333, 128], T, 2 * G, 2, D, 32, seed=40 * T + G)
    _run(api, [260, 5, 77], T, G, 1, D, 128, seed=50 * T + G, nodes=[0, T, max(T - 1, 1)], tree=T > 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 4), (2, 4), (1, 8), (4, 4), (2, 16), (17, 4)])
def test_scores_that_grow_along_the_cache(api, T, G, D):
    """The maximum moves again and again: a row's largest scores are in its last pages."""
    lens, width, page = [2300, 640, 129], 36, 64
    c = _cache(api, lens, width, 1, page, D, 60 + T)
    for b in range(len(lens)):
        for p in range(-(-lens[b] // page)):
            c.k_scale[int(c.page_table[b, p])] = 2.0 ** (-9 + p // 4)
    q, k, v = _new(len(lens), T, G, 1, D, 61 + T, 0.5)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v, c, ln)
    assert api.device_fault_flags() == 0
    _check(out, q, k, v, c, lens)


def _check_whole(out, q, k, v, c, lens):
    """As _check, for blocks of finite values: a sequence's rows and heads at once."""
    B, T, Hq, D = q.shape
    H, page = k.shape[2], c.k.shape[2]
    scale = D ** -0.5
    for b in range(B):
        n = int(lens[b])
        pages = c.page_table[b, :-(-n // page)].long()

        def old(codes, s):  # [H, n, D]
            x = codes[pages].double() * s[pages].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(H, -1, D)[:, :n]

        K = torch.cat([old(c.k, c.k_scale), k[b].double().transpose(0, 1)], 1)
        V = torch.cat([old(c.v, c.v_scale), v[b].double().transpose(0, 1)], 1)
        vs = c.v_scale[pages].double().t().repeat_interleave(page, 1)[:, None, :n]
        Q = q[b].double().view(T, H, Hq // H, D).permute(1, 0, 2, 3).reshape(H, -1, D)
        see = torch.cat([torch.ones(T, n, dtype=torch.bool, device=DEV),
                         _see(None, b, T)], 1).repeat_interleave(Hq // H, 0)
        z = (Q @ K.transpose(1, 2) * scale).masked_fill(~see, -math.inf)
        p = torch.softmax(z, 2)
        ref = p @ V
        got = out[b].double().view(T, H, Hq // H, D).permute(1, 0, 2, 3).reshape(H, -1, D)
        a_old, a_new = p[..., :n] @ V[:, :n].abs(), p[..., n:] @ V[:, n:].abs()
        mag = (Q.abs() @ K.abs().transpose(1, 2)).masked_fill(~see, 0).amax(2, keepdim=True) * scale
        big = z.masked_fill(~see, 0).abs().amax(2, keepdim=True)
        d = (D + 8) * 2.0 ** -24 * mag + 4 * 2.0 ** -24 * big + 2.0 ** -11 * 2.0 ** -1
        if n:
            d = d + 2.0 ** -17 * scale * Q.abs().amax(2, keepdim=True) * \
                K[:, :n].abs().sum(2).amax(1)[:, None, None]
        top = torch.cat([p[..., :n] * vs, p[..., n:]], 2).amax(2, keepdim=True)
        tol = 2.0 ** -11 * a_old + 2.0 ** -8 * a_new + (n + T) * 2.0 ** -25 * 448 * top \
            + 2 * d * (a_old + a_new) + 2.0 ** -8 * ref.abs() + 1e-38
        bad = ~((got - ref).abs() <= tol)
        assert not bad.any(), (b, float(((got - ref).abs() / tol).max()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 4), (1, 16), (5, 4), (8, 4), (9, 4), (16, 4), (17, 4)])
def test_many_sequences_of_one_tile(api, T, G, D):
    """A CTA goes through several items in a row that have a single tile each: the queries of
    one may not be replaced before every warp has taken them."""
    lens = [1 + 37 * b % 128 for b in range(200)]
    c = _cache(api, lens, 1, 4, 128, D, seed=70 + T)
    q, k, v = _new(200, T, 4 * G, 4, D, 71 + T)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v, c, ln)
    torch.cuda.synchronize()
    assert api.device_fault_flags() == 0
    _check_whole(out, q, k, v, c, lens)


@pytest.mark.parametrize("T,G,D", [(1, 3, 64), (1, 8, 128), (2, 8, 64), (5, 4, 128),
                                   (10, 4, 64), (20, 4, 128)])
@pytest.mark.parametrize("n,at", [(100000, 0), (131072, 131071), (262145, 7)])
def test_a_dominating_token_of_value_zero(api, T, G, D, n, at):
    """One cached token has 99% of the weight and value 0: the output is what the others,
    each of a weight of 1 / (99 n) of that token's, add up to. More sequences (of the same
    pages) than CTAs, so that hardly one is split into parts with maxima of their own.

    Relative bound, all values being positive: half a bfloat16 step of the output (2^-8),
    the weights' rounding to half with the largest scaled to 2^9 or more (2^-11, or half
    of a subnormal step, 2^-25 of 2^9 / (99 n)), twice the error of the dominating score
    s < 18 in nats ((D + 8) 2^-24 s, 4 * 2^-24 s and the query parts' 2^-17 s: one element
    of the key is not 0), and float32 sums, 2^-11 as above.
    """
    B, page, width = 200, 128, -(-n // 128)
    g = torch.Generator(device=DEV).manual_seed(n + T)
    table = torch.randperm(width, generator=g, device=DEV).int().repeat(B, 1)
    c = api.kv_cache(table, width, 1, page, D)
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(0.5)
    # 1 to 2 in steps of e4m3
    c.v.copy_(1 + torch.randint(0, 9, c.v.shape, generator=g, device=DEV) / 8)
    pid, slot = int(table[0, at // page]), at % page
    c.k[pid, 0, slot, 0] = 16.0
    c.v[pid, 0, slot] = 0.0
    q, k, v = _new(B, T, G, 1, D, 90)
    q.zero_()
    q[..., 0] = math.log(99 * n) / 16
    s = float(q[0, 0, 0, 0]) * 16  # as rounded
    k.zero_()
    k[..., 0] = -16.0  # the new tokens' weights are (99 n)^-2 of the dominating one's
    ln = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v.abs(), c, ln, scale=1.0)
    assert api.device_fault_flags() == 0
    vals = (c.v[table[0].long(), 0].double() * 0.5).reshape(-1, D)[:n].sum(0)
    off = out.double() / (vals / (math.exp(s) + (n - 1))) - 1
    tol = 2.0 ** -8 + max(2.0 ** -11, 99 * n * 2.0 ** -34) + \
        2 * 18 * ((D + 12) * 2.0 ** -24 + 2.0 ** -17) + 2.0 ** -11
    assert float(off.abs().max()) <= tol


@pytest.mark.parametrize("T,n,D,G", [(1000, 0, 128, 2), (1021, 4000, 64, 4), (4096, 0, 64, 1),
                                     (4096, 4001, 128, 1)])
def test_blocks_up_to_the_longest(api, T, n, D, G):
    lens = [n, 17]
    c = _cache(api, lens, max(1, -(-n // 64)), 1, 64, D, seed=100 + T)
    q, k, v = _new(2, T, G, 1, D, 101 + n)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v, c, ln)
    assert api.device_fault_flags() == 0
    _check_whole(out, q, k, v, c, lens)
    # a tree that is one chain is the same block
    chain = (torch.arange(T, device=DEV) - 1).int().repeat(2, 1)
    assert torch.equal(api.block_attention(q, k, v, c, ln, parent=chain), out)


def test_as_many_sequences_as_are_accepted(api):
    B, page, D = 65535, 16, 64
    g = torch.Generator(device=DEV).manual_seed(110)
    c = api.kv_cache(torch.randint(0, 300, (B, 2), generator=g, device=DEV).int(), 300, 1, page, D)
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes.copy_((torch.randn(codes.shape, generator=g, device=DEV) * 90).clamp(-448, 448))
        scale.fill_(2.0 ** -6)
    q, k, v = _new(B, 1, 1, 1, D, 111)
    lens = [b % 33 for b in range(B)]
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = api.block_attention(q, k, v, c, ln)
    assert api.device_fault_flags() == 0
    some = list(range(0, B, 997)) + [B - 2, B - 1]
    sub = api.KvCache(c.k, c.v, c.k_scale, c.v_scale, c.page_table[some].contiguous())
    _check_whole(out[some], q[some], k[some], v[some], sub, [lens[b] for b in some])
