"""Appends to the paged 8-bit cache (need a B200).

Scales are powers of two and the codes' rounding is exact arithmetic, so every
byte has to equal the float64 form's.
"""

import math

import pytest
import torch

from tests.eight_bit import FP8, kv_append, same_codes

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_decoding_b200 import api as A
    return A


def _cache(api, B, width, H, page, D, seed, spare=2):
    """A cache with random pages; its table uses them in random order."""
    g = torch.Generator().manual_seed(seed)
    N = B * width + spare
    c = api.kv_cache(torch.randperm(N, generator=g)[:B * width].view(B, width).int().to(DEV),
                     N, H, page, D)
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes.copy_((torch.randn(codes.shape, generator=g) * 100).clamp(-448, 448).to(FP8))
        scale.copy_(2.0 ** torch.randint(-9, -5, scale.shape, generator=g).float())
    return c


def _new(B, T, H, D, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(B, T, H, D, generator=g) * std).bfloat16() for _ in range(2)]


def _run(api, c, k, v, start, count=None, rows=None):
    want = [kv_append(codes, s, x, c.page_table, start, count, rows)
            for codes, s, x in ((c.k, c.k_scale, k), (c.v, c.v_scale, v))]

    def dev(t):
        return None if t is None else torch.as_tensor(t, dtype=torch.int32, device=DEV)

    api.kv_append(c, k.to(DEV), v.to(DEV), dev(start), count=dev(count), rows=dev(rows))
    torch.cuda.synchronize()
    for (codes, s), (wc, ws) in zip(((c.k, c.k_scale), (c.v, c.v_scale)), want):
        assert torch.equal(s.cpu(), ws)
        assert same_codes(codes, wc)


@pytest.mark.parametrize("page,D,H", [(16, 64, 1), (32, 128, 3), (64, 128, 8), (128, 64, 2),
                                      (128, 128, 1)])
@pytest.mark.parametrize("T", [1, 5, 17, 150])
def test_append(api, page, D, H, T):
    B, width = 4, -(-(3 * page + T) // page)
    c = _cache(api, B, width, H, page, D, seed=page + T)
    start = torch.tensor([0, 1, page - 1, 2 * page + 3])
    k, v = _new(B, T, H, D, seed=T)
    k[1] *= 100  # the scale grows: the page's earlier tokens move
    v[2] *= 1e-3  # it does not
    _run(api, c, k, v, start)
    _run(api, c, *_new(B, T, H, D, seed=T + 1), start, count=torch.tensor([T, 0, T // 2, T + 9]))


def test_calls_in_pieces_equal_one_call(api):
    """Cut into calls of 1, 6 and 33 tokens a prompt leaves the same scales, and the same codes
    but for those that a growing scale has moved into e4m3's subnormal range."""
    k, v = _new(2, 40, 2, 64, seed=3)
    table = torch.tensor([[0, 1, 2], [5, 4, 3]], dtype=torch.int32, device=DEV)
    one, cut = (api.kv_cache(table, 6, 2, 16, 64) for _ in range(2))
    api.kv_append(one, k.to(DEV), v.to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV))
    at = 0
    for n in (1, 6, 33):
        api.kv_append(cut, k[:, at:at + n].contiguous().to(DEV),
                      v[:, at:at + n].contiguous().to(DEV),
                      torch.full((2,), at, dtype=torch.int32, device=DEV))
        at += n
    assert torch.equal(one.k_scale, cut.k_scale) and torch.equal(one.v_scale, cut.v_scale)
    a, b = one.k.cpu().float(), cut.k.cpu().float()
    # half a subnormal step (2^-9 / 2) for each of the two roundings that may differ
    assert torch.all((a == b) | ((a - b).abs() <= 2.0 ** -9) & (a.abs() < 2.0 ** -5))


def test_rows_of_a_tree(api):
    c = _cache(api, 3, 4, 2, 16, 128, seed=9)
    k, v = _new(3, 29, 2, 128, seed=9)
    rows = torch.tensor([[0, 3, 7, 28], [0, 1, 1, 2], [0, 29, -1, 5]])
    _run(api, c, k, v, torch.tensor([14, 3, 40]), count=torch.tensor([4, 2, 4]), rows=rows)


def test_zeros_infinities_and_nan(api):
    c = _cache(api, 3, 2, 2, 16, 64, seed=11)
    k, v = _new(3, 6, 2, 64, seed=11)
    k[0] = 0
    k[1, 2, 0, 5], k[1, 3, 0, 6], k[1, 4, 1, 7] = math.inf, -math.inf, math.nan
    v[2] = torch.finfo(torch.bfloat16).max
    v[1] = math.nan
    k[2] = 2.0 ** -133  # a subnormal bfloat16: the scale stops at 2^-126
    _run(api, c, k, v, torch.tensor([0, 0, 0]))
    _run(api, c, *_new(3, 6, 2, 64, seed=12), torch.tensor([6, 6, 6]))


def test_what_is_skipped(api):
    """Starts below zero and past the table, tokens past its end, page ids outside the pool."""
    c = _cache(api, 5, 2, 1, 16, 64, seed=13)
    c.page_table[3, 0] = -1
    c.page_table[4, 1] = c.k.shape[0]
    k, v = _new(5, 20, 1, 64, seed=13)
    _run(api, c, k, v, torch.tensor([-1, 33, 25, 0, 3]))
    _run(api, c, k, v, torch.tensor([-2 ** 31, 2 ** 31 - 1, 32, 16, 16]),
         count=torch.tensor([20, 20, 20, -5, 2 ** 31 - 1]))


def test_empty_calls(api):
    c = _cache(api, 2, 2, 1, 16, 64, seed=14)
    before = c.k.clone()
    z = torch.zeros(2, dtype=torch.int32, device=DEV)
    e = torch.empty(2, 0, 1, 64, dtype=torch.bfloat16, device=DEV)
    api.kv_append(c, e, e, z)
    c0 = api.KvCache(c.k, c.v, c.k_scale, c.v_scale, c.page_table[:0])
    api.kv_append(c0, e[:0], e[:0], z[:0])
    assert torch.equal(before.view(torch.uint8), c.k.view(torch.uint8))


def test_codes_behind_the_32_bit_offset(api):
    """A pool of more than 2^31 codes: pages at its end are reached."""
    H, page, D = 8, 128, 128
    N = (1 << 31) // (H * page * D) + 3
    table = torch.tensor([[N - 1, N - 2]], dtype=torch.int32, device=DEV)
    c = api.kv_cache(table, N, H, page, D)
    k, v = _new(1, 130, H, D, seed=15)
    api.kv_append(c, k.to(DEV), v.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    small = api.kv_cache(torch.tensor([[1, 0]], dtype=torch.int32, device=DEV), 2, H, page, D)
    api.kv_append(small, k.to(DEV), v.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    for n in ("k", "v", "k_scale", "v_scale"):
        a, b = getattr(c, n)[-2:].view(torch.uint8), getattr(small, n).view(torch.uint8)
        assert torch.equal(a, b), n


def test_refusals(api):
    c = _cache(api, 2, 2, 2, 16, 64, seed=16)
    k, v = (t.to(DEV) for t in _new(2, 4, 2, 64, seed=16))
    z = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        api.kv_append(c, k.float(), v.float(), z)
    with pytest.raises(TypeError):
        api.kv_append(c, k, v, z.long())
    with pytest.raises(ValueError):
        api.kv_append(c, k, v, z[:1])
    with pytest.raises(ValueError):
        api.kv_append(c, k[:, :, :1].contiguous(), v[:, :, :1].contiguous(), z)
    with pytest.raises(ValueError):
        api.kv_append(c, k.transpose(1, 2), v.transpose(1, 2), z)
    with pytest.raises(ValueError):
        api.kv_append(c, k.cpu(), v, z)
    with pytest.raises(ValueError):
        api.kv_cache(c.page_table, 4, 2, 48, 64)
    with pytest.raises(api.UnoError):
        bad = api.KvCache(*(t[:, :, :8].contiguous() for t in (c.k, c.v)), c.k_scale, c.v_scale,
                          c.page_table)
        api.kv_append(bad, k, v, z)
