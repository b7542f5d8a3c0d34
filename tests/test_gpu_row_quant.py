"""RMS norm with residual and 8-bit rows, and the row quantiser (need a B200).

Against float64. Tolerances: the sum of squares is at most 32 chained float32
additions per thread and 10 shuffle steps, so its relative error is below
42 * 2^-24 and the row factor's below 21 * 2^-24; with the handful of other
float32 operations a normed value is within 32 * 2^-24 < 2e-6 relative. An 8-bit
value may then be off by half a step plus 127 * 2 * 2e-6 < 6e-4 steps, a
value in the rows' dtype by half a step of that type.
"""

import math

import pytest
import torch

from tests.eight_bit import rms_norm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 2e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_decoding_b200 import api as A
    return A


def _rows(M, d, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, d, generator=g) * std).to(DT[dtype])


def _check_q(q, scale, y, ref_scale):
    q, scale = q.cpu().double(), scale.cpu().double()
    assert torch.all((scale - ref_scale).abs() <= REL * ref_scale)
    t = y / torch.where(ref_scale > 0, ref_scale, 1.0)[:, None]
    assert float((q - t).abs().max()) <= 0.5 + 6e-4
    assert float(q.abs().max()) <= 127


SHAPES = [(1, 1), (3, 7), (1, 4096), (5, 33), (17, 255), (9, 256), (4, 1000), (300, 4096),
          (2, 4088), (7, 8191), (3, 8200), (300, 12288), (2, 20011), (2, 32768), (1, 32767),
          (1030, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,d", SHAPES)
def test_rms_norm(api, M, d, dtype):
    x, res, w = _rows(M, d, dtype, 1), _rows(M, d, dtype, 2, 2.0), _rows(1, d, dtype, 3)[0] + 1
    for r in (None, res):
        got = api.rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=None if r is None else r.to(DEV),
                           want_y=True)
        h, y, scale = rms_norm(x, w, 1e-5, r)
        assert torch.equal(got.h.cpu(), h)
        _check_q(got.q, got.scale, y, scale)
        half = torch.finfo(DT[dtype]).eps / 2
        assert torch.all((got.y.cpu().double() - y).abs() <= (half + 2 * REL) * y.abs() + 1e-37)
    only_y = api.rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=res.to(DEV), want_y=True,
                          want_q=False)
    assert only_y.q is None and torch.equal(only_y.y, got.y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,d", SHAPES)
def test_quantize_rows(api, M, d, dtype):
    x = _rows(M, d, dtype, 4, 30.0)
    q, scale = api.quantize_rows(x.to(DEV))
    _check_q(q, scale, x.double(), x.double().abs().amax(1) / 127)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_zeros_of_tiny_and_of_huge_values(api, dtype):
    x = _rows(6, 264, dtype, 5)
    x[0] = 0
    x[1] *= 1e-38    # 127 / max passes float32
    x[2] = 0
    x[2, 17] = -2.5  # one value
    x[3] *= 1e30     # the maximum is finite, the sum of squares is not
    q, scale = api.quantize_rows(x.to(DEV))
    assert float(scale[0]) == 0 and int(q[0].abs().max()) == 0
    assert int(q[2, 17]) == -127 and int(q[2].abs().sum()) == 127
    ref = x.double().abs().amax(1) / 127
    # a scale below float32's normal range is off by half a subnormal step
    assert torch.all((scale.cpu().double() - ref).abs() <= REL * ref + 2.0 ** -150)
    t = x[1].double() / ref[1]
    assert float((q[1].cpu().double() - t).abs().max()) <= 0.5 + 6e-4
    r = api.rms_norm(x.to(DEV), torch.ones(264, dtype=DT[dtype], device=DEV), 1e-6)
    assert float(r.scale[0]) == 0 and int(r.q[0].abs().max()) == 0
    assert math.isnan(float(r.scale[3])) and int(r.q[3].abs().max()) == 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d", [40, 41, 4096])
def test_a_non_finite_row_is_marked_and_the_others_are_not(api, bad, d):
    x = _rows(5, d, "bf16", 6)
    x[2, d - 1] = bad
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    for q, scale in (api.quantize_rows(x.to(DEV)),
                     (lambda r: (r.q, r.scale))(api.rms_norm(x.to(DEV), w, 1e-6))):
        assert torch.isnan(scale).tolist() == [False, False, True, False, False]
        assert int(q[2].abs().max()) == 0 and int(q[3].abs().max()) == 127


def test_empty_and_refusals(api):
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    r = api.rms_norm(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), w, 1e-6)
    assert r.q.shape == (0, 64) and r.scale.shape == (0,)
    x = torch.ones(2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        api.rms_norm(x, w.float(), 1e-6)
    with pytest.raises(ValueError):
        api.rms_norm(x, w, 1e-6, residual=x[:1])
    with pytest.raises(ValueError):
        api.rms_norm(x, w, 1e-6, want_q=False)
    with pytest.raises(ValueError):
        api.quantize_rows(x.t())
    with pytest.raises(api.UnoError):
        api.rms_norm(x, w, -1.0)
    with pytest.raises(api.UnoError):  # rows not on a 16-byte boundary
        api.quantize_rows(torch.ones(65, dtype=torch.bfloat16, device=DEV)[1:].view(1, 64))
    with pytest.raises(api.UnoError):
        api.quantize_rows(torch.ones(1, 32769, dtype=torch.bfloat16, device=DEV))


def test_streams_and_a_captured_graph(api):
    x, w = _rows(300, 4096, "bf16", 7).to(DEV), torch.ones(4096, dtype=torch.bfloat16, device=DEV)
    want = api.rms_norm(x, w, 1e-6)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = api.rms_norm(x, w, 1e-6)
    s.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = api.rms_norm(x, w, 1e-6)
    x.copy_(_rows(300, 4096, "bf16", 8))
    g.replay()
    want = api.rms_norm(x, w, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)


@pytest.mark.parametrize("M,d", [(300, 512), (300, 16384), (300, 16392), (4, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_rows_among_many(api, M, d, dtype):
    """Zeros, tiny, one value, infinities and NaN in each way that rows are taken."""
    x = _rows(M, d, dtype, 9)
    x[0] = 0
    x[1] *= 1e-38
    x[2] = 0
    x[2, d - 1] = 3.0
    bad = [3] if M < 6 else [3, 4, 5]
    for r, v in zip(bad, (math.nan, -math.inf, math.inf)):
        x[r, d // 2] = v
    q, scale = api.quantize_rows(x.to(DEV))
    ok = torch.ones(M, dtype=torch.bool)
    ok[bad] = False
    assert torch.equal(torch.isnan(scale).cpu(), ~ok)
    assert int(q[bad].abs().max()) == 0 and float(scale[0]) == 0 and int(q[0].abs().max()) == 0
    ref = x[ok].double().abs().amax(1) / 127
    assert torch.all((scale.cpu()[ok].double() - ref).abs() <= REL * ref + 2.0 ** -150)
    t = x[ok].double() / torch.where(ref > 0, ref, 1.0)[:, None]
    assert float((q.cpu()[ok].double() - t).abs().max()) <= 0.5 + 6e-4


@pytest.mark.parametrize("M,d", [(4, 512), (300, 512), (300, 4096), (300, 41)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_binade_where_127_over_the_maximum_nears_float32s_end(api, M, d, dtype):
    # maxima of 2^-126 to 2^-115: 127 / max passes float32 below 127 / FLT_MAX, just under 2^-121
    for e in range(-126, -114):
        x = _rows(M, d, dtype, 100 - e).clamp(-1.5, 1.5) * 2.0 ** e
        x[:, 0] = 1.75 * 2.0 ** e
        x[1, 1] = 0
        q, scale = api.quantize_rows(x.to(DEV))
        ref = x.double().abs().amax(1) / 127
        # the scale is a subnormal number: half a step of 2^-149
        assert torch.all((scale.cpu().double() - ref).abs() <= REL * ref + 2.0 ** -150), e
        assert float((q.cpu().double() - x.double() / ref[:, None]).abs().max()) <= 0.5 + 6e-4, e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_without_eps_of_rows_whose_squares_vanish(api, dtype):
    x = _rows(4, 264, dtype, 30)
    x[1] = 0
    x[2] *= 1e-30
    w = torch.ones(264, dtype=DT[dtype])
    r = api.rms_norm(x.to(DEV), w.to(DEV), 0.0)
    assert torch.isnan(r.scale).tolist() == [False, True, True, False]
    assert int(r.q[1:3].abs().max()) == 0
    _, y, scale = rms_norm(x[3:], w, 0.0)
    _check_q(r.q[3:], r.scale[3:], y, scale)


# (M, d) of each way in which rows are taken: element by element, in 16-byte pieces with one,
# two and four to a thread, packed
WAYS = [(128, 41), (128, 8193), (128, 64), (256, 4096), (384, 4096), (384, 16392)]


@pytest.mark.parametrize("e", [0, -40, 60, -119, -120, -121, -125])
@pytest.mark.parametrize("M,d", WAYS)
def test_bfloat16_rows_are_rounded_exactly(api, M, d, e):
    """127 x / max in 64 bits is exact where it is a half and at least 2^-17 x from one
    elsewhere. Each mantissa of the maximum; half of it is 63.5 steps: 64, to the even side."""
    g = torch.Generator().manual_seed(M + d + e)
    top = (1 + torch.arange(M) % 128 / 128).double() * 2.0 ** e
    x = (torch.randn(M, d, generator=g).clamp(-3, 3).double() / 3 * top[:, None]).bfloat16()
    x[:, 0], x[:, 1], x[:, d - 1], x[:, d // 2] = top, -top / 2, top / 2, -top / 4
    assert torch.equal(x.double().abs().amax(1), top)
    q, _ = api.quantize_rows(x.to(DEV))
    want = torch.round(x.double() * 127 / top[:, None])
    assert torch.all(want[:, 1] == -64) and torch.all(want[:, d - 1] == 64)
    assert torch.equal(q.cpu().double(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,d", WAYS)
def test_half_of_the_maximum_is_64_steps(api, M, d, dtype):
    g = torch.Generator().manual_seed(M + d)
    x = (torch.randn(M, d, generator=g) / 16).clamp(-0.9, 0.9).to(DT[dtype])
    top = (1 + torch.rand(M, generator=g)).to(DT[dtype])
    x[:, 0], x[:, 1], x[:, d - 1] = top, -top / 2, top / 2
    w = torch.ones(d, dtype=DT[dtype], device=DEV)
    for q in (api.quantize_rows(x.to(DEV))[0], api.rms_norm(x.to(DEV), w, 1e-6).q):
        q = q.cpu()
        assert torch.all(q[:, 0] == 127) and torch.all(q[:, 1] == -64)
        assert torch.all(q[:, d - 1] == 64)
