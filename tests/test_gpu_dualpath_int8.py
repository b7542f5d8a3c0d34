"""The dual-pathway linear on 8-bit integers (needs a B200).

Against float64. The integer sums are exact, so y_ar is off by the three
float32 roundings of (sum, x scale, w scale) and the output's own; y_draft also by
T's rounding to bf16 (half a step, 2^-8) and r float32 additions, which the
tensor core may truncate (2^-22 each), both relative to |T| |Bm|^T.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_decoding_b200 import api as A
    return A


def _inputs(M, d_in, d_out, r, seed, lo=-127):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def q(n):
        return torch.randint(lo, 128, (n, d_in), generator=g, device=DEV, dtype=torch.int8)

    def s(n, c):
        return (torch.rand(n, generator=g, device=DEV) + 0.5) * c

    d = dict(xq=q(M), x_scale=s(M, 0.02), Wq=q(d_out), w_scale=s(d_out, 1e-4))
    if r:
        d.update(Aq=q(r), a_scale=s(r, 1e-4), scale=2.0,
                 Bm=(torch.randn(d_out, r, generator=g, device=DEV) * 0.05).bfloat16())
    return d


def _reference(d, gate=None):
    """(y_ar, y_draft, |T| |Bm|^T) in float64 on the GPU: the sums of integers are exact
    there too (a sum of 0 stays 0), the scales come after them."""

    def scaled(w, s):
        return (d["xq"].double() @ w.double().t()) * d["x_scale"].double()[:, None] * s.double()

    y = scaled(d["Wq"], d["w_scale"])
    if "Bm" not in d:
        return y, None, None
    t = d["scale"] * scaled(d["Aq"], d["a_scale"])
    if gate is not None:
        t = t * (gate != 0).double()[:, None]
    return y, y + t @ d["Bm"].double().t(), t.abs() @ d["Bm"].double().abs().t()


def _check(y_ar, y_draft, d, out_dtype, gate=None):
    ref, ref_d, spread = _reference(d, gate)
    half = torch.finfo(out_dtype).eps / 2
    if y_ar is not None:
        assert y_ar.dtype == out_dtype
        assert torch.all((y_ar.double() - ref).abs() <= (half + 4 * 2.0 ** -24) * ref.abs())
    if ref_d is None:
        assert y_draft is None
        return
    r = d["Bm"].shape[1]
    tol = (half * 1.01 + 2.0 ** -22) * ref_d.abs() + 4 * 2.0 ** -24 * ref.abs() + \
        (2.0 ** -8 + r * 2.0 ** -22) * 1.01 * spread
    assert torch.all((y_draft.double() - ref_d).abs() <= tol)


SHAPES = [
    (1, 16, 1, 8), (1, 4096, 1024, 128), (3, 48, 17, 16), (17, 512, 4096, 128),
    (33, 144, 129, 40), (64, 1024, 300, 256), (65, 2064, 1000, 24), (128, 128, 128, 8),
    (129, 4096, 4104, 128), (200, 272, 77, 64), (256, 640, 520, 128),
    (257, 128, 256, 8), (300, 144, 333, 40), (512, 2064, 1000, 256), (1088, 1024, 4096, 128),
    (1000, 528, 1031, 72), (2049, 256, 264, 16),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,d_in,d_out,r", SHAPES)
def test_both_paths(api, M, d_in, d_out, r, out):
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    d = _inputs(M, d_in, d_out, r, seed=M + d_in)
    y_ar, y_dr = api.dualpath_linear_int8(**d, out_dtype=t)
    torch.cuda.synchronize()
    _check(y_ar, y_dr, d, t)
    # the paths one by one give the same bits
    only = {k: d[k] for k in ("xq", "x_scale", "Wq", "w_scale")}
    a, none = api.dualpath_linear_int8(**only, out_dtype=t)
    none2, b = api.dualpath_linear_int8(**d, out_dtype=t, want_ar=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None
    assert torch.equal(a, y_ar) and torch.equal(b, y_dr)
    assert api.device_fault_flags() == 0


@pytest.mark.parametrize("M,d_in,d_out,r", [(17, 256, 384, 64), (300, 256, 520, 32),
                                            (300, 256, 333, 32)])
def test_gate(api, M, d_in, d_out, r):
    d = _inputs(M, d_in, d_out, r, seed=M)
    gate = (torch.arange(M, device=DEV) % 17 != 0).to(torch.uint8) * 3
    y_ar, y_dr = api.dualpath_linear_int8(**d, gate=gate)
    torch.cuda.synchronize()
    _check(y_ar, y_dr, d, torch.bfloat16, gate)
    assert torch.equal(y_ar[gate == 0], y_dr[gate == 0])
    both = api.dualpath_linear_int8(**d, gate=gate.bool())[1]
    assert torch.equal(both, y_dr)


def test_sums_are_exact_at_the_largest_depth(api):
    """65536 products of (-128)^2: 2^30, past float32's integers, and every int8 value."""
    d = _inputs(5, 65536, 24, 0, seed=1, lo=-128)
    d["xq"][0] = -128
    d["Wq"][3] = -128
    d["x_scale"][:] = 1
    d["w_scale"][:] = 1
    y, _ = api.dualpath_linear_int8(**d, out_dtype=torch.float32)
    ref = (d["xq"].double() @ d["Wq"].double().t()).float()
    assert float(y[0, 3]) == 2.0 ** 30
    assert torch.equal(y, ref)


@pytest.mark.parametrize("M", [40, 400])
def test_a_row_with_a_nan_scale_stays_alone(api, M):
    d = _inputs(M, 256, 200, 32, seed=2)
    want = api.dualpath_linear_int8(**d)
    d["x_scale"][7] = float("nan")
    got = api.dualpath_linear_int8(**d)
    for w, g in zip(want, got):
        assert torch.isnan(g[7]).all()
        keep = torch.arange(M, device=DEV) != 7
        assert torch.equal(w[keep], g[keep])


def test_empty_and_refusals(api):
    d = _inputs(4, 64, 40, 16, seed=3)
    e = api.dualpath_linear_int8(d["xq"][:0], d["x_scale"][:0], d["Wq"], d["w_scale"])[0]
    assert e.shape == (0, 40)

    def bad(exc, drop=(), **kw):
        args = {k: v for k, v in {**d, **kw}.items() if k not in drop}
        with pytest.raises(exc):
            api.dualpath_linear_int8(**args)

    bad(ValueError, drop=("Bm",))
    bad(ValueError, drop=("a_scale",))
    bad(ValueError, drop=("Aq", "a_scale", "Bm"), want_ar=False)
    bad(ValueError, drop=("Aq", "a_scale", "Bm"), gate=torch.ones(4, device=DEV).bool())
    bad(TypeError, xq=d["xq"].float())
    bad(TypeError, Bm=d["Bm"].float())
    bad(TypeError, out_dtype=torch.float16)
    bad(ValueError, x_scale=d["x_scale"][:3])
    bad(ValueError, Wq=d["Wq"][:, :48])
    bad(ValueError, gate=torch.ones(3, device=DEV).bool())
    bad(api.UnoError, xq=d["xq"][:, :40].contiguous(), Wq=d["Wq"][:, :40].contiguous(),
        Aq=d["Aq"][:, :40].contiguous())
    bad(api.UnoError, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_two_streams_and_captured_graphs(api):
    """Calls on two streams, and two captured graphs replayed side by side, share nothing."""
    ds = [_inputs(M, 512, 1032, 64, seed=M) for M in (40, 400)]
    want = [api.dualpath_linear_int8(**d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[], []]
    for _ in range(10):
        for i, d in enumerate(ds):
            with torch.cuda.stream(streams[i]):
                got[i].append(api.dualpath_linear_int8(**d))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.dualpath_linear_int8(**d))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o[0].zero_()
            o[1].zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    assert api.device_fault_flags() == 0


@pytest.mark.parametrize("M,d_in,d_out,r", [(1, 4096, 1024, 128), (40, 1024, 512, 32),
                                            (1088, 1024, 4096, 128), (300, 256, 256, 64)])
def test_whatever_the_workspace_holds(api, M, d_in, d_out, r):
    """Its flags may hold what a caller can guess of the next call's from those of the last:
    with all operands 0 the flags are the only words that a call leaves that are not."""
    from lossless_decoding_b200._lib import lib
    d = _inputs(M, d_in, d_out, r, seed=M)
    want = api.dualpath_linear_int8(**d)
    zero = {k: torch.zeros_like(v) if torch.is_tensor(v) else v for k, v in d.items()}
    need = int(lib.uno_dualpath_int8_workspace_bytes(M, d_in, d_out, r))
    ws = torch.zeros((need + 7) // 8, dtype=torch.int64, device=DEV)
    w32 = ws.view(torch.int32)
    for guess in ("the same", "32-bit words", "64-bit words"):
        ws.zero_()
        api.dualpath_linear_int8(**zero, workspace=ws)
        at32, at64 = w32 != 0, ws != 0
        assert at32.any()
        if guess == "32-bit words":
            w32 += 1
        elif guess == "64-bit words":
            ws += 1
        # everything else: large halves of floats, and large integers
        if guess == "64-bit words":
            ws[~at64] = 0x7F007F007F007F00
        else:
            w32[~at32] = 0x7F007F00
        got = api.dualpath_linear_int8(**d, workspace=ws)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b), guess
    assert api.device_fault_flags() == 0


@pytest.mark.parametrize("M,d_in,d_out,r,out", [(20011, 272, 1000, 16, "bf16"), (8192, 1024, 513, 128, "f32"),
                                                (5, 4096, 151936, 128, "bf16")])
def test_many_rows_and_many_columns(api, M, d_in, d_out, r, out):
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    d = _inputs(M, d_in, d_out, r, seed=M)
    gate = (torch.arange(M, device=DEV) % 3 != 0).to(torch.uint8)
    y_ar, y_dr = api.dualpath_linear_int8(**d, gate=gate, out_dtype=t)
    _check(y_ar, y_dr, d, t, gate)
    assert api.device_fault_flags() == 0
