"""Argument checks of the 8-bit entry points (host side, no GPU)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from lossless_decoding_b200.build import build_library
    build_library()
    from lossless_decoding_b200._lib import lib as L
    return L


FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4098)


def _name(st):
    from lossless_decoding_b200._lib import STATUS
    return STATUS[st]


def test_rms_norm_args(lib):
    def call(x=FAKE, w=FAKE, eps=1e-6, M=4, d=64, dtype=0, h=None, y=None, q=FAKE, scale=FAKE):
        return _name(lib.uno_rms_norm(x, None, w, eps, M, d, dtype, h, y, q, scale, None))

    assert call(dtype=2) == "UNO_ERR_DTYPE"
    assert call(M=-1) == call(d=0) == call(d=32769) == call(M=(1 << 24) + 1) == "UNO_ERR_SIZE"
    assert call(eps=-1.0) == call(eps=float("nan")) == call(eps=float("inf")) == "UNO_ERR_SIZE"
    assert call(x=None) == call(w=None) == call(q=None) == call(scale=None) == "UNO_ERR_NULL"
    assert call(x=ODD) == call(w=ODD) == call(q=ODD) == call(y=ODD) == "UNO_ERR_ALIGN"
    assert call(M=0, x=None, w=None, q=None, scale=None) == "UNO_OK"


def test_quantize_rows_args(lib):
    def call(x=FAKE, M=4, d=64, dtype=0, q=FAKE, scale=FAKE):
        return _name(lib.uno_quantize_rows(x, M, d, dtype, q, scale, None))

    assert call(dtype=-1) == "UNO_ERR_DTYPE"
    assert call(d=0) == call(d=40000) == "UNO_ERR_SIZE"
    assert call(x=None) == call(q=None) == call(scale=None) == "UNO_ERR_NULL"
    assert call(x=ODD) == call(q=ODD) == "UNO_ERR_ALIGN"
    assert call(M=0, x=None, q=None, scale=None) == "UNO_OK"


def test_kv_append_args(lib):
    def call(k=FAKE, start=FAKE, count=None, rows=None, B=2, T=4, n=4, H=2, D=64, page=16,
             table=FAKE, width=3, N=6, codes=FAKE, scale=FAKE):
        return _name(lib.uno_kv_append(k, FAKE, start, count, rows, B, T, n, H, D, page, table,
                                       width, N, codes, FAKE, scale, FAKE, None))

    for bad in (dict(B=-1), dict(B=65536), dict(T=-1), dict(n=-1), dict(n=5), dict(H=0),
                dict(H=1025), dict(D=96), dict(page=48), dict(width=-1), dict(N=-1),
                dict(width=1 << 27), dict(T=(1 << 20) + 1), dict(rows=FAKE, n=(1 << 20) + 1),
                dict(B=65535, T=1 << 20, n=1 << 20, page=16)):
        assert call(**bad) == "UNO_ERR_SIZE", bad
    for bad in (dict(k=None), dict(start=None), dict(table=None), dict(codes=None),
                dict(scale=None)):
        assert call(**bad) == "UNO_ERR_NULL", bad
    for bad in (dict(k=ODD), dict(codes=ODD), dict(start=ODD), dict(count=ODD), dict(rows=ODD),
                dict(table=ODD), dict(scale=ODD)):
        assert call(**bad) == "UNO_ERR_ALIGN", bad
    assert call(B=0, k=None) == call(T=0, n=0, k=None) == "UNO_OK"


def test_dualpath_int8_args(lib):
    def call(x=FAKE, xs=FAKE, W=FAKE, ws=FAKE, A=FAKE, as_=FAKE, Bm=FAKE, ya=FAKE, yd=FAKE, M=4,
             d_in=64, d_out=40, r=16, dtype=0, work=FAKE, nbytes=1 << 30):
        return _name(lib.uno_dualpath_linear_int8(x, xs, W, ws, A, as_, Bm, 2.0, None, ya, yd, M,
                                                  d_in, d_out, r, dtype, work, nbytes, None))

    assert call(dtype=2) == "UNO_ERR_DTYPE"
    for bad in (dict(M=-1), dict(d_in=0), dict(d_in=40), dict(d_in=65552), dict(d_out=0),
                dict(r=12), dict(r=264), dict(r=0), dict(r=-8)):
        assert call(**bad) == "UNO_ERR_SIZE", bad
    for bad in (dict(x=None), dict(xs=None), dict(W=None), dict(ws=None), dict(A=None),
                dict(as_=None), dict(Bm=None), dict(ya=None, yd=None)):
        assert call(**bad) == "UNO_ERR_NULL", bad
    for bad in (dict(x=ODD), dict(xs=ODD), dict(W=ODD), dict(ws=ODD), dict(A=ODD), dict(as_=ODD),
                dict(Bm=ODD), dict(ya=ODD), dict(yd=ODD), dict(work=ODD)):
        assert call(**bad) == "UNO_ERR_ALIGN", bad
    assert call(work=None) == call(nbytes=64) == "UNO_ERR_WORKSPACE"
    assert call(M=0, x=None) == "UNO_OK"
    assert lib.uno_dualpath_int8_workspace_bytes(17, 4096, 1000, 128) >= 17 * 128 * 2
    assert lib.uno_dualpath_int8_workspace_bytes(17, 4096, 1000, 0) > 0
    assert lib.uno_dualpath_int8_workspace_bytes(17, 4090, 1000, 0) == 0


def test_the_operand_type_of_the_8_bit_call_is_no_dtype_of_the_others(lib):
    for code in (2, 3, -1, -8):
        assert lib.uno_dualpath_workspace_bytes(16, 64, 64, 8, code) == 0
        assert _name(lib.uno_dualpath_linear(FAKE, FAKE, FAKE, FAKE, 2.0, FAKE, FAKE, 16, 64, 64,
                                             8, code, FAKE, 1 << 30, None)) == "UNO_ERR_DTYPE"


def test_block_attention_args(lib):
    def call(q=FAKE, k=FAKE, lens=FAKE, parent=None, nn=None, scale=0.1, B=2, T=4, Hq=4, H=2, D=64,
             page=16, table=FAKE, width=3, N=6, codes=FAKE, ks=FAKE, out=FAKE, work=FAKE,
             nbytes=1 << 30):
        return _name(lib.uno_block_attention(q, k, FAKE, lens, parent, nn, scale, B, T, Hq, H, D,
                                             page, table, width, N, codes, FAKE, ks, FAKE, out,
                                             work, nbytes, None))

    for bad in (dict(B=-1), dict(B=65536), dict(T=-1), dict(T=4097), dict(Hq=3), dict(Hq=1),
                dict(H=0), dict(Hq=16386, H=2), dict(D=80), dict(page=24), dict(width=-1),
                dict(N=-1), dict(N=1 << 27), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == "UNO_ERR_SIZE", bad
    for bad in (dict(q=None), dict(k=None), dict(lens=None), dict(table=None), dict(codes=None),
                dict(ks=None), dict(out=None)):
        assert call(**bad) == "UNO_ERR_NULL", bad
    for bad in (dict(q=ODD), dict(k=ODD), dict(lens=ODD), dict(parent=ODD), dict(nn=ODD),
                dict(table=ODD), dict(codes=ODD), dict(ks=ODD), dict(out=ODD), dict(work=ODD)):
        assert call(**bad) == "UNO_ERR_ALIGN", bad
    assert call(work=None) == call(nbytes=64) == "UNO_ERR_WORKSPACE"
    assert call(B=0, q=None) == call(T=0, q=None) == "UNO_OK"
    assert lib.uno_block_attention_workspace_bytes(64, 17, 32, 8, 128) > 0
    assert lib.uno_block_attention_workspace_bytes(64, 17, 33, 8, 128) == 0
    assert lib.uno_block_attention_workspace_bytes(64, 17, 32, 8, 96) == 0


def test_an_append_to_an_empty_pool_or_table_writes_nothing(lib):
    """Their tensors have no storage, so no pointers; the attention takes them too."""
    def call(table, width, N, codes, scale):
        return _name(lib.uno_kv_append(FAKE, FAKE, FAKE, None, None, 2, 4, 4, 2, 64, 16, table,
                                       width, N, codes, codes, scale, scale, None))

    assert call(None, 0, 6, FAKE, FAKE) == call(FAKE, 3, 0, None, None) == "UNO_OK"
    assert call(None, 0, 0, None, None) == "UNO_OK"
    assert call(None, 3, 6, FAKE, FAKE) == call(FAKE, 3, 6, None, FAKE) == "UNO_ERR_NULL"
