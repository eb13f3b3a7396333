"""Refusals of the paged calls: every bad argument is an SRFTKV_ERR_INVALID with a message before any GPU work, so
these run without one."""

import ctypes
import os

import pytest
import torch

import int8_kv_cache_srft_gb300 as K


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from int8_kv_cache_srft_gb300 import build

        build.build()
    return K.library()


def pages(codes=256, scales=256, lam=None, n_pages=4, H=2, page_size=16, d=128, group=16, bits=4, transform=0, fmt=0):
    return K._Pages(codes, scales, lam, n_pages, H, page_size, d, group, bits, transform, fmt)


def batch(table=16, lens=16, cu=16, B=2, max_pages=4, total_q=2, max_q=1, max_seq_len=0):
    return K._PagedBatch(table, lens, cu, B, max_pages, total_q, max_q, max_seq_len)


def codec(lib, k, v, quantize=True, xk=16, xks=0, xv=16, xvs=0, slots=16, n=4, dtype=0):
    fn = lib.srft_kv_quantize_paged if quantize else lib.srft_kv_dequantize_paged
    p = lambda s: None if s is None else ctypes.pointer(s)  # noqa: E731
    return fn(p(k), xk, xks, p(v), xv, xvs, slots, n, dtype, 1, None)


def attn(lib, k, v, b, q=16, qs=0, out=32, os_=0, dtype=0, Hq=8, sm=0.0, window=0, ws=16, nws=1 << 30):
    p = lambda s: None if s is None else ctypes.pointer(s)  # noqa: E731
    return lib.q4kv_paged_attention(q, qs, out, os_, dtype, Hq, p(k), p(v), p(b), sm, window, 1, ws, nws, None)


BAD_PAGES = [dict(d=96), dict(d=512), dict(group=8), dict(group=24), dict(group=256), dict(page_size=8),
             dict(page_size=24), dict(page_size=512), dict(n_pages=0), dict(H=0), dict(bits=3), dict(bits=16),
             dict(transform=2), dict(fmt=3), dict(codes=None), dict(scales=None), dict(codes=8), dict(scales=4),
             dict(lam=8), dict(n_pages=1 << 30, H=4)]


@pytest.mark.parametrize("quantize", [True, False])
@pytest.mark.parametrize("case", BAD_PAGES)
def test_codec_refuses_bad_pages(lib, case, quantize):
    for k, v in ((pages(**case), None), (None, pages(**case))):
        assert codec(lib, k, v, quantize) == K.SRFTKV_ERR_INVALID
        assert b"paged" in lib.srftkv_last_error()


@pytest.mark.parametrize("case", [dict(xk=None), dict(xk=8), dict(xks=100), dict(xks=260), dict(xks=-256), dict(xv=4),
                                  dict(slots=None), dict(slots=12), dict(n=-1), dict(dtype=2), dict(n=1 << 30)])
def test_codec_refuses_bad_rows(lib, case):
    assert codec(lib, pages(), pages(), **case) == K.SRFTKV_ERR_INVALID


@pytest.mark.parametrize("case", [dict(n_pages=5), dict(H=4), dict(page_size=32), dict(d=64), dict(group=32)])
def test_sides_share_their_sizes(lib, case):
    assert codec(lib, pages(), pages(**case)) == K.SRFTKV_ERR_INVALID
    assert attn(lib, pages(), pages(**case), batch()) == K.SRFTKV_ERR_INVALID


def test_codec_needs_a_side_and_takes_an_empty_call(lib):
    assert codec(lib, None, None) == K.SRFTKV_ERR_INVALID
    assert codec(lib, pages(), pages(bits=8, fmt=1), n=0, slots=None) == K.SRFTKV_OK


@pytest.mark.parametrize("case", BAD_PAGES)
def test_attention_refuses_bad_pages(lib, case):
    assert attn(lib, pages(**case), pages(**case), batch()) == K.SRFTKV_ERR_INVALID
    assert attn(lib, pages(), pages(**{k: v for k, v in case.items()}), batch()) == K.SRFTKV_ERR_INVALID


@pytest.mark.parametrize("case", [dict(B=-1), dict(max_pages=0), dict(total_q=-1), dict(max_q=-1), dict(max_q=3),
                                  dict(max_q=0), dict(max_seq_len=65), dict(max_seq_len=-1), dict(table=None),
                                  dict(lens=None), dict(table=2), dict(lens=6), dict(cu=2), dict(cu=None, total_q=1),
                                  dict(max_pages=1 << 28), dict(B=40000, total_q=40000),
                                  dict(total_q=1 << 30, max_q=1)])
def test_attention_refuses_bad_batches(lib, case):
    assert attn(lib, pages(), pages(), batch(**case)) == K.SRFTKV_ERR_INVALID


@pytest.mark.parametrize("case", [dict(q=None), dict(q=8), dict(out=None), dict(out=8), dict(qs=1000), dict(qs=1028),
                                  dict(os_=512), dict(dtype=2), dict(Hq=0), dict(Hq=7), dict(Hq=258), dict(window=-1),
                                  dict(sm=float("nan")), dict(sm=float("inf"))])
def test_attention_refuses_bad_arguments(lib, case):
    assert attn(lib, pages(), pages(), batch(), **case) == K.SRFTKV_ERR_INVALID


def test_attention_refuses_mixed_scale_formats_and_missing_sides(lib):
    assert attn(lib, pages(fmt=0), pages(fmt=1), batch()) == K.SRFTKV_ERR_INVALID
    assert attn(lib, None, pages(), batch()) == K.SRFTKV_ERR_INVALID
    assert attn(lib, pages(), None, batch()) == K.SRFTKV_ERR_INVALID
    assert attn(lib, pages(), pages(), None) == K.SRFTKV_ERR_INVALID


def test_empty_batches_are_no_ops(lib):
    assert attn(lib, pages(), pages(), batch(B=0, total_q=0, max_q=0)) == K.SRFTKV_OK
    assert attn(lib, pages(), pages(), batch(total_q=0, max_q=0)) == K.SRFTKV_OK


def test_binding_checks_tensors():
    c, s = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, 8)
    K.Pages(c, s, 4, 128, 16).to_c()
    for bad in (dict(codes=c[..., :32]), dict(scales=s.half()), dict(bits=8), dict(group=32), dict(d=64),
                dict(lam=torch.ones(2, 64)), dict(codes=c.float()), dict(codes=c.transpose(0, 1))):
        with pytest.raises(K.SrftKvError) as e:
            K.Pages(**{**dict(codes=c, scales=s, bits=4, d=128, group=16), **bad}).to_c()
        assert e.value.code == K.SRFTKV_ERR_INVALID
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    assert K.PagedBatch(t, n).to_c().total_q == 3
    for bad in (dict(block_table=t.long()), dict(seq_lens=n[:2]), dict(cu_q=n, total_q=3),
                dict(cu_q=torch.zeros(4, dtype=torch.int32)), dict(block_table=t[:, ::2])):
        with pytest.raises(K.SrftKvError):
            K.PagedBatch(**{**dict(block_table=t, seq_lens=n), **bad}).to_c()
    p, slots = K.Pages(c, s, 4, 128, 16), torch.zeros(3, dtype=torch.int64)
    x = torch.zeros(3, 2, 128, dtype=torch.float16)
    for k, xk, sl in ((p, x.float(), slots), (p, x[:2], slots), (p, x[:, :, ::2], slots), (p, x, slots.int()),
                      (p, x.transpose(0, 1).contiguous().transpose(0, 1), slots), (None, None, slots)):
        with pytest.raises(K.SrftKvError) as e:
            K.srft_kv_quantize_paged(k, xk, None, None, sl, 1)
        assert e.value.code == K.SRFTKV_ERR_INVALID
    with pytest.raises(K.SrftKvError):
        K.q4kv_paged_attention(x.float(), x, p, p, K.PagedBatch(t, n), 0.0, 0, 1, c)
    with pytest.raises(K.SrftKvError):  # a side without its rows
        K.srft_kv_quantize_paged(p, None, None, None, slots, 1)
    with pytest.raises(K.SrftKvError, match="overlap"):  # one row for all tokens: its stride is 0
        K.srft_kv_quantize_paged(p, x[:1].expand(3, 2, 128), None, None, slots, 1)
    one = torch.zeros(1, 2, 128, dtype=torch.float16)
    with pytest.raises(K.SrftKvError, match="overlap"):
        K.q4kv_paged_attention(one.expand(3, 2, 128), x, p, p, K.PagedBatch(t, n), 0.0, 0, 1, c)
