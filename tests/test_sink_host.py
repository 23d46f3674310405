"""Refusals of the attention with sinks and of reading back: on the host, before anything is enqueued (no GPU)."""
import ctypes as C

import pytest
import torch

import mixed_precision_quantized_kvq_b200 as kvq
from test_abi import L, _fake_cache

OK, BAD, UNSUP = kvq.KVQ_OK, kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED
BUF = C.create_string_buffer(4096)
P = (C.addressof(BUF) + 255) & ~255
ROW = 32 * 128


def decode(lay=None, cache=None, q=P, qt=1, stride=ROW, lens=P, max_len=8, sinks=4, span=64, scale=0.1, out=P, lse=P):
    lay, (c, keep) = lay or L(), (cache or _fake_cache())
    return kvq.lib().kvq_sink_decode_attention(C.byref(lay.c()), C.byref(c), q, qt, stride, lens, max_len, sinks, span,
                                               C.c_float(scale), out, lse, None)


def prefill(lay=None, cache=None, q=P, qt=1, stride=ROW, cu=P, lens=P, max_q=8, sinks=4, span=64, scale=0.1, out=P, lse=P):
    lay, (c, keep) = lay or L(), (cache or _fake_cache())
    return kvq.lib().kvq_sink_prefill_attention(C.byref(lay.c()), C.byref(c), q, qt, stride, cu, lens, max_q, sinks, span,
                                                C.c_float(scale), out, lse, None)


def back(lay=None, cache=None, first=P, cu=P, lens=P, max_rows=8, k=P, v=P, dt=1):
    lay, (c, keep) = lay or L(), (cache or _fake_cache())
    return kvq.lib().kvq_read_back(C.byref(lay.c()), C.byref(c), first, cu, lens, max_rows, k, v, dt, None)


SHARED = [dict(q=None), dict(q=P + 8), dict(qt=2), dict(qt=-1), dict(stride=ROW - 8), dict(stride=ROW + 4),
          dict(stride=-ROW), dict(stride=0), dict(qt=0, stride=ROW + 2), dict(stride=1 << 41), dict(lens=None), dict(sinks=-1),
          dict(span=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(out=None), dict(out=P + 2), dict(lse=P + 2),
          dict(lay=L(window=-1))]


@pytest.mark.parametrize("kw", SHARED + [dict(max_len=-1)])
def test_decode_refuses(kw):
    assert decode(**kw) == BAD


@pytest.mark.parametrize("kw", SHARED + [dict(cu=None), dict(max_q=-1)])
def test_prefill_refuses(kw):
    assert prefill(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(first=None), dict(cu=None), dict(lens=None), dict(max_rows=-1),
                                dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 4), dict(dt=3)])
def test_read_back_refuses(kw):
    assert back(**kw) == BAD


@pytest.mark.parametrize("call", [decode, prefill, back])
def test_layouts_and_caches_are_checked(call):
    assert call(lay=L(k_bits=3)) == UNSUP
    assert call(lay=L(head_dim=96)) == UNSUP
    assert call(lay=L(k_per_channel=True, k_group=128)) == UNSUP
    assert call(cache=_fake_cache(window=False)) == BAD
    c, keep = _fake_cache()
    c.v_meta += 4
    assert call(cache=(c, keep)) == BAD
    c, keep = _fake_cache(batch=65536)
    assert call(cache=(c, keep)) == UNSUP
    c, keep = _fake_cache(batch=0)
    assert call(cache=(c, keep)) == OK


def test_read_back_bound_on_rows():
    assert back(max_rows=2 ** 31 - 1) == UNSUP
    assert back(max_rows=65533 * 64 + 1) == UNSUP


def test_nothing_to_do():
    assert prefill(max_q=0) == OK
    assert back(max_rows=0) == OK
    assert prefill(max_q=0, q=None, out=None) == OK


def test_binding_checks_before_the_call():
    lay = kvq.Layout(128, 32, 8, window=16)
    z = lambda: torch.zeros(64, dtype=torch.uint8)  # noqa: E731
    c = kvq.PagedCache(z(), z(), z(), z(), z(), z(), torch.zeros((2, 4), dtype=torch.int32), 8)
    lens, cu = torch.ones(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((2, 32, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.sink_decode_attention(lay, c, q, lens, 8, 4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.sink_prefill_attention(lay, c, q, cu, lens, 8, 4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.read_back(lay, c, lens, cu, lens, 2, 2)
    for bad, why in ((q[:1], "shape"), (q[:, :31], "shape"), (q.transpose(0, 1), "shape"), (q.half(), "CUDA tensor"),
                     (torch.zeros((2, 32, 256), dtype=torch.bfloat16)[:, :, ::2], "contiguous"),
                     (torch.zeros((2, 32, 160), dtype=torch.bfloat16)[:, :, :128], "contiguous")):
        with pytest.raises(ValueError, match=why):
            kvq.sink_decode_attention(lay, c, bad, lens, 8, 4, 64)
    with pytest.raises(ValueError, match="share a dtype"):
        kvq.kvq_read_back(lay, c, lens, cu, lens, 2, torch.zeros((2, 8, 128)), torch.zeros((2, 8, 128)).bfloat16())
