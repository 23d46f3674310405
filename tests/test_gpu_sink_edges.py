"""The attention with sinks at its edges, against fp64 numpy over the oracle's cache: clusters whose CTAs have no
tile, weights far below the largest, value scales far apart, scores of single tokens, queries with
NaN, caches that are elsewhere, first calls from several threads."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mixed_precision_quantized_kvq_b200 as kvq
import sink_reference as ref
import workloads as wl
from gpu_harness import Pair, torch_raw
from test_gpu_sink import INF, build, check_attention, i32, poison, small

pytestmark = pytest.mark.gpu


def widen(pair, pages):
    """A page table for `pages` pages a sequence, as a program that serves long sequences has it from the start."""
    wide = np.full((pair.pt.shape[0], pages), -1, np.int32)
    wide[:, : pair.pt.shape[1]] = pair.pt
    pair.pt = wide
    pair.gcache.page_table = torch.from_numpy(wide).cuda()


JOINED = {
    "bf16": dict(window=16),
    "fp32": dict(in_dtype=wl.DT_F32),
    "rotated": dict(rotate_keys=True, window=40),
    "rotated_fp32_d64": dict(rotate_keys=True, head_dim=64, v_group=64, in_dtype=wl.DT_F32),
    "groups16": dict(k_group=16, v_group=32),
    "per_channel": dict(k_per_channel=True, window=16),
    "per_channel_d64": dict(k_per_channel=True, head_dim=64, k_group=64, v_group=64),
}


# (kv-heads, sequences) that leave room for clusters of 8, 4 and 2 on 148 SMs: three blocks of rows a pair
@pytest.mark.parametrize("hkv,batch,ctas", [(1, 3, 8), (4, 3, 4), (4, 6, 2)])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("layout", list(JOINED))
def test_clusters_with_more_ctas_than_tiles(layout, long, hkv, batch, ctas):
    """First prompts of up to 130 positions (one to three tiles) under a page table of 512 pages, both blocks of a CTA in
    use, alone and beside a long sequence: right, and the same bits in each of 200 launches."""
    g, sms = 4, torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 148:
        pairs = 3 * hkv * batch                  # blocks of 64 queries for the 130
        assert pairs * ctas <= sms and (ctas == 8 or pairs * ctas * 2 > sms)
    w = small(batch=batch, num_kv_heads=hkv, num_q_heads=g * hkv, **JOINED[layout])
    lens = np.array([130, 97, 40, 64, 128, 75][:batch])
    n = lens.copy()
    if long:
        lens[0] = 3000
    pair = build(w, lens)
    widen(pair, 512)
    poison(pair)
    first, first_lse = check_attention(pair, n, 4, 2048, False)
    raw, _ = ref.queries(w, int(n.sum()))
    q, cu = torch_raw(raw), i32(np.concatenate([[0], np.cumsum(n)]))
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        out, lse = kvq.sink_prefill_attention(pair.glay, pair.gcache, q, cu, pair.glens, int(n.max()), 4, 2048)
        differ += (out != first).sum() + (lse != first_lse).sum()
    assert int(differ) == 0


@pytest.mark.parametrize("layout", ["groups16", "per_channel", "per_channel_d64"])
def test_single_tokens_in_clusters_with_more_ctas_than_tiles(layout):
    """Single tokens of the layouts that take the same kernel."""
    w = small(batch=3, num_kv_heads=1, num_q_heads=8, **JOINED[layout])
    pair = build(w, [130, 1, 40])
    widen(pair, 512)
    poison(pair)
    raw, f = ref.queries(w, 3)
    q = torch_raw(raw)
    first, first_lse = kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 512 * 64, 4, 4096)
    want, want_lse, tol, tol_l = ref.attention(pair.ocache, pair.pt, pair.signs, f, np.ones(3, int), pair.lens, 4, 4096,
                                               w.head_dim ** -0.5, True, True)
    ref.check_bf16(first.float().cpu().numpy(), want, tol=tol)
    ref.check_lse(first_lse.cpu().numpy(), want_lse, tol_l)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        out, lse = kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 512 * 64, 4, 4096)
        differ += (out != first).sum() + (lse != first_lse).sum()
    assert int(differ) == 0


# ---------------------------------------------------------------- weights far below the largest

FAR = {
    "exact_codes": dict(),
    "d64": dict(head_dim=64, v_group=64),
    "groups16": dict(k_group=16, v_group=32),
    "per_channel": dict(k_per_channel=True),
}


@pytest.mark.parametrize("low,high", [(20, 26), (26, 30)])
@pytest.mark.parametrize("form", ["token", "chunk shared by a cluster", "chunk"])
@pytest.mark.parametrize("layout", list(FAR))
def test_one_page_far_above_the_others(layout, form, low, high):
    """A first page of weight 1 and value 0, and 30000 positions 2^-low to 2^-high below it with values around 1: what
    they add up to is the whole output.  Keys are constant over their groups, values over a position, and queries have
    one channel, so scores, keys and values are exact and the weights' rounding to fp16 is all that counts.  With the
    largest weight at 2^8 or more, each is off by at most 2^-11 of itself or half a subnormal step, 2^-25:
        |out error| <= 2^-11 sum a |v| + 2^-33 a_max sum |v|
    and the fp32 sums add to the former: about 500 tiles' sums of the weights and 4 products a tile, each off by at most
    2^-23 of the whole: 2^-14 + 2^-12."""
    w = small(batch=1, num_kv_heads=1, num_q_heads=2, **FAR[layout])
    L, d, r = 30016, w.head_dim, np.random.default_rng(5)
    key = np.repeat(-r.integers(low * 8, high * 8, L // 64) / 8.0, 64)   # constant over a page: 1/8 is a bf16 step there
    val = r.integers(32, 97, L) / 64.0
    key[:64], val[:64] = 0.0, 0.0
    pair = Pair(w, np.array([L], np.int32))
    pair.lens[:] = 0
    pair.glens.zero_()
    rows = lambda x: wl.bf16_bits(np.repeat(x.astype(np.float32), d).reshape(L, 1, d))  # noqa: E731
    pair.append(rows(key), rows(val), np.array([0, L]))
    pair.compare_cache()
    n = np.array([1 if form == "token" else 40])
    q = np.zeros((int(n[0]), 2, d), np.float32)
    q[:, :, 3] = 1.0
    raw, scale, cu = torch_raw(wl.bf16_bits(q)), float(np.log(2.0)), i32([0, n[0]])
    if form == "token":
        out, lse = kvq.sink_decode_attention(pair.glay, pair.gcache, raw, pair.glens, L, 64, INF, scale)
    else:                                        # (a bound of 20000 queries: blocks enough for every SM)
        out, lse = kvq.sink_prefill_attention(pair.glay, pair.gcache, raw, cu, pair.glens, 40 if "cluster" in form else 20000,
                                              64, INF, scale)
    want, want_lse = ref.attention(pair.ocache, pair.pt, None, q.astype(np.float64), n, pair.lens, 64, INF, scale)
    tol = (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -14) * want + 2.0 ** -33 * np.exp(-want_lse)[:, :, None] * val.sum()
    ref.check_bf16(out.float().cpu().numpy(), want, tol=tol)
    ref.check_lse(lse.cpu().numpy(), want_lse, np.full(want_lse.shape, 2.0 ** -14))



@pytest.mark.parametrize("large", [0, 7])
@pytest.mark.parametrize("vb,vg,d", [(1, 32, 128), (2, 32, 128), (4, 16, 128), (8, 64, 128), (2, 16, 64), (8, 32, 64)])
def test_value_groups_of_different_scales(vb, vg, d, large):
    """Single tokens over exact codes: values of the first group around 2^large and of the others around 2^-6, weights from
    1 down to 2^-24.  Keys and queries as above (scores are exact).  The bound of the two roundings to fp16, of a weight
    and of its product with the scale, and of fp32 sums over 64 pages of 4 products at 2^-23 each (2^-15, and as much
    again for the rest):
        2^-11 sum a (|v| + |code*scale|) + 2^-14 sum a (|code*scale| + |zero|)
        + 2^(s-36) a_max sum (|code*scale| + |zero| + c)"""
    w = small(batch=1, num_kv_heads=1, num_q_heads=3, head_dim=d, v_bits=vb, v_group=vg)
    L, r = 4096, np.random.default_rng(7)
    key = np.repeat(-r.integers(10 * 8, 24 * 8, L // 64) / 8.0, 64)
    key[:64] = 0.0
    val = r.standard_normal((L, d)) * np.where(np.arange(d) < vg, 2.0 ** large, 2.0 ** -6)
    val[:64] *= 2.0 ** -4                                     # the largest weights' values do not hide the others'
    pair = Pair(w, np.array([L], np.int32))
    pair.lens[:] = 0
    pair.glens.zero_()
    pair.append(wl.bf16_bits(np.repeat(key.astype(np.float32), d).reshape(L, 1, d)),
                wl.bf16_bits(val.astype(np.float32).reshape(L, 1, d)), np.array([0, L]))
    pair.compare_cache()
    q = np.zeros((1, 3, d), np.float32)
    q[:, :, 3] = 1.0
    out, lse = kvq.sink_decode_attention(pair.glay, pair.gcache, torch_raw(wl.bf16_bits(q)), pair.glens, L, 64, INF,
                                         float(np.log(2.0)))
    want, want_lse = ref.attention(pair.ocache, pair.pt, None, q.astype(np.float64), np.ones(1, int), pair.lens, 64, INF,
                                   float(np.log(2.0)))
    v = pair.ocache.dequantize(pair.lens, L)[1][0, 0].astype(np.float64)
    groups = v.reshape(L, d // vg, vg)
    zero = np.repeat(groups.min(-1), vg, -1)                  # code 0 is a group's smallest value
    s = max(0.0, np.ceil(np.log2((groups.max(-1) - groups.min(-1)).max() / (2 ** vb - 1)) + 1e-3))
    code = v - zero
    a = np.exp(key * np.log(2.0))
    a /= a.sum()
    c = {1: 129, 2: 771, 4: 255, 8: 255}[vb]
    tol = (2.0 ** -11 * (a @ (np.abs(v) + code)) + 2.0 ** -14 * (a @ (code + np.abs(zero)))
           + 2.0 ** (s - 36) * a.max() * (code + np.abs(zero) + c).sum(0))
    ref.check_bf16(out.float().cpu().numpy()[0], want[0], tol=np.broadcast_to(tol, want[0].shape))
    ref.check_lse(lse.cpu().numpy(), want_lse, np.full(want_lse.shape, 2.0 ** -14))



# ---------------------------------------------------------------- scores of single tokens

SINGLE = {
    "exact_codes": dict(),
    "exact_codes_rotated": dict(rotate_keys=True, window=40),
    "groups16": dict(k_group=16, v_group=32, window=16),
    "groups16_d64": dict(k_group=16, head_dim=64, v_group=64),
    "groups16_rotated": dict(k_group=16, rotate_keys=True, window=40),
    "per_channel": dict(k_per_channel=True, window=16),
    "per_channel_g16": dict(k_per_channel=True, k_group=16),
    "per_channel_d64": dict(k_per_channel=True, k_group=64, head_dim=64, v_group=64),
}


@pytest.mark.parametrize("kb", [1, 2, 4, 8])
@pytest.mark.parametrize("length", [200, 5000])
@pytest.mark.parametrize("layout", list(SINGLE))
def test_single_tokens_have_fp32_scores(layout, length, kb):
    """lse of single tokens where every fp16 rounding would go the same way: keys 1 and 1 + 3*2^-13 (a quarter of their groups
    the latter), queries 1 + 2^-12 with as much again from channel to channel.  Keys and queries count to 2^-22 of
    themselves (or half of fp16's smallest step, 2^-25), products are exact, and the fp32 sums of a score have up to 40
    terms (products of 16 channels, of the two parts, of 32-channel units), each off by up to 2^-23 of the magnitudes'
    sum:
        |score error| <= |sm_scale| (sum |q_j k_j| (2^-21 + 40 * 2^-23) + sum |q_j| 2^-25)
    and lse by as much and its own fp32 steps.  (Rounded to fp16, keys alone would move it by 8e-4.)"""
    w = small(batch=2, num_kv_heads=2, num_q_heads=6, in_dtype=wl.DT_F32, k_bits=kb, **SINGLE[layout])
    lens, d, r = np.array([length, 77], np.int32), w.head_dim, np.random.default_rng(11)
    pair = Pair(w, lens)
    pair.lens[:] = 0
    pair.glens.zero_()
    total = int(lens.sum())
    k = np.where(r.random((total, 2, d)) < 0.25, 1.0 + 3 * 2.0 ** -13, 1.0).astype(np.float32)
    v = r.standard_normal((total, 2, d)).astype(np.float32)
    pair.append(k, v, np.array([0, length, total], np.int32))
    if w.rotate_keys:                            # (fp32 rotations differ in their last bits: the GPU's codes are the cache)
        for name in ("k_codes", "k_meta", "v_codes", "v_meta", "k_win", "v_win"):
            o = getattr(pair.ocache, name).view(np.uint8).ravel()
            if getattr(pair.gcache, name) is not None:
                o[:] = pair.gpu_bytes(name)[: o.size]
    q = (1.0 + 2.0 ** -12 * (1 + np.arange(d) % 2 * 2.0 ** -8) + np.zeros((2, 6, d))).astype(np.float32)
    scale = d ** -0.5
    out, lse = kvq.sink_decode_attention(pair.glay, pair.gcache, torch_raw(q), pair.glens, length, 4, 3000)
    _, want = ref.attention(pair.ocache, pair.pt, pair.signs, q.astype(np.float64), np.ones(2, int), pair.lens, 4, 3000, scale)
    keys = np.abs(pair.ocache.dequantize(pair.lens, length)[0].astype(np.float64))
    D = np.zeros((2, 6))
    for b in range(2):
        paged = np.arange(lens[b]) < ref.paged_len(pair.olay, lens[b])
        for h in range(6):
            x, qh = keys[b, h // 3, : lens[b]], np.abs(q[b, h].astype(np.float64))
            turned = np.zeros(lens[b])
            if w.rotate_keys:
                # codes and zero points are larger than the keys they add up to; a rotated query's channel is off by ten
                # steps of sums that are at most sum |q| / sqrt(d)
                x = np.where(paged[:, None], 3 * np.repeat(x.reshape(lens[b], -1, w.k_group).max(-1), w.k_group, -1), x)
                turned = paged * 10 * 2.0 ** -24 * qh.sum() / np.sqrt(d) * x.sum(-1)
            rot = np.abs((q[b, h] * pair.signs) @ ref.hadamard(d)) if w.rotate_keys else qh
            mag = np.where(paged, x @ rot, x @ qh)
            D[b, h] = scale * (mag * (2.0 ** -21 + 40 * 2.0 ** -23) + np.maximum(rot.sum(), qh.sum()) * 2.0 ** -25 + turned).max()
    ref.check_lse(lse.cpu().numpy(), want, D + 2.0 ** -21 * (1 + np.abs(want)))



@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
@pytest.mark.parametrize("kb", [1, 2, 4, 8])
@pytest.mark.parametrize("d,kg", [(64, 32), (64, 64), (128, 32), (128, 128)])
def test_sums_over_raw_codes(d, kg, kb, dtype):
    """One position, so that lse is its score: 64 keys that are codes times a scale, eight random queries each.  The
    products of bf16 queries and codes are exact; an fp32 query's two parts are 2^-22 of it off; the score then has at
    most 16 sums (four products of a unit of 32 channels, two of them low; four units), each off by 2^-24 of the
    magnitudes' sum:
        |error| <= (2^-22 + 2^-20) sum |q_j k_j|, and half a step of the result."""
    B, r = 64, np.random.default_rng(1)
    w = small(batch=B, num_kv_heads=1, num_q_heads=8, head_dim=d, k_bits=kb, k_group=kg, v_group=64, in_dtype=wl.DT_F32)
    pair = Pair(w, np.ones(B, np.int32))
    pair.lens[:] = 0
    pair.glens.zero_()
    code = r.integers(0, 2 ** kb, (B, 1, d // kg, kg)) * 1.0
    code[..., 0], code[..., 1] = 0, 2 ** kb - 1
    scale = r.integers(1, 256, (B, 1, d // kg, 1)) / 16.0
    k = (code * scale).reshape(B, 1, d).astype(np.float32)
    pair.append(k, np.zeros_like(k), np.arange(B + 1, dtype=np.int32))
    pair.compare_cache()
    q = r.standard_normal((B, 8, d)).astype(np.float32)
    raw = q
    if dtype == wl.DT_BF16:
        raw = wl.bf16_bits(q)
        q = wl.bf16_to_f32(raw)
    _, lse = kvq.sink_decode_attention(pair.glay, pair.gcache, torch_raw(raw), pair.glens, 1, 0, 1, 1.0)
    kk = pair.ocache.dequantize(pair.lens, 1)[0][:, 0, 0].astype(np.float64)
    want = np.einsum("bhd,bd->bh", q.astype(np.float64), kk)
    ref.check_lse(lse.cpu().numpy(), want, (2.0 ** -22 + 2.0 ** -20) * np.einsum("bhd,bd->bh", np.abs(q), kk)
                  + 2.0 ** -22 * np.abs(want))



@pytest.mark.parametrize("d", [64, 128])
def test_fp32_queries_against_the_ring(d):
    """One position in the ring, so that lse is its score.  Queries whose first two bf16 parts leave the same 0.75 * 2^-16 in
    every channel; three parts hold all of them.  Keys of one sign; a score has at most 24 sums (three parts of eight
    products of 16 channels), each off by 2^-24 of it: 2^-19, and half a step of the result."""
    B, r = 16, np.random.default_rng(2)
    w = small(batch=B, num_kv_heads=1, num_q_heads=8, head_dim=d, v_group=64, window=64, in_dtype=wl.DT_F32)
    pair = Pair(w, np.ones(B, np.int32))
    pair.lens[:] = 0
    pair.glens.zero_()
    k = (r.integers(64, 128, (B, 1, d)) / 64.0).astype(np.float32)
    pair.append(k, np.zeros_like(k), np.arange(B + 1, dtype=np.int32))
    pair.compare_cache()
    q = np.full((B, 8, d), 1.0 + 2.0 ** -8 + 0.75 * 2.0 ** -16, np.float32)
    _, lse = kvq.sink_decode_attention(pair.glay, pair.gcache, torch_raw(q), pair.glens, 1, 0, 1, 1.0)
    want = np.einsum("bhd,bd->bh", q.astype(np.float64), k[:, 0].astype(np.float64))
    ref.check_lse(lse.cpu().numpy(), want, (2.0 ** -19 + 2.0 ** -23) * want)


# ---------------------------------------------------------------- NaN

@pytest.mark.parametrize("form", ["token", "chunk shared by a cluster", "chunk"])
@pytest.mark.parametrize("layout", list(JOINED))
def test_a_query_with_nan(layout, form):
    """Its outputs and lse are NaN in every form (an lse of -inf would say that it saw nothing); the other heads and rows
    keep their bits; a query that sees nothing has 0 and -inf whatever it holds."""
    w = small(batch=2, num_kv_heads=2, num_q_heads=6, **JOINED[layout])
    pair = build(w, [700, 90])
    n = np.array([1, 1] if form == "token" else [60, 33])
    raw, _ = ref.queries(w, int(n.sum()))
    q, cu = torch_raw(raw), i32(np.concatenate([[0], np.cumsum(n)]))

    def call(span):
        if form == "token":
            return kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 700, 4 if span else 0, span)
        bound = 60 if "cluster" in form else 20000
        return kvq.sink_prefill_attention(pair.glay, pair.gcache, q, cu, pair.glens, bound, 4 if span else 0, span)

    out, lse = (t.clone() for t in call(600))
    bad = torch.zeros_like(lse, dtype=torch.bool)
    for row, head, channel in ((0, 1, 5), (0, 3, 0), (int(n.sum()) - 1, 5, w.head_dim - 1)):
        q[row, head, channel] = float("nan")
        bad[row, head] = True
    got, got_lse = call(600)
    assert torch.all(got[bad].isnan()) and torch.all(got_lse[bad].isnan())
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])
    got, got_lse = call(0)
    assert torch.all(got == 0) and torch.all(got_lse == -float("inf"))



# ---------------------------------------------------------------- refused on the host

@pytest.mark.parametrize("name", ["page_table", "k_codes", "v_codes", "k_meta", "v_meta", "k_win", "v_win", "rot_signs"])
def test_a_cache_on_another_device(name):
    """A buffer of the cache in host memory, or a page table of 64-bit numbers, is refused before anything is launched."""
    w = small(batch=2, rotate_keys=True, window=40)
    pair = build(w, [100, 90])
    q, cu = torch_raw(ref.queries(w, 2)[0]), i32([0, 1, 2])

    def refused(match):
        with pytest.raises(ValueError, match=match):
            kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 100, 4, 50)
        with pytest.raises(ValueError, match=match):
            kvq.sink_prefill_attention(pair.glay, pair.gcache, q, cu, pair.glens, 1, 4, 50)
        with pytest.raises(ValueError, match=match):
            kvq.read_back(pair.glay, pair.gcache, i32([0, 0]), cu, pair.glens, 2, 1)

    holder = pair.glay if name == "rot_signs" else pair.gcache
    kept = getattr(holder, name)
    setattr(holder, name, kept.cpu())
    refused("is on cpu")
    if name == "page_table":
        setattr(holder, name, kept.long())
        refused("int32")
    setattr(holder, name, kept)
    kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 100, 4, 50)


# ---------------------------------------------------------------- threads

THREADS = """
import threading
import numpy as np, torch
from test_gpu_sink import build, i32, small
import mixed_precision_quantized_kvq_b200 as kvq
import sink_reference as ref
from gpu_harness import torch_raw

pairs = [build(small(batch=2, **kw), [300, 90]) for kw in (dict(window=16), dict(k_per_channel=True, window=16))]
q, cu = torch_raw(ref.queries(pairs[0].w, 100)[0]), i32([0, 60, 100])
start, got, failed = threading.Barrier(8), [None] * 8, []

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            got[i] = [t for p in pairs for t in (
                *kvq.sink_decode_attention(p.glay, p.gcache, q[:2], p.glens, 300, 4, 100),
                *kvq.sink_prefill_attention(p.glay, p.gcache, q, cu, p.glens, 60, 4, 100),
                kvq.prefill_attention(p.glay, p.gcache, q, cu, p.glens, 60)[0])]
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        failed.append(e)

torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))
"""


def test_first_calls_from_several_threads():
    """A process whose threads make the first call of every kernel side by side, each on its own stream."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", THREADS], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
