"""GPU parity of the attention with sinks and a sliding span, and of reading
the cache back, against fp64 numpy over the oracle's cache."""
import numpy as np
import pytest
import torch

import mixed_precision_quantized_kvq_b200 as kvq
import sink_reference as ref
import workloads as wl
from gpu_harness import Pair, torch_raw

pytestmark = pytest.mark.gpu

INF = 2 ** 31 - 1


def small(**kw):
    base = dict(name="sink", batch=4, num_q_heads=8, num_kv_heads=2, head_dim=128, seq_len=0, k_bits=4, v_bits=2,
                k_group=32, v_group=128, window=0, ragged=(1, 500), shuffle_pages=True,
                outliers=("random", 4, 10.0), seed=23)
    base.update(kw)
    return wl.Workload(**base)


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def build(w, lens):
    pair = Pair(w, np.asarray(lens, np.int32))
    pair.prefill(with_f32=False)
    if w.rotate_keys:
        # the rotation before quantizing is fp32 on the GPU: a code may differ from the oracle's, which here only has to
        # hold the same cache
        for name in ("k_codes", "k_meta", "v_codes", "v_meta", "k_win", "v_win"):
            o = getattr(pair.ocache, name).view(np.uint8).ravel()
            if getattr(pair.gcache, name) is not None:
                o[:] = pair.gpu_bytes(name)[: o.size]
    else:
        pair.compare_cache()
    return pair


def poison(pair):
    """Everything that no position uses becomes NaN: fp16 metadata, ring slots and the codes beside them."""
    w, lay = pair.w, pair.olay
    used = np.zeros((pair.num_pages, 64), bool)
    for b in range(w.batch):
        for x in range(ref.paged_len(lay, pair.lens[b])):
            pg = pair.pt[b, x // 64]
            if pg >= 0:
                used[pg, x % 64] = True
    H, d = w.num_kv_heads, w.head_dim
    free = torch.from_numpy(~used).cuda()
    vm = pair.gcache.v_meta[: pair.num_pages * H * 64 * (d // w.v_group) * 4].view(pair.num_pages, H, 64, -1)
    vm.masked_fill_(free[:, None, :, None], 0xFF)
    if not w.k_per_channel:
        km = pair.gcache.k_meta[: pair.num_pages * H * 64 * (d // w.k_group) * 4].view(pair.num_pages, H, 64, -1)
        km.masked_fill_(free[:, None, :, None], 0xFF)
    if lay.ring_slots:
        R = lay.ring_slots
        live = np.zeros((w.batch, R), bool)
        for b in range(w.batch):
            live[b, np.arange(ref.paged_len(lay, pair.lens[b]), pair.lens[b]) % R] = True
        dead = torch.from_numpy(~live).cuda()
        for t in (pair.gcache.k_win, pair.gcache.v_win):
            t[: w.batch * H * R * d * 2].view(w.batch, H, R, d * 2).masked_fill_(dead[:, None, :, None], 0xFF)


def exact_codes(w):
    """Layouts whose single-token kernel multiplies the codes themselves; the others round keys and values to fp16."""
    return w.k_group >= 32 and not w.k_per_channel


def check_attention(pair, n, sinks, span, decode, step=0, stride=None, scale=None):
    """One call against the reference; rows of skipped sequences stay as they were."""
    w = pair.w
    scale = w.head_dim ** -0.5 if scale is None else scale
    rows = int(np.sum(n))
    raw, q = ref.queries(w, rows, step)
    tq = torch_raw(raw)
    if stride:
        wide = torch.full((rows, stride), float("nan"), dtype=tq.dtype, device="cuda")
        wide[:, : tq.shape[1] * tq.shape[2]] = tq.flatten(1)
        tq = wide[:, : tq.shape[1] * tq.shape[2]].unflatten(1, tq.shape[1:])
    out = torch.full((rows, w.num_q_heads, w.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, w.num_q_heads), 7.0, device="cuda")
    if decode:
        kvq.kvq_sink_decode_attention(pair.glay, pair.gcache, tq, pair.glens, int(pair.lens.max()), sinks, span, scale,
                                      out, lse)
        n = np.ones(w.batch, np.int64)
    else:
        cu = np.concatenate([[0], np.cumsum(n)])
        kvq.kvq_sink_prefill_attention(pair.glay, pair.gcache, tq, i32(cu), pair.glens, int(np.max(n)), sinks, span,
                                       scale, out, lse)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_l = ref.attention(pair.ocache, pair.pt, pair.signs, q, n, pair.lens, sinks, span, scale,
                                               w.in_dtype == wl.DT_BF16, True)
    if decode and exact_codes(w):
        tol, tol_l = 1e-3 + 1e-3 * np.abs(want), 1e-3 + 1e-3 * np.abs(want_lse)
    got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
    skipped = np.isnan(want_lse)
    if decode:                                   # an empty sequence has an answer here
        want[skipped], want_lse[skipped], tol[skipped] = 0.0, -np.inf, 0.0
        skipped = np.zeros_like(skipped)
    assert np.all(got[skipped] == 7.0) and np.all(got_lse[skipped] == 7.0)
    ref.check_bf16(got[~skipped], want[~skipped], tol=tol[~skipped])
    ref.check_lse(got_lse[~skipped], want_lse[~skipped], tol_l[~skipped])
    return out, lse


LAYOUTS = {
    "plain": dict(),
    "ring": dict(window=100),
    "d64_g3": dict(head_dim=64, num_q_heads=6, v_group=64, window=16),
    "g1_groups128": dict(num_q_heads=2, k_group=128, v_group=32),
    "g8_groups64": dict(num_q_heads=16, k_group=64, v_group=64, window=64),
    "g7_groups16": dict(num_q_heads=14, k_group=16, v_group=16, window=5),
    "rotated": dict(rotate_keys=True, window=40, outliers=("student_t", 4, 10.0, 3.0)),
    "d64_rotated": dict(rotate_keys=True, head_dim=64, v_group=32, window=70),
    "per_channel": dict(k_per_channel=True, window=16),
    "per_channel_d64": dict(k_per_channel=True, head_dim=64, k_group=64, v_group=64, num_q_heads=10),
    "fp32": dict(in_dtype=wl.DT_F32, window=33, num_q_heads=16),
}
SPANS = [(0, 0), (5, 0), (0, 1), (4, 64), (64, 200), (70, 1), (INF, 3), (0, INF), (9, 333)]


@pytest.mark.parametrize("sinks,span", SPANS)
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_decode(layout, sinks, span):
    w = small(**LAYOUTS[layout], batch=6)
    pair = build(w, [0, 1, 64, 333, 500, 130])
    poison(pair)
    check_attention(pair, np.ones(6, int), sinks, span, True)


@pytest.mark.parametrize("sinks,span", SPANS)
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_prefill(layout, sinks, span):
    w = small(**LAYOUTS[layout], batch=6)
    pair = build(w, [0, 1, 64, 333, 500, 130])
    poison(pair)
    check_attention(pair, np.array([0, 1, 3, 257, 33, 130]), sinks, span, False)


@pytest.mark.parametrize("kb", [1, 2, 4, 8])
@pytest.mark.parametrize("vb", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_bit_widths(kb, vb, d):
    w = small(k_bits=kb, v_bits=vb, head_dim=d, v_group=d, window=10, batch=2)
    pair = build(w, [300, 70])
    check_attention(pair, np.ones(2, int), 3, 150, True)
    check_attention(pair, np.array([140, 9]), 3, 150, False)
    wp = w.with_(k_per_channel=True)
    pair = build(wp, [300, 70])
    check_attention(pair, np.ones(2, int), 3, 150, True)
    check_attention(pair, np.array([140, 9]), 3, 150, False)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 300])
def test_chunk_lengths(n):
    w = small(window=64, num_q_heads=10, batch=2)
    pair = build(w, [700, n])
    check_attention(pair, np.array([n, n]), 4, 128, False)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 63, 64, 65, 127, 128, 129, 191, 200])
def test_lengths(length):
    for window in (0, 1, 64, 300):
        w = small(window=window, batch=1)
        pair = build(w, [length])
        check_attention(pair, np.ones(1, int), 2, 100, True)
        check_attention(pair, np.array([length]), 2, 100, False)


def test_long_context_split():
    """Few pairs and a long span: the span is shared between many blocks."""
    w = small(batch=1, window=128, num_kv_heads=1, num_q_heads=4)
    pair = build(w, [20000])
    check_attention(pair, np.ones(1, int), 4, INF, True)
    check_attention(pair, np.ones(1, int), 4, 9001, True)
    check_attention(pair, np.array([100]), 4, INF, False)


@pytest.mark.parametrize("kw", [dict(k_per_channel=True, window=16), dict(k_group=16), dict(rotate_keys=True, window=40),
                                dict(head_dim=64, v_group=64, window=128)])
def test_shared_tiles(kw):
    """Few rows and many tiles: a chunk's (or, where codes are not multiplied as they are, a token's) tiles are shared by
    the CTAs of a cluster; one of the sequences has fewer tiles than there are CTAs, one nothing to see."""
    w = small(batch=3, num_kv_heads=1, num_q_heads=3, **kw)
    pair = build(w, [5000, 0, 100])
    poison(pair)
    for sinks, span in ((4, INF), (70, 3001), (0, 0)):
        check_attention(pair, np.ones(3, int), sinks, span, True)
        check_attention(pair, np.array([90, 0, 3]), sinks, span, False)
        check_attention(pair, np.array([1, 0, 1]), sinks, span, False)


def test_released_pages():
    """Pages between the sinks and the span are released: same answers; a released page that would be seen counts
    as absent; table entries out of range are absent too."""
    w = small(batch=3, window=16)
    pair = build(w, [700, 650, 90])
    a, al = check_attention(pair, np.ones(3, int), 4, 128, True)
    c, cl = check_attention(pair, np.array([60, 1, 5]), 4, 128, False)
    for b, L in enumerate((700, 650)):
        pair.pt[b, 1:(L - 60 - 127) // 64] = -1
    pair.gcache.page_table = torch.from_numpy(pair.pt).cuda()
    poison(pair)
    for x, y in zip((a, al, c, cl), (*check_attention(pair, np.ones(3, int), 4, 128, True),
                                     *check_attention(pair, np.array([60, 1, 5]), 4, 128, False))):
        assert torch.equal(x, y)
    for bad in (-1, -7, pair.num_pages, INF):
        pair.pt[0, 9] = bad
        pair.gcache.page_table = torch.from_numpy(pair.pt).cuda()
        pair.pt[0, 9] = -1
        check_attention(pair, np.ones(3, int), 4, 200, True)
        check_attention(pair, np.array([60, 1, 5]), 4, 200, False)
    pair.pt[:] = -1                                      # nothing but the ring is left
    pair.gcache.page_table = torch.from_numpy(pair.pt).cuda()
    check_attention(pair, np.ones(3, int), 4, INF, True)
    check_attention(pair, np.array([60, 1, 5]), 4, 5, False)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32])
def test_query_rows_of_a_wider_projection(dtype):
    w = small(window=20, in_dtype=dtype)
    pair = build(w, [100, 300, 64, 7])
    check_attention(pair, np.ones(4, int), 4, 64, True, stride=(8 + 2 * 2) * 128)
    check_attention(pair, np.array([50, 129, 0, 7]), 4, 64, False, stride=(8 + 2 * 2) * 128)


def test_skipped_sequences_and_scales():
    w = small(window=20)
    pair = build(w, [100, 3, 64, 7])
    check_attention(pair, np.array([50, 5, 0, 7]), 4, 64, False)       # five queries for three positions
    for scale in (0.0, -0.1, 0.2):
        check_attention(pair, np.ones(4, int), 4, 64, True, scale=scale)
        check_attention(pair, np.array([50, 1, 0, 7]), 4, 64, False, scale=scale)


def test_lengths_above_the_bound_are_clamped():
    w = small(batch=2, window=0)
    pair = build(w, [300, 200])
    raw, _ = ref.queries(w, 2)
    q = torch_raw(raw)
    a, la = kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 250, 4, 64)
    pair.glens.clamp_(max=250)
    b, lb = kvq.sink_decode_attention(pair.glay, pair.gcache, q, pair.glens, 250, 4, 64)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_small_values_and_large():
    """Keys and values far from unit scale keep their relative accuracy."""
    for factor in (2.0 ** -9, 2.0 ** 8):
        w = small(batch=2, window=32, in_dtype=wl.DT_F32)
        pair = Pair(w, np.array([500, 300], np.int32))
        kr, vr, _, _, cu, _ = wl.prefill(w, pair.lens, with_f32=False)
        pair.lens[:] = 0
        pair.glens.zero_()
        pair.append((kr * np.float32(factor)).astype(np.float32), (vr * np.float32(factor)).astype(np.float32), cu)
        pair.compare_cache()
        for n, decode in ((np.ones(2, int), True), (np.array([40, 200]), False)):
            raw, q = ref.queries(w, int(n.sum()))
            scale = 128 ** -0.5 / factor
            if decode:
                out, _ = kvq.sink_decode_attention(pair.glay, pair.gcache, torch_raw(raw), pair.glens, 500, 4, 200, scale)
            else:
                out, _ = kvq.sink_prefill_attention(pair.glay, pair.gcache, torch_raw(raw), i32([0, 40, 240]), pair.glens,
                                                    200, 4, 200, scale)
            want, _, tol, _ = ref.attention(pair.ocache, pair.pt, None, q, n, pair.lens, 4, 200, scale, False, True)
            tol = 1e-3 + 1e-3 * np.abs(want / factor) if decode else tol / factor
            ref.check_bf16(out.float().cpu().numpy() / factor, want / factor, tol=tol)


# ---------------------------------------------------------------- reading back

def check_back(pair, first, n, dtype):
    cu = np.concatenate([[0], np.cumsum(n)])
    k, v = kvq.read_back(pair.glay, pair.gcache, i32(first), i32(cu), pair.glens, int(cu[-1]), int(np.max(n)), dtype)
    want = ref.rows_back(pair.ocache, pair.pt, pair.signs, first, n, pair.lens)
    half = 2.0 ** -24 if dtype == torch.float32 else ref.HALF_BF16
    # rotated keys: log2(d) fp32 additions and two products, each off by half a step of a partial sum that is at most
    # sqrt(d) times the row's norm in magnitude before the division by sqrt(d)
    d = pair.w.head_dim
    for got, x, turn in ((k, want[0], pair.signs is not None), (v, want[1], False)):
        got = got.double().cpu().numpy()
        sum_err = (np.log2(d) + 2) * 2.0 ** -24 * np.linalg.norm(x, axis=-1, keepdims=True) if turn else 0.0
        lim = half * np.abs(x) + 2.0 ** -24 * np.abs(x) + sum_err * (1 + half)
        assert np.all(np.abs(got - x) <= lim)
    return k, v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_read_back(layout, dtype):
    w = small(**LAYOUTS[layout], batch=6)
    pair = build(w, [0, 1, 64, 333, 500, 130])
    poison(pair)
    check_back(pair, [0, 0, 10, 0, 401, 63], [3, 1, 40, 333, 99, 2], dtype)
    # out of range at either end, nothing at all, far away
    check_back(pair, [-5, 0, 60, -1000, 499, INF - 3], [9, 0, 70, 100, 3, 5], dtype)
    pair.pt[3, 2] = -1
    pair.gcache.page_table = torch.from_numpy(pair.pt).cuda()
    check_back(pair, [0, 0, 0, 100, 0, 0], [0, 0, 0, 150, 0, 0], dtype)


@pytest.mark.parametrize("kb,vb", [(1, 8), (2, 4), (8, 1), (4, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_read_back_bit_widths(kb, vb, d):
    for pc in (False, True):
        w = small(k_bits=kb, v_bits=vb, head_dim=d, v_group=d, window=10, batch=2, k_per_channel=pc)
        pair = build(w, [300, 70])
        check_back(pair, [1, 0], [299, 70], torch.float32)


def test_read_back_skips_longer_runs():
    w = small(batch=2)
    pair = build(w, [300, 200])
    k = torch.full((30, 2, 128), 7.0, device="cuda")
    v = torch.full_like(k, 7.0)
    kvq.kvq_read_back(pair.glay, pair.gcache, i32([5, 6]), i32([0, 10, 30]), pair.glens, 15, k, v)
    assert torch.all(k[10:] == 7.0) and torch.all(v[10:] == 7.0) and not torch.any(k[:10] == 7.0)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kw", [dict(window=32), dict(rotate_keys=True, window=8), dict(k_per_channel=True, window=16)])
def test_serving_with_released_pages(kw):
    """A prompt in chunks, then decode steps, with a physical pool that holds only what the span and the sinks need:
    pages are released as they fall out of the span and mapped again for new positions.  Then the visible rows are
    read back and appended to a cache of another layout, bit for bit what the oracle makes of them."""
    sinks, span, P = 4, 150, 64
    w = small(batch=2, ragged=None, **kw)
    total = 700
    kr, vr, _, _ = zip(*(wl.seq_kv(w, b, total) for b in range(2)))
    pool = 2 * 8
    pair = Pair(w, np.array([total, total], np.int32))       # the oracle keeps every page
    free = list(range(pool))
    gpt = np.full_like(pair.pt, -1)
    cache = kvq.PagedCache.allocate(pair.glay, torch.from_numpy(gpt).cuda(), pool)
    pair.gcache, pair.lens = cache, np.zeros(2, np.int32)
    pair.glens.zero_()
    steps = [90, 128, 61, 100] + [1] * 8 + [77] + [1] * 5
    for i, m in enumerate(steps):
        L = int(pair.lens[0])
        for b in range(2):
            for lp in range(gpt.shape[1]):
                # the queries to come sit at L and later
                if gpt[b, lp] >= 0 and lp * P >= sinks and (lp + 1) * P - 1 <= L - span and (lp + 1) * P <= L - w.window:
                    free.append(int(gpt[b, lp]))
                    gpt[b, lp] = -1
            for lp in range(max(0, L - w.window - w.k_group) // P, (max(0, L + m - w.window) + P - 1) // P):
                if gpt[b, lp] < 0:
                    gpt[b, lp] = free.pop()
        cache.page_table.copy_(torch.from_numpy(gpt))
        pair.append(np.concatenate([x[L:L + m] for x in kr]), np.concatenate([x[L:L + m] for x in vr]),
                    np.array([0, m, 2 * m], np.int32))
        raw, q = ref.queries(w, 2 * m, i)
        if m == 1:
            out, lse = kvq.sink_decode_attention(pair.glay, cache, torch_raw(raw), pair.glens, L + m, sinks, span)
        else:
            out, lse = kvq.sink_prefill_attention(pair.glay, cache, torch_raw(raw), i32([0, m, 2 * m]), pair.glens, m, sinks,
                                                  span)
        want, want_lse, tol, tol_l = ref.attention(pair.ocache, pair.pt, pair.signs, q, [m, m], pair.lens, sinks, span,
                                                   128 ** -0.5, True, True)
        if m == 1 and exact_codes(w):
            tol, tol_l = None, None
        ref.check_bf16(out.float().cpu().numpy(), want, tol=tol)
        ref.check_lse(lse.cpu().numpy(), want_lse, tol_l)
    L = int(pair.lens[0])
    n = [span, span]
    k, v = kvq.read_back(pair.glay, cache, i32([L - span] * 2), i32([0, span, 2 * span]), pair.glens, 2 * span, span)
    wk, wv = ref.rows_back(pair.ocache, pair.pt, pair.signs, [L - span] * 2, n, pair.lens)
    ref.check_bf16(k.float().cpu().numpy(), wk)
    ref.check_bf16(v.float().cpu().numpy(), wv)
    other = Pair(small(batch=2, k_bits=2, window=0), np.array(n, np.int32))
    other.lens[:] = 0
    other.glens.zero_()
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    other.append(bits(k), bits(v), np.array([0, span, 2 * span], np.int32))
    other.compare_cache()


def test_streams_and_graphs():
    """Two calls at once on two streams; each form captured and replayed over new cache contents."""
    w = small(window=16)
    pair = build(w, [300, 500, 64, 129])
    n = np.array([40, 3, 64, 1])
    cu = i32(np.concatenate([[0], np.cumsum(n)]))
    q1, q2 = (torch_raw(ref.queries(w, m)[0]) for m in (4, int(n.sum())))
    first, rows = i32([0, 9, 1, 100]), i32([0, 30, 130, 160, 190])

    def calls():
        return (*kvq.sink_decode_attention(pair.glay, pair.gcache, q1, pair.glens, 500, 4, 100),
                *kvq.sink_prefill_attention(pair.glay, pair.gcache, q2, cu, pair.glens, 64, 4, 100),
                *kvq.read_back(pair.glay, pair.gcache, first, rows, pair.glens, 190, 100))

    want = [t.clone() for t in calls()]
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for _ in range(3):
        for s in side:
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    q1.mul_(-1)
    q2.mul_(0.5)
    pair.glens.sub_(1)
    graph.replay()
    again = [t.clone() for t in held]
    fresh = list(calls())
    for i in (2, 3):                 # sequence 2 now holds 63 positions for its 64 queries: skipped, rows not written
        again[i], fresh[i] = (torch.cat((t[:43], t[107:])) for t in (again[i], fresh[i]))
    assert all(torch.equal(a, b) for a, b in zip(again, fresh))
    assert not torch.equal(again[0], want[0])
