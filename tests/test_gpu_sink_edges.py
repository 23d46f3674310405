"""The attention with sinks where its parts meet: clusters whose CTAs have no tile, against fp64 numpy over the
oracle's cache."""
import numpy as np
import pytest
import torch

import mixed_precision_quantized_kvq_b200 as kvq
import sink_reference as ref
import workloads as wl
from gpu_harness import torch_raw
from test_gpu_sink import build, check_attention, i32, poison, small

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
