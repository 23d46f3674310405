"""Workloads of the attention with sinks and a sliding span over the quantized
paged cache, and of reading the cache back.

Three operators, each with a plain form in elementary torch operations:

* decode: one query per sequence, at the sequence's newest position.
* prefill: a chunk of new queries per sequence, its newest positions.
* read_back: a run of cached positions as dense rows in the model's basis.

A query at position t sees the cached positions p <= t with p < sinks or
t - p < span.  Pages that no query of a sequence sees any more are absent
from its page table (-1), as in a server that has released them.

The cache is made here from the seed alone: pages of codes and fp16 metadata
by the min/max group rule, and the bf16 ring of the newest positions.
"""
import math

import torch

own = False

PAGE = 64

# bit widths of keys and values: the pairs of the bit-allocation sweep
BITS = ((8, 8), (4, 4), (4, 2), (2, 4), (2, 2), (1, 2))


def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, hq=32, hkv=8, d=128, kb=4, vb=2, kg=32, vg=128, window=128, rotate=False,
             per_channel=False, len_lo=4096, len_hi=4096, n_lo=1, n_hi=1, sinks=4, span=4096, q="bf16", out="bf16",
             lse=False)
    c.update(kw)
    return c


def listed():
    return [
        # one short chat on one sequence: the latency of a single call
        _case("decode_b1_short", "decode", len_lo=301, len_hi=301, span=256, window=64, lse=True),
        # a layer with 32 query and 8 kv-heads, 16 long-running sequences, 4096 newest tokens and four sinks
        _case("decode_b16_span4096", "decode", batch=16, len_lo=9000, len_hi=30000, lse=True),
        # a ragged serving batch, five query heads per kv-head, a short span
        _case("decode_b64_ragged_g5", "decode", batch=64, hq=40, len_lo=512, len_hi=16384, window=64, span=2048, sinks=64),
        # rotated keys, no span limit, no bf16 window, fp32 queries
        _case("decode_b32_rotated_full", "decode", batch=32, len_lo=8000, len_hi=8192, window=0, rotate=True,
              sinks=0, span=1 << 30, q="fp32"),
        # one very long sequence at 8 bits
        _case("decode_b1_long_k8v8", "decode", kb=8, vb=8, len_lo=131072, len_hi=131072, sinks=16, span=1 << 30),
        # a short follow-up question on one sequence, small heads
        _case("prefill_b1_n33_d64", "prefill", hq=8, hkv=2, d=64, vg=64, len_lo=777, len_hi=777, n_lo=33, n_hi=33,
              span=500, window=16),
        # the 512-query chunk at 4096 cached tokens, 16 sequences
        _case("prefill_b16_n512", "prefill", batch=16, len_lo=4608, len_hi=4608, n_lo=512, n_hi=512),
        # a long prompt's 2048-query chunk far into its sequence
        _case("prefill_b4_n2048_far", "prefill", batch=4, len_lo=30000, len_hi=32768, n_lo=2048, n_hi=2048, sinks=64),
        # many sequences with a few new tokens each (follow-ups, speculative drafts), rotated keys
        _case("prefill_b32_few_rotated", "prefill", batch=32, hq=40, len_lo=100, len_hi=6000, n_lo=1, n_hi=60, rotate=True,
              span=1024, window=64),
        # whole prompts without a span limit, key groups along positions
        _case("prefill_b2_whole_per_channel", "prefill", batch=2, len_lo=2500, len_hi=3000, n_lo=2500, n_hi=3000, kg=64,
              vg=64, window=32, per_channel=True, sinks=0, span=1 << 30),
        # a few hundred rows of some sequences, rotated keys, in fp32
        _case("read_back_b8_rotated", "read_back", batch=8, len_lo=900, len_hi=1500, n_lo=1, n_hi=300, rotate=True, out="fp32"),
        # the last 4096 rows of 16 sequences in bf16
        _case("read_back_b16_4096", "read_back", batch=16, len_lo=9000, len_hi=30000, n_lo=4096, n_hi=4096),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("decode", "prefill", "read_back"))
    kb, vb = rng.choice(BITS)
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8))
    g = rng.choice((1, 2, 3, 4, 5, 7, 8))
    per_channel = rng.random() < 0.15
    kg = rng.choice((16, 32, 64) if per_channel else tuple(x for x in (16, 32, 32, 64, 128) if x <= d))
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, kb=kb, vb=vb, kg=kg, vg=rng.choice(tuple(x for x in (32, 64, 128, 128) if x <= d)),
             window=rng.choice((0, 16, 64, 100, 128)), rotate=not per_channel and rng.random() < 0.25, per_channel=per_channel,
             sinks=rng.choice((0, 1, 4, 64, 100)), q=rng.choice(("bf16", "bf16", "fp32")), out="bf16", lse=False)
    if op == "decode":
        c["batch"] = log(1, 64)
        c["len_hi"] = log(64, min(131072, 400000 // c["batch"]))
        c["n_lo"] = c["n_hi"] = 1
        c["lse"] = rng.random() < 0.5
    elif op == "prefill":
        c["batch"] = log(1, 16)
        c["n_hi"] = log(1, min(2048, 8192 // c["batch"]))
        c["n_lo"] = max(1, int(c["n_hi"] * rng.random()))
        c["len_hi"] = c["n_hi"] + log(1, 6000)
    else:
        c["batch"] = log(1, 16)
        c["n_hi"] = log(1, 4096)
        c["n_lo"] = max(1, int(c["n_hi"] * rng.random()))
        c["len_hi"] = c["n_hi"] + log(1, 20000)
        c["out"] = rng.choice(("bf16", "fp32"))
    c["len_lo"] = max(c["n_hi"], int(c["len_hi"] * rng.uniform(0.3, 1.0)))
    c["span"] = 1 << 30 if op == "prefill" and rng.random() < 0.3 else max(1, log(32, 16384))
    return c


# ---------------------------------------------------------------- sizes of a case (no randomness, no tensors)

def _spread(lo, hi, count, phase):
    """`count` whole numbers spread over [lo, hi]."""
    return [lo + int((hi - lo + 1) * ((phase + 0.6180339887498949 * i) % 1.0)) for i in range(count)]


def _sizes(case):
    """Lengths, new rows and what is visible of every sequence: (len, n, first visible of the span, sinks in front)."""
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"], 0.99)
    ns = _spread(case["n_lo"], case["n_hi"], case["batch"], 0.5)
    rows = []
    for L, n in zip(lens, ns):
        n = min(n, L)
        lo = max(0, L - n) if case["op"] == "read_back" else max(0, L - n + 1 - case["span"])
        rows.append((L, n, lo, 0 if case["op"] == "read_back" else min(case["sinks"], lo)))
    return rows


def _paged(case, L):
    q = max(0, L - case["window"])
    return q - q % case["kg"] if case["per_channel"] else q


def _ring(case):
    return case["window"] + (case["kg"] - 1 if case["per_channel"] else 0)


def work(case):
    d, hkv, hq = case["d"], case["hkv"], case["hq"]
    groups = d / case["vg"] + (d / case["kg"])      # per-channel groups hold as many values per scale
    paged_bytes = d * (case["kb"] + case["vb"]) / 8 + 4 * groups
    b = f = 0.0
    for L, n, lo, ns in _sizes(case):
        Q = _paged(case, L)
        in_pages = min(ns, Q) + max(0, Q - lo)
        in_ring = L - lo + ns - in_pages
        b += hkv * (in_pages * paged_bytes + in_ring * 4 * d)
        if case["op"] == "read_back":
            b += hkv * n * d * 2 * (4 if case["out"] == "fp32" else 2)
            f += hkv * (in_pages * d * 4 + (in_pages * d * math.log2(d) if case["rotate"] else 0))
            continue
        b += n * hq * (d * ((4 if case["q"] == "fp32" else 2) + 2) + (4 if case["lse"] else 0))
        pairs = 0
        for t in (range(L - n, L) if n <= 64 else ()):
            pairs += min(t + 1, case["span"]) + min(case["sinks"], max(0, t + 1 - case["span"]))
        if n > 64:                                   # the same sum, closed
            s, k = case["span"], case["sinks"]
            full = sum(t + 1 for t in range(L - n, min(L, s)))
            t0 = max(L - n, s)
            pairs = full + max(0, L - t0) * s + sum(min(k, t + 1 - s) for t in range(t0, min(L, s + k))) + k * max(0, L - max(t0, s + k))
        f += 4.0 * d * hq * pairs
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the cache, as a program has it before the call

def _bits16(x):
    return x.view(torch.int16).to(torch.int32) & 0xFFFF


def _round_down(x):
    h = x.to(torch.float16)
    low = torch.nextafter(h.float(), torch.full_like(x, -math.inf))   # one fp32 step lower rounds to h or below it
    step = (h.float().abs() * 2.0 ** -10).clamp_min(2.0 ** -24)
    return torch.where(h.float() > x, (low - step * 0.75).to(torch.float16), h)


def _round_up(x):
    return -_round_down(-x)


def _quantize(x, bits, group):
    """Groups of `group` along the last axis: codes (uint8), metadata words (scale, zero as int16 pairs)."""
    g = x.unflatten(-1, (-1, group))
    zero = _round_down(g.amin(-1))
    scale = _round_up((g.amax(-1) - zero.float()) / (2 ** bits - 1))
    s = scale.float().unsqueeze(-1)
    q = torch.where(s > 0, ((g - zero.float().unsqueeze(-1)) / s).round(), torch.zeros_like(g)).clamp_(0, 2 ** bits - 1)
    return q.flatten(-2).to(torch.uint8), torch.stack((scale, zero), -1).view(torch.int16)


def _pack(codes, bits):
    """Little-endian bit packing along the last axis: rows of bytes."""
    per = 8 // bits
    c = codes.unflatten(-1, (-1, per)).to(torch.int32)
    return (c << (torch.arange(per, device=c.device, dtype=torch.int32) * bits)).sum(-1).to(torch.uint8)


def _chunked(rows):
    """[pages][heads][n][bytes] rows as 16-byte chunks, chunk-major."""
    ch = min(16, rows.shape[-1])
    return rows.unflatten(-1, (-1, ch)).movedim(-2, -3).contiguous()


def _hadamard(d, device):
    h = torch.ones((1, 1), device=device)
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(d)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    B, H, d, kb, vb = case["batch"], case["hkv"], case["d"], case["kb"], case["vb"]
    sizes = _sizes(case)
    # page table: only pages with a position that some query sees (or that is read back); the others were released
    table = [[] for _ in range(B)]
    for b, (L, n, lo, ns) in enumerate(sizes):
        Q = _paged(case, L)
        table[b] = [lp for lp in range(-(-Q // PAGE)) if lp * PAGE < ns or (lp + 1) * PAGE > lo]
    pages = max(1, sum(len(t) for t in table))
    ids = torch.randperm(pages, generator=gen, device=dev).tolist()
    width = max(1, max(-(-L // PAGE) for L, _, _, _ in sizes))
    pt = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, t in enumerate(table):
        if t:
            pt[b, t] = torch.tensor(ids[at:at + len(t)], dtype=torch.int32)
        at += len(t)

    loud = torch.stack([torch.randperm(d, generator=gen, device=dev)[:4] for _ in range(H)])   # outlier channels
    signs = torch.where(torch.rand(d, generator=gen, device=dev) < 0.5, -1, 1).to(torch.int8)
    had = _hadamard(d, dev)

    def keys(*shape):
        k = torch.randn((*shape, H, d), generator=gen, device=dev)
        return k.scatter(-1, loud.expand(*shape, H, 4), 10 * k.gather(-1, loud.expand(*shape, H, 4))).bfloat16()

    parts = [[], [], [], []]
    for p0 in range(0, pages, 256):
        m = min(256, pages - p0)
        k = keys(m, PAGE).float().transpose(1, 2)                               # [m][H][64][d]
        v = torch.randn((m, H, PAGE, d), generator=gen, device=dev).bfloat16().float()
        if case["rotate"]:
            k = (k * signs) @ had
        if case["per_channel"]:
            code, meta = _quantize(k.transpose(-1, -2), kb, case["kg"])         # along positions, [m][H][d][64]
            meta = meta.transpose(2, 3).contiguous()                            # [m][H][64/kg][d]
        else:
            code, meta = _quantize(k, kb, case["kg"])
        parts[0].append(_chunked(_pack(code, kb)))
        parts[1].append(meta)
        code, meta = _quantize(v, vb, case["vg"])
        parts[2].append(_chunked(_pack(code.transpose(-1, -2), vb)))
        parts[3].append(meta)
    k_codes, k_meta, v_codes, v_meta = (torch.cat(x) for x in parts)

    R = _ring(case)
    k_win = keys(B, max(R, 1)).transpose(1, 2).contiguous()
    v_win = torch.randn((B, H, max(R, 1), d), generator=gen, device=dev).bfloat16()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cu = [0]
    for _, n, _, _ in sizes:
        cu.append(cu[-1] + n)
    qt = torch.float32 if case["q"] == "fp32" else torch.bfloat16
    return dict(case=case, k_codes=k_codes, k_meta=k_meta, v_codes=v_codes, v_meta=v_meta,
                k_win=k_win if R else None, v_win=v_win if R else None, page_table=pt.to(dev), pages=pages,
                signs=signs, hadamard=had, lens=ints([s[0] for s in sizes]), cu=ints(cu), rows=cu[-1],
                first=ints([s[0] - s[1] for s in sizes]),
                max_len=max(s[0] for s in sizes), max_n=max(s[1] for s in sizes),
                seen=max(s[0] - s[2] + s[3] for s in sizes),
                q=None if case["op"] == "read_back" else torch.randn((cu[-1], case["hq"], d), generator=gen, device=dev).to(qt))


# ---------------------------------------------------------------- plain forms

def _unpack(rows, bits):
    """[...][bytes] -> [...][codes], fp32."""
    per = 8 // bits
    shift = torch.arange(per, device=rows.device, dtype=torch.uint8) * bits
    return ((rows.unsqueeze(-1) >> shift) & (2 ** bits - 1)).flatten(-2).float()


def _scale_zero(meta, group):
    m = meta.view(torch.float16).float().repeat_interleave(group, -2)
    return m[..., 0], m[..., 1]


def _gather(s, pos):
    """Keys (in the domain of their storage) and values [B][H][S][d] of positions pos [B][S], which of them live in
    pages, and which of them are there at all.  Positions out of range give zeros."""
    c = s["case"]
    B = pos.shape[0]
    lens = s["lens"].long().unsqueeze(1)
    Q = (lens - c["window"]).clamp_min(0)
    Q = Q - Q % c["kg"] if c["per_channel"] else Q
    paged = pos < Q
    page = s["page_table"].long().gather(1, (pos // PAGE).clamp(0, s["page_table"].shape[1] - 1))
    here = (pos >= 0) & (pos < lens) & (~paged | (page >= 0))
    page, slot = page.clamp_min(0), pos % PAGE
    kc, km, vc, vm = s["k_codes"], s["k_meta"], s["v_codes"], s["v_meta"]

    def of_run(codes, bits):     # channel runs [pages][H][chunks][d][bytes]: the slot's code in every channel
        at = slot * bits // 8
        ch = codes.shape[-1]
        byte = codes[page, :, at // ch, :, at % ch].to(torch.int32)              # [B][S][H][d]
        return ((byte >> (slot * bits % 8).to(torch.int32)[:, :, None, None]) & (2 ** bits - 1)).float()

    if c["per_channel"]:
        m = km[page, :, slot // c["kg"]].view(torch.float16).float()            # [B][S][H][d][2]
        k = torch.addcmul(m[..., 1], of_run(kc, c["kb"]), m[..., 0])
    else:
        z = _scale_zero(km[page, :, slot], c["kg"])                             # [B][S][H][d]
        k = torch.addcmul(z[1], _unpack(kc[page, :, :, slot].flatten(-2), c["kb"]), z[0])
    z = _scale_zero(vm[page, :, slot], c["vg"])
    v = torch.addcmul(z[1], of_run(vc, c["vb"]), z[0])
    if s["k_win"] is not None:
        ring = (pos.clamp_min(0) % s["k_win"].shape[2])
        b = torch.arange(B, device=pos.device).unsqueeze(1)
        sel = paged[:, :, None, None]
        k = torch.where(sel, k, s["k_win"][b, :, ring].float())
        v = torch.where(sel, v, s["v_win"][b, :, ring].float())
    ok = here[:, :, None, None]
    k, v = torch.where(ok, k, 0.0), torch.where(ok, v, 0.0)
    return k.transpose(1, 2), v.transpose(1, 2), paged, here


def _plain_attention(s):
    c = s["case"]
    B, H, d, g, n, dev = c["batch"], c["hkv"], c["d"], c["hq"] // c["hkv"], s["max_n"], s["q"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    count = cu[1:] - cu[:-1]
    lo = (lens - count + 1 - c["span"]).clamp_min(0)
    ns = lo.clamp_max(c["sinks"])
    i = torch.arange(s["seen"], device=dev).unsqueeze(0)
    pos = torch.where(i < ns.unsqueeze(1), i, lo.unsqueeze(1) + i - ns.unsqueeze(1))           # [B][S]
    k, v, paged, here = _gather(s, pos)
    # queries padded to [B][H][n*g][d]
    row = (cu[:-1, None] + torch.arange(n, device=dev)).clamp_max(s["rows"] - 1)
    q = s["q"].float()[row].unflatten(2, (H, g)).permute(0, 2, 1, 3, 4).reshape(B, H, n * g, d)
    x = q @ k.transpose(-1, -2)
    if c["rotate"]:
        x = torch.where(paged[:, None, None, :], ((q * s["signs"]) @ s["hadamard"]) @ k.transpose(-1, -2), x)
    t = (lens - count)[:, None] + torch.arange(n, device=dev)                                   # [B][n]
    far = t[:, :, None] - pos[:, None, :]
    sees = here[:, None, :] & (far >= 0) & ((far < c["span"]) | (pos < c["sinks"])[:, None, :])
    sees = sees.repeat_interleave(g, 1)[:, None]                                                # [B][1][n*g][S]
    x = torch.where(sees, x * d ** -0.5, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = w.sum(-1, keepdim=True)
    o = (w @ v) / torch.where(total > 0, total, 1.0)
    b = torch.repeat_interleave(torch.arange(B, device=dev), count, output_size=s["rows"])
    at = torch.arange(s["rows"], device=dev) - cu[:-1][b]
    o = o.unflatten(2, (n, g))[b, :, at].flatten(1, 2).bfloat16()                               # [rows][Hq][d]
    if not c["lse"]:
        return {"out": o}
    lse = (top + torch.log(total)).squeeze(-1).unflatten(2, (n, g))[b, :, at].flatten(1, 2)
    return {"out": o, "lse": lse}


def _plain_read_back(s):
    c = s["case"]
    dev = s["lens"].device
    cu = s["cu"].long()
    b = torch.repeat_interleave(torch.arange(c["batch"], device=dev), cu[1:] - cu[:-1], output_size=s["rows"])
    at = torch.arange(s["rows"], device=dev) - cu[:-1][b]
    pos = s["first"].long().unsqueeze(1) + torch.arange(s["max_n"], device=dev)
    k, v, paged, here = _gather(s, pos)
    if c["rotate"]:
        k = torch.where(paged[:, None, :, None], (k @ s["hadamard"]) * s["signs"], k)
    t = torch.float32 if c["out"] == "fp32" else torch.bfloat16
    return {"k": k[b, :, at].to(t), "v": v[b, :, at].to(t)}


# ---------------------------------------------------------------- the framework's calls

def _handles(s):
    """The layout and the cache object that a program keeps for as long as it keeps the cache."""
    if "handles" not in s:
        import mixed_precision_quantized_kvq_b200 as kvq
        c = s["case"]
        lay = kvq.Layout(c["d"], c["hq"], c["hkv"], c["kb"], c["vb"], c["kg"], c["vg"], PAGE, c["window"], c["rotate"],
                         s["signs"] if c["rotate"] else None, c["per_channel"])
        s["handles"] = (kvq, lay, kvq.PagedCache(s["k_codes"], s["v_codes"], s["k_meta"], s["v_meta"], s["k_win"],
                                                 s["v_win"], s["page_table"], s["pages"]))
    return s["handles"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_read_back(s) if c["op"] == "read_back" else _plain_attention(s)
    kvq, lay, cache = _handles(s)
    if c["op"] == "read_back":
        k, v = kvq.read_back(lay, cache, s["first"], s["cu"], s["lens"], s["rows"], s["max_n"],
                             dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16)
        return {"k": k, "v": v}
    if c["op"] == "decode":
        o, lse = kvq.sink_decode_attention(lay, cache, s["q"], s["lens"], s["max_len"], c["sinks"], c["span"],
                                           want_lse=c["lse"])
    else:
        o, lse = kvq.sink_prefill_attention(lay, cache, s["q"], s["cu"], s["lens"], s["max_n"], c["sinks"], c["span"],
                                            want_lse=c["lse"])
    return {"out": o, "lse": lse} if c["lse"] else {"out": o}


# ---------------------------------------------------------------- the definition in 64 bits, one sequence and head at a time

def _dense(s, b, h):
    """fp64 keys and values [len][d] of one sequence and kv-head in the model's basis, and which positions exist."""
    c = s["case"]
    d, kb, vb, kg, vg = c["d"], c["kb"], c["vb"], c["kg"], c["vg"]
    L = int(s["lens"][b])
    Q = _paged(c, L)
    dev = s["lens"].device
    k = torch.zeros((L, d), dtype=torch.float64, device=dev)
    v = torch.zeros_like(k)
    have = torch.zeros(L, dtype=torch.bool, device=dev)
    table = s["page_table"][b]
    lps = torch.nonzero(table[: -(-Q // PAGE)] >= 0).flatten()
    if lps.numel():
        phys = table[lps].long()

        def bits_of(codes, n, bits, rows):          # codes of one head: [pages][rows][n] whole numbers
            x = codes[phys, h].movedim(1, 2).reshape(len(phys), rows, -1)
            x = (x.unsqueeze(-1) // (2 ** torch.arange(8, device=dev, dtype=torch.uint8))) % 2           # single bits
            x = x.reshape(len(phys), rows, n, bits).double()
            return (x * 2.0 ** torch.arange(bits, device=dev, dtype=torch.float64)).sum(-1)

        f16 = lambda m: m.view(torch.float16).double()  # noqa: E731
        if c["per_channel"]:
            m = f16(s["k_meta"][phys, h])                                        # [p][64/kg][d][2]
            m = m.repeat_interleave(kg, 1)
            kk = bits_of(s["k_codes"], PAGE, kb, d).transpose(1, 2) * m[..., 0] + m[..., 1]
        else:
            m = f16(s["k_meta"][phys, h]).repeat_interleave(kg, 2)               # [p][64][d][2]
            kk = bits_of(s["k_codes"], d, kb, PAGE) * m[..., 0] + m[..., 1]
        m = f16(s["v_meta"][phys, h]).repeat_interleave(vg, 2)
        vv = bits_of(s["v_codes"], PAGE, vb, d).transpose(1, 2) * m[..., 0] + m[..., 1]
        if c["rotate"]:      # the transform is its own inverse up to the signs
            hd = torch.round(s["hadamard"].double() * math.sqrt(d)) / math.sqrt(d)
            kk = (kk @ hd) * s["signs"].double()
        at = (lps[:, None] * PAGE + torch.arange(PAGE, device=dev)).flatten()
        sel = at < Q
        k[at[sel]], v[at[sel]], have[at[sel]] = kk.reshape(-1, d)[sel], vv.reshape(-1, d)[sel], True
    if Q < L:
        at = torch.arange(Q, L, device=dev)
        k[at], v[at], have[at] = s["k_win"][b, h, at % _ring(c)].double(), s["v_win"][b, h, at % _ring(c)].double(), True
    return k, v, have


def exact(case, seed):
    s = prepare(case, seed)
    H, d, g = case["hkv"], case["d"], case["hq"] // case["hkv"]
    cu = s["cu"].tolist()
    dev = s["lens"].device
    if case["op"] == "read_back":
        k = torch.zeros((cu[-1], H, d), dtype=torch.float64, device=dev)
        v = torch.zeros_like(k)
        for b in range(case["batch"]):
            f = int(s["first"][b])
            for h in range(H):
                kk, vv, _ = _dense(s, b, h)
                k[cu[b]:cu[b + 1], h], v[cu[b]:cu[b + 1], h] = kk[f:f + cu[b + 1] - cu[b]], vv[f:f + cu[b + 1] - cu[b]]
        return {"k": k, "v": v}
    out = torch.zeros((cu[-1], H * g, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((cu[-1], H * g), dtype=torch.float64, device=dev)
    for b in range(case["batch"]):
        a, e = cu[b], cu[b + 1]
        L = int(s["lens"][b])
        p = torch.arange(L, device=dev)
        for h in range(H):
            k, v, have = _dense(s, b, h)
            for r in range(a, e, 256):
                m = min(e, r + 256) - r
                t = L - (e - a) + (r - a) + torch.arange(m, device=dev)[:, None]
                hide = ~(have & (p <= t) & ((p < case["sinks"]) | (t - p < case["span"])))
                q = s["q"][r:r + m, h * g:(h + 1) * g].double()
                x = torch.einsum("mgd,pd->gmp", q, k) / math.sqrt(d)
                x = x.masked_fill(hide, -math.inf)
                lse[r:r + m, h * g:(h + 1) * g] = torch.logsumexp(x, -1).T
                out[r:r + m, h * g:(h + 1) * g] = torch.einsum("gmp,pd->mgd", torch.softmax(x, -1).nan_to_num(0.0), v)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
