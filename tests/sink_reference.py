"""Attention with sinks and a sliding span, and rows read back, in fp64 numpy
over the oracle's cache (whose bytes the CUDA cache must equal bit for bit)."""
from __future__ import annotations

import numpy as np

import oracle
import workloads as wl

HALF_BF16 = 2.0 ** -8          # a bf16 rounding is off by at most half a step of 2^-7, relative


def paged_len(lay, L: int) -> int:
    q = max(0, int(L) - lay.window)
    return q - q % lay.k_group if lay.k_per_channel else q


def hadamard(d: int) -> np.ndarray:
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(d)


def present(lay, page_table, b: int, L: int) -> np.ndarray:
    """Which positions of sequence b are there: ring positions, and those whose page is mapped."""
    x = np.arange(L)
    ok = x >= paged_len(lay, L)
    lp = x // 64
    inside = lp < page_table.shape[1]
    ok[inside] |= page_table[b, lp[inside]] >= 0
    return ok


def attention(cache: oracle.Cache, page_table, signs, q, n, lens, sinks: int, span: int, scale: float, exact_q=True,
              want_tol=False):
    """q fp64 [sum n][Hq][d]; n queries per sequence, its newest.  Returns out, lse (fp64).  Sequences with
    n > lens are skipped (nan rows).  With want_tol also how far out and lse may be off where keys, values and weights
    are rounded to fp16, each by at most u = 2^-11 of itself (and 2^-25, half a subnormal step), and the query too
    unless exact_q:
        |score error| <= D = max over visible t of scale * sum_j |q_j| (|k_tj| (u or 2u) + 2^-25),
        so every weight is off by a factor within exp(+-2D) and lse by at most D;
        |out error| <= (exp(2D) - 1) sum_t a_t |v_t - o|  +  (2u + 2^-25) sum_t a_t |v_t|  (weights, values).
    fp32 sums add 2^-24 per term of the same sums: a factor 1.1 on both covers 400 of them in a row at random signs."""
    u, tol_o, tol_l = 2.0 ** -11, np.zeros(q.shape), np.zeros(q.shape[:2])
    lay = cache.layout
    g, d = lay.num_q_heads // lay.num_kv_heads, lay.head_dim
    k, v = cache.dequantize(lens, max(1, int(np.max(lens))))
    out = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    rot = q if signs is None else (q * signs) @ hadamard(d)
    r0 = 0
    for b in range(len(n)):
        L, m = int(lens[b]), int(n[b])
        if m > L:
            r0 += m
            continue
        t = (L - m + np.arange(m))[:, None]
        x = np.arange(L)[None, :]
        sees = (x <= t) & ((x < sinks) | (t - x < span)) & present(lay, page_table, b, L)[None, :]
        paged = x[0] < paged_len(lay, L)
        for h in range(lay.num_q_heads):
            some = sees.any(0)[:, None]                     # what no query sees may hold anything
            kk = np.where(some, k[b, h // g, :L].astype(np.float64), 0.0)
            vv = np.where(some, v[b, h // g, :L].astype(np.float64), 0.0)
            s = np.where(paged, rot[r0:r0 + m, h] @ kk.T, q[r0:r0 + m, h] @ kk.T) * scale
            s = np.where(sees, s, -np.inf)
            top = s.max(-1, keepdims=True, initial=-np.inf)
            w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            tot = w.sum(-1, keepdims=True)
            out[r0:r0 + m, h] = np.where(tot > 0, (w @ vv) / np.where(tot > 0, tot, 1.0), 0.0)
            with np.errstate(divide="ignore"):
                lse[r0:r0 + m, h] = (top + np.log(tot))[:, 0]
            if want_tol:
                qq = np.abs(rot[r0:r0 + m, h]) if signs is not None else np.abs(q[r0:r0 + m, h])
                kr = kk if signs is None else np.where(paged[:, None], kk, (kk * signs) @ hadamard(d))
                D = abs(scale) * (qq @ np.abs(kr).T * u * (1 if exact_q and signs is None else 2)
                                  + qq.sum(-1, keepdims=True) * 2.0 ** -25)
                D = np.where(sees, D, 0.0).max(-1, keepdims=True, initial=0.0)
                a = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 0.0)
                o = out[r0:r0 + m, h]
                spread = a @ np.abs(vv) + np.abs(o) if m * L > 20000 else (
                    a[:, :, None] * np.abs(vv[None] - o[:, None])).sum(1)
                tol_o[r0:r0 + m, h] = 1.1 * (np.expm1(2 * D) * spread + (2 * u + 2.0 ** -25) * (a @ np.abs(vv)))
                tol_l[r0:r0 + m, h] = 1.1 * D[:, 0] + 2.0 ** -20 * (1 + np.abs(np.where(tot > 0, lse[r0:r0 + m, h][:, None], 0))[:, 0])
        r0 += m
    return (out, lse, tol_o, tol_l) if want_tol else (out, lse)


def rows_back(cache: oracle.Cache, page_table, signs, first, n, lens):
    """fp64 keys and values [sum n][Hkv][d] of positions first[b] .. first[b]+n[b]-1 in the model's basis."""
    lay = cache.layout
    k, v = cache.dequantize(lens, max(1, int(np.max(lens))))
    ko = np.zeros((int(np.sum(n)), lay.num_kv_heads, lay.head_dim))
    vo = np.zeros_like(ko)
    r = 0
    for b in range(len(n)):
        ok = present(lay, page_table, b, int(lens[b]))
        for i in range(int(n[b])):
            x = int(first[b]) + i
            if 0 <= x < lens[b] and ok[x]:
                kk = k[b, :, x].astype(np.float64)
                if signs is not None and x < paged_len(lay, lens[b]):
                    kk = (kk @ hadamard(lay.head_dim)) * signs
                ko[r], vo[r] = kk, v[b, :, x]
            r += 1
    return ko, vo


def queries(w: wl.Workload, rows: int, step: int = 0):
    """Query rows: (raw array for the library, fp64 values)."""
    raw, f = wl.chunk_queries(w, rows, step)
    return raw, f.astype(np.float64)


def check_bf16(got, want, what="out", tol=None):
    """|got - want| <= tol (default: 1e-3 + 1e-3*|want|, the bound of the kernels that take exact codes) + half a bf16
    step of the value that is rounded, which is at most |want| plus that bound."""
    got = np.asarray(got, np.float64)
    tol = 1e-3 + 1e-3 * np.abs(want) if tol is None else tol
    lim = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(want) + 1e-30
    err = np.abs(got - want)
    assert got.shape == want.shape
    if got.size and not np.all(err <= lim):
        i = np.unravel_index(np.nanargmax(np.where(np.isnan(err), np.inf, err - lim)), err.shape)
        raise AssertionError(f"{what}: worst at {i}: got {got[i]!r} want {want[i]!r} (max err {np.nanmax(err):.3e})")


def check_lse(got, want, tol=None):
    got = np.asarray(got, np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin) and np.all(got[~fin] == want[~fin])
    tol = 1e-3 + 1e-3 * np.abs(want) if tol is None else tol
    assert np.all(np.abs(got[fin] - want[fin]) <= tol[fin])
