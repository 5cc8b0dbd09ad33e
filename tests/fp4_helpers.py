"""Plain 64-bit forms that the 4-bit cache's tests compare with, and the tolerances that follow
from the kernels' roundings."""
import numpy as np

import workloads

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def bf16_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rows_of(kv, layout, ps, slots):
    """Rows at cache slots (page * ps + offset) of a uint8 cache [pages, page_bytes], in float64."""
    slots = np.asarray(slots, np.int64)
    nope, rb = workloads._NOPE[layout], workloads._ROW_BYTES[layout]
    p, o = slots // ps, slots % ps
    raw = kv[p[:, None], (o * rb)[:, None] + np.arange(rb)]
    if layout == 0:
        return bf16_f64(np.ascontiguousarray(raw).view(np.uint16))
    assert layout >= 3
    sc = kv[p[:, None], (ps * rb + o * 16)[:, None] + np.arange(nope // 32)].astype(np.float64)
    code = np.stack([raw[:, :nope // 2] & 15, raw[:, :nope // 2] >> 4], -1).reshape(-1, nope)
    scale = np.where(sc == 255, np.nan, np.exp2(sc - 127))
    pe = bf16_f64(np.ascontiguousarray(raw[:, nope // 2:]).view(np.uint16))
    return np.concatenate([E2M1[code] * np.repeat(scale, 32, axis=1), pe], 1)


def attend(q, k, scale, sink=None):
    """q [M, D], k [n, D] (float64), sink [M] or None -> out [M, 512], lse [M], and what the errors go by: the
    weighted mean of |V| and the largest sum of |q_i k_i| behind a score (times scale)."""
    M = q.shape[0]
    if k.shape[0] == 0:
        return np.zeros((M, 512)), np.full(M, -np.inf), np.zeros((M, 512)), 0.0
    s = q @ k.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    lse = (m + np.log(l))[:, 0]
    d = l if sink is None else l + np.exp(sink[:, None] - m)
    p = p / d
    return p @ k[:, :512], lse, p @ np.abs(k[:, :512]), float((np.abs(q) @ np.abs(k).T).max() * scale)


def decode(w, kv, rows_for, scale=None):
    """The whole decode of workload w over cache kv: rows_for(t) gives token t's cache slots; scale: the
    kernels' fp32 one unless given."""
    c = w.cfg
    scale = float(np.float32(c.sm_scale)) if scale is None else scale
    T, N, D = w.q.shape
    q = bf16_f64(w.q)
    out, lse = np.zeros((T, N, 512)), np.zeros((T, N))
    mean, terms = np.zeros((T, N, 512)), 0.0
    for t in range(T):
        k = rows_of(kv, c.layout, c.page_size, rows_for(t))
        sink = None if w.sink is None else w.sink.astype(np.float64)
        out[t], lse[t], mean[t], a = attend(q[t], k, scale, sink)
        terms = max(terms, a)
    return out, lse, mean, terms


def dense_slots(w):
    c = w.cfg

    def rows(t):
        b, i = divmod(t, c.sq)
        L = int(w.seqlens[b])
        n = max(0, L - c.sq + i + 1) if c.causal else L
        j = np.arange(n)
        return w.block_table[b, j // c.page_size].astype(np.int64) * c.page_size + j % c.page_size

    return rows


def listed_slots(w):
    c = w.cfg

    def rows(t):
        b = t // c.sq
        j = w.indices[t].astype(np.int64)
        j = j[(j >= 0) & (j < w.seqlens[b])]
        return w.block_table[b, j // c.page_size].astype(np.int64) * c.page_size + j % c.page_size

    return rows


def assert_decode(out, lse, ref, what=""):
    """Bounds, elementwise, from the roundings on the way (u = 2^-8: half a bf16 step relative to the
    value, at most):
      scores   bf16 products are exact in fp32; adding D <= 576 of them in any order loses at most
               D 2^-23 of the sum of their magnitudes: d = 576 * 2^-23 * max sum |q k| scale, absolute;
      weights  e^s is then off by a factor within 1 +- (d + 2^-20) (the exponential and the fp32 sums), the
               normaliser by as much, and each weight is rounded to bf16: (u + 2 (d + 2^-20)) * mean |V|;
      output   rounded to bf16 once: u * |out|. Split partials are fp32 and add 2^-20 of mean |V|.
    """
    ref_out, ref_lse, mean, terms = ref
    u, d = 2.0 ** -8, 576 * 2.0 ** -23 * terms + 2.0 ** -20
    assert d < 0.05, f"{what}: scores of this size say nothing ({d:.3g})"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty), f"{what}: which rows are empty"
    assert np.all(out[empty] == 0), f"{what}: empty rows must be zero"
    # one subnormal bf16 step and 2^-20 of the mean for the merge
    tol = (u + 2.1 * d + 2.0 ** -20) * mean + u * np.abs(ref_out) + 1e-38
    over = np.abs(out - ref_out) - tol
    assert np.all(over <= 0), (f"{what}: off by {np.abs(out - ref_out).max():.3g}, {over.max():.3g} over the bound at "
                               f"{np.unravel_index(np.argmax(over), over.shape)}")
    if (~empty).any():
        off = np.abs(lse[~empty] - ref_lse[~empty])
        assert np.all(off <= 2 * d + 2.0 ** -20 * np.abs(ref_lse[~empty]) + 2.0 ** -20), f"{what}: lse {off.max():.3g}"
