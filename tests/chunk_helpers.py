"""Plain forms in 64 bits of the chunk's operators, and what their results may be off by.

A rounding to bf16 is off by at most H = 2^-8 of the value. Sums of n terms in fp32 are taken to be off by n 2^-23 of the sum
of the terms' magnitudes (a tensor core may cut a product's low bits instead of rounding them)."""
import numpy as np
import torch

import mla_paged_latent_gb300 as mla

H = 2.0 ** -8
DEV = "cuda"


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


class Cache:
    """Paged rows of the requests, written by the library's own write and read back in 64 bits."""

    def __init__(self, g, lens, layout, page, scale=1.0, spare=1):
        per = [-(-n // page) for n in lens]
        pages = sum(per) + spare
        self.layout, self.page, self.lens, self.pages = layout, page, list(lens), pages
        self.data = torch.zeros(pages, mla.mla_page_bytes(layout, page), dtype=torch.uint8, device=DEV)
        self.table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32, device=DEV)
        order = torch.randperm(pages, generator=g, device=DEV).int()
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        slots = torch.arange(pages * page, dtype=torch.int32, device=DEV)
        mla.mla_kv_write(normal(g, pages * page, 576, scale=scale), slots, self.data, layout, page)

    def rows(self, b):
        n = self.lens[b]
        if n == 0:
            return torch.zeros(0, 576, dtype=torch.float64, device=DEV)
        pos = torch.arange(n, device=DEV)
        slots = (self.table[b].long()[pos // self.page] * self.page + pos % self.page).int()
        out = torch.empty(n, 576, dtype=torch.bfloat16, device=DEV)
        mla.mla_kv_read(self.data, self.layout, self.page, slots, out)
        return out.double()


def chunk_reference(q, cache, new, w, scale, causal):
    """(out, lse, out's bound, lse's bound) in 64 bits.

    Bounds. K's rounding moves a score by at most e = H scale sum_d |q_d k_d| over the 128 NoPE elements, and fp32 sums of 192
    products by 192 2^-23 of scale sum_d |q_d k_d|. A weight then changes by a factor of at most e^(2 e) of the largest e of
    the row, its rounding to bf16 and V's by H each, the exponential and the sums over n rows by 2^-18 + n 2^-23, and the
    result is rounded: in all sum_j p_j |v_j| (e^(2 e) (1 + H)^2 (1 + ...) - 1) + H |out|. lse moves by e, and by the
    logarithm's and the sum's own 2^-18 + n 2^-23 and 2^-22 of the largest score."""
    scale = float(np.float32(scale))
    out = torch.zeros(q.shape[0], q.shape[1], 128, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64, device=DEV)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for b, n in enumerate(new):
        rows, length = cache.rows(b), cache.lens[b]
        x = q[at:at + n].double()
        if length > 0 and n > 0:
            hidden = torch.zeros(n, length, dtype=torch.bool, device=DEV)
            if causal:
                hidden = torch.arange(length, device=DEV) > (length - n + torch.arange(n, device=DEV))[:, None]
            for h in range(q.shape[1]):
                k = torch.cat([rows[:, :512] @ w[h, :128].double().T, rows[:, 512:]], 1)
                v = rows[:, :512] @ w[h, 128:].double().T
                s = (x[:, h] @ k.T * scale).masked_fill(hidden, -torch.inf)
                mag = x[:, h, :128].abs() @ k[:, :128].abs().T * scale
                all_mag = mag + x[:, h, 128:].abs() @ k[:, 128:].abs().T * scale
                e = (H * mag + 192 * 2.0 ** -23 * all_mag + 512 * 2.0 ** -23 * mag).masked_fill(hidden, 0).amax(1)
                top = s.amax(1)
                seen = top > -torch.inf
                p = torch.exp(s - torch.where(seen, top, 0.0)[:, None])
                total = p.sum(1)
                p = p / torch.where(seen, total, 1.0)[:, None]
                own = 2.0 ** -18 + length * 2.0 ** -23
                out[at:at + n, h] = p @ v
                grow = torch.exp(2 * e) * (1 + H) ** 2 * (1 + own) ** 2 - 1
                bound[at:at + n, h] = (p @ v.abs()) * grow[:, None] + H * out[at:at + n, h].abs() + 1e-30
                lse[at:at + n, h] = torch.where(seen, torch.log(total) + top, -torch.inf)
                lse_bound[at:at + n, h] = e + own + 2.0 ** -22 * torch.where(seen, top, 0.0).abs()
        at += n
    return out, lse, bound, lse_bound


def run_chunk(q, cache, new, w, scale, causal=True, lse=True, num_sms=None, kv_budget=mla.KV_BUDGET, table=None):
    plan = mla.mla_chunk_plan(new, cache.lens, q.shape[1], causal=causal, kv_budget=kv_budget, num_sms=num_sms)
    sched = torch.from_numpy(plan.sched).to(DEV)
    ws = mla.alloc_workspace(plan.workspace_bytes)
    ws[256:].fill_(255)  # NaN, were it read
    out = torch.full((q.shape[0], q.shape[1], 128), 7.0, dtype=torch.bfloat16, device=DEV)
    sums = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    mla.mla_chunk_attention(q, cache.data, cache.layout, cache.page, cache.table if table is None else table, w, scale, plan,
                            sched, ws, out, sums)
    return out, sums, plan, ws
