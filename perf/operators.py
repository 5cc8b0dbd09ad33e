"""Operators of the 4-bit latent cache: their plain forms, and the framework's calls.

attend   paged MLA attention over a cache whose NoPE part is held in e2m1 (4 bits) with one
         ue8m0 scale per 32 elements: dense, causal draft tokens, top-k lists, slot windows.
store    new rows quantised and written into their pages, then read back by slot as bf16.
append   per-head RMSNorm and RoPE of the queries and, for the same tokens, RMSNorm, RoPE and
         the cache write of the KV rows; the written rows are read back by slot.

A page holds page_size rows, then one 16-byte scale slot per row; its size is a multiple of the
row's. A row is its NoPE codes, two per byte (even element in the low nibble), then 64 bf16
RoPE elements: 448 / 2 + 128 = 352 bytes ("448", K = V = 512 wide) or 512 / 2 + 128 = 384 bytes
("512", K = 576 wide, V = its first 512).
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NOPE = {"448": 448, "512": 512}
WIDTH = {"448": 512, "512": 576}
ROW = {"448": 352, "512": 384}
LAYOUT = {"448": 3, "512": 4}  # MLA_KV_FP4_448_UE8M0, MLA_KV_FP4_512_UE8M0


# ------------------------------------------------------------------------------- cases
def listed():
    dense = dict(op="attend", mode="dense", sink=False, causal=False, topk=0)
    return [
        # two short requests on few heads: what one call costs when there is nearly nothing to read
        dict(dense, name="two short requests", row="512", batch=2, tokens=1, heads=16, page=16, lo=37, hi=130,
             spread="ends"),
        # a decode batch at 128 heads, page-64 cache, contexts of 1K to 8K
        dict(dense, name="decode 64 x 128 heads", row="512", batch=64, tokens=1, heads=128, page=64, lo=1024, hi=8192,
             spread="even"),
        # a decode batch at 64 heads with a sink and contexts of very different lengths
        dict(dense, name="decode 128 x 64 heads, sink", row="448", batch=128, tokens=1, heads=64, page=64, lo=512,
             hi=32768, spread="log", sink=True),
        # speculative verify: four draft tokens a request, causal among themselves
        dict(dense, name="verify 32 x 4 tokens", row="512", batch=32, tokens=4, heads=128, page=64, lo=2052, hi=16388,
             spread="even", causal=True),
        # sparse attention: 2048 listed rows of a 64K context, a tenth of each list unused
        dict(dense, name="top 2048 of 65536", row="512", batch=64, tokens=1, heads=128, page=64, lo=65536, hi=65536,
             spread="even", mode="topk", topk=2048),
        # one long request alone: the work has to be split over the long axis
        dict(dense, name="one request of 131071", row="512", batch=1, tokens=1, heads=128, page=64, lo=131071,
             hi=131071, spread="even"),
        # sliding-window layers: every token reads 96 consecutive slots
        dict(dense, name="window of 96", row="448", batch=128, tokens=1, heads=64, page=64, lo=512, hi=8192,
             spread="log", sink=True, mode="window", topk=96),
        # the new rows of one decode step, already normalised
        dict(op="store", name="store 64 rows", row="512", rows=64, page=64),
        # the rows of a long prompt
        dict(op="store", name="store 65000 rows", row="448", rows=65000, page=64),
        # one decode step: queries prepared and rows appended (rotation only, as the absorbed queries take it)
        dict(op="append", name="append 64 x 128 heads", row="512", rows=64, heads=128, page=64, max_pos=8192,
             norm=False),
        # a verify step of 32 x 4 drafts at 64 heads, queries normalised per head
        dict(op="append", name="append 128 x 64 heads, norm", row="448", rows=128, heads=64, page=64, max_pos=32768,
             norm=True),
        # a prompt's chunk
        dict(op="append", name="append 8192 x 128 heads", row="512", rows=8192, heads=128, page=64, max_pos=65536,
             norm=True),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    row = rng.choice(("448", "512"))
    page = rng.choice((8, 16, 32, 64, 128))
    kind = rng.choice(("dense", "dense", "verify", "topk", "window", "store", "append", "append"))
    if kind == "store":
        return dict(op="store", row=row, rows=_log(rng, 1, 60000), page=page)
    if kind == "append":
        heads = rng.choice((8, 16, 24, 64, 128))
        return dict(op="append", row=row, rows=_log(rng, 1, 8000 * 128 // max(heads, 64)), heads=heads, page=page,
                    max_pos=_log(rng, 1000, 100000), norm=rng.random() < 0.5)
    heads = rng.choice((8, 16, 20, 64, 128))
    tokens = rng.randint(2, 6) if kind == "verify" else 1
    if kind in ("topk", "window"):
        heads = rng.choice((16, 64, 128))
        batch = _log(rng, 1, 96)
        hi = _log(rng, 200, 20000)
        topk = _log(rng, 16, 2000) if kind == "topk" else rng.randint(2, min(2 * page, hi))
        return dict(op="attend", mode=kind, row=row, batch=batch, tokens=1, heads=heads, page=page,
                    lo=min(hi, rng.randint(0, 300)), hi=hi, spread="even", sink=rng.random() < 0.5, causal=False,
                    topk=topk)
    batch = _log(rng, 1, 96)
    hi = _log(rng, max(tokens, 3), min(120000, 600000 // (batch * tokens)))
    return dict(op="attend", mode="dense", row=row, batch=batch, tokens=tokens, heads=heads, page=page,
                lo=rng.choice((0, _log(rng, 1, hi))), hi=hi, spread=rng.choice(("even", "log", "ends")), sink=rng.random() < 0.5,
                causal=kind == "verify", topk=0)


def _lengths(c):
    """The requests' lengths: the same for every seed, so that the work is the case's."""
    lo, hi, n = c["lo"], c["hi"], c["batch"]
    if c["spread"] == "ends":
        return np.array([lo if i % 2 == 0 else hi for i in range(n)], np.int32)
    at = (np.arange(n) + 0.5) / n
    v = lo + (hi - lo) * at if c["spread"] == "even" else max(lo, 1) * (hi / max(lo, 1)) ** at
    return np.random.RandomState(n).permutation(np.rint(v)).astype(np.int32)


def _listed_rows(c):
    """Rows that one token of a top-k or window case reads: entries past a request's length are left out."""
    n = np.minimum(_lengths(c), c["topk"])
    return np.minimum(n, c["topk"] - c["topk"] // 10) if c["mode"] == "topk" else n


def work(case):
    c, width, row = case, WIDTH[case["row"]], ROW[case["row"]] + 16
    if c["op"] == "store":  # read, written, read back as bf16
        return {"bytes": float(c["rows"] * (2 * width + 2 * row + 2 * width + 8)), "flops": float(c["rows"] * width * 4)}
    if c["op"] == "append":
        elems = c["rows"] * (c["heads"] + 1) * width
        return {"bytes": float(4 * elems + c["rows"] * (2 * row + 2 * width + 12)), "flops": float(8 * elems)}
    rows = int(_lengths(c).sum() if c["mode"] == "dense" else _listed_rows(c).sum())
    t = c["batch"] * c["tokens"] * c["heads"]
    lists = 4 * c["batch"] * c["topk"]
    return {"bytes": float(rows * row + t * (2 * width + 1024 + 4) + lists),
            "flops": 2.0 * rows * c["heads"] * c["tokens"] * (width + 512)}


# ------------------------------------------------------------------------------- inputs
def _codes(x):
    """x [n, groups, 32] fp32 -> (codes, ue8m0 bytes, their values): the smallest e with 6 * 2^e >= amax, e2m1
    codes rounded to nearest with ties to the even code."""
    amax = x.abs().amax(-1).clamp_min(1e-10)
    m, k = torch.frexp(amax)  # amax = m * 2^k, and 6 = 0.75 * 2^3
    e = (k - torch.where(m <= 0.75, 3, 2)).clamp(-127, 127)
    a = torch.ldexp(x.abs(), -e[..., None])
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    grid = torch.tensor(E2M1, device=x.device)
    value = torch.ldexp(torch.copysign(grid[code], x), e[..., None])
    return (code + 8 * torch.signbit(x).int()).to(torch.uint8), (e + 127).to(torch.uint8), value


def _quantised(rows, kind):
    """bf16 rows [n, width] -> the values that the cache holds for them, fp32."""
    nope = NOPE[kind]
    x = rows.float()
    v = _codes(x[:, :nope].reshape(-1, nope // 32, 32))[2]
    return torch.cat([v.reshape(-1, nope), x[:, nope:]], 1)


def _pages(rows, kind, pages, page):
    """bf16 rows [pages * page, width] -> the cache, uint8 [pages, page_bytes]."""
    nope, rb = NOPE[kind], ROW[kind]
    cache = torch.zeros(pages, -(-page * (rb + 16) // rb) * rb, dtype=torch.uint8, device="cuda")
    code, scale, _ = _codes(rows[:, :nope].float().reshape(-1, nope // 32, 32))
    code = code.reshape(-1, nope // 2, 2)
    row = cache[:, :page * rb].view(pages, page, rb)
    row[..., :nope // 2] = (code[..., 0] | code[..., 1] << 4).view(pages, page, -1)
    row[..., nope // 2:] = rows[:, nope:].contiguous().view(torch.uint8).view(pages, page, 128)
    cache[:, page * rb:page * (rb + 16)].view(pages, page, 16)[..., :nope // 32] = scale.view(pages, page, -1)
    return cache


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _latent(g, n, width):
    """Latent rows: channels of different magnitudes, as a trained projection gives them."""
    return (_normal(g, n, width) * torch.exp(0.3 * _normal(g, width))).to(torch.bfloat16)


def _table(max_pos):
    """Per position 32 interleaved (cos, sin) pairs; the angles in 64 bits."""
    angle = torch.outer(torch.arange(max_pos, dtype=torch.float64, device="cuda"),
                        10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32))
    return torch.stack([angle.cos(), angle.sin()], -1).reshape(max_pos, 64).float()


def prepare(case, seed):
    c, kind, width = dict(case), case["row"], WIDTH[case["row"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] != "attend":
        n, page = c["rows"], c["page"]
        pages = -(-n // page) + 1
        s["cache"] = torch.zeros(pages, -(-page * (ROW[kind] + 16) // ROW[kind]) * ROW[kind], dtype=torch.uint8,
                                 device="cuda")
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:n].int()
        s["back"] = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
        s["rows"] = _latent(g, n, width)
        if c["op"] == "append":
            heads = c["heads"]
            s["positions"] = torch.randint(c["max_pos"], (n,), generator=g, device="cuda", dtype=torch.int32)
            s["freqs"] = _table(c["max_pos"])
            s["kv_weight"] = (1 + 0.2 * _normal(g, 512)).to(torch.bfloat16)
            s["q_weight"] = (1 + 0.2 * _normal(g, 512)).to(torch.bfloat16) if c["norm"] else None
            if kind == "512":
                # the absorbed part comes from a product batched over heads, the RoPE part is the end of each
                # head of another projection
                s["q_nope"] = _normal(g, heads, n, 512).to(torch.bfloat16).transpose(0, 1)
                s["q_pe"] = _normal(g, n, heads, 192).to(torch.bfloat16)[..., 128:]
            else:
                q = _normal(g, n, heads, 512).to(torch.bfloat16)
                s["q_nope"], s["q_pe"] = q[..., :448], q[..., 448:]
            s["q"] = torch.empty(n, heads, width, dtype=torch.bfloat16, device="cuda")
        return s
    lens, batch, tokens, heads, page = _lengths(c), c["batch"], c["tokens"], c["heads"], c["page"]
    per = -(-lens.astype(np.int64) // page)
    pages = max(1, int(per.sum()))
    table = torch.full((batch, max(1, int(per.max()))), -1, dtype=torch.int32, device="cuda")
    mine = torch.arange(table.shape[1], device="cuda") < torch.from_numpy(per).cuda()[:, None]
    table[mine] = torch.randperm(pages, generator=g, device="cuda")[:int(per.sum())].int()
    s["table"], s["lens"] = table, torch.from_numpy(lens).cuda()
    s["cache"] = _pages(_latent(g, pages * page, width), kind, pages, page)
    s["q"] = _normal(g, batch * tokens, heads, width).to(torch.bfloat16)
    s["sink"] = _normal(g, heads) if c["sink"] else None
    s["scale"] = 1 / math.sqrt(512 if kind == "448" else 192)
    topk = c["topk"]
    if c["mode"] == "topk":  # distinct positions of each request, then -1
        s["indices"] = torch.full((batch, topk), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(_listed_rows(c).tolist()):
            s["indices"][b, :n] = torch.randperm(int(lens[b]), generator=g, device="cuda")[:n].int()
    if c["mode"] == "window":  # consecutive slots, straddling two pages where the request has them
        n = torch.from_numpy(_listed_rows(c)).cuda()
        u = torch.rand(2, batch, generator=g, device="cuda")
        room = (2 if pages > 1 else 1) * page - n  # within two pages: a window has at most two runs
        first = (u[0] * max(1, pages - 1)).int() * page + (u[1] * (room.clamp_max(page - 1) + 1)).int()
        at = torch.arange(topk, device="cuda", dtype=torch.int32)
        s["indices"] = torch.where(at < n[:, None], first[:, None] + at, -1).int()
        s["counts"] = n.int()
    if own:
        import mla_paged_latent_gb300 as mla
        plan = mla.mla_decode_plan(lens, tokens, heads, topk)
        s["plan"] = plan
        s["sched"], s["splits"] = torch.from_numpy(plan.sched).cuda(), torch.from_numpy(plan.num_splits).cuda()
        s["workspace"] = mla.alloc_workspace(plan.workspace_bytes)
        s["out"] = torch.empty(batch * tokens, heads, 512, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(batch * tokens, heads, device="cuda")
        s["runs"] = torch.empty(batch, 4, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _rows_at(s, slot):
    """The cache's rows at slots [...] as fp32 [..., width]; rows at negative slots are zero."""
    c = s["case"]
    nope, rb, page = NOPE[c["row"]], ROW[c["row"]], c["page"]
    pages = s["cache"].shape[0]
    at = slot.reshape(-1).clamp_min(0).int()
    rows = s["cache"][:, :page * rb].view(pages, page, rb)[at // page, at % page]
    scale = s["cache"][:, page * rb:page * (rb + 16)].view(pages, page, 16)[at // page, at % page, :nope // 32]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    pair = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], 1)  # byte -> (low, high)
    v = torch.index_select(pair, 0, rows[:, :nope // 2].reshape(-1).int()).view(-1, nope // 32, 32)
    v = v * torch.exp2(scale.float() - 127)[..., None]
    k = torch.cat([v.view(-1, nope), rows[:, nope // 2:].contiguous().view(torch.bfloat16).float()], 1)
    return (k * (slot.reshape(-1, 1) >= 0)).view(*slot.shape, -1)


def _attend(s):
    c = s["case"]
    batch, tokens, heads, page = c["batch"], c["tokens"], c["heads"], c["page"]
    if c["mode"] == "window":
        slot = s["indices"]
    else:
        pos = s["indices"] if c["mode"] == "topk" else torch.arange(
            max(1, c["hi"]), device="cuda", dtype=torch.int32).expand(batch, -1)
        in_reach = (pos >= 0) & (pos < s["lens"][:, None])
        block = (pos // page).clamp(0, s["table"].shape[1] - 1)
        slot = torch.where(in_reach, torch.gather(s["table"], 1, block.long()) * page + pos % page, -1)
    k = _rows_at(s, slot)
    q = s["q"].float().view(batch, tokens * heads, -1)
    score = torch.bmm(q, k.transpose(1, 2)).mul_(s["scale"]).view(batch, tokens, heads, -1)
    seen = (slot >= 0)[:, None, None, :]
    if c["causal"]:
        last = s["lens"][:, None] - tokens + torch.arange(tokens, device="cuda", dtype=torch.int32)
        seen = seen & (torch.arange(slot.shape[1], device="cuda") <= last[..., None])[:, :, None, :]
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    if s["sink"] is not None:
        total = torch.where(total > 0, total + (s["sink"][:, None] - top).exp(), total)
    out = torch.bmm(p.view(batch, tokens * heads, -1), k[..., :512])
    out = out.view(batch, tokens, heads, 512) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16).view(-1, heads, 512), lse.view(-1, heads)


def _norm(x, weight, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight


def _rotate(x, angle):
    """Adjacent pairs of x [n, ..., 64] by their tokens' (cos, sin) pairs, angle [n, 64]."""
    cos, sin = angle[:, 0::2], angle[:, 1::2]
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)


def _append(s):
    kind = s["case"]["row"]
    angle = s["freqs"][s["positions"]]
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float()
    rows = s["rows"].float()
    rows = torch.cat([_norm(rows[:, :512], s["kv_weight"].float(), 1e-6), rows[:, 512:]], -1)
    if s["q_weight"] is not None:
        q = torch.cat([_norm(q[..., :512], s["q_weight"].float(), 1e-6), q[..., 512:]], -1)
    nope = NOPE[kind]
    q = torch.cat([q[..., :nope], _rotate(q[..., nope:], angle)], -1).to(torch.bfloat16)
    rows = torch.cat([rows[:, :nope], _rotate(rows[:, nope:], angle)], -1).to(torch.bfloat16)
    return q, _quantised(rows, kind).to(torch.bfloat16)


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "attend":
            return _attend(s)
        return _append(s) if c["op"] == "append" else _quantised(s["rows"], c["row"]).to(torch.bfloat16)
    import mla_paged_latent_gb300 as mla
    layout, page = LAYOUT[c["row"]], c["page"]
    if c["op"] == "store":
        mla.mla_kv_write(s["rows"], s["slots"], s["cache"], layout, page)
        mla.mla_kv_read(s["cache"], layout, page, s["slots"], s["back"])
        return s["back"]
    if c["op"] == "append":
        mla.mla_qkv_norm_rope(s["q_nope"], s["q_pe"], s["rows"], s["slots"], s["positions"], s["kv_weight"], 1e-6,
                              s["freqs"], s["q"], s["cache"], layout, page, q_norm_weight=s["q_weight"],
                              q_eps=1e-6 if c["norm"] else None)
        mla.mla_kv_read(s["cache"], layout, page, s["slots"], s["back"])
        return s["q"], s["back"]
    plan = s["plan"]
    if c["mode"] == "window":
        mla.mla_swa_plan(s["indices"], page, 1, s["runs"], topk_lengths=s["counts"])
        mla.mla_decode_runs(s["q"], s["cache"], layout, page, s["runs"], c["topk"], 1, s["scale"], s["sched"],
                            s["splits"], plan.num_partitions, plan.total_splits, s["workspace"], s["out"], s["lse"],
                            sink=s["sink"])
    else:
        mla.mla_decode(s["q"], s["cache"], layout, page, s["table"], s["lens"], c["tokens"], s["scale"], s["sched"],
                       s["splits"], plan.num_partitions, plan.total_splits, s["workspace"], s["out"], s["lse"],
                       sink=s["sink"], indices=s.get("indices"), causal=c["causal"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------- in 64 bits
def _exact_row(cache, page, rb, nope, slots):
    """Rows at slots [n] in 64 bits, from their bytes: sign, two exponent bits, one mantissa bit."""
    base = cache.view(-1)
    p, o = slots // page, slots % page
    start = p * cache.shape[1] + o * rb
    raw = base[start[:, None] + torch.arange(rb, device="cuda")]
    scale = base[(p * cache.shape[1] + page * rb + o * 16)[:, None] + torch.arange(nope // 32, device="cuda")]
    code = torch.stack([raw[:, :nope // 2] & 15, raw[:, :nope // 2] >> 4], -1).reshape(-1, nope)
    ee, m = (code >> 1 & 3).double(), (code & 1).double()
    v = torch.where(ee == 0, m * 0.5, (1 + m * 0.5) * torch.exp2(ee - 1)) * torch.where(code >= 8, -1.0, 1.0)
    v = v * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)
    pe = raw[:, nope // 2:].int()
    bits = (pe[:, 0::2] << 16 | pe[:, 1::2] << 24).contiguous().view(torch.float32)
    return torch.cat([v, bits.double()], 1)


def _exact_bf16(x):
    """64-bit values rounded once to bfloat16 (to nearest, ties to even), kept in 64 bits."""
    _, k = torch.frexp(x)
    step = torch.exp2((k.double() - 8).clamp_min(-133))
    return torch.round(x / step) * step


def _exact_held(rows, nope):
    """What a cache holds of 64-bit rows: every code's value for the group's scale, the nearest taken."""
    x = rows[:, :nope].reshape(-1, 32)
    amax = x.abs().amax(1).clamp_min(float(np.float32(1e-10)))
    step = torch.exp2(torch.ceil(torch.log2(amax / 6)).clamp(-127, 127))
    step = torch.where(6 * step < amax, step * 2, torch.where(3 * step >= amax, step / 2, step))
    a = (x.abs() / step[:, None]).clamp_max(6)
    # the grid's spacing is 0.5 up to 2, 1 up to 4, 2 up to 6; torch.round takes ties to the even multiple
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.round(a / unit) * unit * step[:, None] * torch.sign(x)
    return torch.cat([v.reshape(-1, nope), rows[:, nope:]], 1)


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = case, case["row"]
    nope = NOPE[kind]
    if c["op"] == "store":
        return _exact_held(s["rows"].double(), nope)
    if c["op"] == "append":
        pair = torch.view_as_complex(s["freqs"].double().view(-1, 32, 2))[s["positions"].long()]
        eps = float(np.float32(1e-6))

        def one(x, weight, pair):
            x = x.double().clone()
            if weight is not None:
                x[..., :512] *= weight.double() / torch.sqrt((x[..., :512] ** 2).mean(-1, keepdim=True) + eps)
            z = torch.view_as_complex(x[..., nope:].reshape(*x.shape[:-1], 32, 2)) * pair
            x[..., nope:] = torch.view_as_real(z).flatten(-2)
            return x

        q = torch.cat([one(torch.cat([s["q_nope"][i:i + 512], s["q_pe"][i:i + 512]], -1), s["q_weight"],
                           pair[i:i + 512, None]) for i in range(0, c["rows"], 512)])
        return q, _exact_held(_exact_bf16(one(s["rows"], s["kv_weight"], pair)), nope)
    batch, tokens, heads = c["batch"], c["tokens"], c["heads"]
    out = torch.zeros(batch, tokens, heads, 512, dtype=torch.float64, device="cuda")
    lse = torch.full((batch, tokens, heads), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(batch):
        if c["mode"] == "dense":
            pos = torch.arange(lens[b], device="cuda")
        else:
            pos = s["indices"][b].long()
            pos = pos[(pos >= 0) & (pos < lens[b])] if c["mode"] == "topk" else pos[:int(s["counts"][b])]
        if pos.numel() == 0:
            continue
        slots = pos if c["mode"] == "window" else s["table"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]
        k = _exact_row(s["cache"], c["page"], ROW[kind], nope, slots)
        for t in range(tokens):
            n = max(0, lens[b] - tokens + t + 1) if c["causal"] else k.shape[0]
            if n == 0:
                continue
            x = s["q"][b * tokens + t].double() @ k[:n].T * float(np.float32(s["scale"]))
            lse[b, t] = torch.logsumexp(x, 1)
            weight = torch.exp(x - lse[b, t][:, None])
            if s["sink"] is not None:
                weight /= 1 + torch.exp(s["sink"].double() - lse[b, t])[:, None]
            out[b, t] = weight @ k[:n, :512]
    return out.view(-1, heads, 512), lse.view(-1, heads)
