"""Operators of a chunk of new tokens: their plain forms, and the framework's calls.

chunk    attention of a ragged batch of new tokens over the paged latent cache in its per-head form: row c of the cache
         (512 wide, and 64 RoPE elements that all heads share) gives head h the key [W_k[h] c | rope] and the value
         W_v[h] c, 192 and 128 wide.
axes     queries and KV rows rotated by positions of several axes (time, height, width), the queries normalised where
         asked, the rows normalised and appended to the cache, then read back by slot.
linear   matrix product with bias, activation and residual: act(x W^T + bias) + residual.
"""
import math

import numpy as np
import torch

own = False

# name: MLA_KV_* layout, NoPE elements, elements of a group with one scale, bytes of a row and of its scale slot
CACHES = {"bf16": (0, 512, 0, 1152, 0), "fp8_448": (1, 448, 64, 576, 8), "fp8_512": (2, 512, 64, 640, 8),
          "fp4_448": (3, 448, 32, 352, 16), "fp4_512": (4, 512, 32, 384, 16)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ACTIVATIONS = {"none": None, "silu": "silu", "gelu": "gelu"}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # two short prompts on few heads: what a call costs when there is nearly nothing to do
        dict(op="chunk", name="two short prompts", cache="bf16", page=16, heads=16, new="37 130", context="0 0",
             causal=True),
        # a whole prompt at 128 heads
        dict(op="chunk", name="prompt of 8191", cache="fp8_512", page=64, heads=128, new="8191", context="0", causal=True),
        # a chunk of a long prompt, most of it cached already
        dict(op="chunk", name="2048 after 32768", cache="bf16", page=64, heads=128, new="2048", context="32768", causal=True),
        # a mixed batch: prompts and chunks of different lengths, one with a single token
        dict(op="chunk", name="eight ragged chunks", cache="fp4_512", page=32, heads=64,
             new="1 65 300 1500 700 129 1024 33", context="9000 0 4097 0 12345 700 2048 16000",
             causal=True),
        # a short chunk of a long document on few heads: the work has to be split over the context
        dict(op="chunk", name="200 after 65536, 16 heads", cache="bf16", page=64, heads=16, new="200", context="65536",
             causal=True),
        # tokens of images: per-head queries of a prompt, three axes with a section each
        dict(op="axes", name="image tokens 8192 x 128", cache="bf16", page=64, width=192, rows=8192, heads=128,
             sections="8 12 12", interleaved=False, norm=False, max_pos=16384),
        # one decode step after a video: absorbed queries, pairs of the three axes in turn
        dict(op="axes", name="decode step 64 x 128", cache="fp8_512", page=64, width=576, rows=64, heads=128,
             sections="12 10 10", interleaved=True, norm=False, max_pos=32768),
        # a prompt's rows whose RoPE part lies inside the normalised row, queries normalised per head
        dict(op="axes", name="prompt 4099 x 64, norm", cache="fp4_448", page=64, width=512, rows=4099, heads=64,
             sections="16 8 8", interleaved=False, norm=True, max_pos=8192),
        # the output projection of 128 heads in a decode step of one request, and of 64
        dict(op="linear", name="project 1 token", rows=1, inner=16384, outer=8192, bias=False, act="none", residual=True),
        dict(op="linear", name="project 64 tokens", rows=64, inner=16384, outer=8192, bias=False, act="none",
             residual=True),
        # the same of a chunk
        dict(op="linear", name="project 4096 tokens", rows=4096, inner=16384, outer=8192, bias=False, act="none",
             residual=True),
        # odd sizes, every part of the epilogue but the residual
        dict(op="linear", name="bias and gelu, 1001 tokens", rows=1001, inner=1544, outer=6152, bias=True, act="gelu",
             residual=False),
    ]


def _text(numbers):
    return " ".join(str(n) for n in numbers)


def _numbers(text):
    return [int(n) for n in text.split()]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "axes", "linear"))
    if op == "linear":
        inner, outer = 8 * _log(rng, 8, 2048), 8 * _log(rng, 8, 2048)
        rows = _log(rng, 1, min(8192, 2 * 10 ** 11 // (inner * outer)))
        return dict(op=op, rows=rows, inner=inner, outer=outer, bias=rng.random() < 0.5,
                    act=rng.choice(("none", "silu", "gelu")), residual=rng.random() < 0.5)
    page = rng.choice((8, 16, 32, 64, 128))
    if op == "axes":
        width = rng.choice((192, 192, 576, 512))
        cache = rng.choice(("fp8_448", "fp4_448") if width == 512 else ("bf16", "fp8_512", "fp4_512"))
        cut = sorted(rng.randint(0, 32) for _ in range(rng.randint(0, 3)))
        heads = rng.choice((8, 16, 24, 64, 128))
        return dict(op=op, cache=cache, page=page, width=width, rows=_log(rng, 1, 8000 * 64 // max(heads, 64)), heads=heads,
                    sections=_text(b - a for a, b in zip([0] + cut, cut + [32])), interleaved=rng.random() < 0.5,
                    norm=width != 192 and rng.random() < 0.5, max_pos=_log(rng, 1000, 100000))
    heads = rng.choice((8, 16, 20, 64, 128))
    batch = _log(rng, 1, 12)
    new = [_log(rng, 1, 4096 // batch) for _ in range(batch)]
    context = [rng.choice((0, _log(rng, 1, 32000 // batch))) for _ in range(batch)]
    return dict(op=op, cache=rng.choice(("bf16", "fp8_512", "fp4_512")), page=page, heads=heads, new=_text(new), context=_text(context),
                causal=rng.random() < 0.8)


def _pairs(case):
    """(query, row) pairs that a head computes."""
    n = np.array(_numbers(case["new"]), np.int64)
    c = np.array(_numbers(case["context"]), np.int64)
    return n * c + (n * (n + 1) // 2 if case["causal"] else n * n)


def work(case):
    if case["op"] == "linear":
        t, k, m = case["rows"], case["inner"], case["outer"]
        return {"bytes": 2.0 * (t * k + k * m + t * m * (2 if case["residual"] else 1) + (m if case["bias"] else 0)),
                "flops": 2.0 * t * k * m}
    _, nope, _, row, slot = CACHES[case["cache"]]
    if case["op"] == "axes":
        t, width = case["rows"], nope + 64
        queries = t * case["heads"] * case["width"]
        return {"bytes": float(4 * queries + t * (2 * width + 2 * (row + slot) + 2 * width + 4 * (len(_numbers(case["sections"])) + 1))),
                "flops": float(6 * 64 * t * (case["heads"] + 1) + (4 * queries if case["norm"] else 0))}
    n, heads = np.array(_numbers(case["new"]), np.int64), case["heads"]
    rows, pairs = n + np.array(_numbers(case["context"]), np.int64), _pairs(case)
    # the per-head form, or the absorbed one where that is less: 576 + 512 wide, the queries taken to the latent and back
    per_head = 640 * pairs + 2 * 512 * 256 * rows
    absorbed = 2176 * pairs + 2 * 512 * 256 * n
    return {"bytes": float(rows.sum() * (row + slot) + n.sum() * heads * 2 * (192 + 128) + heads * 256 * 512 * 2),
            "flops": float(heads * np.minimum(per_head, absorbed).sum())}


# ------------------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _page_bytes(kind, page):
    _, _, _, row, slot = CACHES[kind]
    return -(-page * (row + slot) // row) * row


def _quantise(x, kind):
    """x [n, groups, elements] fp32 -> (codes, their values, scale bytes) of a cache: the smallest exponent e with
    largest * 2^e >= the group's magnitude, codes rounded to nearest even."""
    four = kind.startswith("fp4")
    amax = x.abs().amax(-1).clamp_min(1e-10)
    m, k = torch.frexp(amax)  # amax = m 2^k; 6 = 0.75 2^3, 448 = 0.875 2^9
    e = (k - torch.where(m <= (0.75 if four else 0.875), 3 if four else 9, 2 if four else 8)).clamp(-127, 127)
    y = torch.ldexp(x, -e[..., None])
    if four:
        a = y.abs()
        code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
                + (a >= 3.5).int() + (a > 5.0).int())
        held = torch.copysign(torch.tensor(E2M1, device=x.device)[code], y)
        code = (code + 8 * torch.signbit(y).int()).to(torch.uint8)
    else:
        code = y.to(torch.float8_e4m3fn)
        held, code = code.float(), code.view(torch.uint8)
    return code, torch.ldexp(held, e[..., None]), (e + 127).to(torch.uint8)


def _held(rows, kind):
    """What a cache holds of bf16 rows [n, width], fp32."""
    _, nope, group, _, _ = CACHES[kind]
    x = rows.float()
    if group:
        x = torch.cat([_quantise(x[:, :nope].reshape(-1, nope // group, group), kind)[1].reshape(-1, nope), x[:, nope:]], 1)
    return x


def _pages(rows, kind, pages, page):
    """bf16 rows [pages * page, width] -> the cache, uint8 [pages, page_bytes]."""
    _, nope, group, row, slot = CACHES[kind]
    cache = torch.zeros(pages, _page_bytes(kind, page), dtype=torch.uint8, device="cuda")
    at = cache[:, :page * row].view(pages, page, row)
    if not group:
        at.copy_(rows.view(torch.uint8).view(pages, page, row))
        return cache
    code, _, scale = _quantise(rows[:, :nope].float().reshape(-1, nope // group, group), kind)
    code = code.reshape(-1, nope)
    if kind.startswith("fp4"):
        code = code[:, 0::2] | code[:, 1::2] << 4
    at[..., :code.shape[1]] = code.view(pages, page, -1)
    at[..., code.shape[1]:] = rows[:, nope:].contiguous().view(torch.uint8).view(pages, page, 128)
    slots = cache[:, page * row:page * (row + slot)].view(pages, page, slot)
    slots[..., :nope // group] = scale.view(pages, page, -1)
    return cache


def _axis_of_pair(case):
    """The axis that turns each of the 32 pairs: sections one after another, or the axes in turn while they last."""
    left = _numbers(case["sections"])
    if not case["interleaved"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while len(out) < 32:
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _table(max_pos):
    """Per position 32 interleaved (cos, sin) pairs; the angles in 64 bits."""
    angle = torch.outer(torch.arange(max_pos, dtype=torch.float64, device="cuda"),
                        10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32))
    return torch.stack([angle.cos(), angle.sin()], -1).reshape(max_pos, 64).float()


def prepare(case, seed):
    c = dict(case)
    for key in ("new", "context", "sections"):
        if key in c:
            c[key] = _numbers(c[key])
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "linear":
        t, k, m = c["rows"], c["inner"], c["outer"]
        s["x"] = _normal(g, t, k).to(torch.bfloat16)
        s["weight"] = (_normal(g, m, k) / math.sqrt(k)).to(torch.bfloat16)
        s["bias"] = _normal(g, m).to(torch.bfloat16) if c["bias"] else None
        s["residual"] = _normal(g, t, m).to(torch.bfloat16) if c["residual"] else None
        s["out"] = torch.empty(t, m, dtype=torch.bfloat16, device="cuda")
        return s
    layout, nope, _, _, _ = CACHES[c["cache"]]
    page, heads, width = c["page"], c["heads"], nope + 64
    if c["op"] == "axes":
        n, axes = c["rows"], len(c["sections"])
        pages = -(-n // page) + 1
        s["cache"] = torch.zeros(pages, _page_bytes(c["cache"], page), dtype=torch.uint8, device="cuda")
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:n].int()
        s["back"] = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
        s["rows"] = (_normal(g, n, width) * torch.exp(0.3 * _normal(g, width))).to(torch.bfloat16)
        # a grid of tokens row by row, frame after frame, from a start on: the axes count at different rates
        first = torch.randint(c["max_pos"] // 2, (axes, 1), generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        rate = [28 * 28, 28, 1, 7][:axes]
        s["positions"] = torch.stack([(first[a] + at // rate[a]) % c["max_pos"] for a in range(axes)]).int()
        s["axes"] = _axis_of_pair(case)
        s["freqs"] = _table(c["max_pos"])
        s["kv_weight"] = (1 + 0.2 * _normal(g, 512)).to(torch.bfloat16)
        s["q_weight"] = (1 + 0.2 * _normal(g, 512)).to(torch.bfloat16) if c["norm"] else None
        if c["width"] == 576:
            # the absorbed part comes from a product batched over heads, the RoPE part is the end of each head of
            # another projection
            s["q_nope"] = _normal(g, heads, n, 512).to(torch.bfloat16).transpose(0, 1)
            s["q_pe"] = _normal(g, n, heads, 192).to(torch.bfloat16)[..., 128:]
        else:
            q = _normal(g, n, heads, c["width"]).to(torch.bfloat16)
            s["q_nope"], s["q_pe"] = q[..., :-64], q[..., -64:]
        s["q"] = torch.empty(n, heads, c["width"], dtype=torch.bfloat16, device="cuda")
        return s
    lens = [a + b for a, b in zip(c["new"], c["context"])]
    per = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(per), generator=g, device="cuda").int()
    for b, n in enumerate(per):
        table[b, :n] = order[sum(per[:b]):sum(per[:b]) + n]
    s["table"], s["lens"] = table, lens
    s["cache"] = _pages((_normal(g, sum(per) * page, width) * torch.exp(0.3 * _normal(g, width))).to(torch.bfloat16),
                        c["cache"], sum(per), page)
    s["q"] = _normal(g, sum(c["new"]), heads, 192).to(torch.bfloat16)
    s["weight"] = (_normal(g, heads, 256, 512) / math.sqrt(512)).to(torch.bfloat16)
    s["scale"] = 1 / math.sqrt(192)
    if own:
        import mla_paged_latent_gb300 as mla
        s["plan"] = mla.mla_chunk_plan(c["new"], lens, heads, causal=c["causal"])
        s["sched"] = torch.from_numpy(s["plan"].sched).cuda()
        s["workspace"] = mla.alloc_workspace(s["plan"].workspace_bytes)
        s["out"] = torch.empty(sum(c["new"]), heads, 128, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _request_rows(s, b):
    """The cached rows of request b, fp32 [length, 576]."""
    c = s["case"]
    _, nope, group, row, slot = CACHES[c["cache"]]
    page, n = c["page"], s["lens"][b]
    mine = s["cache"][s["table"][b, :-(-n // page)].long()]
    raw = mine[:, :page * row].reshape(-1, row)[:n]
    if not group:
        return raw.contiguous().view(torch.bfloat16).float()
    scale = mine[:, page * row:page * (row + slot)].reshape(-1, slot)[:n, :nope // group]
    if c["cache"].startswith("fp4"):
        grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        code = raw[:, :nope // 2]
        v = torch.stack([grid[(code & 15).int()], grid[(code >> 4).int()]], -1).reshape(-1, nope)
    else:
        code = raw[:, :nope]
        v = code.contiguous().view(torch.float8_e4m3fn).float()
    v = v.view(n, -1, group) * torch.exp2(scale.float() - 127)[..., None]
    return torch.cat([v.reshape(n, nope), raw[:, -128:].contiguous().view(torch.bfloat16).float()], 1)


def _chunk(s):
    c = s["case"]
    heads, outs, at = c["heads"], [], 0
    for b, n in enumerate(c["new"]):
        rows, length = _request_rows(s, b), s["lens"][b]
        q = s["q"][at:at + n].float().transpose(0, 1)
        at += n
        step = max(1, min(heads, (1 << 28) // (n * length)))
        hidden = None
        if c["causal"]:
            last = length - n + torch.arange(n, device="cuda")
            hidden = torch.arange(length, device="cuda") > last[:, None]
        part = []
        for h in range(0, heads, step):
            w = s["weight"][h:h + step].float()
            k = torch.matmul(rows[:, :512], w[:, :128].transpose(1, 2))
            v = torch.matmul(rows[:, :512], w[:, 128:].transpose(1, 2))
            score = torch.matmul(q[h:h + step, :, :128], k.transpose(1, 2))
            score += torch.matmul(q[h:h + step, :, 128:], rows[:, 512:].T)
            score *= s["scale"]
            if hidden is not None:
                score.masked_fill_(hidden, -math.inf)
            score = score.sub_(score.amax(-1, keepdim=True)).exp_()
            total = score.sum(-1, keepdim=True)
            part.append((torch.matmul(score, v) / total).transpose(0, 1))
        outs.append(torch.cat(part, 1))
    return torch.cat(outs).to(torch.bfloat16)


def _norm(x, weight, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight


def _rotate(x, angle):
    """Adjacent pairs of x [n, ..., 64] by their tokens' (cos, sin) pairs, angle [n, 32, 2]."""
    cos, sin = angle[..., 0], angle[..., 1]
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)


def _axes(s):
    c = s["case"]
    nope = CACHES[c["cache"]][1]
    where = s["positions"][torch.tensor(s["axes"], device="cuda")].long()  # [32, n]
    angle = s["freqs"].view(-1, 32, 2)[where, torch.arange(32, device="cuda")[:, None]].transpose(0, 1)
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float()
    if s["q_weight"] is not None:
        q = torch.cat([_norm(q[..., :512], s["q_weight"].float(), 1e-6), q[..., 512:]], -1)
    q = torch.cat([q[..., :-64], _rotate(q[..., -64:], angle)], -1).to(torch.bfloat16)
    rows = s["rows"].float()
    rows = torch.cat([_norm(rows[:, :512], s["kv_weight"].float(), 1e-6), rows[:, 512:]], -1)
    rows = torch.cat([rows[:, :nope], _rotate(rows[:, nope:], angle)], -1).to(torch.bfloat16)
    return q, _held(rows, c["cache"]).to(torch.bfloat16)


def _linear(s):
    y = s["x"].float() @ s["weight"].float().T
    if s["bias"] is not None:
        y += s["bias"].float()
    if s["case"]["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif s["case"]["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if s["residual"] is not None:
        y += s["residual"].float()
    return y.to(torch.bfloat16)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"chunk": _chunk, "axes": _axes, "linear": _linear}[c["op"]](s)
    import mla_paged_latent_gb300 as mla
    if c["op"] == "linear":
        mla.mla_linear(s["x"], s["weight"], s["out"], bias=s["bias"], activation=ACTIVATIONS[c["act"]],
                       residual=s["residual"])
        return s["out"]
    layout = CACHES[c["cache"]][0]
    if c["op"] == "axes":
        mla.mla_qkv_norm_rope_axes(s["q_nope"], s["q_pe"], s["rows"], s["slots"], s["positions"], s["axes"],
                                   s["kv_weight"], 1e-6, s["freqs"], s["q"], s["cache"], layout, c["page"],
                                   q_norm_weight=s["q_weight"], q_eps=1e-6 if c["norm"] else None)
        mla.mla_kv_read(s["cache"], layout, c["page"], s["slots"], s["back"])
        return s["q"], s["back"]
    mla.mla_chunk_attention(s["q"], s["cache"], layout, c["page"], s["table"], s["weight"], s["scale"], s["plan"],
                            s["sched"], s["workspace"], s["out"])
    return s["out"]


# ------------------------------------------------------------------------------- in 64 bits
def _exact_rows(cache, kind, page, slots):
    """Rows at slots [n] in 64 bits, from their bytes."""
    _, nope, group, row, slot = CACHES[kind]
    base, p, o = cache.view(-1), slots // page, slots % page
    raw = base[(p * cache.shape[1] + o * row)[:, None] + torch.arange(row, device="cuda")]
    pe = raw[:, row - 128 if group else 0:].int()
    plain = (pe[:, 0::2] << 16 | pe[:, 1::2] << 24).contiguous().view(torch.float32).double()
    if not group:
        return plain
    scale = base[(p * cache.shape[1] + page * row + o * slot)[:, None] + torch.arange(nope // group, device="cuda")]
    if kind.startswith("fp4"):  # sign, two exponent bits, one mantissa bit; bias 1
        code = torch.stack([raw[:, :nope // 2] & 15, raw[:, :nope // 2] >> 4], -1).reshape(-1, nope)
        sign, e, m, bias, steps = code >> 3, (code >> 1 & 3).double(), (code & 1).double(), 1, 2
    else:  # sign, four exponent bits, three mantissa bits; bias 7
        code = raw[:, :nope]
        sign, e, m, bias, steps = code >> 7, (code >> 3 & 15).double(), (code & 7).double(), 7, 8
    v = torch.where(e == 0, m / steps * 2.0 ** (1 - bias), (1 + m / steps) * torch.exp2(e - bias))
    v = torch.where(sign == 1, -v, v) * torch.exp2(scale.double() - 127).repeat_interleave(group, 1)
    return torch.cat([v, plain], 1)


def _exact_bf16(x):
    """64-bit values rounded once to bfloat16 (to nearest, ties to even), kept in 64 bits."""
    _, k = torch.frexp(x)
    step = torch.exp2((k.double() - 8).clamp_min(-133))
    return torch.round(x / step) * step


def _exact_held(rows, kind):
    """What a cache holds of 64-bit rows: every code's value for the group's scale, the nearest taken."""
    _, nope, group, _, _ = CACHES[kind]
    if not group:
        return rows
    four = kind.startswith("fp4")
    largest, least = (6.0, 0.5) if four else (448.0, 2.0 ** -9)
    x = rows[:, :nope].reshape(-1, group)
    amax = x.abs().amax(1).clamp_min(float(np.float32(1e-10)))
    step = torch.exp2(torch.ceil(torch.log2(amax / largest)).clamp(-127, 127))
    step = torch.where(largest * step < amax, step * 2, torch.where(largest / 2 * step >= amax, step / 2, step))
    a = (x.abs() / step[:, None]).clamp_max(largest)
    # the codes' spacing: the least value's, up to twice a mantissa's worth of it, then doubling with every power of two
    unit = torch.exp2(torch.floor(torch.log2(a.clamp_min(1e-30))) - (1 if four else 3)).clamp_min(least)
    v = torch.round(a / unit) * unit * step[:, None] * torch.sign(x)
    return torch.cat([v.reshape(-1, nope), rows[:, nope:]], 1)


def _exact_axes(s):
    c = s["case"]
    nope, eps = CACHES[c["cache"]][1], float(np.float32(1e-6))
    pair = torch.view_as_complex(s["freqs"].double().view(-1, 32, 2))
    turn = torch.stack([pair[s["positions"][a].long(), i] for i, a in enumerate(s["axes"])], 1)

    def one(x, weight, turn):
        x = x.double().clone()
        if weight is not None:
            x[..., :512] *= weight.double() / torch.sqrt((x[..., :512] ** 2).mean(-1, keepdim=True) + eps)
        z = torch.view_as_complex(x[..., -64:].reshape(*x.shape[:-1], 32, 2)) * turn
        x[..., -64:] = torch.view_as_real(z).flatten(-2)
        return x

    q = torch.cat([one(torch.cat([s["q_nope"][i:i + 512], s["q_pe"][i:i + 512]], -1), s["q_weight"],
                       turn[i:i + 512, None]) for i in range(0, c["rows"], 512)])
    return q, _exact_held(_exact_bf16(one(s["rows"], s["kv_weight"], turn)), c["cache"])


def _exact_linear(s):
    c, out = s["case"], []
    for i in range(0, c["outer"], 1024):
        y = torch.einsum("tk,mk->tm", s["x"].double(), s["weight"][i:i + 1024].double())
        if s["bias"] is not None:
            y = y + s["bias"][i:i + 1024].double()
        if c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        out.append(y if s["residual"] is None else y + s["residual"][:, i:i + 1024].double())
    return torch.cat(out, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s)
    if case["op"] == "axes":
        return _exact_axes(s)
    new = s["case"]["new"]
    out = torch.empty(sum(new), case["heads"], 128, dtype=torch.float64, device="cuda")
    scale, at = float(np.float32(s["scale"])), 0
    for b, n in enumerate(new):
        length = s["lens"][b]
        pos = torch.arange(length, device="cuda")
        row = _exact_rows(s["cache"], case["cache"], case["page"],
                          s["table"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"])
        latent, rope = row[:, :512], row[:, 512:]
        for h in range(case["heads"]):
            w = s["weight"][h].double()
            x = torch.cat([latent @ w[:128].T, rope], 1) @ s["q"][at:at + n, h].double().T * scale  # [length, n]
            if case["causal"]:
                x[length - n:].masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").tril(-1), -math.inf)
            out[at:at + n, h] = torch.softmax(x, 0).T @ (latent @ w[128:].T)
        at += n
    return out
