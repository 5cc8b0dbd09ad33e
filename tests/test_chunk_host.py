"""The chunk's operators without a GPU: the plan covers every query, head and KV tile once, and the entry points refuse what they
do not take before any device work."""
import ctypes

import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
from mla_paged_latent_gb300 import build as mla_build

FAKE, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100008)


def at(mb):
    return ctypes.c_void_p(mb << 20)


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load()


# ------------------------------------------------------------------------------- the plan
def sections(plan):
    i, w = plan.info, plan.sched
    a = 4 * (i.kv_rows // 128)
    b = a + (i.pairs + 1 + 3) // 4 * 4
    c = b + 12 * i.items
    return (w[:a].reshape(-1, 4), w[a:a + i.pairs + 1], w[b:c].reshape(-1, 12), w[c:c + 8 * i.merges].reshape(-1, 8))


def tiles_of(n, length, q0, causal):
    """KV tiles that the 512 queries from q0 on see."""
    last = min(q0 + 512, n) - 1
    lim = min(length, length - n + last + 1) if causal else length
    return max(0, -(-lim // 128))


@pytest.mark.parametrize("seed", range(20))
def test_every_query_and_tile_once(lib, seed):
    rng = np.random.default_rng(seed)
    batch = int(rng.integers(1, 12))
    q = rng.choice([0, 1, 5, 128, 129, 512, 513, 2000], batch)
    kv = rng.choice([0, 1, 127, 128, 129, 3000, 20000], batch)
    heads, causal, sms = int(rng.choice([1, 7, 16])), bool(rng.integers(2)), int(rng.choice([2, 8, 152]))
    plan = mla.mla_chunk_plan(q, kv, heads, causal, num_sms=sms)
    i = plan.info
    kv_tiles, pairs, items, merges = sections(plan)
    blocks = -(-kv // 128) * (q > 0)  # of a request without queries no row is read
    q_start, kv_start = np.cumsum(q) - q, 128 * (np.cumsum(blocks) - blocks)
    of = np.repeat(np.arange(batch), blocks)
    assert np.array_equal(kv_tiles[:, 0], of) and np.array_equal(kv_tiles[:, 2], kv[of])
    assert np.array_equal(kv_tiles[:, 1], 128 * np.arange(len(of)) - kv_start[of])
    assert (i.tokens, i.kv_rows, i.heads, i.group) == (q.sum(), 128 * blocks.sum(), heads, heads)
    assert i.pairs <= max(1, sms // 2) and pairs[0] == 0 and pairs[-1] == i.items
    assert (np.diff(pairs) > 0).all()
    request = {int(q_start[b]): b for b in range(batch) if q[b]}  # those without queries have no items
    seen, parts = {}, {}
    for qs, n, ks, length, q0, head, t0, t1, slot, *_ in items.tolist():
        b = request[qs]
        assert (n, ks, length) == (q[b], kv_start[b], kv[b])
        seen.setdefault((b, q0, head), []).append((t0, t1))
        if slot >= 0:
            parts.setdefault((b, q0, head), []).append(slot)
    want = {(b, q0, h) for b in range(batch) for q0 in range(0, int(q[b]), 512) for h in range(heads)}
    assert set(seen) == want
    for (b, q0, h), ranges in seen.items():
        ranges.sort()
        assert ranges[0][0] == 0 and ranges[-1][1] == tiles_of(int(q[b]), int(kv[b]), q0, causal)
        assert all(x[1] == y[0] for x, y in zip(ranges, ranges[1:]))
        assert (len(ranges) > 1) == ((b, q0, h) in parts)
    used, starts = 0, []
    assert len(merges) == len(parts)
    for token, rows, h, first, n, *_ in merges.tolist():
        b = int(np.searchsorted(q_start, token, "right")) - 1
        while q[b] == 0 or token >= q_start[b] + q[b]:
            b -= 1
        q0 = token - int(q_start[b])
        assert rows == min(512, int(q[b]) - q0) and sorted(parts[b, q0, h]) == [first + rows * k for k in range(n)]
        used += n * rows
        starts.append((first, n * rows))
    assert used == plan.slots
    starts.sort()
    assert all(x + n <= y for (x, n), (y, _) in zip(starts, starts[1:]))


@pytest.mark.parametrize("heads, budget, group", [(16, 0, 1), (16, 512 * 128, 1), (16, 5 * 512 * 128, 4), (7, 3 * 512 * 128, 3),
                                                  (20, 1 << 40, 20)])
def test_groups_of_heads(lib, heads, budget, group):
    plan = mla.mla_chunk_plan([10], [100], heads, kv_budget=budget, num_sms=152)
    assert plan.group == group
    assert plan.workspace_bytes < 256 + 128 * 1152 + 512 + 128 * 512 * group + 64 * group + 512 + 516 * plan.slots


def test_plan_refuses(lib):
    for q, kv, heads in (([1], [-1], 4), ([-1], [1], 4), ([1], [1], 0), ([1], [1], 5000), ([], [], 4),
                         ([1 << 30, 1 << 30], [1, 1], 4), ([1], [2 ** 31 - 1], 4)):
        with pytest.raises(mla.MlaError):
            mla.mla_chunk_plan(q, kv, heads, num_sms=152)
    with pytest.raises(ValueError):
        mla.mla_chunk_plan([1, 2], [3], 4, num_sms=152)
    with pytest.raises(ValueError):
        mla.mla_chunk_plan([1], [3], 4, kv_budget=-1, num_sms=152)
    for q, kv in (([2 ** 32 + 1], [2 ** 32 + 3]), ([1.5], [3]), ([1], [2.5])):
        with pytest.raises(ValueError, match="whole numbers"):
            mla.mla_chunk_plan(q, kv, 4, num_sms=152)
    info = mla._ChunkInfo()
    one = np.array([700], np.int32)
    buf = np.zeros(8, np.int32)
    rc = lib.mla_chunk_plan(one.ctypes.data, one.ctypes.data, 1, 4, 1, 1 << 30, 152, buf.ctypes.data, 8, ctypes.byref(info))
    assert rc == -6 and info.sched_words > 8 and not buf.any()
    assert lib.mla_chunk_plan(one.ctypes.data, one.ctypes.data, 1, 4, 1, 1 << 30, 152, None, 0, ctypes.byref(info)) == 0
    assert lib.mla_chunk_plan(None, one.ctypes.data, 1, 4, 1, 1 << 30, 152, None, 0, ctypes.byref(info)) == -1


# ------------------------------------------------------------------------------- refusals
def chunk_rc(lib, **over):
    plan = over.pop("plan", None) or mla.mla_chunk_plan([100], [300], 4, num_sms=152)
    a = dict(q=at(1), kv=at(16), layout=0, num_pages=40, page=16, table=at(2), max_pages=40, w=at(3), scale=0.1, info=plan.info,
             sched=at(6), ws=at(32), ws_bytes=plan.workspace_bytes, out=at(8), lse=at(9))
    a.update(over)
    info = None if a["info"] is None else ctypes.byref(a["info"])
    return lib.mla_chunk_attention(a["q"], a["kv"], a["layout"], a["num_pages"], a["page"], a["table"], a["max_pages"], a["w"],
                                   a["scale"], info, a["sched"], a["ws"], a["ws_bytes"], a["out"], a["lse"], None)


def test_chunk_attention_refuses(lib):
    for name in ("q", "kv", "table", "w", "sched", "ws", "out", "info"):
        assert chunk_rc(lib, **{name: None}) == -1, name
    for name in ("q", "kv", "w", "sched", "out", "ws"):
        assert chunk_rc(lib, **{name: ODD}) == -1, name
    assert chunk_rc(lib, out=ctypes.c_void_p((8 << 20) + 16)) == -1   # 32-byte stores
    assert chunk_rc(lib, ws=ctypes.c_void_p((32 << 20) + 128)) == -1
    assert chunk_rc(lib, layout=1) == -2 and chunk_rc(lib, layout=3) == -2   # 512-wide rows
    assert b"512-wide" in lib.mla_last_error()
    assert chunk_rc(lib, layout=9) == -1
    assert chunk_rc(lib, page=12) == -2 and chunk_rc(lib, page=4) == -2
    assert chunk_rc(lib, num_pages=0) == -1 and chunk_rc(lib, max_pages=0) == -1
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert chunk_rc(lib, scale=bad) == -1
    plan = mla.mla_chunk_plan([100], [300], 4, num_sms=152)
    assert chunk_rc(lib, ws_bytes=plan.workspace_bytes - 1) == -3
    # overlaps of what is written with what is read, and with one another
    for name in ("q", "kv", "table", "w", "sched"):
        where = {"q": 1, "kv": 16, "table": 2, "w": 3, "sched": 6}[name]
        for out in ("out", "lse", "ws"):
            assert chunk_rc(lib, **{out: at(where)}) == -1, (name, out)
    assert chunk_rc(lib, lse=at(8)) == -1 and chunk_rc(lib, ws=at(8)) == -1 and chunk_rc(lib, ws=at(9)) == -1
    # a plan that was not made here
    for field, value in (("batch", 0), ("tokens", -1), ("kv_rows", 100), ("group", 5), ("sched_words", 3), ("heads", 0)):
        plan = mla.mla_chunk_plan([100], [300], 4, num_sms=152)
        setattr(plan.info, field, value)
        assert chunk_rc(lib, plan=plan) == -1, field
    assert chunk_rc(lib, plan=mla.mla_chunk_plan([0, 0], [300, 4], 4, num_sms=152)) == 0   # nothing to do


def linear_rc(lib, **over):
    a = dict(x=at(1), xs=64, w=at(2), bias=at(3), res=at(4), rs=128, act=0, rows=4, inner=64, outer=128, out=at(5), os=128,
             status=at(6))
    a.update(over)
    return lib.mla_linear(a["x"], a["xs"], a["w"], a["bias"], a["res"], a["rs"], a["act"], a["rows"], a["inner"], a["outer"],
                          a["out"], a["os"], a["status"], None)


def test_linear_refuses(lib):
    assert linear_rc(lib, rows=0, x=None) == 0
    for name in ("x", "w", "out"):
        assert linear_rc(lib, **{name: None}) == -1, name
    for name in ("x", "w", "bias", "res", "out"):
        assert linear_rc(lib, **{name: ODD}) == -1, name
    assert linear_rc(lib, status=ctypes.c_void_p(0x600002)) == -1
    assert linear_rc(lib, rows=-1) == -1 and linear_rc(lib, inner=0) == -1 and linear_rc(lib, outer=0) == -1
    assert linear_rc(lib, inner=60, xs=64) == -2 and linear_rc(lib, outer=100, rs=104, os=104) == -2
    assert linear_rc(lib, act=3) == -1 and linear_rc(lib, act=-1) == -1
    for name, wide in (("xs", 64), ("rs", 128), ("os", 128)):
        assert linear_rc(lib, **{name: wide - 8}) == -1 and linear_rc(lib, **{name: wide + 4}) == -1, name
        assert linear_rc(lib, **{name: -wide}) == -1 and linear_rc(lib, rows=1 << 30, **{name: 1 << 35}) == -1
    for name in ("x", "w", "bias"):
        assert linear_rc(lib, out=linear_at[name]) == -1, name
    assert linear_rc(lib, out=at(4), os=136) == -1                       # the residual's memory, but not element for element
    assert linear_rc(lib, out=ctypes.c_void_p((4 << 20) + 256)) == -1    # a row further


linear_at = {"x": at(1), "w": at(2), "bias": at(3)}


def axes_rc(lib, **over):
    a = dict(qn=at(1), qns=4 * 192, qnh=192, qp=ctypes.c_void_p((1 << 20) + 256), qps=4 * 192, qph=192, width=192, norm=0, qw=None,
             qe=0.0, raw=at(2), rs=576, slots=at(3), pos=at(4), n_axes=3, axes=[0] * 8 + [1] * 12 + [2] * 12, kw=at(5), ke=1e-6,
             freqs=at(6), max_pos=100, T=5, N=4, out=at(7), kv=at(16), layout=0, num_pages=8, page=16, status=None)
    a.update(over)
    axes = None if a["axes"] is None else (ctypes.c_int32 * 32)(*a["axes"])
    return lib.mla_qkv_norm_rope_axes(a["qn"], a["qns"], a["qnh"], a["qp"], a["qps"], a["qph"], a["width"], a["norm"], a["qw"],
                                      a["qe"], a["raw"], a["rs"], a["slots"], a["pos"], a["n_axes"], axes, a["kw"], a["ke"],
                                      a["freqs"], a["max_pos"], a["T"], a["N"], a["out"], a["kv"], a["layout"], a["num_pages"],
                                      a["page"], a["status"], None)


def test_axes_refuses(lib):
    assert axes_rc(lib, T=0, qn=None) == 0
    assert axes_rc(lib, T=-1) == -1
    for name in ("qn", "qp", "raw", "slots", "pos", "axes", "kw", "freqs", "out", "kv"):
        assert axes_rc(lib, **{name: None}) == -1, name
    assert axes_rc(lib, n_axes=0) == -2 and axes_rc(lib, n_axes=5) == -2
    assert axes_rc(lib, n_axes=2) == -1                                  # pairs of axis 2
    assert axes_rc(lib, axes=[-1] + [0] * 31) == -1
    assert axes_rc(lib, width=512) == -1 and axes_rc(lib, width=200) == -1
    assert axes_rc(lib, layout=1) == -1                                  # 192-wide queries beside 512-wide rows
    assert axes_rc(lib, layout=7) == -1
    assert axes_rc(lib, norm=1, qe=1e-6) == -2                           # 192-wide queries are not normalised
    assert axes_rc(lib, qw=at(8)) == -1
    assert axes_rc(lib, ke=-1.0) == -1 and axes_rc(lib, ke=float("nan")) == -1
    assert axes_rc(lib, page=12) == -1 and axes_rc(lib, max_pos=0) == -1 and axes_rc(lib, N=0) == -1
    for name in ("qns", "qnh", "qps", "qph", "rs"):
        assert axes_rc(lib, **{name: 100}) == -1, name
    for name in ("qn", "qp", "raw", "kw", "freqs", "out", "kv"):
        assert axes_rc(lib, **{name: ODD}) == -1, name
    # q_out over its inputs other than row for row, and over the cache; three rows of positions, not one, are looked at
    assert axes_rc(lib, out=ctypes.c_void_p((1 << 20) + 384)) == -1
    assert axes_rc(lib, out=at(16)) == -1 and axes_rc(lib, out=at(2)) == -1
    assert axes_rc(lib, pos=ctypes.c_void_p((7 << 20) - 48)) == -1


class On:
    """A tensor as far as the binding looks before its call: it claims to live on a device."""
    is_cuda = True
    shape = (2, 2, 2)
    dtype = None

    def __init__(self, d):
        self.device, self.get_device = f"cuda:{d}", lambda: d
        self.data_ptr, self.numel = (lambda: 256), (lambda: 1 << 20)


def calls(plan):
    return {
        "mla_qkv_norm_rope_axes": lambda t: (t[0], t[1], t[2], t[3], t[4], [0] * 32, t[5], 1e-6, t[6], t[7], t[8], 4, 64),
        "mla_chunk_attention": lambda t: (t[0], t[1], 0, 64, t[2], t[3], 0.1, plan, t[4], t[5], t[6], t[7]),
        "mla_linear": lambda t: (t[0], t[1], t[2], t[3], None, t[4], t[5]),
    }


@pytest.mark.parametrize("name", ["mla_qkv_norm_rope_axes", "mla_chunk_attention", "mla_linear"])
def test_tensors_of_another_device_are_refused(name, monkeypatch, lib):
    plan = mla.mla_chunk_plan([1], [1], 1, num_sms=2)

    class Lib:
        def __getattr__(self, entry):
            raise AssertionError(f"{entry} was reached")

    monkeypatch.setattr(mla, "load", lambda path=None: Lib())
    monkeypatch.setattr(mla, "_stream", lambda s: None)
    monkeypatch.setattr(mla, "_torch_c", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    call, args = getattr(mla, name), calls(plan)[name]
    with pytest.raises(ValueError, match="current device"):
        call(*args([On(1)] * 9))
    used = args(list(range(100, 109)))
    for i in [x - 100 for x in used if isinstance(x, int) and x >= 100]:
        tensors = [On(0)] * 9
        tensors[i] = On(1)
        with pytest.raises(ValueError, match="one device|current device"):
            call(*args(tensors))


def test_the_binding_names_what_is_wrong(lib, monkeypatch):
    """Types, shapes and layouts, on CPU tensors that claim the current device."""
    monkeypatch.setattr(mla, "_require_one_device", lambda *t: None)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x, w, y = bf(3, 64), bf(16, 64), bf(3, 16)
    for args, kw, what in (((x.float(), w, y), {}, "x must be"), ((x, bf(16, 72), y), {}, "weight"), ((x, w.T, y), {}, "weight"),
                           ((x, w, bf(3, 24)), {}, "out"), ((x, w, y), dict(bias=bf(8)), "bias"),
                           ((x, w, y), dict(residual=bf(4, 16)), "residual"), ((x, w, y), dict(activation="relu"), "activation"),
                           ((bf(64, 3).T, w, y), {}, "adjacent"), ((x[0], w, y), {}, "two dimensions"),
                           ((x, w, y), dict(status=torch.zeros(1, dtype=torch.uint8)), "status")):
        with pytest.raises(ValueError, match=what):
            mla.mla_linear(*args, **kw)
    plan = mla.mla_chunk_plan([3], [5], 2, num_sms=152)
    good = dict(q=bf(3, 2, 192), kv=torch.zeros(2, 8 * 1152, dtype=torch.uint8), table=i32(1, 4), w=bf(2, 256, 512),
                sched=torch.from_numpy(plan.sched), ws=torch.zeros(plan.workspace_bytes, dtype=torch.uint8), out=bf(3, 2, 128),
                lse=torch.zeros(3, 2))
    for name, bad, what in (("q", bf(4, 2, 192), "q must"), ("q", bf(3, 2, 384)[..., ::2], "q must be contiguous"),
                            ("kv", torch.zeros(2, 100, dtype=torch.uint8), "kv_cache"), ("table", i32(2, 4), "block_table"),
                            ("w", bf(2, 512, 256), "w_kv"), ("sched", i32(7), "sched"), ("out", bf(3, 2, 192), "out"),
                            ("lse", bf(3, 2), "lse"), ("ws", good["ws"].view(torch.int8), "workspace")):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError, match=what):
            mla.mla_chunk_attention(a["q"], a["kv"], 0, 8, a["table"], a["w"], 0.1, plan, a["sched"], a["ws"], a["out"], a["lse"])
    good = dict(qn=bf(3, 2, 128), qp=bf(3, 2, 64), raw=bf(3, 576), slots=i32(3), pos=i32(3, 3), axes=[0] * 32, kw=bf(512),
                freqs=torch.zeros(9, 64), out=bf(3, 2, 192), kv=torch.zeros(2, 8 * 1152, dtype=torch.uint8))
    for name, bad, what in (("qn", bf(3, 2, 100), "q_nope"), ("qp", bf(3, 2, 32), "q_pe"), ("raw", bf(3, 512), "kv_raw"),
                            ("slots", i32(4), "slots"), ("pos", i32(3), "positions"), ("pos", i32(3, 4), "positions"),
                            ("pos", i32(3, 3).long(), "positions"), ("axes", [0] * 31, "32 pairs"),
                            ("axes", [2 ** 32] + [0] * 31, "axes below 4"), ("kw", bf(256), "kv_norm_weight"),
                            ("freqs", torch.zeros(9, 32), "freqs"), ("out", bf(3, 2, 576), "q_out")):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError, match=what):
            mla.mla_qkv_norm_rope_axes(a["qn"], a["qp"], a["raw"], a["slots"], a["pos"], a["axes"], a["kw"], 1e-6, a["freqs"],
                                       a["out"], a["kv"], 0, 8)


def test_axes_that_change_are_read_again(monkeypatch):
    """One entry changed in place between two calls; and what is no whole number."""
    monkeypatch.setattr(mla, "_require_one_device", lambda *t: None)
    seen = []

    class Lib:
        def mla_qkv_norm_rope_axes(self, *args):
            seen.append(list(args[15]))
            return 0

        def mla_page_bytes(self, layout, page, out):
            out._obj.value = 8 * 1152
            return 0

    monkeypatch.setattr(mla, "load", lambda path=None: Lib())
    monkeypatch.setattr(mla, "_stream", lambda s: None)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    call = lambda axes: mla.mla_qkv_norm_rope_axes(  # noqa: E731
        bf(3, 2, 128), bf(3, 2, 64), bf(3, 576), i32(3), i32(3, 3), axes, bf(512), 1e-6, torch.zeros(9, 64), bf(3, 2, 192),
        torch.zeros(2, 8 * 1152, dtype=torch.uint8), 0, 8)
    axes = list(torch.arange(32) % 3)
    call(axes)
    axes[5].fill_(0)
    call(axes)
    want = [i % 3 for i in range(32)]
    assert seen[0] == want and seen[1] == want[:5] + [0] + want[6:]
    call(np.arange(32) % 3)
    assert seen[2] == want
    with pytest.raises(TypeError):
        call([0.0] * 32)
