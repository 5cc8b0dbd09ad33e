"""Calls on one stream, each reading what the one just ahead of it writes into memory that both sides use again and
again: every reader has the newest bytes, although its kernel may be on the SMs before the writer has ended."""
import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
import workloads
from gpu_helpers import DeviceWorkload

pytestmark = pytest.mark.gpu
STEPS = 40


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_paged_latent_gb300 import build
    build.build()
    mla.load()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _rows(n, width, i):
    """bf16 rows that every layout holds exactly: each group of 32 has one magnitude, a power of two."""
    g = torch.Generator(device="cuda").manual_seed(1000 + i)
    e = torch.randint(-3, 4, (n, width // 32, 1), generator=g, device="cuda").float()
    s = torch.randint(0, 2, (n, width // 32, 32), generator=g, device="cuda").float() * 2 - 1
    return (s * torch.exp2(e)).reshape(n, width).to(torch.bfloat16)


@pytest.mark.parametrize("layout", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("n", [3, 500, 9000])
def test_rows_read_behind_their_write(layout, n):
    """The same slots written and read in turn; two sets of slots share the sectors of their scales."""
    width, ps = workloads._DQK[layout], 64
    kv = torch.zeros(2 * n // ps + 2, mla.mla_page_bytes(layout, ps), dtype=torch.uint8, device="cuda")
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = [2 * at, 2 * at + 1]
    rows = [_rows(n, width, i) for i in range(4)]
    back = [torch.zeros(n, width, dtype=torch.bfloat16, device="cuda") for _ in range(STEPS)]
    torch.cuda.synchronize()
    for i in range(STEPS):
        mla.mla_kv_write(rows[i % 4], slots[i % 2], kv, layout, ps)
        mla.mla_kv_read(kv, layout, ps, slots[i % 2], back[i])
    torch.cuda.synchronize()
    for i in range(STEPS):
        # a 64-element group of the fp8 layouts spans two magnitudes, at most 2^6 apart: both exact in e4m3
        assert torch.equal(back[i], rows[i % 4]), i
    # rows read become rows written, of another cache
    kv2 = torch.zeros_like(kv)
    a, b = torch.zeros_like(rows[0]), torch.zeros_like(rows[0])
    for i in range(STEPS):
        mla.mla_kv_write(rows[i % 4], slots[0], kv, layout, ps)
        mla.mla_kv_read(kv, layout, ps, slots[0], a)
        mla.mla_kv_write(a, slots[1], kv2, layout, ps)
        mla.mla_kv_read(kv2, layout, ps, slots[1], b)
        back[i].copy_(b)
    for i in range(STEPS):
        assert torch.equal(back[i], rows[i % 4]), i


@pytest.mark.parametrize("layout,heads", [(1, 64), (2, 128), (3, 16), (3, 64), (3, 128), (4, 64), (4, 128), (0, 64), (0, 128)])
@pytest.mark.parametrize("listed", [False, True])
def test_decode_behind_the_write_of_its_rows(layout, heads, listed):
    """A short decode behind each write, its partials merged behind it: the outputs of the calls in a row are those of
    the same calls with a synchronisation between them, bit for bit."""
    cfg = (workloads.sparse(batch=4, heads=heads, seqlens=(300, 90, 64, 200), layout=layout, topk=150, page_size=16,
                            min_splits=2, new_rows=False) if listed else
           workloads.dsv3(batch=4, heads=heads, seqlens=(300, 90, 64, 200), len_dist="fixed", layout=layout, page_size=16,
                          new_rows=False))
    w = workloads.generate(cfg)
    slots = np.concatenate([w.block_table[b, np.arange(L) // 16] * 16 + np.arange(L) % 16
                            for b, L in enumerate(w.seqlens)]).astype(np.int32)
    rows = [_rows(slots.size, workloads._DQK[layout], 10 + i) for i in range(3)]
    d = DeviceWorkload(w)
    d.make_plan(min_splits=2)
    at = _cuda(slots)
    apart = []
    for i in range(3):
        mla.mla_kv_write(rows[i], at, d.kv, layout, 16)
        torch.cuda.synchronize()
        d.decode()
        torch.cuda.synchronize()
        apart.append((d.out.clone(), d.lse.clone()))
    assert not torch.equal(apart[0][0], apart[1][0])
    outs = [(torch.zeros_like(d.out), torch.zeros_like(d.lse)) for _ in range(STEPS)]
    torch.cuda.synchronize()
    for i in range(STEPS):
        d.out, d.lse = outs[i]
        mla.mla_kv_write(rows[i % 3], at, d.kv, layout, 16)
        d.decode()
    assert mla.mla_read_status(d.ws) == 0
    for i in range(STEPS):
        assert torch.equal(outs[i][0], apart[i % 3][0]) and torch.equal(outs[i][1], apart[i % 3][1]), i


@pytest.mark.parametrize("layout,heads", [(1, 64), (3, 64), (3, 128), (4, 20)])
def test_windows_behind_their_plan(layout, heads):
    """Runs planned into the same memory for other windows each time, the decode right behind."""
    ps, T, window = 64, 150, 96
    w = workloads.generate(workloads.dsv4(batch=T, seqlens=(200,) * T, len_dist="fixed", heads=heads, layout=layout,
                                          page_size=ps, new_rows=False))
    d = DeviceWorkload(w)
    rng = np.random.default_rng(7)
    pages = w.kv_cache.shape[0]
    idx = [_cuda((rng.integers(0, pages - 1, (T, 1)) * ps + rng.integers(0, 32, (T, 1)) + np.arange(window)).astype(np.int32))
           for _ in range(3)]
    plan = mla.mla_decode_plan(np.full(T, window, np.int32), 1, heads, window)
    ws, sched, ns = mla.alloc_workspace(plan.workspace_bytes), _cuda(plan.sched), _cuda(plan.num_splits)
    runs = torch.zeros(T, 4, dtype=torch.int32, device="cuda")

    def call(i, out, lse, apart):
        mla.mla_swa_plan(idx[i % 3], ps, 1, runs)
        if apart:
            torch.cuda.synchronize()
        mla.mla_decode_runs(d.q, d.kv, layout, ps, runs, window, 1, w.cfg.sm_scale, sched, ns, plan.num_partitions,
                            plan.total_splits, ws, out, lse, sink=d.sink)

    def outputs():
        return torch.zeros(T, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, heads, device="cuda")

    apart = [outputs() for _ in range(3)]
    for i in range(3):
        call(i, *apart[i], True)
        torch.cuda.synchronize()
    assert not torch.equal(apart[0][0], apart[1][0])
    outs = [outputs() for _ in range(STEPS)]
    torch.cuda.synchronize()
    for i in range(STEPS):
        call(i, *outs[i], False)
    assert mla.mla_read_status(ws) == 0
    for i in range(STEPS):
        assert torch.equal(outs[i][0], apart[i % 3][0]) and torch.equal(outs[i][1], apart[i % 3][1]), i
