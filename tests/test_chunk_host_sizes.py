"""Chunk plans at the ends of their ranges, without a GPU."""
import ctypes
import time

import numpy as np
import pytest

import mla_paged_latent_gb300 as mla
from mla_paged_latent_gb300 import build as mla_build


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load()


def test_more_units_than_an_index_holds_are_refused(lib):
    """Requests without a cached row need no space for K and V, so nothing else bounds their units: one a request and head, of 12
    words each. Refused before they are made."""
    q, kv = np.ones(44000, np.int32), np.zeros(44000, np.int32)
    info = mla._ChunkInfo()
    start = time.monotonic()
    rc = lib.mla_chunk_plan(q.ctypes.data, kv.ctypes.data, 44000, 4096, 1, 1 << 33, 152, None, 0, ctypes.byref(info))
    assert rc == -2 and b"units" in lib.mla_last_error()
    assert time.monotonic() - start < 5  # (of 25 to make them)
    with pytest.raises(mla.MlaError, match="units"):
        mla.mla_chunk_plan(q, kv, 4096, num_sms=152)


def test_many_requests_without_rows_are_planned(lib):
    plan = mla.mla_chunk_plan(np.ones(20000, np.int32), np.zeros(20000, np.int32), 16, num_sms=152)
    assert plan.info.items == 320000 and plan.info.merges == 0 and plan.info.kv_rows == 0


def test_the_longest_request(lib):
    """2^31 - 512 rows or queries are the end; just below it the plan's sums hold."""
    plan = mla.mla_chunk_plan([5], [2 ** 31 - 640], 1, kv_budget=0, num_sms=152)
    assert plan.info.kv_rows == 2 ** 31 - 640 and plan.workspace_bytes > 1152 * (2 ** 31 - 640)
    for q, kv in (([1], [2 ** 31 - 512]), ([2 ** 31 - 512], [1])):
        with pytest.raises(mla.MlaError, match="too many"):
            mla.mla_chunk_plan(q, kv, 1, num_sms=152)
