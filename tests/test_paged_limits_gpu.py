"""The paged KV cache at its limits on the GPU, against the float64 oracle."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import oracle
from block_sparse_approximate_b200 import binding as bd
from block_sparse_approximate_b200.pipeline import PagedServing
from tests.test_paged_gpu import DEV, _i32

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_plan_around_the_default_shared_memory_limit(lib):
    # The prefix sums of 2419 .. 2457 requests fit a CTA's default shared memory only without the kernel's static
    # arrays.  A process of its own, from few requests to many: a larger call's launch attribute would stay.
    code = textwrap.dedent("""
        import numpy as np, torch, oracle
        from block_sparse_approximate_b200 import binding as bd
        i32 = lambda a: torch.from_numpy(np.asarray(a)).to(device="cuda", dtype=torch.int32)
        for S in (2048, 2049, 2418, 2419, 2440, 2457, 2458, 4096, 2440):
            r = np.random.RandomState(S)
            ctx, new = np.zeros(S, int), r.randint(0, 3, S)
            held, table, ring, state = np.zeros(S, int), np.full((S, 2), -1), r.permutation(S), np.array([7, S])
            d = [i32(a) for a in (held, table, ring, state)]
            got = bd.paged_plan(i32(ctx), i32(new), *d, 2 * S, 16)
            ref = oracle.paged_plan(ctx, new, held, table, ring, state, 2 * S, 16)
            for x, y in zip((*got, *d), ref):
                np.testing.assert_array_equal(x.cpu().numpy(), y, err_msg=str(S))
        print("plans ok")
    """)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "plans ok" in r.stdout, r.stdout + r.stderr


def test_plan_of_its_own_lengths_is_refused(lib):
    # kv_len as the next step's ctx_len: read and written by the call
    eng = PagedServing(requests=3, max_pages=4, pages=16, page=16, tokens=40, Hq=2, Hkv=1, d=64)
    eng.plan(_i32([0, 0, 0]), _i32([15, 16, 1]))
    state = (eng.held, eng.table, eng.free_pages, eng.free_state, eng.q_start, eng.kv_len, eng.slots)
    before = [x.clone() for x in state]
    with pytest.raises(bd.SparseAttnError, match="kv_len and ctx_len overlap"):
        eng.plan(eng.kv_len, _i32([1, 1, 1]))
    assert all(torch.equal(x, y) for x, y in zip(state, before))
    ctx = eng.kv_len.clone()                        # the caller's own copy serves
    q_start, kv_len, slots = eng.plan(ctx, _i32([1, 1, 1]))
    assert kv_len.tolist() == [16, 17, 2] and eng.held.tolist() == [1, 2, 1]


@pytest.mark.parametrize("S,tokens", [(5, 40), (1500, 3000)])
def test_plan_of_adjacent_arrays(lib, S, tokens):
    # the arrays lie behind one another in one buffer, without a gap: nothing overlaps
    r = np.random.RandomState(S)
    width, P = 3, 2 * S
    new = r.randint(0, 3, S)
    first = [np.zeros(S, int), new, np.zeros(S, int), np.full((S, width), -1), r.permutation(P), np.array([P - 2, P]),
             np.zeros(S + 1, int), np.zeros(S, int)]
    n = sum(a.size for a in first)
    flat = torch.zeros(2 * tokens + n, device=DEV, dtype=torch.int32)
    at, views = 2 * tokens, []
    for a in first:
        v = flat[at:at + a.size].view(a.shape)
        v.copy_(_i32(a))
        views.append(v)
        at += a.size
    ctx_d, new_d, held, table, ring, state, q_start, kv_len = views
    slots = flat[:2 * tokens].view(torch.int64)
    bd.paged_plan(ctx_d, new_d, held, table, ring, state, tokens, 16, q_start=q_start, kv_len=kv_len, slots=slots)
    ref = oracle.paged_plan(*first[:6], tokens, 16)
    for x, y in zip((q_start, kv_len, slots, held, table, ring, state), ref):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
    assert ctx_d.count_nonzero() == 0 and np.array_equal(new_d.cpu().numpy(), new)
