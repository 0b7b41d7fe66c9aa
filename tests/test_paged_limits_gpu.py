"""The paged KV cache at its limits on the GPU, against the float64 oracle."""
import os
import subprocess
import sys
import textwrap

import pytest

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
