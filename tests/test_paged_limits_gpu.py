"""The paged KV cache at its limits on the GPU, against the float64 oracle.

Tolerances are those of test_paged_gpu's assert_attention, for fp32 too where
masked keys are not finite, unless a test derives its own.
"""
import math
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
from tests._parity import assert_no_device_error, np64
from tests.test_paged_gpu import BF, DEV, F32, Case, _i32, assert_attention

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


def planted(c, s, key):
    """The pool's page and offset of a request's key."""
    page = c.Kc.shape[2]
    return int(c.table[s, key // page]), key % page


@pytest.mark.parametrize("dtype,d,Hq", [(BF, 128, 8), (BF, 64, 2), (F32, 128, 8), (F32, 64, 2), (F32, 64, 16)])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_scores_above_float32(lib, dtype, d, Hq, n):
    # q.k is finite and scale q.k is not: such a row is NaN, wherever the key lies; the other KV head's scores are 0
    c = Case([300, 40, 2000], [n, n, n], Hq, 2, d, 32, dtype, seed=31, poison=False)
    c.scale = 8.0
    c.Q = torch.zeros_like(c.Q)
    c.Q[..., 0] = 2.0 ** 63
    c.Kc[..., 0] = 0.0
    for s, key in ((0, 5), (1, 40), (2, 1500)):
        pid, off = planted(c, s, key)
        c.Kc[pid, 0, off, 0] = 2.0 ** 63
    out = c.run()
    torch.cuda.synchronize()
    assert_no_device_error()
    assert out[:, :Hq // 2].isnan().all()
    c.Kc[..., 0] = 0.0                             # (the oracle has no such rows; weights are equal and exact)
    O, A, seen = c.oracle()
    w = 2.0 ** -8 if dtype == BF else 2.0 ** -24   # the weight's and the output's rounding
    bound = (w + 2 * (2.0 ** -21 + seen[:, None, None] * 2.0 ** -24)) * A + 2 * w * np.abs(O)
    assert (np.abs(np64(out) - O) <= bound)[:, Hq // 2:].all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_rows_whose_scores_are_all_minus_infinity(lib, dtype, d, n):
    # one KV head's keys score -inf (K holds it): its rows are zero, the other head's are as ever
    c = Case([200, 2500, 3], [n, n, n], 4, 2, d, 16, dtype, seed=33, poison=False)
    c.Q = c.Q.clone()
    c.Q[..., 0] = 1.0
    O, A, seen = c.oracle()
    c.Kc[:, 1, :, 0] = float("-inf")
    out = c.run(out=torch.full((c.T, 4, d), 7.0, device=DEV, dtype=dtype))
    assert (out[:, 2:] == 0).all()
    c.Kc[:, 1, :, 0] = 0.0
    out[:, 2:] = torch.from_numpy(O[:, 2:]).to(DEV).to(dtype)
    assert_attention(out, O, A, seen, c, 7.0)


def test_scale_whose_logarithm_base_2_overflows_is_refused(lib):
    c = Case([5], [1], 2, 1, 64, 16, BF, seed=32, poison=False)
    c.scale = 3e38
    with pytest.raises(bd.SparseAttnError, match="scale"):
        c.run()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("low", [-1e4, float("-inf")])
@pytest.mark.parametrize("dtype,d,lens", [
    (BF, 128, "whole"), (BF, 64, "split"), (BF, 128, "split"), (BF, 128, "chunk"), (BF, 64, "chunk"),
    (F32, 64, "whole"), (F32, 128, "split"), (F32, 64, "chunk")])
def test_values_under_vanishing_weights(lib, dtype, d, lens, low, bad):
    # A key that rows see with a weight of 0 holds a value that is not finite: its column is not finite, whether
    # the key's tile is seen whole (5, 130) or in part (the last keys), in whole items, split ones and chunks
    ctx, new = {"whole": ([260] * 300, [1] * 300), "split": ([9000, 700], [1, 2]),
                "chunk": ([300, 0], [150, 200])}[lens]
    c = Case(ctx, new, 4, 2, d, 16, dtype, seed=34, poison=False)
    c.Q = c.Q.clone()
    c.Q[..., 0] = 8.0
    clean = c.Kc.clone()
    keys = {0: (5, 130), 1: (c.kv[1] - 1,)}
    hit = np.zeros(c.T, bool)
    for s, at in keys.items():
        for key in at:
            pid, off = planted(c, s, key)
            c.Kc[pid, :, off, 0] = low
            first = c.kv[s] - new[s]
            hit[c.q_start[s] + max(0, key - first):c.q_start[s + 1]] = True
    # every row keeps a key of its own beside the planted ones
    O, A, seen = c.oracle()
    for s, at in keys.items():
        for key in at:
            pid, off = planted(c, s, key)
            c.Vc[pid, :, off, 9] = bad
    out = c.run()
    torch.cuda.synchronize()
    assert_no_device_error()
    assert not out[torch.from_numpy(hit).to(DEV)][..., 9].isfinite().any()
    if math.isnan(bad):
        assert out[torch.from_numpy(hit).to(DEV)][..., 9].isnan().all()
    want = torch.from_numpy(O).to(DEV).to(dtype)
    out[torch.from_numpy(hit).to(DEV), :, 9] = want[torch.from_numpy(hit).to(DEV), :, 9]
    c.Kc = clean                                   # (the largest score that counts is one of these)
    assert_attention(out, O, A, seen, c, 7.0)


@pytest.mark.parametrize("dtype,d,group", [(F32, 128, 1), (F32, 128, 2), (F32, 64, 4), (F32, 64, 1), (F32, 128, 4),
                                           (BF, 128, 4), (BF, 64, 1)])
@pytest.mark.parametrize("window", [0, 1, 70, 200])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_masked_keys_that_are_not_finite(lib, dtype, d, group, window, bad):
    # K and V of some keys are not finite: rows that do not see them (earlier tokens; with a window also later ones)
    # are right to the type's own tolerance, rows that see them are not finite
    c = Case([200, 130, 63, 500, 260], [2, 3, 40, 130, 8], 2 * group, 2, d, 16, dtype, seed=35, window=window, pad=1)
    out = torch.full((c.T, 2 * group, d), 7.0, device=DEV, dtype=dtype)
    O, A, seen = c.oracle()
    clean = c.Kc.clone()
    hit = np.zeros(c.T, bool)
    for s, back in enumerate((0, 1, 20, 64, 3)):   # the key is `back` tokens before the request's last
        key = int(c.kv[s]) - 1 - back
        pid, off = planted(c, s, key)
        c.Vc[pid, :, off] = bad
        c.Kc[pid, :, off, 3] = bad
        first = key - (int(c.kv[s]) - (c.q_start[s + 1] - c.q_start[s]))
        rows = np.arange(c.q_start[s + 1] - c.q_start[s])
        hit[c.q_start[s]:c.q_start[s + 1]] = (rows >= first) & ((window == 0) | (rows < first + window))
    c.run(out=out)
    torch.cuda.synchronize()
    assert_no_device_error()
    mask = torch.from_numpy(hit).to(DEV)
    assert not out[mask].isfinite().any()
    out[mask] = torch.from_numpy(O).to(DEV).to(dtype)[mask]
    c.Kc = clean
    assert_attention(out, O, A, seen, c, 7.0)


def test_serving_steps_in_fp32_are_close(lib):
    # chunks, single tokens, a step back and a refused request, each step to fp32's tolerance
    r = np.random.RandomState(36)
    Hq, Hkv, d, page, T = 6, 2, 64, 16, 80
    eng = PagedServing(requests=3, max_pages=12, pages=30, page=page, tokens=T, Hq=Hq, Hkv=Hkv, d=d, dtype=F32)
    eng.Kcache.fill_(float("nan"))
    eng.Vcache.fill_(float("nan"))
    hist, length = [np.zeros((2, 0, Hkv, d)) for _ in range(3)], np.zeros(3, int)
    for at, new in ((None, [40, 1, 0]), (None, [30, 1, 33]), (None, [1, 1, 1]), ([50, -1, 20], [2, 70, 3]),
                    (None, [3, 0, 76])):
        for s, a in enumerate(at or ()):
            if a >= 0:
                length[s], hist[s] = a, hist[s][:, :a]
        fused = torch.from_numpy(r.randn(T, Hq + 2 * Hkv, d)).to(DEV).to(F32)
        Q, K, V = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        eng.plan(_i32(length), _i32(new))
        out = np64(eng.attend(Q, K, V, 0.125))
        rows = np.concatenate([[0], np.cumsum(new)])
        assert eng.kv_len.tolist() == (length + new).tolist()
        for s in range(3):
            a, b = rows[s], rows[s + 1]
            hist[s] = np.concatenate([hist[s], np.stack([np64(K[a:b]), np64(V[a:b])])], axis=1)
            length[s] += new[s]
            if a == b:
                continue
            k, v = (x.transpose(1, 0, 2)[None] for x in hist[s])
            O, A, _ = oracle.paged_attention(np64(Q[a:b]), k, v, [[0]], [0, b - a], [length[s]], 0.125)
            largest = np.sqrt((np64(Q[a:b]) ** 2).sum(-1)).max() * np.sqrt((k ** 2).sum(-1)).max() * 0.125
            w = (d + 4) * 2.0 ** -24 * largest + 2.0 ** -21 + length[s] * 2.0 ** -24
            assert (np.abs(out[a:b] - O) <= 2 * w * A + 2.0 ** -23 * np.abs(O) + 1e-30).all(), (new, s)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_table_entries_leave_the_other_requests_exact(lib, dtype):
    # entries outside the pool under one request's keys: the others' bits are those without them
    c = Case([100, 90, 300], [40, 1, 3], 4, 2, 64, 32, dtype, seed=37, poison=False)
    want = c.run()
    c.table[0, 1], c.table[0, 2] = 1 << 30, -5
    out = c.run()
    torch.cuda.synchronize()
    assert_no_device_error()
    assert torch.equal(out[40:], want[40:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pages,width", [(0, 3), (4, 0), (0, 0)])
def test_no_pages(lib, dtype, pages, width):
    # a pool or a table without pages holds no key: every row of a request is zero
    Kc = torch.zeros(pages, 2, 16, 64, device=DEV, dtype=dtype)
    Q = torch.randn(6, 4, 64, device=DEV).to(dtype)
    out = torch.full_like(Q, 7.0)
    bd.paged_attn_fwd(Q, Kc, Kc.clone(), _i32(np.zeros((2, width))), _i32([0, 1, 5]), _i32([9, 40]), 0.125, out=out)
    torch.cuda.synchronize()
    assert_no_device_error()
    assert (out[:5] == 0).all() and (out[5:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_without_rows_or_requests(lib, dtype):
    Kc = torch.ones(3, 2, 16, 64, device=DEV, dtype=dtype)
    before = Kc.clone()
    none = torch.empty(0, 2, 64, device=DEV, dtype=dtype)
    bd.paged_append(none, none, torch.empty(0, device=DEV, dtype=torch.int64), Kc, Kc.clone())
    assert torch.equal(Kc, before)
    table, kv = _i32([[0, 1]]), _i32([20])
    assert bd.paged_attn_fwd(none, Kc, Kc, table, _i32([0, 0]), kv, 0.125).shape == (0, 2, 64)
    out = torch.full((3, 2, 64), 7.0, device=DEV, dtype=dtype)
    bd.paged_attn_fwd(torch.ones_like(out), Kc, Kc, _i32(np.zeros((0, 2))), _i32([0]), _i32([]), 0.125, out=out)
    assert (out == 7.0).all()
    # a plan without rows in its arrays still hands pages back, and refuses rows
    held, ring, state = _i32([2]), _i32([2, 0, 0]), _i32([0, 1])
    q_start, kv_len, slots = bd.paged_plan(_i32([5]), _i32([0]), held, table, ring, state, 0, 16)
    assert q_start.tolist() == [0, 0] and kv_len.tolist() == [5] and held.tolist() == [1] and slots.numel() == 0
    assert table.tolist() == [[0, -1]] and state.tolist() == [0, 2] and ring.tolist()[:2] == [2, 1]
    assert bd.paged_plan(_i32([5]), _i32([1]), held, table, ring, state, 0, 16)[1].tolist() == [0]


def test_many_requests_captured(lib):
    # plan, append and fp32 attention of 2440 requests in a graph, replayed with other lengths
    S, page, T = 2440, 16, 2600
    r = np.random.RandomState(38)
    eng = PagedServing(requests=S, max_pages=3, pages=2 * S, page=page, tokens=T, Hq=2, Hkv=1, d=64, dtype=F32)
    ctx_d, new_d = _i32(np.zeros(S)), _i32(np.zeros(S))
    fused = torch.zeros(T, 4, 64, device=DEV)
    Q, K, V = fused[:, :2], fused[:, 2:3], fused[:, 3:]

    def step():
        eng.plan(ctx_d, new_d)
        eng.attend(Q, K, V, 0.125)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                      # nothing to do yet: lengths are zero
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    length, rows = np.zeros(S, int), [[np.zeros((0, 64))] * 2 for _ in range(S)]
    for _ in range(3):
        new = r.randint(0, 2, S)
        new[r.randint(0, S, 20)] = r.randint(2, 12, 20)
        ctx_d.copy_(_i32(length))
        new_d.copy_(_i32(new))
        fused.copy_(torch.from_numpy(r.randn(T, 4, 64)).to(DEV))
        g.replay()
        out, q, k, v = (np64(x) for x in (eng.out, Q, K, V))
        assert eng.kv_len.tolist() == (length + new).tolist()
        q_start = np.concatenate([[0], np.cumsum(new)])
        length += new
        for s in range(S):
            a, b = q_start[s], q_start[s + 1]
            rows[s] = [np.concatenate([x, y[a:b, 0]]) for x, y in zip(rows[s], (k, v))]
            if a == b:
                continue
            O, A, _ = oracle.paged_attention(q[a:b], *(x[None, None] for x in rows[s]), [[0]], [0, b - a], [length[s]],
                                             0.125)
            largest = np.sqrt((q[a:b] ** 2).sum(-1)).max() * np.sqrt((rows[s][0] ** 2).sum(-1)).max() * 0.125
            w = 68 * 2.0 ** -24 * largest + 2.0 ** -21 + length[s] * 2.0 ** -24
            assert (np.abs(out[a:b] - O) <= 2 * w * A + 2.0 ** -23 * np.abs(O) + 1e-30).all(), s
    assert_no_device_error()
