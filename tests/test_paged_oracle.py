"""Pins of the paged cache's oracle, and the C ABI's refusals (no GPU needed)."""

import numpy as np
import pytest
import torch

import oracle
from block_sparse_approximate_b200 import binding as bd

FAKE = 0x10000  # never dereferenced: validation fails (or returns) before any launch


def test_attention_of_one_whole_request_is_causal_attention():
    r = np.random.RandomState(0)
    n, Hq, Hkv, d, page = 37, 6, 2, 16, 8
    Q, K, V = r.randn(n, Hq, d), r.randn(n, Hkv, d), r.randn(n, Hkv, d)
    ids = r.permutation(9)[:5]
    Kc, Vc = np.full((9, Hkv, page, d), np.nan), np.full((9, Hkv, page, d), np.nan)
    table = np.full((1, 6), -1)
    table[0, :5] = ids
    slots = [ids[t // page] * page + t % page for t in range(n)]
    Kc, Vc = oracle.paged_append(K, V, slots, Kc, Vc)
    O, A, seen = oracle.paged_attention(Q, Kc, Vc, table, [0, n], [n], d ** -0.5)
    t = lambda x: torch.from_numpy(x).transpose(0, 1).repeat_interleave(Hq // x.shape[1], 0)  # noqa: E731
    ref = torch.nn.functional.scaled_dot_product_attention(t(Q), t(K), t(V), is_causal=True).transpose(0, 1).numpy()
    np.testing.assert_allclose(O, ref, rtol=1e-12, atol=1e-13)
    assert (np.abs(O) <= A + 1e-12).all() and seen.tolist() == list(range(1, n + 1))
    # a chunk of the last rows gives the whole prompt's last rows
    Oc, _, _ = oracle.paged_attention(Q[30:], Kc, Vc, table, [0, 7], [n], d ** -0.5)
    np.testing.assert_allclose(Oc, ref[30:], rtol=1e-12, atol=1e-13)
    # a window as wide as the request changes nothing; width 1 gives the value itself
    Ow, _, _ = oracle.paged_attention(Q, Kc, Vc, table, [0, n], [n], d ** -0.5, window=n)
    np.testing.assert_array_equal(Ow, O)
    O1, _, _ = oracle.paged_attention(Q, Kc, Vc, table, [0, n], [n], d ** -0.5, window=1)
    np.testing.assert_allclose(O1, V.repeat(Hq // Hkv, axis=1), rtol=1e-12)


@pytest.mark.parametrize("seed", range(4))
def test_plan_keeps_every_page_once(seed):
    r = np.random.RandomState(seed)
    S, width, P, page, tokens = 9, 7, 30, 16, 120
    held, table = np.zeros(S, int), np.full((S, width), -1)
    ring, state = r.permutation(P), np.array([0, P])
    length = np.zeros(S, int)
    refused = 0
    for step in range(40):
        ctx = np.where(r.rand(S) < 0.2, length // 2, length)     # some are shortened, some end
        ctx = np.where(r.rand(S) < 0.1, 0, ctx)
        new = r.randint(0, 40, S) * (r.rand(S) < 0.6)
        q, kv, slots, held, table, ring, state = oracle.paged_plan(ctx, new, held, table, ring, state, tokens, page)
        free = ring[(state[0] + np.arange(state[1])) % P]
        owned = table[np.arange(width)[None, :] < held[:, None]]
        assert sorted(np.concatenate([free, owned]).tolist()) == list(range(P))
        assert (table[np.arange(width)[None, :] >= held[:, None]] == -1).all()
        live = slots[slots >= 0]
        assert len(set(live.tolist())) == len(live)
        for s in range(S):
            mine = slots[q[s]:q[s + 1]]
            if kv[s] == ctx[s] + new[s]:
                assert held[s] == -(-kv[s] // page)
                length[s] = kv[s]
                if len(mine) == new[s]:
                    assert set((mine // page).tolist()) <= set(table[s, :held[s]].tolist())
            else:
                refused += 1
                assert (mine == -1).all()
    assert refused > 0


def test_binding_mirrors_paged_shape():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    txt = open(os.path.join(root, "include", "sparseattn.h")).read()
    body = re.search(r"typedef struct \{([^{}]*)\} sa_paged_shape;", txt).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for line in re.findall(r"int32_t ([^;]*);", body) for n in re.split(r",\s*", line)]
    assert names == [n for n, _ in bd.PagedShape._fields_]


def test_plan_refusals(lib):
    f = lib.sa_paged_plan

    def call(sh, args=(FAKE,) * 2, rest=(FAKE,) * 7):
        return f(*args, sh, *rest, None)
    ok = dict(S=4, T=8, Hq=1, Hkv=1, d=64, page=16, P=32, max_pages=4)
    sh = lambda **kw: bd.PagedShape(**{**ok, **kw})  # noqa: E731
    assert call(sh(S=-1)) == bd.SA_ERR_INVALID_ARG
    assert call(sh(S=0)) == bd.SA_ERR_INVALID_ARG
    assert call(sh(P=0)) == bd.SA_ERR_INVALID_ARG
    assert call(sh(max_pages=0)) == bd.SA_ERR_INVALID_ARG
    assert call(sh(page=48)) == bd.SA_ERR_UNSUPPORTED
    assert call(sh(page=256)) == bd.SA_ERR_UNSUPPORTED
    assert call(sh(S=4097)) == bd.SA_ERR_UNSUPPORTED
    assert call(sh(max_pages=(1 << 26) + 1)) == bd.SA_ERR_UNSUPPORTED
    assert call(sh(), args=(None, FAKE)) == bd.SA_ERR_INVALID_ARG
    for k in range(7):
        rest = [FAKE] * 7
        rest[k] = None
        assert call(sh(), rest=rest) == bd.SA_ERR_INVALID_ARG, k
        rest[k] = FAKE + 2
        assert call(sh(), rest=rest) == bd.SA_ERR_ALIGNMENT, k
    assert call(sh(), rest=[FAKE] * 6 + [FAKE + 4]) == bd.SA_ERR_ALIGNMENT    # slots are 8 bytes wide


def test_append_refusals(lib):
    f = lib.sa_paged_append
    ok = dict(S=0, T=8, Hq=4, Hkv=4, d=64, page=16, P=32, max_pages=0)

    def call(kw={}, K=FAKE, V=FAKE, ks=256, vs=256, dtype=1, slots=FAKE, Kc=FAKE, Vc=FAKE):
        return f(K, V, ks, vs, dtype, bd.PagedShape(**{**ok, **kw}), slots, Kc, Vc, None)
    assert call(dict(T=0)) == bd.SA_OK
    assert call(dict(P=0)) == bd.SA_OK
    assert call(dict(T=-1)) == bd.SA_ERR_INVALID_ARG
    assert call(dict(Hkv=0)) == bd.SA_ERR_INVALID_ARG
    assert call(dict(d=96)) == bd.SA_ERR_UNSUPPORTED
    assert call(dict(page=8)) == bd.SA_ERR_UNSUPPORTED
    assert call(dtype=2) == bd.SA_ERR_UNSUPPORTED
    assert call(K=None) == call(V=None) == call(slots=None) == call(Kc=None) == call(Vc=None) == bd.SA_ERR_INVALID_ARG
    assert call(ks=255) == call(vs=128) == bd.SA_ERR_INVALID_ARG      # rows would overlap
    assert call(ks=260) == call(K=FAKE + 8) == call(Vc=FAKE + 4) == call(slots=FAKE + 4) == bd.SA_ERR_ALIGNMENT
    assert call(dict(P=1 << 30)) == bd.SA_ERR_UNSUPPORTED


def test_attention_refusals(lib):
    f = lib.sa_paged_attn_fwd
    ok = dict(S=4, T=8, Hq=8, Hkv=4, d=128, page=16, P=32, max_pages=4)

    def call(kw={}, Q=FAKE, qs=1024, Kc=FAKE, Vc=FAKE, dtype=1, q_start=FAKE, kv=FAKE, tab=FAKE, window=0, O=FAKE,
             ws=FAKE, n=None, scale=0.1):
        sh = bd.PagedShape(**{**ok, **kw})
        n = lib.sa_paged_attn_workspace_size(sh) if n is None else n
        return f(Q, qs, Kc, Vc, dtype, sh, q_start, kv, tab, window, scale, O, ws, n, None)
    assert call(dict(T=0)) == bd.SA_OK and call(dict(S=0)) == bd.SA_OK
    assert call(dict(Hq=6)) == bd.SA_ERR_INVALID_ARG
    assert call(dict(Hq=0)) == bd.SA_ERR_INVALID_ARG
    assert call(dict(d=80)) == bd.SA_ERR_UNSUPPORTED
    assert call(dict(page=24)) == bd.SA_ERR_UNSUPPORTED
    assert call(dict(S=5000)) == bd.SA_ERR_UNSUPPORTED
    assert call(dict(T=1 << 28)) == bd.SA_ERR_UNSUPPORTED             # T * Hq rows
    assert call(dtype=7) == bd.SA_ERR_UNSUPPORTED
    assert call(dict(Hq=4 * 129), qs=1 << 20) == bd.SA_ERR_UNSUPPORTED   # query heads per KV head, bf16
    assert call(window=-1) == bd.SA_ERR_INVALID_ARG
    for scale in (0.0, -0.1, float("inf"), float("nan")):
        assert call(scale=scale) == bd.SA_ERR_INVALID_ARG, scale
    for name in ("Q", "Kc", "Vc", "q_start", "kv", "tab", "O"):
        assert call(**{name: None}) == bd.SA_ERR_INVALID_ARG, name
    for name in ("Q", "Kc", "Vc", "O"):
        assert call(**{name: FAKE + 8}) == bd.SA_ERR_ALIGNMENT, name
    for name in ("q_start", "kv", "tab"):
        assert call(**{name: FAKE + 1}) == bd.SA_ERR_ALIGNMENT, name
    assert call(qs=1000) == bd.SA_ERR_INVALID_ARG and call(qs=1028) == bd.SA_ERR_ALIGNMENT
    assert call(ws=None) == bd.SA_ERR_WORKSPACE
    assert call(n=lib.sa_paged_attn_workspace_size(bd.PagedShape(**ok)) - 1) == bd.SA_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == bd.SA_ERR_ALIGNMENT
    assert "workspace" in lib.sa_last_error().decode()


def test_workspace_size():
    size = bd.paged_attn_workspace_size
    assert size(4, 8, 6, 4, 128, 16, 32, 4) == 0                      # Hq % Hkv
    assert 0 < size(1, 1, 32, 8, 128, 64, 100, 100) < 3 << 20
    assert size(64, 1 << 16, 32, 8, 128, 64, 100, 100) <= 39 << 20    # the documented bound


def test_binding_refuses_host_tensors_and_wrong_layouts():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        bd.paged_plan(i(2), i(2), i(2), i(2, 3), i(8), i(2), 4, 16)
    with pytest.raises(ValueError, match="table"):
        bd.paged_plan(i(2), i(2), i(2), i(3, 3), i(8), i(2), 4, 16)
    x = torch.zeros(4, 2, 64)
    c = torch.zeros(3, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        bd.paged_append(x, x, torch.zeros(4, dtype=torch.int64), c, c)
    with pytest.raises(ValueError, match=r"\[T,Hkv,d\]"):
        bd.paged_append(x, x[:3], torch.zeros(4, dtype=torch.int64), c, c)
    with pytest.raises(ValueError, match="contiguous"):
        bd._paged_rows(x.transpose(1, 2), "x")
    assert bd._paged_rows(torch.zeros(4, 9, 64)[:, 2:5], "x") == 9 * 64
    with pytest.raises(ValueError, match="q_start"):
        bd.paged_attn_fwd(x, c, c, i(2, 3), i(2), i(2), 1.0)
    for window in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="window"):
            bd.paged_attn_fwd(x, c, c, i(2, 3), i(3), i(2), 1.0, window=window)


def test_plan_refuses_arrays_that_overlap(lib):
    # the lengths that a call writes are not those that it reads: every pair of arrays of which one is written
    S, T, P, width = 8, 32, 64, 4
    sizes = dict(ctx=4 * S, new=4 * S, held=4 * S, table=4 * S * width, ring=4 * P, state=8, q_start=4 * (S + 1),
                 kv_len=4 * S, slots=8 * T)
    sh = bd.PagedShape(S=S, T=T, Hq=1, Hkv=1, d=64, page=16, P=P, max_pages=width)
    names = list(sizes)
    for a in names:
        for b in names:
            if a == b or {a, b} == {"ctx", "new"}:
                continue
            at = {n: FAKE + 0x1000 * k for k, n in enumerate(names)}
            for shift in (0, (sizes[a] - 1) // 8 * 8 if b == "slots" else sizes[a] - 4):
                at[b] = at[a] + shift              # b begins with a, or within its last elements
                status = lib.sa_paged_plan(at["ctx"], at["new"], sh, *(at[n] for n in names[2:]), None)
                assert status == bd.SA_ERR_INVALID_ARG, (a, b, shift)
                assert "overlap" in lib.sa_last_error().decode(), (a, b)


def test_attention_refuses_a_scale_that_overflows_in_base_2(lib):
    # (without a workspace, so that no call gets as far as a launch)
    sh = bd.PagedShape(S=4, T=8, Hq=8, Hkv=4, d=128, page=16, P=32, max_pages=4)
    for dtype in (0, 1):
        for scale, status in ((2.3e38, bd.SA_ERR_WORKSPACE), (2.4e38, bd.SA_ERR_INVALID_ARG),
                              (3.4e38, bd.SA_ERR_INVALID_ARG)):
            assert lib.sa_paged_attn_fwd(FAKE, 1024, FAKE, FAKE, dtype, sh, FAKE, FAKE, FAKE, 0, scale, FAKE, None, 0,
                                         None) == status, scale


def test_binding_refuses_sizes_beyond_32_bits():
    # sizes that the C struct's fields would cut: a view of one element stands for the large tensor
    big = (1 << 32) + 4
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    many = lambda t, *s: t[:1].expand(*s)  # noqa: E731
    x, c = torch.zeros(4, 2, 64), torch.zeros(3, 2, 16, 64)
    slots = torch.zeros(1, dtype=torch.int64)
    for call in (lambda: bd.paged_plan(i(2), i(2), i(2), i(2, 3), i(8), i(2), big, 16, slots=many(slots, big)),
                 lambda: bd.paged_plan(i(2), i(2), i(2), i(2, 3), i(8), i(2), 4, (1 << 32) + 16),
                 lambda: bd.paged_plan(i(2), i(2), i(2), i(2, 3), many(i(1), big), i(2), 4, 16),
                 lambda: bd.paged_plan(i(2), i(2), i(2), many(i(1, 1), 2, big), i(8), i(2), 4, 16),
                 lambda: bd.paged_append(many(x, big, 2, 64), many(x, big, 2, 64), many(slots, big), c, c),
                 lambda: bd.paged_attn_fwd(many(x, big, 2, 64), c, c, i(2, 3), i(3), i(2), 1.0),
                 lambda: bd.paged_attn_fwd(x, c, c, many(i(1, 1), 2, big), i(3), i(2), 1.0),
                 lambda: bd.paged_attn_workspace_size(4, big, 8, 4, 128, 16, 32, 4)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
