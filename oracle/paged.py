"""Plain float64 CPU oracle of the paged KV cache: plan, append, attention.

TEST INFRASTRUCTURE: only the tests and ``__graft_entry__.smoke()`` use this
module.  It shares no code with the CUDA library.

Definitions.  A request s has ctx tokens in its pages and brings new rows; its
pages become ceil((ctx + new) / page).  Missing pages are taken from the free
ring in request order, surplus ones go back behind the ring's tail.  Row i of
a request with n rows and kv keys has position kv - n + i and sees the keys
max(0, p - window + 1) .. p; its output is softmax attention over exactly
these, 0 when there are none.

Pins (``tests/test_paged_oracle.py``): attention over one full-length request
equals torch's causal scaled_dot_product_attention; the plan's ring and table
hold every page exactly once after any sequence of steps, and a request's
slots are distinct and inside its own pages.
"""

import numpy as np


def paged_plan(ctx, new, held, table, ring, state, tokens, page):
    """Returns (q_start, kv_len, slots, held, table, ring, state) as new int64 arrays."""
    held, table, ring = (np.array(a, dtype=np.int64) for a in (held, table, ring))
    S, width = table.shape
    P = len(ring)
    head, count = int(state[0]), int(state[1])
    q_start = np.zeros(S + 1, dtype=np.int64)
    kv_len = np.zeros(S, dtype=np.int64)
    slots = np.full(tokens, -1, dtype=np.int64)
    asked = taken = 0
    returned = []
    row = 0
    for s in range(S):
        c, n = int(ctx[s]), int(new[s])
        begin, row = row, row + max(0, n)
        q_start[s + 1] = min(row, tokens)
        want = -((-(c + n)) // page)
        if c < 0 or n < 0 or want > width or (n > 0 and row > tokens):
            continue
        if want > held[s]:
            asked += want - int(held[s])
            if asked > count:
                continue
            while held[s] < want:
                table[s, held[s]] = ring[(head + taken) % P]
                taken += 1
                held[s] += 1
        for cell in range(want, int(held[s])):
            returned.append(table[s, cell])
            table[s, cell] = -1
        held[s] = want
        kv_len[s] = c + n
        for i in range(n):
            slots[begin + i] = table[s, (c + i) // page] * page + (c + i) % page
    for k, pid in enumerate(returned):
        ring[(head + count + k) % P] = pid
    return (q_start, kv_len, slots, held, table, ring,
            np.array([(head + taken) % P, count - taken + len(returned)], dtype=np.int64))


def paged_append(K, V, slots, Kc, Vc):
    """Kc, Vc [P,Hkv,page,d] with the rows K, V [T,Hkv,d] written to their slots, as new arrays."""
    Kc, Vc = np.array(Kc), np.array(Vc)
    P, _, page, _ = Kc.shape
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if 0 <= slot < P * page:
            Kc[slot // page, :, slot % page] = K[t]
            Vc[slot // page, :, slot % page] = V[t]
    return Kc, Vc


def paged_attention(Q, Kc, Vc, table, q_start, kv_len, scale, window=0):
    """float64 (O, A, seen): O [T,Hq,d] (rows of no request: NaN), A = Σ p |v|
    / Σ p elementwise (what a relative error of the weights p can move), and
    the number of visible keys of each row (-1: a row of no request)."""
    Q = np.asarray(Q, dtype=np.float64)
    T, Hq, d = Q.shape
    P, Hkv, page, _ = Kc.shape
    g = Hq // Hkv
    O = np.full((T, Hq, d), np.nan)
    A = np.zeros((T, Hq, d))
    seen = np.full(T, -1, dtype=np.int64)
    for s in range(len(kv_len)):
        a, b, kv = int(q_start[s]), int(q_start[s + 1]), int(kv_len[s])
        n = b - a
        if n <= 0:
            continue
        first = max(0, kv - n - window + 1) if window > 0 else 0
        cells = np.arange(first // page, -(-kv // page))
        base = first // page * page
        ids = np.asarray(table[s])[cells].astype(np.int64)
        k = np.asarray(Kc[ids], dtype=np.float64).transpose(1, 0, 2, 3).reshape(Hkv, -1, d)
        v = np.asarray(Vc[ids], dtype=np.float64).transpose(1, 0, 2, 3).reshape(Hkv, -1, d)
        for i in range(n):
            p = kv - n + i
            lo = max(0, p - window + 1) if window > 0 else 0
            seen[a + i] = max(0, p + 1 - lo)
            if p < 0:
                O[a + i] = 0.0
                continue
            kk, vv = k[:, lo - base:p + 1 - base], v[:, lo - base:p + 1 - base]
            z = scale * np.einsum("hgd,hkd->hgk", Q[a + i].reshape(Hkv, g, d), kk)
            e = np.exp(z - z.max(axis=-1, keepdims=True))
            e /= e.sum(axis=-1, keepdims=True)
            O[a + i] = np.einsum("hgk,hkd->hgd", e, vv).reshape(Hq, d)
            A[a + i] = np.einsum("hgk,hkd->hgd", e, np.abs(vv)).reshape(Hq, d)
    return O, A, seen
