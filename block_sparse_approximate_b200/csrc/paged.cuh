// Paged KV cache: what the plan, the append and the attention kernels share.
//
// The cache is a pool of P pages, [P][Hkv][page][d] for K and for V; request s
// owns the pages table[s][0 .. ceil(len / page)).  The rows of all requests'
// new tokens are packed one behind the other; request s has the rows
// q_start[s] .. q_start[s+1].
//
// Work division of the attention.  The query rows of one (request, KV head)
// are numbered token-major, r = token * group + (query head within the
// group), so that a tile of consecutive rows shares its keys.  An item is such
// a tile (Params::bm rows); its keys are the span its rows can see, walked in
// tiles of BN keys.  The items of all requests are laid on one line, each as long as its
// cost, and the line is cut into equal shares, one per CTA: a share starts
// and ends anywhere, also inside an item.  A CTA that holds all key tiles of
// an item writes its output; otherwise each CTA writes a partial state
// (unnormalised sums, row maxima and sums) and paged_combine_kernel merges
// them in key order.  Every CTA derives the line from q_start and kv_len by
// itself, so no lengths are read by the host and a captured graph follows
// them.
#pragma once

#include "common.cuh"

namespace sa {
namespace paged {

constexpr int kMaxRequests = 4096;

// Division of 0 <= n < 2^31 by a divisor that the host knows, as a
// multiplication (the method with a rounded-up reciprocal of Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, mul, shift;
  explicit FastDiv(uint32_t divisor) : d(divisor), mul(1), shift(0) {
    while (((uint64_t)1 << shift) < d) ++shift;
    mul = (uint32_t)(((((uint64_t)1 << shift) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};

struct Params {
  const int32_t* q_start;   // [S+1]
  const int32_t* kv_len;    // [S]
  const int32_t* table;     // [S][max_pages]
  int S, T, Hq, Hkv, group, page_shift, P, max_pages;
  int window;               // 0: none; else below max_pages * page
  int bm, half;             // rows of an item; up to `half` rows are a half item
  FastDiv by_group, by_heads, by_bm;   // of group, Hkv, bm

  // Row r of (the request whose rows start at row0, KV head h) as a row of the
  // packed arrays: token * Hq + query head.
  __device__ __forceinline__ int64_t query_row(int row0, int h, int r) const {
    const int tok = by_group.div(r);
    return (int64_t)(row0 + tok) * Hq + h * group + r - tok * group;
  }
};

// Quotient of non-negative numbers; 32-bit division where both fit (the line is
// cut before the first load, where a 64-bit one's hundred instructions show).
__host__ __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line in equal shares: share c starts at c * each + min(c, rest).
struct Shares {
  int64_t each;
  int32_t rest, parts;
  __device__ __forceinline__ int64_t start(int c) const { return each * c + min(c, rest); }
};

// Partial states in the workspace: slot 2c holds the first item portion of
// CTA c, slot 2c + 1 the last one.  desc[c] describes the split item whose
// first key tile lies with CTA c.
struct Desc {
  int64_t start;            // the item's place on the line
  Shares shares;
  int32_t valid, slot, unit, nt, row0, r0, rv, h;
};

struct Workspace {
  Desc* desc;               // [ctas]
  float* o;                 // [2 ctas][d / 4][rows_cap][4]: lanes of a warp hold rows, so stores coalesce
  float* ml;                // [2 ctas][rows_cap][2]: running maximum (log2 units), sum
  int rows_cap, ctas;
  template <int D>
  __device__ __forceinline__ float4* chunk(int slot, int k) const {   // columns 4k .. 4k + 3 of a slot's rows
    return reinterpret_cast<float4*>(o) + ((size_t)slot * (D / 4) + k) * rows_cap;
  }
  __device__ __forceinline__ float2* state(int slot) const {
    return reinterpret_cast<float2*>(ml) + (size_t)slot * rows_cap;
  }
};

// ---- the items of a request
struct Request {
  int row0, n, len;
};

__device__ __forceinline__ Request load_request(const Params& p, int s) {
  // lengths come from device memory: bounded here, so that no table or row
  // access can leave its array whatever they hold
  const int a = min(max(p.q_start[s], 0), p.T);
  const int b = min(max(p.q_start[s + 1], a), p.T);
  return {a, b - a, min(max(p.kv_len[s], 0), p.max_pages << p.page_shift)};
}

struct Item {
  int r0, rv;        // first row within the request, number of rows
  int p0;            // position of the request's first new token (negative: rows before it see no key)
  int lo, hi;        // keys that some row sees
  int t0, nt;        // their tiles
  int unit;          // cost of a tile
};

// A tiling has BN keys a tile; a tile costs kUnit, of a half item kUnitHalf;
// kOver is an item's own cost in the same unit; a share holds at least
// kMinShare.
template <class TL>
__device__ __forceinline__ Item item_of(const Request& q, const Params& p, int j) {
  Item it;
  it.r0 = j * p.bm;
  it.rv = min(p.bm, q.n * p.group - it.r0);
  it.p0 = q.len - q.n;
  const int p_lo = it.p0 + p.by_group.div(it.r0), p_hi = it.p0 + p.by_group.div(it.r0 + it.rv - 1);
  it.lo = p.window > 0 ? max(0, p_lo - p.window + 1) : 0;
  it.hi = max(0, p_hi + 1);
  it.t0 = it.lo / TL::BN;
  it.nt = it.hi > it.lo ? (it.hi + TL::BN - 1) / TL::BN - it.t0 : 0;
  it.unit = it.rv <= p.half ? TL::kUnitHalf : TL::kUnit;
  return it;
}
template <class TL>
__device__ __forceinline__ int item_cost(const Item& it) { return it.nt * it.unit + TL::kOver; }
__device__ __forceinline__ int items_of(const Request& q, const Params& p) {
  return p.by_bm.div(q.n * p.group + p.bm - 1);
}

// Key tiles of an item that lie before the place x >= 0 of its own stretch.
__device__ __forceinline__ int tiles_before(int64_t x, int nt, int unit) {
  return x >= (int64_t)nt * unit ? nt : (int)((uint32_t)x / (uint32_t)unit);
}

template <class TL>
__device__ __forceinline__ Shares cut_line(int64_t total, int ctas) {
  const int64_t n = total / TL::kMinShare;
  Shares s;
  s.parts = (int)(n < 1 ? 1 : (n < ctas ? n : ctas));
  s.each = quotient(total, s.parts);
  s.rest = (int)(total - s.each * s.parts);
  return s;
}

// Lays the line: pre[s] = the end of request s on it (all threads of a block
// of kThreads; pre and tot in shared memory).  Returns the line's length.
template <class TL, int kThreads>
__device__ int64_t lay_line(const Params& p, int64_t* pre, int64_t* tot) {
  constexpr int NW = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // each request's cost; neighbours go to different warps, since requests of
  // many items are taken by a whole warp, a lane an item
  for (int base = 0; base < p.S; base += kThreads) {
    const int s = base + lane * NW + warp;
    Request q{0, 0, 0};
    if (s < p.S) q = load_request(p, s);
    const int nj = items_of(q, p);
    int64_t c = 0;
    if (nj <= 2)
      for (int j = 0; j < nj; ++j) c += item_cost<TL>(item_of<TL>(q, p, j));
    for (unsigned big = __ballot_sync(0xffffffffu, nj > 2); big; big &= big - 1) {
      const int src = __ffs(big) - 1;
      const Request b{0, __shfl_sync(0xffffffffu, q.n, src), __shfl_sync(0xffffffffu, q.len, src)};
      const int nb = items_of(b, p);
      int64_t sum = 0;
      for (int j = lane; j < nb; j += 32) sum += item_cost<TL>(item_of<TL>(b, p, j));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == src) c = sum;
    }
    if (s < p.S) pre[s] = c * p.Hkv;
  }
  __syncthreads();
  int64_t run = 0;
  for (int base = 0; base < p.S; base += kThreads) {
    const int s = base + threadIdx.x;
    int64_t c = s < p.S ? pre[s] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += y;
    }
    if (lane == 31) tot[warp] = c;
    __syncthreads();
    int64_t off = run, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) off += tot[w];
      all += tot[w];
    }
    if (s < p.S) pre[s] = off + c;
    run += all;
    __syncthreads();
  }
  return run;
}

// Who holds place w of the line: {request, its start, its end} (all threads;
// out in shared memory, to be read behind a barrier).
template <int kThreads>
__device__ __forceinline__ void find_request(const Params& p, const int64_t* pre, int64_t w, int64_t* out) {
  for (int s = threadIdx.x; s < p.S; s += kThreads) {
    const int64_t a = s ? pre[s - 1] : 0, b = pre[s];
    if (a <= w && w < b) {
      out[0] = s;
      out[1] = a;
      out[2] = b;
    }
  }
}

// One warp walks the items of a share.
template <class TL>
struct Walker {
  Request q;
  Item it;
  int s, h, j, nj, cost;
  int64_t start;

  __device__ __forceinline__ void set_item(const Params& p) {
    it = item_of<TL>(q, p, j);
    cost = item_cost<TL>(it);
  }
  // The item that holds place w of the line, 0 <= w < its length; `at`: the
  // request that does (find_request).
  __device__ void find(const Params& p, int at_request, int64_t first, int64_t end, int64_t w) {
    const int lane = threadIdx.x & 31;
    s = at_request;
    q = load_request(p, s);
    const int64_t len = end - first;
    const int64_t head = len >> 31 ? len / p.Hkv : (int64_t)p.by_heads.div((int)len);
    h = p.Hkv == 1 ? 0 : (int)quotient(w - first, head);
    int64_t at = first + h * head;
    nj = items_of(q, p);
    for (j = 0;; j += 32) {
      const int mine = j + lane < nj ? item_cost<TL>(item_of<TL>(q, p, j + lane)) : 0;
      int64_t end = mine;
      if (nj > 1) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += y;
        }
      }
      const unsigned past = __ballot_sync(0xffffffffu, at + end > w);
      if (past) {
        const int src = __ffs(past) - 1;
        start = at + __shfl_sync(0xffffffffu, end - mine, src);
        j += src;
        break;
      }
      at += __shfl_sync(0xffffffffu, end, 31);
      if (j + 32 >= nj) {   // not reached while the line is the sum of its items
        j = nj - 1;
        start = at;
        break;
      }
    }
    set_item(p);
  }
  __device__ __forceinline__ bool next(const Params& p) {
    start += cost;
    if (++j == nj) {
      j = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++s >= p.S) return false;
          q = load_request(p, s);
        } while (q.n == 0);
        nj = items_of(q, p);
      }
    }
    set_item(p);
    return true;
  }
  // Key tiles [ta, tb) of the item in the share [w0, w1); false: none here.
  __device__ __forceinline__ bool portion(int64_t w0, int64_t w1, int& ta, int& tb) const {
    ta = w0 > start ? tiles_before(w0 - start, it.nt, it.unit) : 0;
    tb = tiles_before(w1 - start, it.nt, it.unit);
    return it.nt == 0 ? start >= w0 : ta < tb;
  }
};

// ---- host side
struct Limits {
  // One or two CTAs on each of B200's 148 SMs (right on any other number, where
  // some CTAs would wait for a place)
  static constexpr int kCtas = 148;        // of the tensor-core kernel: one per SM
  static constexpr int kCtasSimt = 296;    // of the CUDA-core kernel: two per SM
};

}  // namespace paged

// The bf16 attention on the tensor cores (paged_attn_tc.cu).
sa_status paged_attn_tc(const void* Q, int64_t q_stride, const void* Kc, const void* Vc, const sa_paged_shape& s,
                        const paged::Params& p, float scale, void* O, const paged::Workspace& ws,
                        cudaStream_t stream);

}  // namespace sa
