// The plan of a serving step on a paged KV cache (block tables and slot maps
// from the requests' lengths) and the write of the new K and V rows.
#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"

namespace sa {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------- plan
// Per request s: want = ceil((ctx + new) / page) pages, need = want - held.
// need > 0 takes pages from the ring's head in request order, need < 0 hands
// the last pages back behind the ring's tail.  Three prefix sums over the
// requests (rows, pages asked for, pages handed back) fix every place; then
// tokens, taken pages and returned pages are independent and each finds its
// request by binary search in the prefix sums, so the work is even however
// the lengths are spread.
//
// A request is refused (kv_len 0, its slots -1, its pages and table row as
// they were) when its lengths are negative, exceed the table row, when its
// rows exceed T, or when the pages asked for up to and including it exceed
// the free ones.  Pages handed back in a step can be taken from the next one
// on: what is read (the ring's free span) and what is written (behind it)
// are then disjoint and the CTAs need no order between them.
//
// One cluster of up to 8 CTAs, each with the prefix sums in its own shared
// memory (S values each, recomputed: cheaper than handing them over); the
// state that every CTA reads (held, free_state) is rewritten by one CTA
// behind a cluster barrier.  Latency-bound: a launch, two dependent loads, a
// block scan.
constexpr int kPlanMaxCluster = 8;

struct Sum3 {
  int64_t rows, ask, give;
};

__device__ __forceinline__ int first_above(const int* end, int n, int x) {
  int a = 0, b = n - 1;
  while (a < b) {
    const int m = (a + b) >> 1;
    if (end[m] > x) b = m;
    else a = m + 1;
  }
  return a;
}

__global__ void __launch_bounds__(1024)
paged_plan_kernel(const int32_t* __restrict__ ctx_len, const int32_t* __restrict__ new_len, int S, int T,
                  int page_shift, int P, int max_pages, int32_t* held, int32_t* table, int32_t* ring,
                  int32_t* free_state, int32_t* __restrict__ q_start, int32_t* __restrict__ kv_len,
                  int64_t* __restrict__ slots) {
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), nctas = (int)cluster.num_blocks();
  extern __shared__ int smem_plan[];
  int* q_end = smem_plan;         // [S] rows up to and including s, at most T
  int* ask_end = q_end + S;       // [S] pages asked for; exact where the request is served
  int* give_end = ask_end + S;    // [S] pages handed back
  int* owned = give_end + S;      // [S] pages held on entry; -1 - that for a refused request
  int* shift_s = owned + S;       // [S] position of a row within its request, less the row
  __shared__ Sum3 tot[32];
  __shared__ int taken_all;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const int page = 1 << page_shift;
  int head = free_state[0] % P;
  if (head < 0) head += P;
  const int count = min(max(free_state[1], 0), P);
  if (tid == 0) taken_all = 0;
  Sum3 run{0, 0, 0};
  for (int base = 0; base < S; base += nthr) {
    const int s = base + tid;
    int64_t ctx = 0, nw = 0;
    int old = 0;
    if (s < S) {
      ctx = ctx_len[s];
      nw = new_len[s];
      old = min(max(held[s], 0), max_pages);
    }
    const int64_t want = (ctx + nw + page - 1) >> page_shift;
    const bool fits = ctx >= 0 && nw >= 0 && want <= max_pages;
    // rows first: a request with rows behind T neither asks nor hands back
    Sum3 x{nw > 0 ? nw : 0, 0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x.rows, o);
      if (lane >= o) x.rows += y;
    }
    if (lane == 31) tot[warp].rows = x.rows;
    __syncthreads();
    int64_t off = run.rows, all = 0;
    for (int w = 0; w < nthr / 32; ++w) {
      if (w < warp) off += tot[w].rows;
      all += tot[w].rows;
    }
    const int64_t rows_incl = off + x.rows;
    run.rows += all;
    const bool fine = s < S && fits && (nw == 0 || rows_incl <= T);
    x.ask = fine && want > old ? want - old : 0;
    x.give = fine && want < old ? old - want : 0;
    const bool asks = x.ask > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t ya = __shfl_up_sync(0xffffffffu, x.ask, o), yg = __shfl_up_sync(0xffffffffu, x.give, o);
      if (lane >= o) {
        x.ask += ya;
        x.give += yg;
      }
    }
    if (lane == 31) {
      tot[warp].ask = x.ask;
      tot[warp].give = x.give;
    }
    __syncthreads();
    int64_t oa = run.ask, og = run.give, aa = 0, ag = 0;
    for (int w = 0; w < nthr / 32; ++w) {
      if (w < warp) {
        oa += tot[w].ask;
        og += tot[w].give;
      }
      aa += tot[w].ask;
      ag += tot[w].give;
    }
    if (s < S) {
      const int64_t ask_incl = oa + x.ask;
      const bool ok = fine && (!asks || ask_incl <= count);
      q_end[s] = (int)min(rows_incl, (int64_t)T);
      ask_end[s] = (int)min(ask_incl, (int64_t)0x7fffffff);
      give_end[s] = (int)(og + x.give);
      owned[s] = ok ? old : -1 - old;
      shift_s[s] = ok ? (int)(ctx + (nw > 0 ? nw : 0) - rows_incl) : 0;
      if (ok && asks) atomicMax(&taken_all, (int)ask_incl);
      if (rank == 0) {
        if (s == 0) q_start[0] = 0;
        q_start[s + 1] = (int)min(rows_incl, (int64_t)T);
        kv_len[s] = ok ? (int)(ctx + nw) : 0;
      }
    }
    run.ask += aa;
    run.give += ag;
    __syncthreads();
  }
  const int rows = S ? q_end[S - 1] : 0;
  const int taken = taken_all, given = (int)run.give;
  const int first = rank * nthr + tid, step = nctas * nthr;
  // (k stays below 2 P unless the state contradicts itself)
  auto ring_at = [&](int64_t k) {
    const int64_t x = head + k;
    return (int)(x < P ? x : x < 2 * (int64_t)P ? x - P : x % P);
  };
  // slots of the new tokens; a page below `owned` stands in the table already,
  // the others are still to come from the ring.  Four rows at a time, so that
  // their searches and loads overlap (the search is a chain of shared-memory
  // reads, the page id a load from L2).
  for (int t0 = first; t0 < T; t0 += 4 * step) {
    const int32_t* at[4];
    int off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u * step;
      at[u] = nullptr;
      if (t >= rows) continue;
      const int s = first_above(q_end, S, t), old = owned[s];
      if (old < 0) continue;
      const int pos = t + shift_s[s], cell = pos >> page_shift;
      off[u] = pos & (page - 1);
      at[u] = cell < old ? table + (size_t)s * max_pages + cell
                         : ring + ring_at((int64_t)(s ? ask_end[s - 1] : 0) + cell - old);
    }
    int id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = at[u] ? *at[u] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (t0 + u * step < T)
        slots[t0 + u * step] = id[u] >= 0 && id[u] < P ? ((int64_t)id[u] << page_shift) + off[u] : -1;
  }
  for (int k = first; k < taken; k += step) {
    const int s = first_above(ask_end, S, k);
    const int cell = owned[s] + k - (s ? ask_end[s - 1] : 0);
    table[(size_t)s * max_pages + cell] = ring[ring_at(k)];
  }
  for (int k = first; k < given; k += step) {
    const int s = first_above(give_end, S, k);
    // the last of the pages that s hands back is its last one
    int32_t* cell = table + (size_t)s * max_pages + owned[s] - (give_end[s] - k);
    ring[ring_at((int64_t)count + k)] = *cell;
    *cell = -1;
  }
  // every CTA has read held and free_state
  if (nctas > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0) {
    for (int s = tid; s < S; s += nthr)
      if (owned[s] >= 0)
        held[s] = owned[s] + (ask_end[s] - (s ? ask_end[s - 1] : 0)) - (give_end[s] - (s ? give_end[s - 1] : 0));
    if (tid == 0) {
      free_state[0] = ring_at(taken);
      free_state[1] = min(count - taken + given, P);
    }
  }
}

// ---------------------------------------------------------------- append
// Kc[slot / page][h][slot % page][:] = K[t][h][:], V alike: a copy, bound by
// memory.  A block takes rows_per_block rows (about 1024 16-byte chunks); a
// thread keeps four chunks of K and four of V in flight.
constexpr int kAppendThreads = 256, kAppendUnroll = 4;

__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const uint4* __restrict__ K, const uint4* __restrict__ V, int64_t k_stride, int64_t v_stride,
                    const int64_t* __restrict__ slots, int T, int Hkv, int vec, int page_shift, int64_t slot_count,
                    int rows_per_block, uint4* __restrict__ Kc, uint4* __restrict__ Vc) {
  pdl_wait();
  pdl_trigger();
  const int row0 = blockIdx.x * rows_per_block;
  const uint32_t per_row = (uint32_t)(Hkv * vec);
  const uint32_t n = (uint32_t)min(rows_per_block, T - row0) * per_row;
  for (uint32_t base = threadIdx.x; base < n; base += kAppendThreads * kAppendUnroll) {
    uint4 a[kAppendUnroll], b[kAppendUnroll];
    int64_t dst[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
      const uint32_t x = base + u * kAppendThreads;
      dst[u] = -1;
      if (x >= n) continue;
      const uint32_t r = x / per_row, c = x % per_row;
      const int64_t slot = slots[row0 + r];
      if (slot < 0 || slot >= slot_count) continue;
      const uint32_t h = c / (uint32_t)vec, e = c % (uint32_t)vec;
      const int64_t page_id = slot >> page_shift;
      dst[u] = ((((page_id * Hkv + h) << page_shift) + (slot & ((1 << page_shift) - 1))) * vec) + e;
      a[u] = __ldg(K + (row0 + (int64_t)r) * k_stride + c);
      b[u] = __ldg(V + (row0 + (int64_t)r) * v_stride + c);
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u)
      if (dst[u] >= 0) {
        Kc[dst[u]] = a[u];
        Vc[dst[u]] = b[u];
      }
  }
}

}  // namespace

sa_status check_paged(const sa_paged_shape& s, const char* fn) {
  const std::string f(fn);
  if (s.S < 0 || s.T < 0 || s.P < 0 || s.max_pages < 0)
    return fail(SA_ERR_INVALID_ARG, f + ": negative size");
  if (s.page != 16 && s.page != 32 && s.page != 64 && s.page != 128)
    return fail(SA_ERR_UNSUPPORTED, f + ": page must be 16, 32, 64 or 128");
  if (s.S > paged::kMaxRequests) return fail(SA_ERR_UNSUPPORTED, f + ": at most 4096 requests");
  if ((int64_t)s.max_pages * s.page > (1 << 30))
    return fail(SA_ERR_UNSUPPORTED, f + ": max_pages * page must not exceed 2^30 tokens");
  if ((int64_t)s.S * s.max_pages > INT32_MAX || s.T > (1 << 30))
    return fail(SA_ERR_UNSUPPORTED, f + ": table or row count exceeds 32-bit indexing");
  return SA_OK;
}

sa_status check_paged_heads(const sa_paged_shape& s, sa_dtype dtype, const char* fn) {
  const std::string f(fn);
  sa_status r = check_paged(s, fn);
  if (r != SA_OK) return r;
  if (dtype != SA_FP32 && dtype != SA_BF16) return fail(SA_ERR_UNSUPPORTED, f + ": dtype must be SA_FP32 or SA_BF16");
  if (s.Hkv <= 0) return fail(SA_ERR_INVALID_ARG, f + ": Hkv must be positive");
  if (s.d != 64 && s.d != 128) return fail(SA_ERR_UNSUPPORTED, f + ": d must be 64 or 128");
  if ((int64_t)s.P * s.Hkv > INT32_MAX || (int64_t)s.T * s.Hkv > INT32_MAX)
    return fail(SA_ERR_UNSUPPORTED, f + ": pages or rows times heads exceed 32-bit indexing");
  return SA_OK;
}

}  // namespace sa

extern "C" sa_status sa_paged_plan(const int32_t* ctx_len, const int32_t* new_len, sa_paged_shape shape, int32_t* held,
                                   int32_t* table, int32_t* free_pages, int32_t* free_state, int32_t* q_start,
                                   int32_t* kv_len, int64_t* slots, void* stream) {
  using namespace sa;
  const char* fn = "sa_paged_plan";
  sa_status r = check_paged(shape, fn);
  if (r != SA_OK) return r;
  if (shape.S == 0) return fail(SA_ERR_INVALID_ARG, "sa_paged_plan: at least one request is required");
  if (shape.P == 0 || shape.max_pages == 0)
    return fail(SA_ERR_INVALID_ARG, "sa_paged_plan: P and max_pages must be positive");
  if (!ctx_len || !new_len || !held || !table || !free_pages || !free_state || !q_start || !kv_len ||
      (shape.T > 0 && !slots))
    return fail(SA_ERR_INVALID_ARG, "sa_paged_plan: every array is required");
  // element-sized accesses only, except that slots are 8 bytes wide
  const void* ptrs[] = {ctx_len, new_len, held, table, free_pages, free_state, q_start, kv_len};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u)
      return fail(SA_ERR_ALIGNMENT, "sa_paged_plan: 32-bit arrays must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(slots) & 7u)
    return fail(SA_ERR_ALIGNMENT, "sa_paged_plan: slots must be 8-byte aligned");
  // The call rewrites its state in place and reads the lengths from several
  // CTAs: an array that is written is no other's memory (kv_len as the next
  // step's ctx_len would be).
  const size_t n = (size_t)shape.S * 4;
  const struct {
    const char* name;
    const void* at;
    size_t bytes;
  } arrays[] = {{"slots", slots, (size_t)shape.T * 8},
                {"kv_len", kv_len, n},
                {"q_start", q_start, n + 4},
                {"free_state", free_state, 8},
                {"free_pages", free_pages, (size_t)shape.P * 4},
                {"table", table, n * shape.max_pages},
                {"held", held, n},
                {"new_len", new_len, n},
                {"ctx_len", ctx_len, n}};
  for (int a = 0; a < 7; ++a)
    for (int b = a + 1; b < 9; ++b) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(arrays[a].at), y = reinterpret_cast<uintptr_t>(arrays[b].at);
      if (x < y + arrays[b].bytes && y < x + arrays[a].bytes)
        return fail(SA_ERR_INVALID_ARG,
                    std::string("sa_paged_plan: ") + arrays[a].name + " and " + arrays[b].name + " overlap");
    }
  // One CTA up to 1024 rows and requests, from there a cluster of a power of
  // two up to 8; 512 threads each (8.4 us for 512 requests and 32615 rows,
  // with 1024 threads, whose scan has twice the warps, 9.4; 4 CTAs 11.4) and
  // 1024 where that saves a pass over the requests.
  const int work = std::max(shape.T, shape.S);
  const int threads = work <= 256 ? 256 : shape.S <= 512 ? 512 : 1024;
  int ctas = 1;
  while (ctas < kPlanMaxCluster && ctas * 1024 < work) ctas *= 2;
  // Static arrays count towards the 48 KB that a CTA has by default, so the
  // opt-in is taken well before the sums alone fill it; always to the same
  // size, since the attribute is shared by all threads that call.
  constexpr int kSums = 5 * sizeof(int), kMostSmem = paged::kMaxRequests * kSums;
  const size_t smem = (size_t)shape.S * kSums;
  if (smem > 40 * 1024 && cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMostSmem) != cudaSuccess)
    return launch_status("cudaFuncSetAttribute(paged_plan_kernel)");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;   // a lone CTA needs no cluster
  const int shift = 31 - __builtin_clz((unsigned)shape.page);
  cudaLaunchKernelEx(&cfg, paged_plan_kernel, ctx_len, new_len, (int)shape.S, (int)shape.T, shift, (int)shape.P,
                     (int)shape.max_pages, held, table, free_pages, free_state, q_start, kv_len, slots);
  return launch_status("paged_plan_kernel");
}

extern "C" sa_status sa_paged_append(const void* K, const void* V, int64_t k_row_stride, int64_t v_row_stride,
                                     sa_dtype dtype, sa_paged_shape shape, const int64_t* slots, void* Kcache,
                                     void* Vcache, void* stream) {
  using namespace sa;
  sa_status r = check_paged_heads(shape, dtype, "sa_paged_append");
  if (r != SA_OK) return r;
  if (shape.T == 0) return SA_OK;   // no rows
  if (!K || !V || !slots || (shape.P > 0 && (!Kcache || !Vcache)))
    return fail(SA_ERR_INVALID_ARG, "sa_paged_append: K, V, slots and the caches are required");
  const int64_t e = (int64_t)dtype_size(dtype), row = (int64_t)shape.Hkv * shape.d;
  if (shape.T > 1 && (k_row_stride < row || v_row_stride < row))
    return fail(SA_ERR_INVALID_ARG, "sa_paged_append: a row stride is smaller than Hkv * d");
  if ((k_row_stride * e) % 16 || (v_row_stride * e) % 16 || !aligned16(K) || !aligned16(V) || !aligned16(Kcache) ||
      !aligned16(Vcache) || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return fail(SA_ERR_ALIGNMENT,
                "sa_paged_append: pointers and row strides must be 16-byte aligned (slots 8-byte aligned)");
  if (shape.P == 0) return SA_OK;   // no slot is valid
  const int vec = (int)(shape.d * e / 16);
  const int64_t per_row = (int64_t)shape.Hkv * vec;
  if (per_row > (1 << 24)) return fail(SA_ERR_UNSUPPORTED, "sa_paged_append: Hkv * d is too large");
  const int rows = (int)std::max<int64_t>(1, kAppendThreads * kAppendUnroll / per_row);
  const int shift = 31 - __builtin_clz((unsigned)shape.page);
  const cudaError_t le = launch_pdl(
      paged_append_kernel, dim3((shape.T + rows - 1) / rows), dim3(kAppendThreads), 0, as_stream(stream),
      static_cast<const uint4*>(K), static_cast<const uint4*>(V), k_row_stride * e / 16, v_row_stride * e / 16, slots,
      shape.T, shape.Hkv, vec, shift, (int64_t)shape.P << shift, rows, static_cast<uint4*>(Kcache),
      static_cast<uint4*>(Vcache));
  if (le != cudaSuccess) return fail(SA_ERR_CUDA, std::string("paged_append_kernel: ") + cudaGetErrorString(le));
  return launch_status("paged_append_kernel");
}
