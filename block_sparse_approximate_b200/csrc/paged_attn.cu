// Attention of new tokens over a paged KV cache: the entry point, the
// CUDA-core kernel for fp32 and the merge of split items.  The bf16 kernel is
// in paged_attn_tc.cu.
#include <algorithm>

#include "paged.cuh"

namespace sa {

sa_status check_paged_heads(const sa_paged_shape& s, sa_dtype dtype, const char* fn);

namespace {

using namespace paged;

// ---------------------------------------------------------------- CUDA-core kernel
// Tiles of 64 rows and 64 keys, 256 threads, two CTAs per SM.  Thread (ty,
// tx) holds scores of rows ty + 16 i and keys tx + 16 j (4 x 4) and outputs of
// the same rows (d / 16 columns); a row's maximum and sum are reduced over
// its 16 tx lanes, in 32 bits as the products are.  K and V of a tile come by
// cp.async, both before the scores, and the scores' exponentials take K's
// place, so that two CTAs fit an SM and one's loads run beside the other's
// products.  Prompts are bound by shared memory's rate and the FMA pipe beside
// it (64 x 64 x 64 products in 2800 cycles an SM, 2048 at the FMA rate); items
// of 9 to 16 rows form only the row group i = 0, smaller ones take few_rows.
constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 64;
struct SimtTiling {
  static constexpr int BN = 64;
  // a tile of at most 16 rows (a half item here) costs about half a full tile
  // (for those of up to 8 rows 1, 2 and 3 measured alike)
  static constexpr int kUnit = 4, kUnitHalf = 2, kOver = 2, kMinShare = 4;
};
constexpr int kPitchP = 68;

__device__ __forceinline__ void store8(float* dst, const float* x, float f) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4] * f, x[5] * f, x[6] * f, x[7] * f);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float* x, float f) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e] * f, x[2 * e + 1] * f);
    w[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(dst) = u;
}

template <int D>
constexpr size_t simt_smem() { return (size_t)(3 * 64 * (D + 4)) * 4; }
static_assert(kPitchP <= 64 + 4, "the exponentials lie in K's tile");

__device__ __forceinline__ void copy16_or_zero(float* dst, const float* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(copy ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct Job {
  int live, s, h, row0, r0, rv, p0, lo, hi, t0, ta, tb, slot;   // slot < 0: the whole item
};

// Items of up to 8 rows (decoding).  The tiling above makes each warp read all
// of K and V from shared memory for its two rows: 8192 cycles a tile for the
// scores of two CTAs, shared memory's rate.  Here the D / 4 lanes that copy a
// row of K or V are the ones that use it, each its own four channels, so the
// groups of lanes run through their keys without a barrier, each with a
// running maximum, sum and output of its own (joined once an item).  32
// sequences of about 1900 keys, 2 KV heads of 128: 42 us with up to 4 rows an
// item, 48 with 5 to 8, against 96 in the tiling above; heads of 64: 22 and 27
// against 52.  At 42 us memory runs at 52% of the copy rate (19 us would be all
// of it) and the schedulers issue in 47% of their cycles: the bound is the
// latency of a CTA's one tile of K and V, refilled once it is consumed, under
// the 16 warps of an SM.
//   scores: a lane's products of KB keys and R rows, KB R = the group's lanes,
//   are summed over the group by halving: lanes exchange half of what they
//   hold, and lane x ends with the sum of pair reversed(x) = key R + row.
//   outputs: a lane's four columns of the R rows; the weights go through
//   shared memory, a group's own.
constexpr int kFewRows = 8;

template <int L>
__host__ __device__ constexpr int reversed(int x) {
  int y = 0;
  for (int o = 1; o < L; o *= 2) y = 2 * y + ((x & o) != 0);
  return y;
}

template <int D, int R, typename LookUp, typename Issue>
__device__ __forceinline__ void few_rows(const Params& p, const Job& jb, float scale2, float* sq, float* sk, float* sv,
                                         LookUp look_up, Issue issue, const float* Kc, const float* Vc, float* O,
                                         const Workspace& ws) {
  constexpr int DP = D + 4, L = D / 4, NG = kSimtThreads / L, IT = 64 / NG, KB = L / R, NB = IT / KB;
  static_assert(KB * R == L && NB * KB == IT, "a batch of keys fills the group");
  static_assert((size_t)NG * R * D <= 2 * 64 * DP && NG * R * 2 <= 64 * DP, "the groups' states fit the tiles");
  static_assert(R <= 16 && 16 * DP + 64 * R <= 64 * DP, "the weights fit behind the queries");
  const int tid = threadIdx.x, x = tid % L, grp = tid / L, e0 = 4 * x;
  // this lane's pair: row and key of a batch
  const int pair = (int)(__brev((unsigned)x) >> (L == 32 ? 27 : 28)), prow = pair % R, pkey = pair / R;
  auto row_last = [&](int r) { return jb.p0 + p.by_group.div(jb.r0 + r); };
  const int last = prow < jb.rv ? row_last(prow) : -1;
  auto sees = [&](int row_end, int key) { return key <= row_end && (p.window == 0 || key > row_end - p.window); };
  float* weights = sq + 16 * DP + grp * (NB * L);   // the group's, behind the queries
  float q[R][4], o[R][4], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[r][c] = 0.f;
  copies_wait<1>();                             // K and the queries have come
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float4 v = *reinterpret_cast<const float4*>(sq + r * DP + e0);
    q[r][0] = v.x * scale2, q[r][1] = v.y * scale2, q[r][2] = v.z * scale2, q[r][3] = v.w * scale2;
  }
  for (int t = jb.ta; t < jb.tb; ++t) {
    const int k0 = (jb.t0 + t) * 64;
    const bool more = t + 1 < jb.tb;
    if (t > jb.ta) copies_wait<1>();            // this lane's own part of K
    if (more) look_up(k0 + 64);
    float s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float v[L];
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(sk + (grp + NG * (b * KB + k)) * DP + e0);
#pragma unroll
        for (int r = 0; r < R; ++r)
          v[k * R + r] = fmaf(q[r][0], y.x, fmaf(q[r][1], y.y, fmaf(q[r][2], y.z, q[r][3] * y.w)));
      }
#pragma unroll
      for (int o2 = 1; o2 < L; o2 *= 2) {
        const bool upper = x & o2;
#pragma unroll
        for (int i = 0; i < L / 2 / o2; ++i) {
          const float low = v[i], high = v[i + L / 2 / o2], give = upper ? low : high, keep = upper ? high : low;
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o2);
        }
      }
      s[b] = sees(last, k0 + grp + NG * (b * KB + pkey)) ? v[0] : -INFINITY;
    }
    if (more) issue(k0 + 64, Kc, sk);
    float mx = s[0];
#pragma unroll
    for (int b = 1; b < NB; ++b) mx = fmaxf(mx, s[b]);
#pragma unroll
    for (int o2 = 1; o2 < KB; o2 *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;     // no key yet: every term is 2^-inf = 0
    const float f = fast_exp2(m - base);
    m = mn;
    l *= f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float e = fast_exp2(s[b] - base);
      weights[b * L + pair] = e;
      l += e;
    }
    __syncwarp();
    if (__any_sync(0xffffffffu, f != 1.f))
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float fr = __shfl_sync(0xffffffffu, f, reversed<L>(r), L);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[r][c] *= fr;
      }
    if (more) copies_wait<1>();                 // this lane's own part of V
    else copies_wait<0>();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float4 y[KB];
      float big = 0.f;
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        y[k] = *reinterpret_cast<const float4*>(sv + (grp + NG * (b * KB + k)) * DP + e0);
        // (0 or NaN)
        big = fmaf(y[k].x, 0.f, fmaf(y[k].y, 0.f, fmaf(y[k].z, 0.f, fmaf(y[k].w, 0.f, big))));
      }
      // 0 times a value that is not finite is not 0: where one was met, a key
      // is left out for the rows that do not see it
      auto product = [&](auto guarded) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          float4 four[R / 4];
#pragma unroll
          for (int r = 0; r < R; r += 4)
            four[r / 4] = *reinterpret_cast<const float4*>(weights + b * L + k * R + r);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float4 z = four[r / 4];
            const float w = (r & 3) == 0 ? z.x : (r & 3) == 1 ? z.y : (r & 3) == 2 ? z.z : z.w;
            if (decltype(guarded)::value &&
                (r >= jb.rv || !sees(row_last(r), k0 + grp + NG * (b * KB + k)))) continue;
            o[r][0] = fmaf(w, y[k].x, o[r][0]);
            o[r][1] = fmaf(w, y[k].y, o[r][1]);
            o[r][2] = fmaf(w, y[k].z, o[r][2]);
            o[r][3] = fmaf(w, y[k].w, o[r][3]);
          }
        }
      };
      if (__any_sync(0xffffffffu, big != 0.f)) product(std::true_type{});
      else product(std::false_type{});
    }
    __syncwarp();
    if (more) issue(k0 + 64, Vc, sv);
  }
#pragma unroll
  for (int o2 = 1; o2 < KB; o2 *= 2) l += __shfl_xor_sync(0xffffffffu, l, o2);
  // the groups' states: outputs over K and V, maxima and sums over the queries
  __syncthreads();
  float2* ml = reinterpret_cast<float2*>(sq);
  if (pkey == 0) ml[grp * R + prow] = make_float2(m, l);
#pragma unroll
  for (int r = 0; r < R; ++r)
    *reinterpret_cast<float4*>(sk + (grp * R + r) * D + e0) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
  __syncthreads();
  const int r = tid / L;                        // four columns of a row each
  if (r >= jb.rv) return;
  float M = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int g = 0; g < NG; ++g) M = fmaxf(M, ml[g * R + r].x);
  const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float2 y = ml[g * R + r];
    const float f = fast_exp2(y.x - base);
    const float4 v = *reinterpret_cast<const float4*>(sk + (g * R + r) * D + e0);
    sum = fmaf(y.y, f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  if (jb.slot < 0) {
    const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
    *reinterpret_cast<float4*>(O + p.query_row(jb.row0, jb.h, jb.r0 + r) * D + e0) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  } else {
    ws.chunk<D>(jb.slot, x)[r] = acc;
    if (x == 0) ws.state(jb.slot)[r] = make_float2(M, sum);
  }
}

template <int D>
__global__ void __launch_bounds__(kSimtThreads, 2)
paged_attn_simt_kernel(const float* __restrict__ Q, int64_t q_stride, const float* __restrict__ Kc,
                       const float* __restrict__ Vc, Params p, float scale2, float* __restrict__ O, Workspace ws) {
  pdl_wait();
  pdl_trigger();
  using TL = SimtTiling;
  constexpr int DP = D + 4, NC = D / 64;        // NC float4 columns of the output per thread
  extern __shared__ __align__(16) float smem_f[];
  float* sq = smem_f;
  float* sk = sq + 64 * DP;
  float* sv = sk + 64 * DP;
  float* sp = sk;                               // after the scores
  __shared__ int64_t tot[kSimtThreads / 32];
  __shared__ Job job;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;

  // the line, laid in the operand buffers before their first use
  int64_t* pre = reinterpret_cast<int64_t*>(smem_f);
  const int64_t total = lay_line<TL, kSimtThreads>(p, pre, tot);
  const Shares shares = cut_line<TL>(total, ws.ctas);
  if (tid == 0) ws.desc[c].valid = 0;
  if (total == 0 || c >= shares.parts) return;
  Walker<TL> w;
  __shared__ int64_t found[3];
  const int64_t w0 = shares.start(c), w1 = shares.start(c + 1);
  find_request<kSimtThreads>(p, pre, w0, found);
  bool more = true;
  __syncthreads();                              // the line is read; its memory becomes the operands'
  if (warp == 0) w.find(p, (int)found[0], found[1], found[2], w0);
  int emitted = 0;
  bool first = true;

  for (;;) {
    if (warp == 0) {
      // the next portion of the share
      int ta = 0, tb = 0;
      bool got = false;
      while (more && !got) {
        if (!first) more = w.next(p);
        first = false;
        if (!more || w.start >= w1) {
          more = false;
          break;
        }
        got = w.portion(w0, w1, ta, tb);
      }
      if (lane == 0) {
        job.live = got;
        if (got) {
          const bool whole = ta == 0 && tb == w.it.nt;
          const int slot = whole ? -1 : 2 * c + (emitted > 0);
          job = Job{1, w.s, w.h, w.q.row0, w.it.r0, w.it.rv, w.it.p0, w.it.lo, w.it.hi, w.it.t0, ta, tb, slot};
          if (!whole && ta == 0)
            ws.desc[c] = Desc{w.start, shares, 1, slot, w.it.unit, w.it.nt, w.q.row0, w.it.r0, w.it.rv, w.h};
        }
      }
      emitted += got;
    }
    __syncthreads();
    const Job jb = job;
    if (!jb.live) return;

    // K and V of the tile at k0; rows outside the item's span and pages outside the pool read as zero
    constexpr int IT = D / 16, RI = kSimtThreads / (D / 4);   // chunks of a thread, RI rows apart
    const int row0 = tid / (D / 4), e0 = 4 * (tid % (D / 4));
    const int mask = (1 << p.page_shift) - 1;
    int id[IT];                                 // pages of this thread's rows of a tile, -1: none
    auto look_up = [&](int k0) {
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const int key = k0 + row0 + RI * k;
        id[k] = -1;
        if (key >= jb.lo && key < jb.hi) id[k] = p.table[(size_t)jb.s * p.max_pages + (key >> p.page_shift)];
      }
    };
    auto issue = [&](int k0, const float* src, float* dst) {
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const bool there = id[k] >= 0 && id[k] < p.P;
        const int64_t at = ((((int64_t)id[k] * p.Hkv + jb.h) << p.page_shift) + ((k0 + row0 + RI * k) & mask)) * D + e0;
        copy16_or_zero(dst + (row0 + RI * k) * DP + e0, src + (there ? at : 0), there);
      }
      copies_commit();
    };
    auto issue_tile = [&](int k0) {
      look_up(k0);
      issue(k0, Kc, sk);
      issue(k0, Vc, sv);
    };
    if (jb.ta < jb.tb) {
      // queries, in the group of the first K tile
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const int r = row0 + RI * k, at = min(r, jb.rv - 1);
        const int tok = p.by_group.div(jb.r0 + at), head = jb.h * p.group + jb.r0 + at - tok * p.group;
        copy16_or_zero(sq + r * DP + e0, Q + (int64_t)(jb.row0 + tok) * q_stride + (int64_t)head * D + e0, r < jb.rv);
      }
      issue_tile((jb.t0 + jb.ta) * 64);
    }
    if (jb.rv <= kFewRows) {
      auto few = [&](auto rows) {
        few_rows<D, decltype(rows)::value>(p, jb, scale2, sq, sk, sv, look_up, issue, Kc, Vc, O, ws);
      };
      if (jb.rv <= 4) few(std::integral_constant<int, 4>{});
      else few(std::integral_constant<int, 8>{});
      __syncthreads();                          // job, queries and the groups' states are read
      continue;
    }
    float m[4], l[4], o[4][NC * 4];
    int last[4];                                // the row's last visible key
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int r = ty + 16 * i;
      last[i] = jb.p0 + p.by_group.div(jb.r0 + min(r, jb.rv - 1));
#pragma unroll
      for (int k = 0; k < NC * 4; ++k) o[i][k] = 0.f;
    }
    // one key tile; NI: row groups of 16 that hold rows
    auto tile = [&](auto ni, int k0) {
      constexpr int NI = decltype(ni)::value;
      float s[NI][4];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int e = 0; e < D; e += 4) {
        float4 a[NI], b[4];
#pragma unroll
        for (int i = 0; i < NI; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * DP + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * DP + e);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
      }
      __syncthreads();                          // K is read; its place takes the exponentials
      // (the rows' reductions side by side, so that their shuffles' latencies overlap)
      float mx[NI], sum[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        mx[i] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = k0 + tx + 16 * j;
          const bool seen = key <= last[i] && (p.window == 0 || key > last[i] - p.window);
          s[i][j] = seen ? s[i][j] * scale2 : -INFINITY;
          mx[i] = fmaxf(mx[i], s[i][j]);
        }
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < NI; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float mn = fmaxf(m[i], mx[i]);
        const float base = mn == -INFINITY ? 0.f : mn;     // no key yet: every term is 2^-inf = 0
        const float f = fast_exp2(m[i] - base);
        m[i] = mn;
        sum[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = fast_exp2(s[i][j] - base);
          sum[i] += e;
          sp[(ty + 16 * i) * kPitchP + tx + 16 * j] = e;
        }
        l[i] *= f;
#pragma unroll
        for (int k = 0; k < NC * 4; ++k) o[i][k] *= f;
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < NI; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);
#pragma unroll
      for (int i = 0; i < NI; ++i) l[i] += sum[i];
      copies_wait<0>();                         // V has come
      // 0 times a value that is not finite is not 0: such a tile takes the
      // products that leave the masked keys out
      bool finite = true;
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(sv + (row0 + RI * k) * DP + e0);
        finite &= fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY;
      }
      const bool guard = __syncthreads_or(!finite);
      auto product = [&](auto guarded) {
#pragma unroll 4
        for (int k = 0; k < 64; k += 4) {
          float4 a[NI];
#pragma unroll
          for (int i = 0; i < NI; ++i) a[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * kPitchP + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            float4 b[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n)
              b[n] = *reinterpret_cast<const float4*>(sv + (k + kk) * DP + 4 * tx + 64 * n);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const float e = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
              // a masked key's term is absent, also where its value is not finite
              if (decltype(guarded)::value) {
                const int key = k0 + k + kk;
                if (key > last[i] || (p.window > 0 && key <= last[i] - p.window)) continue;
              }
#pragma unroll
              for (int n = 0; n < NC; ++n) {
                o[i][4 * n] = fmaf(e, b[n].x, o[i][4 * n]);
                o[i][4 * n + 1] = fmaf(e, b[n].y, o[i][4 * n + 1]);
                o[i][4 * n + 2] = fmaf(e, b[n].z, o[i][4 * n + 2]);
                o[i][4 * n + 3] = fmaf(e, b[n].w, o[i][4 * n + 3]);
              }
            }
          }
        }
      };
      if (guard) product(std::true_type{});
      else product(std::false_type{});
    };
    for (int t = jb.ta; t < jb.tb; ++t) {
      const int k0 = (jb.t0 + t) * 64;
      copies_wait<1>();                         // K has come
      __syncthreads();
      if (jb.rv <= 16) tile(std::integral_constant<int, 1>{}, k0);
      else tile(std::integral_constant<int, 4>{}, k0);
      __syncthreads();                          // V and the exponentials are read
      if (t + 1 < jb.tb) issue_tile(k0 + 64);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      if (r >= jb.rv) continue;
      if (jb.slot < 0) {
        const float inv = l[i] > 0.f ? 1.0f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
        float* dst = O + p.query_row(jb.row0, jb.h, jb.r0 + r) * D + 4 * tx;
#pragma unroll
        for (int n = 0; n < NC; ++n)
          *reinterpret_cast<float4*>(dst + 64 * n) =
              make_float4(o[i][4 * n] * inv, o[i][4 * n + 1] * inv, o[i][4 * n + 2] * inv, o[i][4 * n + 3] * inv);
      } else {
#pragma unroll
        for (int n = 0; n < NC; ++n)
          ws.chunk<D>(jb.slot, tx + 16 * n)[r] =
              make_float4(o[i][4 * n], o[i][4 * n + 1], o[i][4 * n + 2], o[i][4 * n + 3]);
        if (tx == 0) ws.state(jb.slot)[r] = make_float2(m[i], l[i]);
      }
    }
    __syncthreads();                            // job and queries are read
  }
}

// ---------------------------------------------------------------- merge
// Block (c, y) merges 16 columns of the split item that starts in share c:
// the states of its portions, in a fixed order, so the result does not depend
// on which CTA ran first.  A thread takes a row; items of few rows (decoding:
// many portions) give each row several threads, every one of them the
// portions of its residue, joined through shared memory.  Reads a few hundred
// KB to some MB; bound by latency.
constexpr int kCombineThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads)
paged_combine_kernel(Params p, Workspace ws, T* __restrict__ O) {
  pdl_wait();
  pdl_trigger();
  __shared__ int slots[Limits::kCtasSimt + 1];
  __shared__ int count;
  __shared__ float red[kCombineThreads][19];    // maximum, sum, 16 columns
  const Desc d = ws.desc[blockIdx.x];
  if (!d.valid) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the portions' slots, in key order
  if (warp == 0) {
    const int64_t end_tiles = d.start + (int64_t)d.nt * d.unit;
    int n = 1;
    if (lane == 0) slots[0] = d.slot;
    for (int base = blockIdx.x + 1; base < d.shares.parts; base += 32) {
      const int c = base + lane;
      bool in = false, over = true;
      if (c < d.shares.parts) {
        const int64_t a = d.shares.start(c), b = d.shares.start(c + 1);
        over = a >= end_tiles;
        in = !over && tiles_before(a - d.start, d.nt, d.unit) < tiles_before(b - d.start, d.nt, d.unit);
      }
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (in) slots[n + __popc(who & ((1u << lane) - 1u))] = 2 * c;
      n += __popc(who);
      if (__any_sync(0xffffffffu, over)) break;
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int n = count;
  int rows = 16;                                // threads of a residue: a power of two over the rows
  while (rows < d.rv) rows *= 2;
  const int r = tid % rows, pl = tid / rows, step = kCombineThreads / rows;
  const bool mine = r < d.rv;
  float m = -INFINITY, sum = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  if (mine) {
    // Two portions at a time, states and columns in one go: the loads' latency
    // is what a merge of few portions costs (four at a time took registers
    // from the blocks that an SM holds: 30 against 26.5 us for the whole of a
    // small fp32 batch).
    for (int k0 = pl; k0 < n; k0 += 2 * step) {
      float2 ml[2];
      float4 x[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = k0 + j * step;
        ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k >= n) continue;
        ml[j] = ws.state(slots[k])[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] = ws.chunk<D>(slots[k], 4 * blockIdx.y + e)[r];
      }
      // NaN counts as the largest maximum: it belongs into the result
      float most = m;
#pragma unroll
      for (int j = 0; j < 2; ++j) most = most < ml[j].x || ml[j].x != ml[j].x ? ml[j].x : most;
      const float base = most == -INFINITY ? 0.f : most;
      const float f0 = fast_exp2(m - base);
      m = most;
      sum *= f0;
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] *= f0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // (a portion without a visible key adds zeros: nothing is left out, since
        // scores that are all NaN leave a maximum of -inf, and weights of 0 an
        // output that is NaN where a value is infinite)
        const float f = fast_exp2(ml[j].x - base);
        sum = fmaf(ml[j].y, f, sum);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[4 * e] = fmaf(x[j][e].x, f, acc[4 * e]);
          acc[4 * e + 1] = fmaf(x[j][e].y, f, acc[4 * e + 1]);
          acc[4 * e + 2] = fmaf(x[j][e].z, f, acc[4 * e + 2]);
          acc[4 * e + 3] = fmaf(x[j][e].w, f, acc[4 * e + 3]);
        }
      }
    }
    if (step > 1) {
      red[tid][0] = m;
      red[tid][1] = sum;
#pragma unroll
      for (int e = 0; e < 16; ++e) red[tid][2 + e] = acc[e];
    }
  }
  if (step > 1) {
    __syncthreads();
    if (pl > 0 || !mine) return;
    float M = m;
    for (int k = 1; k < step; ++k) M = M < red[tid + k * rows][0] || red[tid + k * rows][0] != red[tid + k * rows][0]
                                           ? red[tid + k * rows][0] : M;
    const float base = M == -INFINITY ? 0.f : M;
    const float f0 = fast_exp2(m - base);
    sum *= f0;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] *= f0;
    for (int k = 1; k < step; ++k) {
      const float* x = red[tid + k * rows];
      const float f = fast_exp2(x[0] - base);
      sum = fmaf(x[1], f, sum);
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = fmaf(x[2 + e], f, acc[e]);
    }
  }
  if (!mine) return;
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
  T* dst = O + p.query_row(d.row0, d.h, d.r0 + r) * D + 16 * blockIdx.y;
#pragma unroll
  for (int e = 0; e < 16; e += 8) store8(dst + e, acc + e, inv);
}

// ---------------------------------------------------------------- host side

// rows an item may hold in the workspace: never more than the call has
int rows_cap(const sa_paged_shape& s, int bm) {
  const int64_t rows = (int64_t)s.T * (s.Hq / s.Hkv);
  return (int)std::min<int64_t>(bm, (rows + 7) / 8 * 8);
}

constexpr size_t kDescBytes = (sizeof(Desc) * Limits::kCtasSimt + 255) / 256 * 256;

size_t workspace_bytes(const sa_paged_shape& s) {
  const size_t tc = (size_t)2 * Limits::kCtas * rows_cap(s, 256);
  const size_t simt = (size_t)2 * Limits::kCtasSimt * rows_cap(s, kSimtRows);
  return kDescBytes + std::max(tc, simt) * (s.d + 2) * sizeof(float);
}

template <int D>
sa_status launch_simt(const void* Q, int64_t q_stride, const void* Kc, const void* Vc, const sa_paged_shape& s,
                      const Params& p, float scale, void* O, const Workspace& ws, cudaStream_t stream) {
  constexpr size_t smem = simt_smem<D>();
  static_assert(smem >= kMaxRequests * sizeof(int64_t), "the line lies in the operand buffers");
  auto kern = paged_attn_simt_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return launch_status("cudaFuncSetAttribute(paged_attn_simt_kernel)");
  const cudaError_t le =
      launch_pdl(kern, dim3(ws.ctas), dim3(kSimtThreads), smem, stream, static_cast<const float*>(Q),
                 q_stride, static_cast<const float*>(Kc), static_cast<const float*>(Vc), p, scale * kLog2e,
                 static_cast<float*>(O), ws);
  if (le != cudaSuccess) return fail(SA_ERR_CUDA, std::string("paged_attn_simt_kernel: ") + cudaGetErrorString(le));
  return launch_status("paged_attn_simt_kernel");
}

template <typename T, int D>
sa_status launch_combine(const Params& p, const Workspace& ws, void* O, cudaStream_t stream) {
  const cudaError_t le = launch_pdl(paged_combine_kernel<T, D>, dim3(ws.ctas, D / 16), dim3(kCombineThreads), 0,
                                    stream, p, ws, static_cast<T*>(O));
  if (le != cudaSuccess) return fail(SA_ERR_CUDA, std::string("paged_combine_kernel: ") + cudaGetErrorString(le));
  return launch_status("paged_combine_kernel");
}

sa_status check_attn_shape(const sa_paged_shape& s, sa_dtype dtype, const char* fn) {
  sa_status r = check_paged_heads(s, dtype, fn);
  if (r != SA_OK) return r;
  if (s.Hq <= 0 || s.Hq % s.Hkv)
    return fail(SA_ERR_INVALID_ARG, std::string(fn) + ": Hq must be a positive multiple of Hkv");
  if ((int64_t)s.T * s.Hq > (1 << 30))
    return fail(SA_ERR_UNSUPPORTED, std::string(fn) + ": T * Hq exceeds 2^30 query rows");
  return SA_OK;
}

}  // namespace
}  // namespace sa

extern "C" size_t sa_paged_attn_workspace_size(sa_paged_shape shape) {
  using namespace sa;
  if (check_attn_shape(shape, SA_BF16, "sa_paged_attn_workspace_size") != SA_OK) return 0;
  return workspace_bytes(shape);
}

extern "C" sa_status sa_paged_attn_fwd(const void* Q, int64_t q_row_stride, const void* Kcache, const void* Vcache,
                                       sa_dtype dtype, sa_paged_shape shape, const int32_t* q_start,
                                       const int32_t* kv_len, const int32_t* table, int32_t window, float scale,
                                       void* O, void* workspace, size_t workspace_bytes_given, void* stream) {
  using namespace sa;
  using namespace sa::paged;
  sa_status r = check_attn_shape(shape, dtype, "sa_paged_attn_fwd");
  if (r != SA_OK) return r;
  if (window < 0) return fail(SA_ERR_INVALID_ARG, "sa_paged_attn_fwd: window must be 0 (none) or positive");
  if (!(scale > 0.f && scale * kLog2e < INFINITY))   // (the kernels' scores are in powers of 2)
    return fail(SA_ERR_INVALID_ARG, "sa_paged_attn_fwd: scale must be positive, and scale * log2(e) finite");
  if (shape.T == 0 || shape.S == 0) return SA_OK;   // no row belongs to a request
  if (!Q || !q_start || !kv_len || !O || (shape.P > 0 && shape.max_pages > 0 && (!Kcache || !Vcache || !table)))
    return fail(SA_ERR_INVALID_ARG, "sa_paged_attn_fwd: Q, caches, q_start, kv_len, table and O are required");
  if (dtype == SA_BF16 && shape.Hq / shape.Hkv > 128)
    return fail(SA_ERR_UNSUPPORTED, "sa_paged_attn_fwd: at most 128 query heads per KV head in bf16");
  const int64_t e = (int64_t)dtype_size(dtype);
  if (shape.T > 1 && q_row_stride < (int64_t)shape.Hq * shape.d)
    return fail(SA_ERR_INVALID_ARG, "sa_paged_attn_fwd: q_row_stride is smaller than Hq * d");
  if (!aligned16(Q) || !aligned16(Kcache) || !aligned16(Vcache) || !aligned16(O) || (q_row_stride * e) % 16)
    return fail(SA_ERR_ALIGNMENT, "sa_paged_attn_fwd: pointers and q_row_stride must be 16-byte aligned");
  for (const void* x : {(const void*)q_start, (const void*)kv_len, (const void*)table})
    if (reinterpret_cast<uintptr_t>(x) & 3u)
      return fail(SA_ERR_ALIGNMENT, "sa_paged_attn_fwd: q_start, kv_len and table must be 4-byte aligned");
  if (!workspace || workspace_bytes_given < workspace_bytes(shape))
    return fail(SA_ERR_WORKSPACE,
                "sa_paged_attn_fwd: workspace missing or smaller than sa_paged_attn_workspace_size()");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(SA_ERR_ALIGNMENT, "sa_paged_attn_fwd: workspace must be 256-byte aligned");
  // a pool or table without pages holds no key: every length reads as 0
  const bool keys = shape.P > 0 && shape.max_pages > 0;
  const int shift = 31 - __builtin_clz((unsigned)shape.page);
  const int most = keys ? shape.max_pages << shift : 0;
  const bool tc = dtype == SA_BF16;
  const int group = shape.Hq / shape.Hkv;
  // tensor cores: 128-row tiles of whole tokens, two to an item
  const int half = tc ? 128 / group * group : 16, bm = tc ? 2 * half : kSimtRows;
  Params p{q_start, kv_len, table, shape.S, shape.T, shape.Hq, shape.Hkv, group, shift, shape.P,
           keys ? shape.max_pages : 0, window >= most ? 0 : window, bm, half, FastDiv(group), FastDiv(shape.Hkv),
           FastDiv(bm)};
  Workspace ws;
  ws.desc = static_cast<Desc*>(workspace);
  ws.rows_cap = rows_cap(shape, tc ? 256 : kSimtRows);
  ws.ctas = tc ? Limits::kCtas : Limits::kCtasSimt;
  ws.o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kDescBytes);
  ws.ml = ws.o + (size_t)2 * ws.ctas * ws.rows_cap * shape.d;
  cudaStream_t st = as_stream(stream);
  if (dtype == SA_FP32) {
    r = shape.d == 128 ? launch_simt<128>(Q, q_row_stride, Kcache, Vcache, shape, p, scale, O, ws, st)
                       : launch_simt<64>(Q, q_row_stride, Kcache, Vcache, shape, p, scale, O, ws, st);
    if (r != SA_OK) return r;
    return shape.d == 128 ? launch_combine<float, 128>(p, ws, O, st) : launch_combine<float, 64>(p, ws, O, st);
  }
  using bf = __nv_bfloat16;
  r = paged_attn_tc(Q, q_row_stride, Kcache, Vcache, shape, p, scale, O, ws, st);
  if (r != SA_OK) return r;
  return shape.d == 128 ? launch_combine<bf, 128>(p, ws, O, st) : launch_combine<bf, 64>(p, ws, O, st);
}
