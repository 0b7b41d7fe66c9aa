// Attention of new tokens over a paged KV cache on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA), bf16, d = 64 or 128.
//
// One persistent CTA per SM walks its share of the line of items (paged.cuh).
// An item is up to two tiles of query rows (token-major, the query heads of
// one KV head side by side; a tile holds as many whole tokens as fit 128 rows,
// so that a TMA box of tokens x heads x 64 channels loads it whatever the group
// size).  Its keys come in tiles of 128, one box per page and 64 channels, so a
// key tile may be gathered from 1 to 8 pages.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  two softmax warpgroups ("streams").  Items of two row
//              tiles: stream s owns tile s and both use every key tile.  Items
//              of one row tile (decoding): both own it, stream s takes the key
//              tiles of its parity, and stream 0 merges the two states.  So one
//              group's softmax overlaps the other's MMAs in either case.
//              Thread r of a group is query row r (TMEM lane r); warps
//              without rows only keep the barriers' count;
//   warp 8     TMA producer: K and V tiles into one ring of slots, the lanes
//              share a tile's boxes;
//   warp 9     MMA issuer: S = Q Kᵀ two steps ahead of O += P V (P read from
//              TMEM, written over S), across item boundaries, so the next
//              item's scores form during the epilogue;
//   warp 10    loads the query tiles (TMA);
//   warp 11    walks the share and hands the items to the others through a
//              ring in shared memory.
// TMEM (512 columns): S_0 [0,128), S_1 [128,256), O_0 [256,384), O_1 [384,512).
//
// Numerics: scores, maxima, sums and O in fp32; the weights are rounded to
// bf16 for P V (their fp32 values enter the row sum), which moves an output
// by at most 2^-8 Σ p|v| / Σ p, the size of the output's own rounding.
//
// Keys that a row does not see: the score is replaced by -inf, and as 0 · inf
// is not 0, the values of an edge tile (one that some row of the item does
// not see whole) are screened before P V: rows of V outside the item's span
// are cleared, and elements that are not finite are cleared and added back
// after the item's store for the rows that see them (add_unbounded), whatever
// their weights: an infinite value whose weight is 0 in float32 gives its
// infinity there and NaN in a tile that is seen whole, never a finite output.
#include "paged.cuh"
#include "tc_util.cuh"

namespace sa {
namespace {

using namespace tc;
using namespace paged;

constexpr int kThreads = 384;
// registers: 256 softmax threads x 216 + 128 others x 72 = 64512 = 384 x 168,
// what the block is launched with (build.py checks ptxas reports 168)
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr uint32_t kSpan = 128 * 128;          // 128 rows x one 128-byte swizzle span
constexpr uint32_t kColO = 256;
constexpr float kLazy = 8.0f;                  // O is rescaled when the maximum grew by more than 2^8
constexpr float kStaleSum = 65536.0f;          // a tile's exponentials sum to less, or its maximum is formed
constexpr int kFewTokens = 4;                  // a query tile of so few tokens is loaded token by token
constexpr int kItems = 4;                      // item ring
constexpr uint32_t kExpBits = 0x7f807f80u, kExpStep = 0x00800080u;   // exponents of two bf16

struct TcTiling {
  static constexpr int BN = 128;
  // a key tile of a two-tile item costs about two 128x128 steps of the tensor
  // pipe, one of a half item its 64 KB from memory
  static constexpr int kUnit = 4, kUnitHalf = 3, kOver = 6, kMinShare = 3;
};

// An item as the walker hands it out.  The softmax warps read its fields here
// when they need them instead of holding them in registers beside a row of S.
struct TileItem {
  int live, s, h, row0, r0, rv, p0, lo, hi, t0, n, slot, paired, qhalf, kt, pad;
  int rows[2], steps[2];                       // of each stream: rows, key tiles
  // tiles t (of 0 .. n - 1) with t >= from or t < to: the stream's rows do not
  // see them whole / some row of the item does not
  struct { int mask_from, mask_to, screen_from, screen_to; } edge[2];
  int pad2[4];
};
static_assert(sizeof(TileItem) == 128, "item ring layout");

// Tiles t >= from hold a key behind position p_first, tiles t < to one left of
// the window of position p_last (t counted from the tile at t0).
__device__ __forceinline__ void edge_range(int p_first, int p_last, int window, int t0, int& from, int& to) {
  from = p_first < 0 ? 0 : max(0, (p_first + 1) / 128 - t0);
  to = window > 0 && p_last - window >= 0 ? max(0, (p_last - window) / 128 + 1 - t0) : 0;
}

template <int D>
struct Lay {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kTile = NH * kSpan;
  static constexpr int NS = D == 128 ? 5 : 10;
  static constexpr int B_QF = 0, B_QE = 2, B_KF = 4, B_KE = B_KF + NS, B_SF = B_KE + NS, B_PR = B_SF + 2,
                       B_OD = B_PR + 2, B_OF = B_OD + 2, B_EX = B_OF + 2, B_IF = B_EX + 1, B_IE = B_IF + kItems,
                       B_FIN = B_IE + kItems, B_QZ = B_FIN + 1, NBAR = B_QZ + 1;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kBarOff = kRing + NS * kTile;
  static constexpr uint32_t kSlotOff = (kBarOff + 8 * NBAR + 15) / 16 * 16;  // tmem base, abort, unbounded
  static constexpr uint32_t kItemOff = kSlotOff + 16;
  static constexpr uint32_t kExOff = kItemOff + 128 * kItems;                 // stream 1's maxima and sums
  static constexpr uint32_t kTotOff = kExOff;                                // lay_line's totals, before the roles
  static constexpr uint32_t kEnd = kExOff + 2 * 128 * 4;
  static constexpr size_t smem_bytes = 1024 + kEnd;
};
static_assert(Lay<128>::smem_bytes <= 232448 && Lay<64>::smem_bytes <= 232448, "shared memory of a CTA");
static_assert(2 * Lay<64>::kTile >= kMaxRequests * sizeof(int64_t), "the line lies in the query tiles");

// The MMAs of one step in one asm block: the converged warp elects a lane
// once and that lane issues them back to back, the operands' descriptors
// advanced by constants (only the start-address field changes, and no carry
// leaves it).  With an election and a descriptor per MMA the issuing warp,
// which shares its scheduler with two softmax warps, was the slowest role of
// the kernel (2700 cycles a step, 1100 of them here).

// S(tmem) = A · B, both K-major tiles of 64-channel spans 16 KB apart.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#define SA_STEP(OFF, ACC)                                                                  \
  "add.s64 ra, %1, " #OFF ";\n\tadd.s64 rb, %2, " #OFF ";\n\t"                             \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ra, rb, %3, {%4, %4, %4, %4}, " #ACC ";\n\t"
  if constexpr (D == 128) {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b64 ra, rb;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, %4, 0;\n\t"
        SA_STEP(0, f) SA_STEP(2, t) SA_STEP(4, t) SA_STEP(6, t)
        SA_STEP(1024, t) SA_STEP(1026, t) SA_STEP(1028, t) SA_STEP(1030, t) "}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(0u) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b64 ra, rb;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, %4, 0;\n\t"
        SA_STEP(0, f) SA_STEP(2, t) SA_STEP(4, t) SA_STEP(6, t) "}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(0u) : "memory");
  }
#undef SA_STEP
}

// O(tmem) (+)= P(tmem) · V, V an MN-major tile of 128 rows: 16 keys a step.
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t pa, uint64_t v, uint32_t idesc, uint32_t accumulate) {
#define SA_STEP(COL, OFF, ACC)                                                             \
  "add.s32 rp, %1, " #COL ";\n\tadd.s64 rv, %2, " #OFF ";\n\t"                             \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [rp], rv, %3, {%5, %5, %5, %5}, " #ACC ";\n\t"
  asm volatile(
      "{\n\t.reg .pred e, f, t;\n\t.reg .b64 rv;\n\t.reg .b32 rp;\n\telect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, %5, 0;\n\t"
      SA_STEP(0, 0, f) SA_STEP(8, 128, t) SA_STEP(16, 256, t) SA_STEP(24, 384, t)
      SA_STEP(32, 512, t) SA_STEP(40, 640, t) SA_STEP(48, 768, t) SA_STEP(56, 896, t) "}"
      ::"r"(d), "r"(pa), "l"(v), "r"(idesc), "r"(accumulate), "r"(0u) : "memory");
#undef SA_STEP
}
__device__ __forceinline__ void mma_commit_w(uint32_t bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
               : "memory");
}

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// A wait of a whole warp, bounded like mbar_wait.  The first try is kept
// short: most waits of the MMA issuer find their barrier complete.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// A value that all lanes of the warp hold, in a form that the compiler knows
// to be uniform (the MMA operands then live in uniform registers).
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// The abort path's own wait: nothing can release it but the copy in flight.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!try_wait(bar, parity) && clock64() - t0 < kWaitCycles / 8) {
  }
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Whether some row of an item (first position p_first, keys below hi) does
// not see the whole tile at k0.
__device__ __forceinline__ bool edge_tile(int p_first, int hi, int window, int k0) {
  return k0 + 127 > p_first || (window > 0 && k0 <= hi - 1 - window);
}

// Adds the values that are not finite, of the keys of edge tiles that a row
// with last key `last` sees, to its stored output (groups of four columns
// `stride` elements apart).  Runs only after such a value was met in this CTA.
template <typename T>
__device__ __noinline__ void add_unbounded(const Params& p, int s, int h, int t0, int n, int p_first, int hi,
                                           const __nv_bfloat16* Vc, int D, int last, T* dst, int stride) {
  for (int t = 0; t < n; ++t) {
    const int k0 = (t0 + t) * 128;
    if (!edge_tile(p_first, hi, p.window, k0)) continue;
    const int a = max(max(k0, 0), p.window > 0 ? last - p.window + 1 : 0), b = min(k0 + 127, last);
    for (int key = a; key <= b; ++key) {
      const int id = p.table[(size_t)s * p.max_pages + (key >> p.page_shift)];
      if (id < 0 || id >= p.P) continue;
      const int64_t row = (((int64_t)id * p.Hkv + h) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
      const __nv_bfloat16* v = Vc + row * D;
      for (int e = 0; e < D; ++e) {
        const float x = __bfloat162float(v[e]);
        T* o = dst + (size_t)(e >> 2) * stride + (e & 3);
        if (!(fabsf(x) < INFINITY)) *o = from_f<T>(to_f(*o) + x);
      }
    }
  }
}

// 64 bytes of a lane's own row; with 32-byte stores where the rows allow them,
// whole sectors, half the passes of 16-byte ones.
__device__ __forceinline__ void store64(void* dst, const uint32_t (&u)[16], bool wide) {
  if (wide) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                   ::"l"(static_cast<char*>(dst) + 32 * k), "r"(u[8 * k]), "r"(u[8 * k + 1]), "r"(u[8 * k + 2]),
                     "r"(u[8 * k + 3]), "r"(u[8 * k + 4]), "r"(u[8 * k + 5]), "r"(u[8 * k + 6]), "r"(u[8 * k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      static_cast<uint4*>(dst)[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __nv_bfloat16* __restrict__ Vc, const Params p, float scale2,
                     __nv_bfloat16* __restrict__ O, const Workspace ws) {
  using L = Lay<D>;
  using TL = TcTiling;
  constexpr int NS = L::NS, NH = L::NH;
  constexpr uint32_t kTile = L::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  // hardware warps 0-3 are the roles 8-11 and come first: the scheduler prefers
  // older warps, and the MMA issuer must not wait behind the softmax (1.5% of
  // the kernel)
  const int hw = uniform((int)(threadIdx.x >> 5)), warp = hw < 4 ? hw + 8 : hw - 4, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kSlotOff + 4);
  volatile int* unbounded_flag = reinterpret_cast<volatile int*>(smem + L::kSlotOff + 8);
  TileItem* items = reinterpret_cast<TileItem*>(smem + L::kItemOff);
  auto bar = [&](int k) { return sb + L::kBarOff + 8u * k; };

  // barriers and TMEM while the previous launch drains
  if (threadIdx.x == 32) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::B_QF + s), 1);
      mbar_init(bar(L::B_QE + s), 1);
      mbar_init(bar(L::B_SF + s), 1);
      mbar_init(bar(L::B_PR + s), 4);
      mbar_init(bar(L::B_OD + s), 1);
      mbar_init(bar(L::B_OF + s), 4);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(L::B_KF + s), 1);
      mbar_init(bar(L::B_KE + s), 1);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(bar(L::B_IF + s), 1);
      mbar_init(bar(L::B_IE + s), 11);         // producer, MMA issuer, query loader, 8 softmax warps
    }
    mbar_init(bar(L::B_EX), 4);
    mbar_init(bar(L::B_FIN), 1);
    mbar_init(bar(L::B_QZ), 8);
    *abort_flag = 0;
    *unbounded_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmQ1);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), 512);
  pdl_wait();
  pdl_trigger();
  // the line, in the memory of the query tiles (loaded after the first item is handed out)
  int64_t* pre = reinterpret_cast<int64_t*>(smem);
  int64_t* found = reinterpret_cast<int64_t*>(smem + L::kTotOff) + kThreads / 32;
  const int64_t total = lay_line<TL, kThreads>(p, pre, reinterpret_cast<int64_t*>(smem + L::kTotOff));
  const Shares shares = cut_line<TL>(total, ws.ctas);
  if (threadIdx.x == 0) ws.desc[c].valid = 0;
  const bool idle = total == 0 || c >= shares.parts;
  if (!idle) find_request<kThreads>(p, pre, shares.start(c), found);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = uniform(*tmem_slot);
  if (idle) {
    if (warp == 0) tmem_dealloc(tbase, 512);
    return;
  }

  // Item n of the ring: wait until it is handed out / give it back.
  auto item_wait = [&](int n) { return warp_wait(bar(L::B_IF + n % kItems), (n / kItems) & 1, abort_flag); };
  auto item_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(L::B_IE + n % kItems));
  };

  if (warp == 11) {
    // ------------------------------------------------------------ walker
    regs_dec<kOtherRegs>();
    const int64_t w0 = shares.start(c), w1 = shares.start(c + 1);
    Walker<TL> w;
    w.find(p, (int)found[0], found[1], found[2], w0);
    int n = 0, qhalf = 1, kt = 0;
    for (bool more = true;;) {
      int ta = 0, tb = 0;
      bool got = false;
      while (more && !got) {
        if (w.start >= w1) more = false;
        else if (!w.portion(w0, w1, ta, tb)) more = w.next(p);
        else if (w.it.nt == 0) {
          // no row of the item sees a key
          for (int x = lane; x < w.it.rv * (D / 8); x += 32) {
            __nv_bfloat16* row = O + p.query_row(w.q.row0, w.h, w.it.r0 + x / (D / 8)) * D;
            *reinterpret_cast<uint4*>(row + 8 * (x % (D / 8))) = make_uint4(0, 0, 0, 0);
          }
          more = w.next(p);
        } else {
          got = true;
        }
      }
      if (n >= kItems && !warp_wait(bar(L::B_IE + n % kItems), ((n / kItems) - 1) & 1, abort_flag)) break;
      const bool whole = ta == 0 && tb == w.it.nt;
      const int slot = whole ? -1 : 2 * c + (n > 0);
      const int paired = w.it.rv <= p.half;
      qhalf = paired ? 1 - qhalf : 1;          // half items alternate the two query tiles
      if (lane == 0) {
        TileItem& to = items[n % kItems];
        to.live = got;
        to.s = w.s;
        to.h = w.h;
        to.row0 = w.q.row0;
        to.r0 = w.it.r0;
        to.rv = w.it.rv;
        to.p0 = w.it.p0;
        to.lo = w.it.lo;
        to.hi = w.it.hi;
        to.t0 = w.it.t0 + ta;
        to.n = tb - ta;
        to.slot = slot;
        to.paired = paired;
        to.qhalf = qhalf;
        to.kt = kt;
        const int p_first = w.it.p0 + p.by_group.div(w.it.r0);
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const int first = paired ? 0 : st * p.half;
          to.rows[st] = min(p.half, w.it.rv - first);
          to.steps[st] = paired ? (tb - ta - st + 1) / 2 : tb - ta;
          auto& e = to.edge[st];
          const int r_first = w.it.r0 + first, r_last = r_first + to.rows[st] - 1;
          edge_range(w.it.p0 + p.by_group.div(r_first), w.it.p0 + p.by_group.div(r_last), p.window, to.t0, e.mask_from,
                     e.mask_to);
          edge_range(p_first, w.it.hi - 1, p.window, to.t0, e.screen_from, e.screen_to);
        }
        if (got && !whole && ta == 0)
          ws.desc[c] = Desc{w.start, shares, 1, slot, w.it.unit, w.it.nt, w.q.row0, w.it.r0, w.it.rv, w.h};
        mbar_arrive(bar(L::B_IF + n % kItems));
      }
      __syncwarp();
      if (!got) break;
      ++n;
      kt += tb - ta;
      more = w.next(p);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ producer
    regs_dec<kOtherRegs>();
    const int page = 1 << p.page_shift;
    const int boxes = (128 >> p.page_shift) * NH;    // of a whole tile
    const int pi = lane / NH, hf = lane % NH;
    const uint32_t box_bytes = (uint32_t)page * 128u;
    int seq = 0;                               // slots filled
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const TileItem it = items[n % kItems];
      item_done(n);
      if (!it.live) break;
      // the pages of a tile are looked up one tile ahead (nothing looks at the
      // loaded id before its tile's turn, so the load is not waited for)
      const int32_t* row = p.table + (size_t)it.s * p.max_pages;
      auto in_span = [&](int t) {
        const int key = (it.t0 + t) * 128 + pi * page;
        return t < it.n && lane < boxes && key < it.hi && key + page > it.lo;
      };
      int id_next = in_span(0) ? row[(it.t0 * 128 + pi * page) >> p.page_shift] : 0;
      for (int t = 0; ok && t < it.n; ++t) {
        const bool mine = in_span(t);
        const int id = id_next;
        if (in_span(t + 1)) id_next = row[((it.t0 + t + 1) * 128 + pi * page) >> p.page_shift];
        // behind the pool: the box is filled with zeros
        const int outer = id >= 0 && id < p.P ? id * p.Hkv + it.h : p.P * p.Hkv;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * box_bytes;
        for (int kv = 0; kv < 2; ++kv) {
          const int s = seq % NS;
          if (!warp_wait(bar(L::B_KE + s), ((seq / NS) & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_expect_tx(bar(L::B_KF + s), bytes);
          __syncwarp();
          if (mine)
            tma_load_3d(sb + L::kRing + s * kTile + hf * kSpan + pi * box_bytes, kv ? &tmV : &tmK, 64 * hf, 0, outer,
                        bar(L::B_KF + s));
          ++seq;
        }
      }
    }
    if (*abort_flag)                           // let the loads in flight land before the CTA goes away
      for (int q = seq > NS ? seq - NS : 0; q < seq; ++q) drain_wait(bar(L::B_KF + q % NS), (q / NS) & 1);
  } else if (warp == 10) {
    // ------------------------------------------------------------ query loader
    regs_dec<kOtherRegs>();
    // A tile of many tokens is one box per 64 channels (rows of other requests
    // behind this one's may come along: a row of S depends on its own row of Q
    // alone, and they are not stored).  A tile of few tokens (decoding) takes
    // its tokens one by one and keeps the other rows zero: the MMAs multiply
    // them all the same, and with zeros the tensor cores draw so much less
    // power that a long run of decoding steps holds a higher clock.  Measured
    // on 128 sequences of up to 8192 keys in such a run, 32 / 8 heads: 401 -> 380 us
    // with 1 token a tile, 403 -> 389 with 4, 441 -> 416 with 5, 455 -> 441
    // with 16, 475 either way with 32.  Against that stand the loads of short
    // batches (16 sequences of 2000 keys): 44 -> 46 us with 4 tokens, 45 -> 47
    // with 16.  The limit of 4 is single tokens and short drafts.
    int loads = 0;                             // bit h: parity of the loads of query tile h
    int dirty[2] = {0, 0};                     // rows of each tile that may not be zero
    bool ok = warp_wait(bar(L::B_QZ), 0, abort_flag);
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const TileItem& it = items[n % kItems];
      if (!it.live) break;
      const int first = it.row0 + p.by_group.div(it.r0), paired = it.paired, qhalf = it.qhalf, head = it.h * p.group;
      const int rows0 = it.rows[0], rows1 = it.rows[1];
      item_done(n);
#pragma unroll
      for (int hx = 0; hx < 2; ++hx) {
        if (paired && hx != qhalf) continue;
        if (!warp_wait(bar(L::B_QE + hx), ((loads >> hx) & 1) ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        loads ^= 1 << hx;
        const int rows = paired || hx == 0 ? rows0 : rows1, tokens = p.by_group.div(rows);
        const int tok = first + (paired ? 0 : hx * p.by_group.div(p.half));
        if (tokens <= kFewTokens) {
          for (int x = rows * 8 + lane; x < dirty[hx] * 8; x += 32)
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
              *reinterpret_cast<uint4*>(smem + hx * kTile + hf * kSpan + 16 * x) = make_uint4(0, 0, 0, 0);
          if (dirty[hx] > rows) fence_async();
          dirty[hx] = rows;
          __syncwarp();
          if (lane == 0) {
            mbar_expect_tx(bar(L::B_QF + hx), (uint32_t)(rows * D * 2));
            for (int k = 0; k < tokens; ++k)
#pragma unroll
              for (int hf = 0; hf < NH; ++hf)
                tma_load_3d(sb + hx * kTile + hf * kSpan + k * p.group * 128, &tmQ1, 64 * hf, head, tok + k,
                            bar(L::B_QF + hx));
          }
        } else {
          dirty[hx] = p.half;
          if (lane == 0) {
            mbar_expect_tx(bar(L::B_QF + hx), (uint32_t)(p.half * D * 2));
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
              tma_load_3d(sb + hx * kTile + hf * kSpan, &tmQ, 64 * hf, head, tok, bar(L::B_QF + hx));
          }
        }
        __syncwarp();
      }
    }
    if (*abort_flag)                           // a completed load's wait returns at once
      for (int hx = 0; hx < 2; ++hx) drain_wait(bar(L::B_QF + hx), ((loads >> hx) & 1) ^ 1);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    // Step x of an item belongs to stream x & 1: two steps per key tile, or
    // one per tile (paired), with a dummy that makes their number even.
    regs_dec<kOtherRegs>();
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t idO = idesc_bf16_f32(128, D, 0, 1);
    // Up to 16 rows (most decoding) take M = 64, whose first 16 rows lie in the
    // same TMEM lanes as those of M = 128: half the multiplications by zero,
    // for the power that they draw (410 -> 387 us, as kFewTokens above)
    constexpr uint32_t idS64 = idesc_bf16_f32(64, 128, 0, 0), idO64 = idesc_bf16_f32(64, D, 0, 1);
    // score cursor: step x of nx of item a, the K slot and its phase
    int a = -1, x = 0, nx = 0, n_a = 0, paired_a = 0, small_a = 0, qh_a = 0, ks = 0, kph = 0;
    int qf = 0, pr = 0, drained = 0;           // bit h / st: parity of the barrier's next completion
    bool end = false;
    auto score_step = [&]() -> bool {          // false on abort; does nothing behind the last item
      if (end) return true;
      if (x == nx) {
        ++a;
        if (!item_wait(a)) return false;
        const TileItem& it = items[a % kItems];
        if (!uniform(it.live)) {
          end = true;
          return true;
        }
        x = 0;
        n_a = uniform(it.n);
        paired_a = uniform(it.paired);
        small_a = uniform(it.rv) <= 16;
        qh_a = uniform(it.qhalf);
        nx = paired_a ? (n_a + 1) / 2 * 2 : 2 * n_a;
      }
      const int st = x & 1;
      if (!paired_a || x < n_a) {
        const int half = paired_a ? qh_a : st;
        if (paired_a ? x == 0 : x < 2) {       // the first step on this query tile
          if (!warp_wait(bar(L::B_QF + half), (qf >> half) & 1, abort_flag)) return false;
          qf ^= 1 << half;
        }
        // (a tile that both streams use was waited for by stream 0's step)
        if ((paired_a || st == 0) && !warp_wait(bar(L::B_KF + ks), kph, abort_flag)) return false;
        tc_fence_after();
        const uint64_t qd = desc_sw128(sb + half * kTile, 16, 1024);
        const uint64_t kd = desc_sw128(sb + L::kRing + ks * kTile, 16, 1024);
        const uint32_t d = tbase + (uint32_t)st * 128;
        mma_scores<D>(d, qd, kd, small_a ? idS64 : idS);
        mma_commit_w(bar(L::B_SF + st));
        if (paired_a || st == 1) {             // the last use of this K tile
          mma_commit_w(bar(L::B_KE + ks));
          ks += 2;
          if (ks >= NS) {
            ks -= NS;
            kph ^= 1;
          }
        }
        if (paired_a ? x == n_a - 1 : x >= nx - 2) mma_commit_w(bar(L::B_QE + half));
      }
      ++x;
      return true;
    };
    int vs = 1, vph = 0;
    bool ok = score_step() && score_step();
    for (int b = 0; ok; ++b) {
      if (!item_wait(b)) break;
      const TileItem& itb = items[b % kItems];
      if (!uniform(itb.live)) break;
      const int n_b = uniform(itb.n), paired_b = uniform(itb.paired), small_b = uniform(itb.rv) <= 16;
      const int real = paired_b ? n_b : 2 * n_b, ny = (real + 1) / 2 * 2;
      for (int y = 0; y < ny; ++y) {
        const int st = y & 1;
        if (y < real) {
          if (y < 2) {                         // this stream's O of an earlier item is read
            if (!warp_wait(bar(L::B_OF + st), ((drained >> st) & 1) ^ 1, abort_flag)) { ok = false; break; }
            drained ^= 1 << st;
          }
          if (!warp_wait(bar(L::B_PR + st), (pr >> st) & 1, abort_flag)) { ok = false; break; }
          pr ^= 1 << st;
          if ((paired_b || st == 0) && !warp_wait(bar(L::B_KF + vs), vph, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t vd = desc_sw128(sb + L::kRing + vs * kTile, kSpan, 1024);
          const uint32_t pa = tbase + (uint32_t)st * 128, od = tbase + kColO + (uint32_t)st * 128;
          mma_values(od, pa, vd, small_b ? idO64 : idO, y >= 2);
          if (paired_b || st == 1) {           // the last use of this V tile
            mma_commit_w(bar(L::B_KE + vs));
            vs += 2;
            if (vs >= NS) {
              vs -= NS;
              vph ^= 1;
            }
          }
          if (y + 2 >= real) mma_commit_w(bar(L::B_OD + st));   // the stream's last step of the item
        }
        // the scores overwrite this stream's P, whose product was issued before
        if (!score_step()) { ok = false; break; }
      }
      item_done(b);
    }
    // every MMA issued above has completed before TMEM is released
    mma_commit_w(bar(L::B_FIN));
    drain_wait(bar(L::B_FIN), 0);
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<kSoftmaxRegs>();
    const int st = warp >> 2, wq = warp & 3, wr = wq * 32 + lane;
    // the query tiles start as zeros (the line that lay there is read)
    for (int x = threadIdx.x - 128; x < (int)(2 * kTile / 16); x += 256)
      reinterpret_cast<uint4*>(smem)[x] = make_uint4(0, 0, 0, 0);
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(L::B_QZ));
    const uint32_t lrow = tbase + ((uint32_t)(wq * 32) << 16);
    const uint32_t s_col = (uint32_t)st * 128, o_col = kColO + (uint32_t)st * 128;
    const bool wide = (reinterpret_cast<uintptr_t>(O) & 31) == 0;
    float* ex = reinterpret_cast<float*>(smem + L::kExOff);   // [2][128]: stream 1's maxima, sums
    int sf = 0, od = 0, exp_ = 0;              // parities of the next completions
    // the last key that this thread's row sees (of the item's last row for a thread without one)
    auto row_last = [&](const TileItem& it) {
      const int r = wr < it.rows[st] ? (it.paired ? 0 : st * p.half) + wr : it.rv - 1;
      return it.p0 + p.by_group.div(it.r0 + r);
    };
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const TileItem& it = items[n % kItems];
      if (!it.live) {
        item_done(n);
        break;
      }
      const int U = it.steps[st];              // this stream's steps
      const bool live_warp = wq * 32 < it.rows[st], mine = wr < it.rows[st];
      float m_used = -INFINITY, l = 0.f;
      for (int u = 0; u < U; ++u) {
        const int t = it.paired ? 2 * u + st : u;
        const bool screen = t >= it.edge[st].screen_from || t < it.edge[st].screen_to;
        const bool mask = t >= it.edge[st].mask_from || t < it.edge[st].mask_to;
        // S is complete, and with it the product P V before it
        if (!warp_wait(bar(L::B_SF + st), sf, abort_flag)) { ok = false; break; }
        sf ^= 1;
        if (screen) {
          // screen the V tile: thread wr takes row wr
          const int seq = 2 * (it.kt + t) + 1, s = seq % NS, key = (it.t0 + t) * 128 + wr;
          if (!warp_wait(bar(L::B_KF + s), (seq / NS) & 1, abort_flag)) { ok = false; break; }
          uint8_t* vrow = smem + L::kRing + s * kTile + wr * 128;
          auto chunk16 = [&](int j) {
            return reinterpret_cast<uint4*>(vrow + (j >> 3) * kSpan + (((j & 7) ^ (wr & 7)) << 4));
          };
          if (key < it.lo || key >= it.hi) {
#pragma unroll
            for (int j = 0; j < 8 * NH; ++j) *chunk16(j) = make_uint4(0, 0, 0, 0);
          } else {
            // an exponent of all ones carries into the half's top bit
            uint32_t hit = 0;
#pragma unroll
            for (int j = 0; j < 8 * NH; ++j) {
              const uint4 y = *chunk16(j);
              hit |= ((y.x & kExpBits) + kExpStep) | ((y.y & kExpBits) + kExpStep) | ((y.z & kExpBits) + kExpStep) |
                     ((y.w & kExpBits) + kExpStep);
            }
            if (hit & 0x80008000u) {
              *unbounded_flag = 1;             // before the values go
              __threadfence_block();
#pragma unroll 1
              for (int j = 0; j < 32 * NH; ++j) {
                uint32_t* w = reinterpret_cast<uint32_t*>(chunk16(j >> 2)) + (j & 3);
                const uint32_t top = ((*w & kExpBits) + kExpStep) & 0x80008000u;
                *w &= ~((top >> 15) * 0xffffu);
              }
            }
          }
          fence_async();
        }
        if (live_warp) {
          tc_fence_after();
          uint32_t v[128];
          float sum = 0.f, factor = 1.f;
          bool need = false;
          // v[e] = the pair e of exponentials as bf16, their sum in sm8
          auto exps = [&](int from, int to, float ng, float (&sm8)[8]) {
#pragma unroll
            for (int e = from; e < to; ++e) {
              float a0, a1;
              ffma2(a0, a1, __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]), scale2, scale2, ng, ng);
              const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
              fadd2(sm8[2 * (e & 3)], sm8[2 * (e & 3) + 1], p0, p1);
              v[e] = pack_bf16(p0, p1);
            }
          };
          auto add8 = [](const float (&x)[8]) {
            return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
          };
          // The maximum only keeps the exponentials in range, and a stale one
          // does as long as the tile's exponentials sum to less than 2^16.  So
          // the tile's own maximum is formed for a row's first keys, for masked
          // tiles and when that check fails (as it does for NaN and inf), and
          // otherwise the exponentials of a quarter of the row run while the
          // next quarter comes from TMEM (6% of the kernel).  Where the check
          // fails in every tile (scores that rise by 12 binary orders each 128
          // keys) the second pass makes the chunk of 4096 rows over 16001 keys
          // 36% slower and decoding 64 sequences 19%.  All exponentials run
          // on MUFU: a share of 1/8 or 3/8 on the FMA pipe, as the block-sparse
          // kernel has, cost 1 and 3%, since the MMA issuer shares that pipe's
          // scheduler.
          bool fresh = mask || __any_sync(0xffffffffu, mine && m_used == -INFINITY);
          if (!fresh) {
            float sm8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            tmem_ld32(lrow + s_col, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k < 3) tmem_ld32(lrow + s_col + 32 * (k + 1), *reinterpret_cast<uint32_t(*)[32]>(&v[32 * (k + 1)]));
              if (mine) exps(16 * k, 16 * k + 16, -m_used, sm8);   // (lanes without a row rest)
              if (k < 3) tmem_wait_ld();
            }
            sum = add8(sm8);
            fresh = !__all_sync(0xffffffffu, sum < kStaleSum || !mine);
          }
          if (fresh) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tmem_ld32(lrow + s_col + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(&v[32 * k]));
            tmem_wait_ld();
            if (mask) {
              const int hi = row_last(it) - (it.t0 + t) * 128, lo = p.window > 0 ? hi - p.window + 1 : 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // the columns 32 k + n that the row sees, bit n
                const int h = hi - 32 * k, w = lo - 32 * k;
                const uint32_t seen = (h >= 31 ? ~0u : h < 0 ? 0u : (2u << h) - 1u) &
                                      (w <= 0 ? ~0u : w > 31 ? 0u : ~0u << w);
                if (__all_sync(0xffffffffu, seen == ~0u)) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((seen >> e) & 1u)) v[32 * k + e] = __float_as_uint(-INFINITY);
              }
            }
            float mx8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 64; ++e)
              mx8[e & 7] = fmax3_nan(mx8[e & 7], __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
            const float mx = fmax3_nan(fmax3_nan(mx8[0], mx8[1], mx8[2]), fmax3_nan(mx8[3], mx8[4], mx8[5]),
                                       fmax3_nan(mx8[6], mx8[7], mx8[7]));
            // a score that is NaN or +inf makes the row NaN (as inf - inf does),
            // whether q.k is so or the scale takes it there
            const float top = mx * scale2, m_tile = top < INFINITY ? top : NAN;
            need = !(m_tile <= m_used + kLazy);
            if (need) {
              factor = fast_exp2(m_used - m_tile);
              m_used = m_tile;
            }
            float sm8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (mine) exps(0, 64, m_used == -INFINITY ? 0.f : -m_used, sm8);   // no key seen yet: p = 2^-inf = 0
            sum = add8(sm8);
          }
          l = l * factor + sum;
          tmem_st32(lrow + s_col, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_st32(lrow + s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          if (u >= 1 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              uint32_t o[32];
              tmem_ld32(lrow + o_col + 32 * k, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
              tmem_st32(lrow + o_col + 32 * k, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_PR + st));
      }
      if (!ok) break;
      if (U > 0) {
        if (!warp_wait(bar(L::B_OD + st), od, abort_flag)) break;
        od ^= 1;
        tc_fence_after();
      }
      const bool paired = it.paired;
      if (paired && st == 1) {
        // hand the state to stream 0 (which gives back O_1)
        if (U > 0) {
          ex[wr] = m_used;
          ex[128 + wr] = l;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::B_EX));
        }
        item_done(n);
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      const bool merge = paired && it.steps[1] > 0;
      if (merge) {
        if (!warp_wait(bar(L::B_EX), exp_, abort_flag)) break;
        exp_ ^= 1;
        tc_fence_after();
        const float m1 = ex[wr], l1 = ex[128 + wr];
        const float M = m_used < m1 || m1 != m1 ? m1 : m_used;     // NaN if either is
        const float base = M == -INFINITY ? 0.f : M;
        f0 = fast_exp2(m_used - base);
        f1 = fast_exp2(m1 - base);
        l = l * f0 + l1 * f1;
        m_used = M;
      }
      const int slot = it.slot, r = (paired ? 0 : st * p.half) + wr;
      const bool whole = slot < 0;
      const float inv = !whole ? 1.f : (l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l));
      __nv_bfloat16* orow = O + p.query_row(it.row0, it.h, it.r0 + r) * D;
      if (live_warp) {
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          // rolled, as the other loops off the tiles' path: code that is not
          // there does not push the tiles' out of the instruction caches (5%)
          uint32_t x[32], y[32];
          tmem_ld32(lrow + o_col + 32 * k, x);
          if (merge) tmem_ld32(lrow + kColO + 128 + 32 * k, y);
          tmem_wait_ld();
          float z[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            z[e] = __uint_as_float(x[e]) * f0;
            if (merge) z[e] = fmaf(__uint_as_float(y[e]), f1, z[e]);
            z[e] *= inv;
          }
          if (!mine) continue;
          if (whole) {
            uint32_t u[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) u[q] = pack_bf16(z[2 * q], z[2 * q + 1]);
            store64(orow + 32 * k, u, wide);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              ws.chunk<D>(slot, 8 * k + q)[r] = make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
          }
        }
        if (mine && !whole) ws.state(slot)[r] = make_float2(m_used, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (merge) mbar_arrive(bar(L::B_OF + 1));
        mbar_arrive(bar(L::B_OF + st));
      }
      if (*unbounded_flag && mine) {
        const int p_first = it.p0 + p.by_group.div(it.r0), last = row_last(it);
        if (whole) add_unbounded(p, it.s, it.h, it.t0, it.n, p_first, it.hi, Vc, D, last, orow, 4);
        else
          add_unbounded(p, it.s, it.h, it.t0, it.n, p_first, it.hi, Vc, D, last,
                        reinterpret_cast<float*>(ws.chunk<D>(slot, 0) + r), 4 * ws.rows_cap);
      }
      item_done(n);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
sa_status launch(const CUtensorMap& mq, const CUtensorMap& mq1, const CUtensorMap& mk, const CUtensorMap& mv,
                 const void* Vc, const Params& p, float scale, void* O, const Workspace& ws, cudaStream_t stream) {
  auto kern = paged_attn_tc_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<D>::smem_bytes) != cudaSuccess)
    return launch_status("cudaFuncSetAttribute(paged_attn_tc_kernel)");
  const cudaError_t le =
      launch_pdl(kern, dim3(ws.ctas), dim3(kThreads), Lay<D>::smem_bytes, stream, mq, mq1, mk, mv,
                 static_cast<const __nv_bfloat16*>(Vc), p, scale * kLog2e, static_cast<__nv_bfloat16*>(O), ws);
  if (le != cudaSuccess) return fail(SA_ERR_CUDA, std::string("paged_attn_tc_kernel: ") + cudaGetErrorString(le));
  return launch_status("paged_attn_tc_kernel");
}

}  // namespace

sa_status paged_attn_tc(const void* Q, int64_t q_stride, const void* Kc, const void* Vc, const sa_paged_shape& s,
                        const paged::Params& p, float scale, void* O, const paged::Workspace& ws,
                        cudaStream_t stream) {
  CUtensorMap mq, mq1, mk, mv;
  uint64_t outer = (uint64_t)s.P * s.Hkv;
  if (p.max_pages == 0) {
    // no pages: every length reads as 0 and nothing is loaded through the maps
    Kc = Vc = ws.o;
    outer = 1;
  }
  if (s.T == 1) q_stride = (int64_t)s.Hq * s.d;   // a single row has no stride
  const uint64_t page_elems = (uint64_t)s.d * s.page;
  if (!make_tmap_bf16_3d(&mq, Q, s.d, s.Hq, s.T, s.d, q_stride, 64, p.group, p.half / p.group) ||
      !make_tmap_bf16_3d(&mq1, Q, s.d, s.Hq, s.T, s.d, q_stride, 64, p.group, 1) ||
      !make_tmap_bf16_3d(&mk, Kc, s.d, s.page, outer, s.d, page_elems, 64, s.page, 1) ||
      !make_tmap_bf16_3d(&mv, Vc, s.d, s.page, outer, s.d, page_elems, 64, s.page, 1))
    return fail(SA_ERR_CUDA, "sa_paged_attn_fwd: cuTensorMapEncodeTiled failed for Q and the caches");
  return s.d == 128 ? launch<128>(mq, mq1, mk, mv, Vc, p, scale, O, ws, stream)
                    : launch<64>(mq, mq1, mk, mv, Vc, p, scale, O, ws, stream);
}

uint32_t paged_tc_error_take() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, tc::g_device_error, sizeof(v)) != cudaSuccess ||
      cudaMemcpyToSymbol(tc::g_device_error, &zero, sizeof(zero)) != cudaSuccess)
    return 0;
  return v;
}

}  // namespace sa
