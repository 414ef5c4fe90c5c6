// Attention of many new tokens over a paged KV cache held in 8 bits on the tcgen05 tensor cores: prompts, chunks of
// prompts, and batches that mix them with decode steps.
//
//   x_t = log2(e) / sqrt(d) s_k(t) q . c_k(t),   o = sum_t 2^x_t s_v(t) c_v(t) / sum_t 2^x_t,   lse = ln sum_t 2^x_t,
//
// c the e4m3 codes of slot t, s_k and s_v the scales of its block of 16 slots. Tiles, items, their cut along the cached
// tokens and the join are those of 16-bit caches (kv_attend_tc.cu); what comes between the cache and the products:
//   * The loaders bring 128 cached tokens' codes by TMA (boxes of a page's tokens) and, with the keys', the tile's 16
//     scales by cp.async, into a ring of code tiles. What lies behind a row's length comes too: it changes nothing, as
//     its scores are masked and its values' codes are replaced by zeros.
//   * A third warpgroup turns code tiles into fp16 tiles, exactly, in the layout that the products read (128-byte
//     swizzle). All products are fp16: bf16 queries are lifted to it in place by the softmax warps when they
//     arrive, each row by a power of two of its own.
//   * s_k multiplies 16 scores of a thread's row at once. With y_t = x_t + log2 s_v(t) and a running maximum of y, the
//     weights 2^(y_t - M) are what c_v is multiplied by, and the sum takes them divided by s_v: one exponential
//     serves both, and the fp16 weights are relative to the largest that enters the product, whatever the scales.
// Bound: the softmax warps' chain from scores to weights to the next scores, of a step for two tiles about 2800 clocks, of which
// the products (four of 128 x 128 x 128) need 2048, and what of the converters does not hide behind it: 2048 new tokens at 65536,
// 8 heads of 128, 4 query rows each, 1604 us and 1.35 of 1.87 PFLOP/s; four prompts of 4096, 32 heads, 535 us. Each instruction counts,
// also in the instruction caches, which the roles share: scales held over a step, inverse scales from the converters, three-way
// maxima, packed sums, and one loop each for loads and products took these from 1783 and 578 (to 1590 and 535; bounds of the
// scores' factors, see kv8.h, take 14 again). Not kept: without the maximum
// ahead of the weights (raised afterwards where 16 weights' sum had left fp16) steps were no shorter, and first ones twice as
// long (806 us for the prompts, against 578); the units' softmax by turns on each scheduler (1831 against 1641, 575 against
// 554); queries loaded behind the next item's first keys (592 against 578).
// A product straight on the codes (kind::f8f6f4) would want the queries and weights in 8 bits too, in two or three terms
// each to keep their precision: as many products as in fp16, and the weights' terms in the softmax, which bounds the
// kernel already.
//
// Pairs (heads of 128, see launch_kv8_attend_tc): two CTAs of a cluster, on neighbouring SMs, share each step's keys and values.
//   * A product then has 256 query rows (tcgen05, cta_group::2), 128 of either CTA. Each holds its own queries, scores,
//     weights and outputs, and half of the other operand: of a step's 128 keys the 64 of its rank, of the values' 128
//     columns 64. So it loads, converts, keeps and reads half of what it would alone for as many products; alone, the
//     converters and the products' operands together keep the shared memory's ports busy.
//   * The first CTA takes the items and hands their numbers to the other. Its MMA warp issues all products, when both
//     CTAs' tiles, weights and queries say so at its barriers; what they complete arrives at the barriers of both.
//   * Whatever happened, the two meet before they end: neither's shared or tensor memory is gone while the other's arrivals
//     or products may still come.
//
// Every wait is bounded; one that gives up records PALU_ERR_TIMEOUT, and all roles wait for their own
// copies and products in flight before tensor memory is freed.
#include "kv8.h"
#include "kv_tc_items.cuh"

namespace palu {
namespace {

constexpr int kThreads = 512;            // two softmax warpgroups; two loader warps, MMA and an idle warp; converters
constexpr int kBlocks = kTile / kKv8Block;

template <int DH, bool PAIR> struct Lay {
  // Registers: launched with 128 a thread; 256 softmax + 128 other + 128 convert = 512 * 128. 2048 tokens at 32768, 32 / 8
  // heads, in bf16 and fp16: 808 and 823 us; with 208, 48 and 48 830 and 828; 184, 72 and 72 836 and 846; with 200, 56 and 56 809
  // and 817, but loaders that are short of registers: 16 tokens of 16 rows at 4096, pages of 64, take 67 us against 58.
  static constexpr int kRegsSoftmax = 192, kRegsOther = 64, kRegsConvert = 64;
  // Query tiles: 64 elements (128 bytes) of all rows, then the next 64. fp16 and code tiles hold the CTA's part: keys as the
  // queries (of a pair's CTA 64 tokens), values by 64 columns of all tokens. Rows of 128 bytes are swizzled.
  static constexpr int kHalf = kTile * 128;             // 64 elements of 128 rows
  static constexpr int kTileB = kHalf * (DH / 64);
  static constexpr int kParts = PAIR ? 2 : 1;           // CTAs that share a tile of keys or values
  static constexpr int kStageB = kTileB / kParts, kKeyHalf = kHalf / kParts;
  static constexpr int kCodeB = kTile * DH / kParts;
  static constexpr int kStages = PAIR ? 6 : DH == 128 ? 3 : 5;   // fp16 tiles
  static constexpr int kCodes = PAIR ? 7 : DH == 128 ? 4 : 8;    // code tiles
  // Scales of key tiles in use. A tile's are written when its place in the ring of kStages tiles is free, and all
  // tiles whose values' products had not ended then count: of the kStages - 1 places before it, and of the values up to
  // three places behind their keys, at most kStages / 2 + 2.
  static constexpr int kScales = DH == 128 && !PAIR ? 4 : 8;
  static constexpr int kOffKv = 2 * kTileB;             // behind two query tiles
  static constexpr int kOffCode = kOffKv + kStages * kStageB;
  static constexpr int kOffBar = kOffCode + kCodes * kCodeB;
  static constexpr int kShared = DH == 128 && !PAIR ? 2048 : 4096;   // barriers, items, scales, lifts
  static constexpr int kSmem = kOffBar + kShared + 1024;    // and alignment
  static constexpr uint32_t kColO = 2 * kTile;          // tensor memory: S (and P) of the units, then O
  static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
};

// a code tile, for the converters: its tokens that are below the row's length, and what it is
struct Info {
  int valid, kind;                        // kind: kKeys, kValues or kEnd
};
constexpr int kKeys = 0, kValues = 1, kEnd = 2;
constexpr int kScaleLanes = 2 * kBlocks;  // lanes that load a key tile's scales

template <int DH, bool PAIR> struct Shared {
  using Y = Lay<DH, PAIR>;
  // of a pair: at the first CTA, from both: full, q_ready, p_full, idx_empty; at both, from the first one's products: empty,
  // q_empty, s_full, o_full, drained; the others from the CTA itself
  uint64_t full[Y::kStages], empty[Y::kStages], code_full[Y::kCodes], code_empty[Y::kCodes], scale_full[Y::kScales];
  uint64_t q_full, q_ready, q_empty, lift_full, x_full, drained;
  uint64_t s_full[2], o_full[2], p_full[2][2];
  uint64_t item_full[2], item_empty[2], idx_full[2], idx_empty[2];
  int idx[2];                             // items' numbers, from the pair's first CTA
  Item item[2];
  Plan plan;
  Info info[Y::kCodes];
  unsigned cut;                           // pieces of cut tiles that this CTA has taken
  uint32_t tmem;
  int abort_flag;
  float raw[Y::kCodes][2][kBlocks];       // scales of keys and values, as they arrive
  float2 scale[Y::kScales][kBlocks];      // s_k and log2 s_v
  float2 part[Y::kScales][kBlocks];       // 1 / s_v, twice
  float lift[kTile];                      // of the queries' rows where both units share a tile
};
template <int DH, bool PAIR> constexpr bool fits = sizeof(Shared<DH, PAIR>) <= Lay<DH, PAIR>::kShared;
static_assert(fits<128, false> && fits<64, false> && fits<128, true>, "shared block");
static_assert(sizeof(JoinShared) <= 2 * Lay<64, false>::kTileB, "in the queries' space");

struct Tc8Params {
  TcParams P;
  const float* k_scale;
  const float* v_scale;
};

// 4 bytes global -> shared; bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp4(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
// this thread's copies so far arrive at the barrier when they have landed
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_addr(bar)), "r"(n) : "memory");
}

// two columns of this warp's lanes of tensor memory
__device__ __forceinline__ void tmem_st2(uint32_t ta, float a, float b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(ta), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float2 tmem_ld2(uint32_t ta) {
  float2 v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\ntcgen05.wait::ld.sync.aligned;"
               : "=f"(v.x), "=f"(v.y)
               : "r"(ta)
               : "memory");
  return v;
}

// Lifts a row of bf16 queries, as TMA left it (two halves of 64 elements, 128-byte swizzle), to fp16 in place.
template <int DH> __device__ __forceinline__ float lift_row(uint8_t* tile, int r) {
  auto at = [&](int c) -> uint4* {
    return reinterpret_cast<uint4*>(tile + c / 8 * (kTile * 128) + r * 128 + ((c % 8 ^ (r & 7)) << 4));
  };
  __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) {
    const uint4 v = *at(c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
  }
  const float lift = lift_of(fmaxf(__low2float(top), __high2float(top)));
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) {
    const uint4 v = *at(c);
    *at(c) = make_uint4(lifted(v.x, lift), lifted(v.y, lift), lifted(v.z, lift), lifted(v.w, lift));
  }
  return lift;
}

// ------------------------------------------------------------------------------------------- of a pair
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t at_cta(const void* p, uint32_t rank) {   // the same place of a CTA of the cluster
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_peer(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(at_cta(bar, rank)) : "memory");
}
// For what lies in tensor memory alone (scores read, weights written). PTX orders those by tcgen05's own fences, whatever the
// arrival's semantics: fence::before_thread_sync puts the warp's tcgen05 operations, which it has waited for, ahead of the
// arrival, and fence::after_thread_sync the products behind the wait. No ordinary memory is handed over here: places of scales
// are written anew three key tiles or more behind the last that reads them. With release the softmax warps waited 1000 clocks.
__device__ __forceinline__ void arrive_peer_relaxed(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(at_cta(bar, rank)) : "memory");
}
__device__ __forceinline__ void st_peer(int* p, int v, uint32_t rank) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_cta(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// tc::mbar_wait_short, with the cluster's order
__device__ __forceinline__ bool wait_pair(uint64_t* b, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, "
        "p;\n}\n"
        : "=r"(ok)
        : "r"(tc::smem_addr(b)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    const uint64_t t = tc::globaltimer();
    if (t0 == 0) {
      t0 = t;
    } else if (t - t0 > limit_ns) {
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_addr(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t base, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// the products issued so far arrive at the barrier of both CTAs
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_addr(bar)),
      "h"(uint16_t(3))
      : "memory");
}
template <bool PAIR> __device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR) commit_pair(bar);
  else tc::umma_commit(bar);
}

// ------------------------------------------------------------------------------------------- attend
template <int DH, bool BF16, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const Tc8Params P8) {
  using Y = Lay<DH, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared<DH, PAIR>& S = *reinterpret_cast<Shared<DH, PAIR>*>(smem + Y::kOffBar);
  volatile int* abort_flag = &S.abort_flag;
  const TcParams& P = P8.P;                    // per_tile: of the rows of a product, 128 or 256
  const KvAttendArgs& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = PAIR ? (int)cta_rank() : 0;
  const int per = P.per_tile / Y::kParts;      // tokens of this CTA's rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < Y::kStages; ++i) {
      tc::mbar_init(&S.full[i], PAIR && rank == 0 ? 5 : 4);   // the converters; the other CTA's MMA warp
      tc::mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < Y::kCodes; ++i) {
      tc::mbar_init(&S.code_full[i], 1 + kScaleLanes);
      tc::mbar_init(&S.code_empty[i], 4);
    }
    for (int i = 0; i < Y::kScales; ++i) tc::mbar_init(&S.scale_full[i], 1);
    tc::mbar_init(&S.q_full, 1);
    tc::mbar_init(&S.q_ready, 8 * Y::kParts);  // the softmax warps have seen, and lifted, the queries
    tc::mbar_init(&S.lift_full, 4);
    tc::mbar_init(&S.q_empty, 1);              // the products that read the queries
    tc::mbar_init(&S.x_full, 4);
    tc::mbar_init(&S.drained, 1);
    for (int u = 0; u < 2; ++u) {
      tc::mbar_init(&S.s_full[u], 1);
      tc::mbar_init(&S.o_full[u], 1);
      for (int k = 0; k < 2; ++k) tc::mbar_init(&S.p_full[u][k], 4 * Y::kParts);
      tc::mbar_init(&S.item_full[u], 1);
      tc::mbar_init(&S.item_empty[u], 10);     // eight softmax warps, the MMA warp, the value loader
      tc::mbar_init(&S.idx_full[u], 1);
      tc::mbar_init(&S.idx_empty[u], 1);
    }
    S.abort_flag = 0;
    S.cut = 0;
    tc::fence_barrier_init();
  }
  if constexpr (PAIR) {                        // both CTAs' barriers are there
    __syncthreads();
    cluster_meet();
    if (warp == 9) tmem_alloc_pair(&S.tmem, 512);
  } else if (warp == 9) {
    tc::tmem_alloc(&S.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = S.tmem;
  grid_wait();                                 // for the plan
  grid_release();

  if (warp >= 12) {
    // ------------------------------------------------------------------ converters
    // 16 codes a lane and step; a warp takes a group of eight rows and 64 of their columns: eight lanes at a time rows a
    // and a ^ 5, whose 16-byte chunks lie in different banks both as codes (128-byte swizzle; rows of 64 bytes lie
    // so without one) and as fp16. All places are a thread's base and constants. Of a pair's tile a warp has 16 keys with
    // both halves of their columns, or 64 columns of 32 values.
    tc::regs_shrink<Y::kRegsConvert>();
    constexpr int kHalves = DH / 64, kEach = kTile / 8 * kHalves / 4 / Y::kParts;   // steps of a warp
    const int c = lane & 3, a7 = (lane >> 3) ^ (lane & 4 ? 5 : 0);       // a7: row of its group of eight
    const uint32_t from = DH == 128 ? uint32_t(a7 * 128 + ((c ^ a7) << 4)) : uint32_t(a7 * 64 + (c << 4));
    const uint32_t from_v = PAIR ? uint32_t(a7 * 64 + (c << 4)) : from;
    const uint32_t to = uint32_t(a7 * 128 + ((2 * c ^ a7) << 4));
    // the warp's first row of a tile of keys, or of values, which a pair's CTA holds by halves
    const int row_k = (warp - 12) * (kEach / kHalves) * 8, row_v = (warp - 12) * 32;
    const int tok_k = PAIR ? rank * 64 + row_k : row_k;
    int sc = 0, st = 0, n_k = 0;
    uint32_t par_c = 0, par = 1;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return __all_sync(0xffffffffu, tc::mbar_wait_short(bar, phase, abort_flag, P.wait_ns));
    };
    for (;;) {
      if (!wait(&S.code_full[sc], par_c)) break;
      const Info info = S.info[sc];
      if (info.kind == kEnd) break;
      const bool keys = info.kind == kKeys, whole = !PAIR || keys;      // rows of whole heads, or of 64 columns
      // the tile's codes are taken while its place is still read by products
      const uint8_t* src = smem + Y::kOffCode + sc * Y::kCodeB + (warp - 12) * (Y::kCodeB / 4);
      uint4 v[kEach];
#pragma unroll
      for (int x = 0; x < kEach; ++x)
        v[x] = *reinterpret_cast<const uint4*>(src + (whole ? x / kHalves * 8 * DH + (from ^ (x % kHalves * 64)) : x * 512 + from_v));
      if (info.valid != kTile) {
        const int valid = info.valid - (keys ? tok_k : row_v) - a7;    // of this thread's rows, those 8 x below it
#pragma unroll
        for (int x = 0; x < kEach; ++x)
          if ((whole ? x / kHalves : x) * 8 >= valid) v[x] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (!wait(&S.empty[st], par)) break;
      if (keys) {
        if (warp == 12) {
          if (lane < kBlocks) {
            const float s_v = scale_or_one(S.raw[sc][1][lane]);
            S.scale[n_k % Y::kScales][lane] = make_float2(scale_or_one(S.raw[sc][0][lane]), lg2(s_v));
            S.part[n_k % Y::kScales][lane] = make_float2(rcp(s_v), rcp(s_v));
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&S.scale_full[n_k % Y::kScales]);
        }
        ++n_k;
      }
      uint8_t* dst = smem + Y::kOffKv + st * Y::kStageB + (whole ? row_k : row_v) * 128;
#pragma unroll
      for (int x = 0; x < kEach; ++x) {
        const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
        uint32_t f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[2 * e] = f16_of_codes(uint16_t(w[e]));
          f[2 * e + 1] = f16_of_codes(uint16_t(w[e] >> 16));
        }
        uint8_t* at = dst + (whole ? x % kHalves * Y::kKeyHalf + x / kHalves * 1024 : x * 1024);
        *reinterpret_cast<uint4*>(at + to) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(at + (to ^ 16)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&S.full[st]);
        tc::mbar_arrive(&S.code_empty[sc]);
      }
      if (++sc == Y::kCodes) {
        sc = 0;
        par_c ^= 1;
      }
      if (++st == Y::kStages) {
        st = 0;
        par ^= 1;
      }
    }
  } else if (warp >= 8) {
    tc::regs_shrink<Y::kRegsOther>();
    if (warp == 8 || warp == 10) {
      // ------------------------------------------------------------------ loaders
      // Warp 8 takes the items and loads Q and K, warp 10 V. Both count every stage of the ring, in the order
      // in which the products take them: K runs one tile ahead of V, two where the units alternate. Copies are
      // issued by one lane with uniform operands.
      const bool keys = warp == 8;
      const CUtensorMap* map = keys ? &tm_k : &tm_v;
      Rows32 rows;
      Plan plan{};
      if (keys) {
        plan = plan_rows(P, rows, blockIdx.x == 0);
        if (lane == 0) S.plan = plan;        // the first item's arrival publishes it
      }
      const int total = plan.items * a.n_kv;
      const int box = P.box, n_box = kTile / box;
      // this CTA's boxes of a tile: of a pair half of the keys, half of the values' columns
      const int x0 = PAIR && keys ? rank * (n_box / 2) : 0, x1 = PAIR && keys ? x0 + n_box / 2 : n_box;
      const int row_b = PAIR && !keys ? DH / 2 : DH, col = PAIR && !keys ? rank * (DH / 2) : 0;
      const int ps = a.pages.page_size, tile_pages = kTile / ps, tile_rest = kTile % ps;
      const int table_pages = int(a.rows.table_pages), n_pages = int(a.pages.n_pages);
      const int oob_slot = n_pages * ps;
      int st = 0, loads_q = 0, seq = 0;    // the ring's next stage; stages counted
      uint32_t par = 1, mine = 0;          // what `code_empty` is waited for; which of the last stages this warp filled
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait_short(bar, phase, abort_flag, P.wait_ns));
        return ok;
      };
      auto across = [&](uint64_t* bar, uint32_t phase) {   // what the pair's other CTA says
        ok = __all_sync(0xffffffffu, wait_pair(bar, phase, abort_flag, P.wait_ns));
        return ok;
      };
      if (lane == 0) {
        if (keys) tc::tma_prefetch(&tm_q);
        tc::tma_prefetch(map);
      }
      for (int i = 0; ok; ++i) {
        Item it{};
        if (keys) {
          if (!wait(&S.item_empty[i & 1], ((i >> 1) & 1) ^ 1)) break;
          int idx = 0;
          if (rank == 0) {
            // the peer's place for the number is free when it has read the one two before
            if (PAIR && i >= 2 && !across(&S.idx_empty[i & 1], ((i >> 1) & 1) ^ 1)) break;
            if (lane == 0) {
              idx = (int)atomicAdd(&P.plan.head->next, 1u);
              if constexpr (PAIR) {
                st_peer(&S.idx[i & 1], idx, 1);
                arrive_peer(&S.idx_full[i & 1], 1);
              }
            }
          } else {
            if (!across(&S.idx_full[i & 1], (i >> 1) & 1)) break;
            if (lane == 0) {
              idx = *(volatile int*)&S.idx[i & 1];
              arrive_peer(&S.idx_empty[i & 1], 0);
            }
          }
          idx = __shfl_sync(0xffffffffu, idx, 0);
          if (idx < total) {
            const int e = idx / a.n_kv;    // never less than the one before
            while (e >= rows.items) {
              rows_load(rows, a.rows, rows.row0 + 32, P.per_tile);
              rows_cut(rows, plan.target);
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, e < rows.item0 + rows.tiles * rows.pieces)) - 1;
            const int in_row = e - __shfl_sync(0xffffffffu, rows.item0, src);
            const int pieces = __shfl_sync(0xffffffffu, rows.pieces, src), tile = in_row / pieces;
            it.b = rows.row0 + src;
            it.h = idx % a.n_kv;
            it.q0 = __shfl_sync(0xffffffffu, rows.q0, src);
            it.n = __shfl_sync(0xffffffffu, rows.n, src);
            it.L = __shfl_sync(0xffffffffu, rows.L, src);
            it.tok0 = (__shfl_sync(0xffffffffu, rows.tiles, src) - 1 - tile) * 2 * P.per_tile;
            it.tiles = it.n - it.tok0 > P.per_tile ? 2 : 1;
            const int last = min(it.n, it.tok0 + it.tiles * P.per_tile) - 1;
            const int steps = steps_of(min(it.L, it.L - it.n + last + 1)), len = (steps + pieces - 1) / pieces;
            it.kv0 = min(steps, in_row % pieces * len);
            it.kv1 = min(steps, it.kv0 + len);
            it.split = pieces > 1 ? __shfl_sync(0xffffffffu, rows.slot0, src) + in_row : -1;
          }
          if (lane == 0) {
            S.item[i & 1] = it;
            tc::mbar_arrive(&S.item_full[i & 1]);
          }
        } else {
          if (!wait(&S.item_full[i & 1], (i >> 1) & 1)) break;
          it = S.item[i & 1];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&S.item_empty[i & 1]);
        }
        const int b = __shfl_sync(0xffffffffu, it.b, 0), L = __shfl_sync(0xffffffffu, it.L, 0);
        const int h = __shfl_sync(0xffffffffu, it.h, 0), tiles = __shfl_sync(0xffffffffu, it.tiles, 0);
        const int kv0 = __shfl_sync(0xffffffffu, it.kv0, 0), kv1 = __shfl_sync(0xffffffffu, it.kv1, 0);
        if (tiles == 0) break;
        if (kv1 == kv0) continue;
        const int32_t* table = a.rows.page_table ? a.rows.page_table + (int64_t)b * table_pages : nullptr;
        if (keys) {
          // the queries' space: read by the last item's products
          if (!wait(&S.q_empty, (loads_q & 1) ^ 1)) break;
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(&S.q_full, uint32_t(tiles) * per * a.g * DH * 2);
            for (int t = 0; t < tiles; ++t)
              for (int c = 0; c < DH / 64; ++c)
                tc::tma_load_3d(smem + t * Y::kTileB + c * Y::kHalf, &tm_q, &S.q_full, c * 64, h * a.g,
                                it.q0 + it.tok0 + t * P.per_tile + rank * per);
          }
          ++loads_q;
          __syncwarp();
        }
        // One tile of 128 cached tokens in boxes of `box` tokens of a page. A lane looks up the slot of its box one tile
        // ahead: the next tile's is 128 tokens on.
        int tb = kv0 * kTile + lane * box;
        int pg = tb / ps, off = tb - pg * ps;   // without a table ps is not exceeded: pg is 0
        int next_page = -1, next_off = 0, next_t = 0;
        auto look = [&]() {
          next_page = table ? -1 : b;
          if (lane < n_box && tb < L && table && pg < table_pages) next_page = table[pg];
          next_off = off;
          next_t = tb;
          tb += kTile;
          pg += tile_pages;
          off += tile_rest;
          if (off >= ps) {
            off -= ps;
            ++pg;
          }
        };
        look();
        auto load = [&](int j) {
          int slot = oob_slot;                   // of this lane's box; outside the pool: zeros
          if (lane < n_box && next_t < L) {
            if (next_page >= 0 && next_page < n_pages) slot = next_page * ps + next_off;
            else record_error(a.err, kCodeDevice, kErrPage, next_t, b);
          }
          // a lane's block of 16 of the tile, the first 8 lanes for the keys' scales, the next 8 for the values'
          const int t16 = lane % kBlocks * kKv8Block;
          const int slot16 = __shfl_sync(0xffffffffu, slot, t16 / box) + t16 % box;
          if (!wait(&S.code_empty[st], par)) return;
          if (lane == 0) {
            S.info[st].valid = min(kTile, L - j * kTile);
            S.info[st].kind = keys ? kKeys : kValues;
          }
          if (keys && lane < kScaleLanes) {
            const bool in = j * kTile + t16 < L && slot16 < oob_slot;
            const int64_t at = in ? (int64_t)(slot16 / kKv8Block) * a.n_kv + h : 0;
            cp4(&S.raw[st][lane / kBlocks][lane % kBlocks], (lane < kBlocks ? P8.k_scale : P8.v_scale) + at, in ? 4 : 0);
            cp_arrive(&S.code_full[st]);
          }
          __syncwarp();
          if (lane == 0) {
            if (!keys) mbar_arrive_n(&S.code_full[st], kScaleLanes);
            tc::mbar_arrive_expect_tx(&S.code_full[st], Y::kCodeB);
          }
          __syncwarp();
          uint8_t* dst = smem + Y::kOffCode + st * Y::kCodeB;
          for (int x = x0; x < x1; ++x) {
            const int sx = __shfl_sync(0xffffffffu, slot, x);
            if (tc::elect_one()) tc::tma_load_3d(dst + (x - x0) * box * row_b, map, &S.code_full[st], col, h, sx);
            __syncwarp();
          }
          mine |= 1u;
          look();
        };
        auto step = [&](bool k_tile, int j) {
          mine <<= 1;
          ++seq;
          if (k_tile == keys && !(P.plan.test_stall && !keys)) load(j);
          if (++st == Y::kCodes) {
            st = 0;
            par ^= 1;
          }
        };
        const int lead = tiles == 1 ? 2 : 1;
#pragma unroll 1
        for (int jk = kv0, jv = kv0; ok && jv < kv1;) {
          const bool k_tile = jk < kv1 && jk - jv < lead;
          step(k_tile, k_tile ? jk++ : jv++);
        }
      }
      if (ok && keys && wait(&S.code_empty[st], par) && lane == 0) {   // the converters' end
        S.info[st].kind = kEnd;
        mbar_arrive_n(&S.code_full[st], 1 + kScaleLanes);
      }
      if (!ok) {   // copies still in flight must land before the CTA exits
        volatile int quiet = 0;
        for (int d = 0; d < Y::kCodes && d < seq; ++d) {
          const int p = seq - 1 - d;
          if (mine >> d & 1u)
            tc::mbar_wait_bounded(&S.code_full[p % Y::kCodes], (p / Y::kCodes) & 1, &quiet, P.wait_ns / 10);
        }
        if (loads_q) tc::mbar_wait_bounded(&S.q_full, (loads_q - 1) & 1, &quiet, P.wait_ns / 10);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------------ MMA
      // The whole warp walks the loop, so that stages and descriptors stay in uniform registers, and one lane
      // issues: from a branch of one thread each product took 80 cycles to issue, longer than it runs. One warp
      // issues for both units, in turn: with a warp each, the units fell into step and waited together.
      // Of a pair, the first CTA's issues for both, and the other's hands on what its converters say.
      const uint32_t id_qk = tc::idesc_f16(kTile * Y::kParts, kTile, false);
      const uint32_t id_pv = tc::idesc_f16(kTile * Y::kParts, DH, false) | tc::kIdescBMajorMN;
      const uint32_t base = tc::smem_addr(smem);
      const uint64_t dq = tc::sdesc_sw128(base, 16, 1024), dk = tc::sdesc_sw128(base + Y::kOffKv, 16, 1024);
      const uint64_t dv = tc::sdesc_sw128(base + Y::kOffKv, Y::kHalf, 1024);
      int st = 0, loads_q = 0;           // the ring's stage that comes next
      uint32_t par = 0, np = 0;          // its phase; the weights' phases of the units, a bit each
      // A wait that gives up only raises the abort flag, at which every later wait gives up at once; the loop
      // looks at the flag once a tile, so that a wait that need not wait costs little more than its test.
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (!tc::mbar_try_wait(bar, phase)) tc::mbar_wait_short(bar, phase, abort_flag, P.wait_ns);
      };
      auto stage = [&]() -> int {        // waits for the next stage of the ring and takes it
        const int s = st;
        if constexpr (PAIR) wait_pair(&S.full[s], par, abort_flag, P.wait_ns);
        else wait(&S.full[s], par);
        if (++st == Y::kStages) {
          st = 0;
          par ^= 1;
        }
        return s;
      };
      // S_u = Q K^T of key stage s; `last`: the item's last product that reads the queries
      auto qk = [&](int u, uint64_t q, int s, bool free, bool last) {
        const uint64_t kd = dk + uint64_t(s) * (Y::kStageB >> 4);
        __syncwarp();
        tc::tc_fence_after();
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint64_t qo = ((k / 4) * Y::kHalf + (k % 4) * 32) >> 4, ko = ((k / 4) * Y::kKeyHalf + (k % 4) * 32) >> 4;
            if constexpr (PAIR) umma_pair(tmem + u * kTile, q + qo, kd + ko, id_qk, k != 0);
            else tc::umma_f16(tmem + u * kTile, q + qo, kd + ko, id_qk, k != 0);
          }
          commit<PAIR>(&S.s_full[u]);
          if (free) commit<PAIR>(&S.empty[s]);
          if (last) commit<PAIR>(&S.q_empty);
        }
      };
      // O_u += P_u V of value stage s, the first half's weights first; `last`: the item's last for the unit
      auto pv = [&](int u, int s, bool first, bool free, bool last) {
        const uint64_t vd = dv + uint64_t(s) * (Y::kStageB >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait(&S.p_full[u][half], np >> u & 1);
          __syncwarp();
          tc::tc_fence_after();
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t o = tmem + Y::kColO + u * DH, w = tmem + u * kTile + half * 32 + k * 8;
              const uint64_t v = vd + half * (8192 >> 4) + ((k * 2048) >> 4);
              if constexpr (PAIR) umma_pair_ts(o, w, v, id_pv, !first || half + k != 0);
              else tc::umma_f16_ts(o, w, v, id_pv, !first || half + k != 0);
            }
            if (half == 1 && free) commit<PAIR>(&S.empty[s]);
            if (half == 1 && last) commit<PAIR>(&S.o_full[u]);
          }
        }
        np ^= 1u << u;
      };
      auto dead = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };
      for (int i = 0;; ++i) {
        wait(&S.item_full[i & 1], (i >> 1) & 1);
        if (dead()) break;
        Item it = S.item[i & 1];
        it.L = __shfl_sync(0xffffffffu, it.L, 0);
        it.n = __shfl_sync(0xffffffffu, it.n, 0);
        it.tok0 = __shfl_sync(0xffffffffu, it.tok0, 0);
        it.tiles = __shfl_sync(0xffffffffu, it.tiles, 0);
        it.kv0 = __shfl_sync(0xffffffffu, it.kv0, 0);
        it.kv1 = __shfl_sync(0xffffffffu, it.kv1, 0);
        if (lane == 0) tc::mbar_arrive(&S.item_empty[i & 1]);
        if (it.tiles == 0) break;
        const int n = it.kv1 - it.kv0;
        if (n == 0) continue;
        if (rank != 0) {
          for (int k = 0; k < 2 * n && !dead(); ++k) {
            const int s = st;
            wait(&S.full[s], par);
            if (++st == Y::kStages) {
              st = 0;
              par ^= 1;
            }
            if (lane == 0) arrive_peer(&S.full[s], 0);
          }
          continue;
        }
        if constexpr (PAIR) wait_pair(&S.q_ready, loads_q & 1, abort_flag, P.wait_ns);
        else wait(&S.q_ready, loads_q & 1);
        ++loads_q;
        // Two tiles of queries: both units over each tile of the cache; unit 0 may see fewer (it stops first). One: the
        // units take the cache's tiles in turn. One loop for both, and for the units, keeps the code short: the warps of
        // other roles on this scheduler wait for their instructions too.
        const bool two = it.tiles == 2;
        const int n0 = two ? unit_steps(it, 0, P.per_tile) : 0;
        int sk = 0, sv = 0;
#pragma unroll 1
        for (int u = 0; u < (two ? 2 : min(n, 2)); ++u) {
          if (!two || u == 0) sk = stage();
          if (!two || u == 1 || n0 > 0)
            qk(u, two && u == 1 ? dq + (Y::kTileB >> 4) : dq, sk, !two || u == 1, two ? u == 1 && n == 1 : u + 1 == n);
        }
#pragma unroll 1
        for (int x = 0; x < (two ? 2 * n : n); ++x) {
          if (dead()) break;
          const int u = x & 1, k = two ? x >> 1 : x, seen = two && u == 0 ? n0 : n, next = two ? k + 1 : k + 2;
          const bool second = !two || u == 1, first = !two || u == 0, more = first && next < n;
          if (first) sv = stage();
          // Before the weights come: a look at a pair's barriers takes 200 clocks. Alone, units in turn over one tile would wait
          // for keys that are converted behind the values that the weights want.
          if (PAIR && more) sk = stage();
          if (k < seen) pv(u, sv, two ? k == 0 : k < 2, second, next >= seen);
          if (!PAIR && more) sk = stage();
          if (next < seen) qk(u, two && u == 1 ? dq + (Y::kTileB >> 4) : dq, sk, second, second && next + 1 == n);
        }
        __syncwarp();
      }
      __syncwarp();
      // every product issued has completed once this commit lands, at both CTAs
      volatile int quiet = 0;
      if (rank == 0 && tc::elect_one()) commit<PAIR>(&S.drained);
      __syncwarp();
      tc::mbar_wait_bounded(&S.drained, 0, &quiet, Y::kParts * P.wait_ns);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    tc::regs_grow<Y::kRegsSoftmax>();
    const int u = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                        // query row of the tile = lane of tensor memory
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + u * kTile, t_o = tmem + lanes + Y::kColO + u * DH;
    int n_s = 0, n_o = 0, n_x = 0, n_q = 0, n_k = 0, n_l = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait_short(bar, par, abort_flag, P.wait_ns));
      tc::tc_fence_after();
      return ok;
    };
    for (int i = 0; ok; ++i) {
      if (!wait(&S.item_full[i & 1], (i >> 1) & 1)) break;
      const Item it = S.item[i & 1];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&S.item_empty[i & 1]);
      if (it.tiles == 0) break;
      if (threadIdx.x == 0 && it.split >= 0) ++S.cut;
      const int tile = it.tiles == 2 ? u : 0;
      const int first_tok = it.tok0 + tile * P.per_tile + (PAIR ? (int)cta_rank() * per : 0);
      const int tok = first_tok + r / a.g;
      const bool live = r < per * a.g && tok < it.n;
      const int vis = it.L - it.n + tok;                         // last slot this row sees
      const int vis_min = it.L - it.n + first_tok;               // every row of the tile sees slots up to here
      const int steps = unit_steps(it, u, P.per_tile);
      const bool exchange = it.tiles == 1 && it.kv1 - it.kv0 > 1;

      float c = a.scale_log2;                                    // of this row's scores: without its lift
      if (it.kv1 > it.kv0) {
        if (!wait(&S.q_full, n_q & 1)) break;                    // both units: neither arrives for an item to come
        if constexpr (BF16) {
          float lift = 1.f;
          if (it.tiles == 2 || u == 0) {
            if (r < per * a.g) lift = lift_row<DH>(smem + tile * Y::kTileB, r);
            if (it.tiles == 1) S.lift[r] = lift;
            tc::fence_async_smem();
          }
          __syncwarp();
          if (it.tiles == 1) {
            if (u == 0 && lane == 0) tc::mbar_arrive(&S.lift_full);
            if (u == 1) {
              if (!wait(&S.lift_full, n_l & 1)) break;
              lift = S.lift[r];
            }
            ++n_l;
          }
          c *= 1.f / lift;                                       // powers of two
        }
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) arrive_peer(&S.q_ready, 0);
          else tc::mbar_arrive(&S.q_ready);
        }
        ++n_q;
      }

      float m = -INFINITY;
      uint64_t l2 = 0;                                           // the sum, in two parts
      for (int k = 0; k < steps; ++k) {
        const int tk = unit_tile(it, u, k), kk = n_k + tk - it.kv0;
        if (!wait(&S.scale_full[kk % Y::kScales], (kk / Y::kScales) & 1)) break;
        if (!wait(&S.s_full[u], n_s & 1)) break;
        ++n_s;
        const float2* sc = S.scale[kk % Y::kScales];
        const float2* part = S.part[kk % Y::kScales];
        const int t0 = tk * kTile;
        if (t0 + kTile - 1 > vis_min) {
          // tokens that a row does not see: masked in tensor memory, so that the common tile's code stays short
          const int lim = vis - t0;
#pragma unroll 1
          for (int x = 0; x < kTile; x += 32) {
            uint32_t w[32];
            tc::tmem_ld32_nowait(t_s + x, w);
            tc::tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 32; ++y) w[y] = x + y > lim ? 0xff800000u : w[y];
            tc::tmem_st32(t_s + x, w);
          }
          tc::tmem_st_wait();
        }
        float s[kTile];
#pragma unroll
        for (int x = 0; x < 4; ++x) tc::tmem_ld32_nowait(t_s + x * 32, reinterpret_cast<uint32_t*>(s) + x * 32);
        tc::tmem_ld_wait();
        float2 z[kBlocks];   // of each 16 scores: s_k c and log2 s_v, held (read again for the weights: 578 us against 562 for the prompts)
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          float y0 = max3(s[b * 16], s[b * 16 + 1], s[b * 16 + 2]), y1 = max3(s[b * 16 + 3], s[b * 16 + 4], s[b * 16 + 5]);
          y0 = max3(y0, s[b * 16 + 6], s[b * 16 + 7]);
          y1 = max3(y1, s[b * 16 + 8], s[b * 16 + 9]);
          y0 = max3(y0, s[b * 16 + 10], s[b * 16 + 11]);
          y1 = max3(y1, s[b * 16 + 12], s[b * 16 + 13]);
          y0 = max3(y0, s[b * 16 + 14], s[b * 16 + 15]);
          z[b] = sc[b];
          z[b].x = factor_of<BF16>(c, z[b].x);
          mx[b & 1] = fmaxf(mx[b & 1], fmaf(fmaxf(y0, y1), z[b].x, z[b].y));
        }
        const float top = softmax_base<false>(fmaxf(mx[0], mx[1]), kLift);
        const bool raise = top > m + kRaise;                     // true on the first finite score
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? top : m;
          const float f = m == -INFINITY ? 0.f : exp2f(m - mn);    // nothing seen yet: sum and output are 0
          m = mn;
          l2 = mul2(l2, pair(f, f));
          if (k > 0) {   // s_full also says that the product before it, into O, has completed
#pragma unroll 1
            for (int x = 0; x < DH; x += 16) {
              uint32_t o[16];
              tc::tmem_ld16_nowait(t_o + x, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc::tmem_st16(t_o + x, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;             // nothing seen yet: every p is 2^-inf = 0
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[16];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float2 zb = z[x * 2 + b];
            const uint64_t c2 = pair(zb.x, zb.x), n2 = pair(zb.y + neg, zb.y + neg);
            uint64_t sum2[2];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const float2 e = unpair(fma2(pair(s[x * 32 + b * 16 + 2 * y], s[x * 32 + b * 16 + 2 * y + 1]), c2, n2));
              const float p0 = ex2(e.x), p1 = ex2(e.y);
              sum2[y & 1] = y < 2 ? pair(p0, p1) : add2(sum2[y & 1], pair(p0, p1));
              p[b * 8 + y] = pack2<false>(p0, p1);
            }
            const float2 inv = part[x * 2 + b];
            l2 = fma2(add2(sum2[0], sum2[1]), pair(inv.x, inv.y), l2);   // without the values' scale
          }
          tc::tmem_st16(t_s + x * 16, p);
          if (x & 1) {                                           // 64 tokens' weights: the product may begin
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR) arrive_peer_relaxed(&S.p_full[u][x >> 1], 0);
              else tc::mbar_arrive(&S.p_full[u][x >> 1]);
            }
          }
        }
      }
      if (!ok) break;
      n_k += it.kv1 - it.kv0;
      float l = unpair(l2).x + unpair(l2).y;

      // the unit's row: O / l, or its partial
      if (steps > 0) {
        if (!wait(&S.o_full[u], n_o & 1)) break;
        ++n_o;
      }
      if (exchange && u == 1) {
        // the other unit finds this one's output where it is, and maximum and sum in place of its scores; the next products
        // into either come behind the other's word that it is ready for another item
        tmem_st2(t_s, m, l);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.x_full);
        continue;
      }
      if (it.tiles == 1 && u == 1) continue;                     // a single step: unit 0 has all of it
      float f0 = 1.f, f1 = 0.f;
      if (exchange) {
        if (!wait(&S.x_full, n_x & 1)) break;
        ++n_x;
        const float2 o1 = tmem_ld2(t_s + kTile);
        const float mn = fmaxf(m, o1.x), b0 = mn == -INFINITY ? 0.f : mn;
        f0 = exp2f(m - b0);
        f1 = exp2f(o1.x - b0);
        l = fmaf(l, f0, o1.y * f1);
        m = mn;
      }
      const int64_t row = (int64_t)(it.q0 + tok) * a.n_heads + it.h * a.g + r % a.g;
      const int64_t slot = (((int64_t)it.split * a.n_kv + it.h) * 2 + tile) * Y::kParts + (PAIR ? (int)cta_rank() : 0);
      if (it.split < 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        f0 *= inv;
        f1 *= inv;
        if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        if (live) a.part_ml[slot * kTile + r] = make_float2(m, l);
      }
#pragma unroll 1
      for (int x = 0; x < DH / 32; ++x) {
        float o[32];
        if (steps > 0) {
          tc::tmem_ld32_nowait(t_o + x * 32, reinterpret_cast<uint32_t*>(o));
          tc::tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] *= f0;
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0.f;
        }
        if (exchange) {
          float o1[32];
          tc::tmem_ld32_nowait(t_o + DH + x * 32, reinterpret_cast<uint32_t*>(o1));
          tc::tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = fmaf(o1[y], f1, o[y]);
        }
        if (it.split >= 0 && live) {
          float4* po = reinterpret_cast<float4*>(a.part_o) + (slot * (DH / 4) + x * 8) * kTile + r;
#pragma unroll
          for (int y = 0; y < 8; ++y) po[y * kTile] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        } else if (it.split < 0 && live) {
          uint16_t* out = static_cast<uint16_t*>(a.out) + row * DH + x * 32;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t w[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) w[z] = pack2<BF16>(o[16 * y + 2 * z], o[16 * y + 2 * z + 1]);
            store32(out + 16 * y, w, P.out_sectors);
          }
        }
      }
      tc::tc_fence_before();
    }
    // The join. Every item has been taken when a CTA comes here, by CTAs that run and wait for none: the wait for
    // their pieces ends whichever CTAs the GPU holds. All warps meet first, also after a wait that gave up.
    const auto any = [](bool bad) { return tc::named_bar_or(1, kJoinWarps * 32, bad); };
    if (!any(!ok) && S.plan.joins > 0) {
      Rows32 rows;
      rows_load(rows, a.rows, 0, P.per_tile);
      if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(&P.plan.head->pieces, S.cut);
        ok = pieces_wait(&P.plan.head->pieces, unsigned(S.plan.slots * a.n_kv * Y::kParts), P.wait_ns);
        if (!ok) *abort_flag = 1;
      }
      // the queries' space is free: nothing is in flight behind the last item
      if (!any(!ok)) join_pieces<DH, BF16, 2 * Y::kParts>(P, S.plan, rows, *reinterpret_cast<JoinShared*>(smem));
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_meet();
  tc::tc_fence_after();
  if (threadIdx.x == 0) {
    if (*abort_flag) record_error(a.err, kCodeTimeout, kErrWait, blockIdx.x, 0);
    // the last CTA to end sets the counters back for the next call; `done` wraps to zero by itself
    __threadfence();
    if (atomicInc(&P.plan.head->done, gridDim.x - 1) == gridDim.x - 1) P.plan.head->next = P.plan.head->pieces = 0;
  }
  if (warp == 9) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tc::tmem_dealloc(tmem, 512);
  }
}

template <int DH, bool BF16, bool PAIR> cudaError_t prepare_tc() {
  return cudaFuncSetAttribute(kv8_attend_tc_kernel<DH, BF16, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Lay<DH, PAIR>::kSmem);
}
template <int DH, bool BF16, bool PAIR> cudaError_t launch_tc(const Kv8AttendArgs& A, const KvTcPlan& t, cudaStream_t st) {
  using Y = Lay<DH, PAIR>;
  const KvAttendArgs& a = A.a;
  Tc8Params P8{};
  P8.k_scale = A.k_scale;
  P8.v_scale = A.v_scale;
  TcParams& P = P8.P;
  P.a = a;
  P.plan = t;
  const int per = kTile / a.g, sms = t.sm_count / Y::kParts;   // tokens of 128 rows; CTAs or pairs
  P.per_tile = per * Y::kParts;
  P.plan.sm_count = sms;
  P.plan.slots = t.slots / Y::kParts;          // a pair's piece stores twice the rows
  P.out_sectors = (uintptr_t)a.out % 32 == 0;
  P.wait_ns = t.wait_ns;
  CUtensorMap tm_q, tm_k, tm_v;
  {
    // queries [token][head][d]: boxes of 64 columns, one group's heads, the tokens of 128 rows
    const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[3] = {DH, (cuuint64_t)a.n_heads, (cuuint64_t)a.rows.n_tokens};
    const cuuint64_t strides[2] = {DH * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)per};
    if (!tma_encode(&tm_q, dt, 3, a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  {
    // codes [slot][kv head][d]. A box lies in one page: the largest power of two (16 and more) that divides a page, and
    // without a table, where a row's tokens lie in a row, a whole tile; of a pair, half a tile at most, and of the values
    // half the columns.
    constexpr int kBox = kTile / Y::kParts;
    P.box = a.rows.page_table ? a.pages.page_size & -a.pages.page_size : kBox;
    P.box = P.box > kBox ? kBox : P.box;
    const cuuint64_t dims[3] = {DH, (cuuint64_t)a.n_kv, (cuuint64_t)(a.pages.n_pages * a.pages.page_size)};
    const cuuint64_t strides[2] = {DH, (cuuint64_t)a.n_kv * DH};
    auto map = [&](CUtensorMap* m, const void* p, int columns) {
      const cuuint32_t box[3] = {(cuuint32_t)columns, 1, (cuuint32_t)P.box};
      const CUtensorMapSwizzle sw = columns == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
      return tma_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p, dims, strides, box, sw);
    };
    if (!map(&tm_k, a.pages.k, DH) || !map(&tm_v, a.pages.v, DH / Y::kParts)) return cudaErrorInvalidValue;
  }
  const int64_t most = ((int64_t)t.tile_cap + P.plan.slots) * a.n_kv;
  const unsigned grid = (unsigned)(most < sms ? most : sms) * Y::kParts;
  return launch_early<Y::kParts>(kv8_attend_tc_kernel<DH, BF16, PAIR>, dim3(grid), kThreads, Y::kSmem, st, tm_q, tm_k, tm_v, P8);
}

// Pairs take where there is enough work for them and its rows fill their tiles, by the call's averages and bounds.
//   * An item of a pair is 512 query rows. Its start, its end and the rows that a causal item computes in vain cost more
//     than an item of 256, so a pair must have at least 40 steps (of two tiles) to do, of which steps over the new tokens
//     themselves count a quarter: 128 tokens of 4 heads, 8 key/value heads, at 8192 (7): 35 us against 33; at 32768 (27): 73 against 75;
//     16 sequences of 256 such tokens at 4096 (107): 251 against 271; four prompts of 2048, 32 heads (27): 186 against 175.
//   * Where a sequence's last item is half empty for want of rows, one CTA alone would have skipped that half. A pair's
//     steps take about 14/15 of the time, which makes up for that from 3584 rows on: 16 sequences at 4096 of 768 rows take
//     240 us by pairs against 208, of 1024 rows 251 against 271.
bool in_pairs(const KvAttendArgs& a, int sms) {
  if (a.head_dim != 128) return false;
  const int64_t rows = ((int64_t)a.rows.n_tokens * a.g + a.rows.batch - 1) / a.rows.batch;
  const int64_t ones = (rows + 2 * kTile - 1) / (2 * kTile), pairs = (ones + 1) / 2;
  const int64_t steps = ((int64_t)a.rows.max_kv_len - (int64_t)a.rows.max_new * 3 / 4) / kTile;
  return 28 * pairs <= 15 * ones && a.rows.batch * pairs * a.n_kv * steps >= (int64_t)40 * (sms / 2);
}

}  // namespace

cudaError_t prepare_kv8_attend_tc(int head_dim, bool bf16) {
  if (head_dim == 64) return bf16 ? prepare_tc<64, true, false>() : prepare_tc<64, false, false>();
  const cudaError_t e = bf16 ? prepare_tc<128, true, false>() : prepare_tc<128, false, false>();
  if (e != cudaSuccess) return e;
  return bf16 ? prepare_tc<128, true, true>() : prepare_tc<128, false, true>();
}

cudaError_t launch_kv8_attend_tc(const Kv8AttendArgs& a, const KvTcPlan& t, cudaStream_t st) {
  if (!tma_available()) return cudaErrorNotSupported;
  if (a.a.head_dim == 64) return a.a.bf16 ? launch_tc<64, true, false>(a, t, st) : launch_tc<64, false, false>(a, t, st);
  if (in_pairs(a.a, t.sm_count)) return a.a.bf16 ? launch_tc<128, true, true>(a, t, st) : launch_tc<128, false, true>(a, t, st);
  return a.a.bf16 ? launch_tc<128, true, false>(a, t, st) : launch_tc<128, false, false>(a, t, st);
}

}  // namespace palu
