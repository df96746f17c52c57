// Attention of many query rows (prompts and their chunks) over the 4-bit paged cache on the
// 5th-generation tensor cores (tcgen05, sm_100a).
//
//   x_ij = q_i . k'_j,  k'_j = scale log2(e) (c_j - z_j) hk_j;   w_ij = 2^(x_ij - m_i + 7)
//   o_i  = sum_j w_ij v_j / sum_j w_ij,  v_j = (c_j - z_j) hv_j
// k', v and w are float16 operands, each rounded once (by at most 2^-11 of it), as in the
// calibrated block's own attention; statistics, sums (of the weights before their rounding) and
// accumulators are float32. (The tensor cores cut their sums off towards zero: of 30000 keys in one
// part o loses 7e-5 of itself, in proportion to the keys.) (Keeping the steps outside the
// products, as kv_rows.cu does, costs three broadcast shared loads per score here: 393 KB a
// tile of keys against 128 B a clock, more than the products' time.) The reference m_i follows
// the row's maximum only when that has grown by more than 2^8, so o is rescaled rarely; in
// exact arithmetic the result is the same.
//
// A pair of CTAs (cluster of 2, cta_group::2) takes 512 query rows of one (request, kv head),
// row r = new token r / G, query head r mod G of the group: two subtiles of 256 rows, whose
// products and softmax alternate (while one subtile's scores become weights, the other's
// products run). Per 128 keys: S = Q K^T (256 x 128 x D), O += P V (256 x D x 128), P straight
// from tensor memory, where it takes S's place. Each CTA expands the keys' codes it contributes
// to the pair's operands: K of 64 keys, V's 64 columns of all 128 keys (for D = 64 the second
// CTA's V half stays zero). The order in which a word yields its 8 values (0 4 1 5 2 6 3 7) is
// kept in both operands (Q is staged in the same order) and undone where o is written.
// Where the items are few for the 74 pairs, a pair takes an equal share of an item's keys and
// leaves o and (m, l) in float32; a second kernel joins the parts in their order (one request
// under 65536 tokens, 8 x 4 heads: 64 new tokens 949 -> 130 us, 128 new ones 1019 -> 141).
// Which item a pair has follows from the lengths on the device, so that requests of another
// kind (a step with one chunk and many single tokens) take no pairs.
// Warp roles (512 threads; registers are shared out again at the start, 200 a softmax thread
// and 56 the others):
//   0-3, 4-7  softmax of subtile 0 / 1, a row a thread; they also stage Q and write o
//   8, 9      expand K; 10, 11 expand V
//   12        MMA issue (leader CTA); TMEM allocation
//   13        bulk copies of the raw cells
// Measured, 8 x 4 heads of 128: a prompt of 8192 tokens 507 us (1.08 PFLOP/s) in a burst at
// 1965 MHz and 568 under load at the power limit (1760 MHz), three chunks of up to 1000 behind
// contexts of up to 16411 533 us (0.96) and 560 (1860 MHz); 32 heads, 2048 tokens 65 us (0.53: 4 to
// 16 tiles of keys do not hide a pair's first 7 us). A step of 128 keys takes 3550 cycles against
// 2048 of products and another 2048 of exponentials (256 rows x 128 keys a CTA, 16 a clock); the
// two meet only partly, a row's chain being read S, maximum, exponentials, write P with no more
// than two subtiles in 512 columns of tensor memory. Tensor cores 56% busy, exponential unit 56%.
// (Steps of 64 keys with two places for each subtile's scores, so that the next are ready when
// a row's weights are done, took 571 us: eight waits and twelve commits a tile of keys in the
// issuing warp.)
// Every mbarrier wait is bounded; on expiry the error flag is raised, every role stops, copies
// and MMAs in flight are drained and both CTAs meet before TMEM is released. Loads never
// multicast.
#include "kv_internal.cuh"

namespace omq {
namespace kv {

static __device__ unsigned g_tiles_error = 0;
static __device__ uint64_t g_tiles_limit_ns = 2000000000ull;

cudaError_t tiles_take_error(unsigned* flag) {
  unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_tiles_error, sizeof(unsigned));
  if (e == cudaSuccess && *flag) e = cudaMemcpyToSymbol(g_tiles_error, &zero, sizeof(unsigned));
  return e;
}
cudaError_t tiles_set_limit(uint64_t ns) {
  return cudaMemcpyToSymbol(g_tiles_limit_ns, &ns, sizeof(ns));
}

namespace {

constexpr int KT = 128;               // keys of a tile
constexpr int NS = 2;                 // expanded K / V stages
constexpr int NR = 3;                 // raw stages
constexpr int THREADS = 512;
constexpr int REGS = 128, REGS_SOFTMAX = 200, REGS_OTHER = 56;   // per thread: launch, after
static_assert(2 * REGS >= REGS_SOFTMAX + REGS_OTHER, "the shares come out of the launch's registers");
constexpr int ROWS = 512;             // query rows of a pair
constexpr float UP = 7.f;             // weights are 2^(x - m_i + UP), at most 2^15 in float16
constexpr float GROW = 8.f;           // growth of a row's maximum (log2) that moves m_i

template <int D>
struct TilesCfg {
  using C = CellT<D>;
  static constexpr int QSUB = 128 * D * 2;               // one subtile's Q rows of a CTA
  static constexpr int KST = 64 * D * 2;                 // K stage: 64 keys
  static constexpr int VST = KT * 64 * 2;                // V stage: 64 columns of 128 keys
  static constexpr int RAW = (KT / kCell) * C::BYTES;
  static constexpr int Q_OFF = 0, K_OFF = 2 * QSUB, V_OFF = K_OFF + NS * KST,
                       RAW_OFF = V_OFF + NS * VST, CTL = RAW_OFF + NR * RAW;
  // barriers
  static constexpr int QF = CTL, KF = QF + 16, KE = KF + 8 * NS, VF = KE + 8 * NS,
                       VE = VF + 8 * NS, SF = VE + 8 * NS, PF = SF + 16, PG = PF + 16, OF = PG + 16,
                       RF = OF + 16, RE = RF + 8 * NR, DR = RE + 8 * NR,
                       // cells that are there per raw stage; cells that are missing per tile
                       MASK = DR + 8, MISS = MASK + 4 * NR, SLOT = MISS + 32, ABORT = SLOT + 4,
                       END = ABORT + 4;
  static constexpr int SMEM = END + 1024;                // + alignment slack
};

__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Arrive on a barrier of CTA `rank`. What the arrivals publish (operands in shared memory, weights
// in TMEM) is read by the tensor cores of the CTA that wrote it, so the release is at CTA scope;
// at cluster scope every arrival waited about 1000 cycles for a memory barrier.
__device__ __forceinline__ void arrive_rank(uint32_t bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_rank(bar, rank)) : "memory");
}
// Bounded wait; also gives up once the CTA's abort flag is set.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         unsigned bit) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  const uint64_t lim = *const_cast<const volatile uint64_t*>(&g_tiles_limit_ns);
  while (!bar_try(bar, parity)) {
    if (*abort_flag) return false;
    if (now_ns() - t0 > lim) {
      atomicOr(&g_tiles_error, bit);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
// float16 operands, float32 accumulator: B K-major or MN-major, N / 8, M / 16.
constexpr uint32_t idesc(int m, int n, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
// The upper word of every operand descriptor here: stride 1024 bytes between 8-row atoms,
// version 1, 128-byte swizzle. The lower word is the address and the leading offset (one
// operand never has a second chunk within an instruction).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescLead = 1u << 16;
// Issued by one lane, with operands that are the same for the whole warp.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b),
      "r"(id), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b),
      "r"(id), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
__device__ __forceinline__ void commit_local(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tm_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
               ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// What expand() needs of a row: the step as two float16, hi + lo 2^-11 (lo as large as hi's last
// bit allows, so that it keeps its own bits down to a step of 2^-14), and 1024 + z, 64 + z (twice
// each). |z| <= 960 is exact in them. The rows beyond (all values 60 times further from zero than
// they spread) and those of smaller steps take the slow path. (With lo as a plain float16 a step
// below 2^-9 was off by up to 2^-25, times c - z: a value row of 0.01 +- 1e-4 by 2.6e-3 of it.
// Chunks of 1000 behind 16411 take 527 us for 523 with the product more; where every step of K
// is around 2^-14, so that warps take both paths, 880.)
constexpr float kSmallStep = 6.103515625e-05f;             // 2^-14
struct RowSteps {
  uint32_t hi, lo, z10, z6;
  float h, z;
  bool slow;
};
__device__ __forceinline__ RowSteps row_steps(float h, float z) {
  RowSteps r;
  const float hi = __half2float(__float2half_rn(h));
  r.hi = pack_h2(hi, hi);
  // (an infinite or NaN step has no remainder)
  const float lo = fabsf(hi) < INFINITY ? (h - hi) * 2048.f : 0.f;
  r.lo = pack_h2(lo, lo);
  r.z10 = pack_h2(-1024.f - z, -1024.f - z);
  r.z6 = pack_h2(-64.f - z, -64.f - z);
  r.h = h;
  r.z = z;
  r.slow = fabsf(z) > 960.f || (h != 0.f && fabsf(h) < kSmallStep);
  return r;
}
// (c - z) h of a word's eight codes in the order 0 4 1 5 2 6 3 7: a code placed in the mantissa
// of 1024 (or, in the next nibble, as 16 c) gives c - z exactly, and with the step in two parts
// the product is rounded once but for 2^-20 of it and, where the second part's product is a
// subnormal, 2^-25.
__device__ __forceinline__ void expand(uint32_t w, const RowSteps& r, uint32_t addr) {
  uint32_t o[4];
  const uint32_t w8 = w >> 8;
  const uint32_t d[4] = {hadd2((w & 0x000F000Fu) | 0x64006400u, r.z10),
                         hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, r.z6),
                         hadd2((w8 & 0x000F000Fu) | 0x64006400u, r.z10),
                         hfma2((w8 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, r.z6)};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = hfma2(d[i], r.hi, hmul2(hmul2(d[i], r.lo), 0x10001000u));
  sts4(addr, o[0], o[1], o[2], o[3]);
}
// The same in float32, rounded once. (A code is read as a number from the mantissa of 2^23: the
// conversion instruction runs on the exponentials' unit.)
__device__ __forceinline__ float slow_value(uint32_t c, float h, float z) {
  return ((__uint_as_float(c | 0x4B000000u) - 8388608.f) - z) * h;
}
__device__ __noinline__ void expand_slow(uint4 w, float h, float z, uint32_t base, int j0, int sw) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const uint32_t u = k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack_h2(slow_value((u >> (4 * i)) & 15u, h, z), slow_value((u >> (4 * i + 16)) & 15u, h, z));
    sts4(base + (((j0 + k) ^ sw) << 4), o[0], o[1], o[2], o[3]);
  }
}
__device__ __forceinline__ void expand4(const uint4& w, const RowSteps& r, uint32_t base, int j0, int sw) {
  if (!r.slow) {
    expand(w.x, r, base + (((j0 + 0) ^ sw) << 4));
    expand(w.y, r, base + (((j0 + 1) ^ sw) << 4));
    expand(w.z, r, base + (((j0 + 2) ^ sw) << 4));
    expand(w.w, r, base + (((j0 + 3) ^ sw) << 4));
  } else {
    expand_slow(w, r.h, r.z, base, j0, sw);
  }
}

// Partial results of pairs that share an item's keys: o (not divided) of part i at
// o[(i D / 4 + column / 4) 512 + row], columns in the operands' order; (reference, sum) at
// ml[512 i + row], the sum 0 where there was no key (o is then not written). desc: the item's
// request and tile, request -1: none.
struct TilesSpace {
  float4* o;
  float2* ml;
  int2* desc;
};

// Row tiles that request b has for this kernel.
__device__ __forceinline__ int req_tiles(const AttnParams& p, int b, int min_rows) {
  const int first = p.cu[b];
  const int n = min(max(p.cu[b + 1] - first, 0), p.max_q);
  if (first < 0 || first >= p.T || n * p.G < min_rows) return 0;
  return (static_cast<int>(min(static_cast<int64_t>(n), p.T - first)) * p.G + ROWS - 1) / ROWS;
}
// The at-th row tile of all requests, in their order, a request's last (it sees the most keys)
// first: (request, tile), request -1 behind the last. For the whole block.
__device__ __forceinline__ int2 find_tile(const AttnParams& p, int at, int min_rows) {
  if (p.n_req == 1) {
    const int n = req_tiles(p, 0, min_rows);
    return at < n ? make_int2(0, n - 1 - at) : make_int2(-1, 0);
  }
  __shared__ int sums[THREADS / 32];
  __shared__ int2 found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) found = make_int2(-1, 0);
  for (int c = 0; c < p.n_req; c += THREADS) {
    const int b = c + threadIdx.x;
    const int n = b < p.n_req ? req_tiles(p, b, min_rows) : 0;
    int end = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += o;
    }
    if (lane == 31) sums[warp] = end;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w == warp) end += all;
      all += sums[w];
    }
    if (at < end && at >= end - n) found = make_int2(b, end - 1 - at);
    __syncthreads();
    if (at < all) break;
    at -= all;
  }
  return found;
}

// Eight results in the operands' order (elements 0 .. 7 stand at 0 2 4 6 1 3 5 7), 16 bits each.
__device__ __forceinline__ uint4 out_eight(const float* v, int dt) {
  uint32_t w[4];
  const int e0[4] = {0, 4, 1, 5}, e1[4] = {2, 6, 3, 7};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (dt == OMQ_F16) {
      w[k] = pack_h2(v[e0[k]], v[e1[k]]);
    } else {
      const __nv_bfloat162 q = __floats2bfloat162_rn(v[e0[k]], v[e1[k]]);
      w[k] = *reinterpret_cast<const uint32_t*>(&q);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    kv_tiles_kernel(AttnParams p, int pieces, int min_rows, TilesSpace ws) {
  using F = TilesCfg<D>;
  using C = CellT<D>;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  // (broadcast, so that the roles' branches are known to be warp-uniform)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + F::ABORT);
  volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + F::MASK);
  volatile uint32_t* miss = reinterpret_cast<volatile uint32_t*>(smem + F::MISS);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + F::SLOT);

  // part of the launch: a share of an item's keys
  const int part = blockIdx.x >> 1;
  const int item = SPLIT ? part / pieces : part;
  const int kvh = item % p.pool.Hkv;

  pdl_wait();
  pdl_launch();
  const int2 at = find_tile(p, item / p.pool.Hkv, min_rows);
  const int b = at.x, tile = at.y;
  if (SPLIT && rank == 0 && threadIdx.x == 0 && part == item * pieces) ws.desc[item] = at;
  if (b < 0) return;                                           // the same for both CTAs
  const int len = min(max(p.lens[b], 0), p.width * p.pool.page);
  const int first = p.cu[b];
  const int n_new = max(p.cu[b + 1] - first, 0);
  const int rows = min(n_new, p.max_q) * p.G;
  const int row0 = tile * ROWS;

  auto row_vis = [&](int r) {
    if (r >= rows || first + r / p.G >= p.T) return 0;
    return p.causal ? min(max(len - n_new + r / p.G + 1, 0), len) : len;
  };
  const int vis_max = row_vis(min(row0 + 511, rows - 1));
  // tiles of keys that the subtiles see
  int nt0 = (row_vis(min(row0 + 255, rows - 1)) + KT - 1) / KT;
  int nt1 = row0 + 256 < rows ? (vis_max + KT - 1) / KT : 0;
  int key0 = 0;                                                // the part's first key
  if (SPLIT) {
    const int share = (max(nt0, nt1) + pieces - 1) / pieces, t0 = (part - item * pieces) * share;
    nt0 = min(max(nt0 - t0, 0), share);
    nt1 = min(max(nt1 - t0, 0), share);
    key0 = t0 * KT;
  }
  const int nt = max(nt0, nt1);
  const int n_cell = (vis_max + kCell - 1) / kCell;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      bar_init(sb + F::QF + 8 * s, 8);        // leader's: four warps of either CTA
      bar_init(sb + F::SF + 8 * s, 1);
      bar_init(sb + F::PF + 8 * s, 8);        // leader's
      bar_init(sb + F::PG + 8 * s, 8);        // leader's
      bar_init(sb + F::OF + 8 * s, 1);
    }
    for (int s = 0; s < NS; ++s) {
      bar_init(sb + F::KF + 8 * s, 4);        // leader's: two warps of either CTA
      bar_init(sb + F::KE + 8 * s, 1);
      bar_init(sb + F::VF + 8 * s, 4);        // leader's
      bar_init(sb + F::VE + 8 * s, 1);
    }
    for (int s = 0; s < NR; ++s) {
      bar_init(sb + F::RF + 8 * s, 1);
      bar_init(sb + F::RE + 8 * s, 4);
    }
    bar_init(sb + F::DR, 1);
    *abort_flag = 0;
    bar_init_fence();
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (D == 64 && rank == 1) {                 // the pair's second V half has no columns
    for (int i = threadIdx.x; i < NS * F::VST / 16; i += THREADS)
      sts4(sb + F::V_OFF + 16 * i, 0u, 0u, 0u, 0u);
    fence_async();
  }
  tc_before();
  __syncthreads();
  cluster_sync_all();
  tc_after();
  // All 512 columns are this pair's, so they start at 0.
  constexpr uint32_t tmem = 0;
  if (*slot != 0) *abort_flag = 1;
  // TMEM columns: S / P of subtile s at 128 s, O of subtile s at 256 + 128 s

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int s = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;                        // row of the CTA's half subtile
    const int row = row0 + 256 * s + 128 * static_cast<int>(rank) + r;
    const int vis = row_vis(row);
    const bool have_row = row < rows && first + row / p.G < p.T;
    const int tok = row / p.G, hq = kvh * p.G + row - tok * p.G;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = lane_base + 128 * s, tO = lane_base + 256 + 128 * s;
    const int my_nt = s ? nt1 : nt0;
    float post = 1.f;                                      // 2^-e of a row staged as q 2^e
    bool any_post = false;
    if (my_nt > 0) {
      const bool f16 = p.dt == OMQ_F16;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) +
          (have_row ? static_cast<int64_t>(first + tok) * p.q_ld + static_cast<int64_t>(hq) * D : 0));
      uint4 u[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) u[i] = have_row ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      float am = 0.f;
      if (!f16) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            am = max3(am, fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u)));
        }
      }
      // float16 queries are exact as they stand, bfloat16 rows whose largest is from 2^-10 to 2^15
      // but for elements below 2^-17, which are taken to 2^-25; other rows are moved by a power
      // of two, taken back from the scores (and are then exact to 2^-39 of their largest)
      int e = 0;
      if (am > 0.f && am < INFINITY && (am >= 32768.f || am < 0.0009765625f)) e = 14 - ilogbf(am);
      e = min(max(e, -126), 126);
      const float up = __int_as_float((e + 127) << 23);
      post = __int_as_float((127 - e) << 23);
      any_post = __any_sync(0xffffffffu, e != 0);
      const uint32_t dst = sb + F::Q_OFF + s * F::QSUB + r * 128;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        if (!f16) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_h2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
        }
        // 0 4 1 5 2 6 3 7
        sts4(dst + (i >> 3) * 16384 + (((i & 7) ^ (r & 7)) << 4), __byte_perm(w[0], w[2], 0x5410),
             __byte_perm(w[0], w[2], 0x7632), __byte_perm(w[1], w[3], 0x5410),
             __byte_perm(w[1], w[3], 0x7632));
      }
      fence_async();
      __syncwarp();
      if (lane == 0) arrive_rank(sb + F::QF + 8 * s, 0);
    }
    // the warp's rows see at least this many keys
    const int vis_warp = __reduce_min_sync(0xffffffffu, have_row ? vis : 0x7fffffff);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < my_nt; ++j) {
      ok = wait_for(sb + F::SF + 8 * s, j & 1, abort_flag, DEV_ERR_EPI_WAIT);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_after();
      // A tile in which some row of the warp hides keys, or whose scores carry a row's power of
      // two, is put right in tensor memory first (a rolled loop: with this in the unrolled code
      // the roles' code missed the instruction cache in 30% of its requests, and 8192 tokens of
      // 8 x 4 heads took 827 us instead of 592).
      const uint32_t gone = miss[j & 7];
      if (any_post || key0 + j * KT + KT > vis_warp || gone != 0) {
        const int lim = vis - key0 - j * KT;
#pragma unroll 1
        for (int c = 0; c < KT; c += 16) {
          float x[16];
          tm_ld16(tS + c, reinterpret_cast<uint32_t*>(x));
          tm_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const bool hide = c + k >= lim || ((gone >> (c >> 4)) & 1u);
            x[k] = hide ? -INFINITY : x[k] * post;
          }
          tm_st16(tS + c, reinterpret_cast<uint32_t*>(x));
        }
        tm_st_wait();
      }
      float x[KT];
#pragma unroll
      for (int c = 0; c < KT; c += 32) tm_ld32(tS + c, reinterpret_cast<uint32_t*>(x + c));
      tm_ld_wait();
      float mx;
      {
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < KT - 4; c += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = max3(m4[k], x[c + k], x[c + 4 + k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], x[KT - 4 + k]);
        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
      const bool grow = mx > m + GROW || (m == -INFINITY && mx > -INFINITY);
      if (__any_sync(0xffffffffu, grow)) {
        const float al = grow ? ex2(m - mx) : 1.f;
        if (grow) m = mx;
        l *= al;
        if (j > 0) {
          // the products so far are in o: wait for the last of them
          ok = wait_for(sb + F::OF + 8 * s, (j - 1) & 1, abort_flag, DEV_ERR_EPI_WAIT);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tm_ld16(tO + c, o);
            tm_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tm_st16(tO + c, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const float2 nref = make_float2(UP - ref, UP - ref);
      float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          const int c = 64 * h + k;
          const float2 u = __fadd2_rn(make_float2(x[c], x[c + 1]), nref);
          const float2 v = __fadd2_rn(make_float2(x[c + 2], x[c + 3]), nref);
          const float2 wu = make_float2(ex2(u.x), ex2(u.y)), wv = make_float2(ex2(v.x), ex2(v.y));
          la = __fadd2_rn(la, wu);
          lb = __fadd2_rn(lb, wv);
          pk[k / 2] = pack_h2(wu.x, wu.y);
          pk[k / 2 + 1] = pack_h2(wv.x, wv.y);
        }
        tm_st16(tS + 32 * h, pk);
        tm_st16(tS + 32 * h + 16, pk + 16);
        if (h == 0) {                                      // the first half's product may start
          tm_st_wait();
          tc_before();
          __syncwarp();
          if (lane == 0) arrive_rank(sb + F::PF + 8 * s, 0);
        }
      }
      la = __fadd2_rn(la, lb);
      l += la.x + la.y;
      tm_st_wait();
      tc_before();
      __syncwarp();
      if (lane == 0) arrive_rank(sb + F::PG + 8 * s, 0);
    }
    // ---- o
    if (ok && my_nt > 0)
      ok = wait_for(sb + F::OF + 8 * s, (my_nt - 1) & 1, abort_flag, DEV_ERR_EPI_WAIT);
    if (SPLIT) {
      if (__all_sync(0xffffffffu, ok)) {
        tc_after();
        const int64_t at_row = row - row0;
        if (have_row) ws.ml[static_cast<int64_t>(part) * ROWS + at_row] = make_float2(m, l);
        float4* dst = ws.o + static_cast<int64_t>(part) * (D / 4) * ROWS + at_row;
        if (my_nt > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tm_ld16(tO + c, o);
            tm_ld_wait();
            if (have_row && l != 0.f) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                dst[static_cast<int64_t>((c + i) / 4) * ROWS] =
                    make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                                __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
            }
          }
        }
      }
    } else if (__all_sync(0xffffffffu, ok)) {
      tc_after();
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      const int64_t orow = static_cast<int64_t>(first + tok) * p.Hq + hq;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (have_row ? orow * D : 0));
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (my_nt > 0) {
          tm_ld32(tO + c, o);
          tm_ld_wait();
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = none ? 0.f : __uint_as_float(o[i]) * inv;
        if (have_row) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) dst[(c + i) / 8] = out_eight(v + i, p.out_dt);
        }
      }
      if (p.lse && have_row)
        p.lse[orow] = none ? -INFINITY : 0.6931471805599453f * ((m == -INFINITY ? 0.f : m) + (__log2f(l) - UP));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == 12) {
    // ---------------------------------------------------------------- MMA issue
    // The whole warp walks the loop, so that addresses and descriptors stay warp-uniform; an
    // elected lane issues each group in a branch of its own: 21 to 26 cycles an instruction.
    // (With the loop inside one lane's branch it was 110 beside four softmax warps of its
    // scheduler, 3600 a tile of keys; with every instruction predicated 66, chunks of 1000 behind
    // 16411 538 us for 527.)
    if (rank == 0 && nt > 0) {
      constexpr uint32_t id_qk = idesc(256, KT, false), id_pv = idesc(256, 128, true);
      const uint32_t leader = elect();
      const uint32_t q_lo = ((sb + F::Q_OFF) >> 4) | kDescLead;
      const uint32_t k_lo = ((sb + F::K_OFF) >> 4) | kDescLead;
      const uint32_t v_lo = ((sb + F::V_OFF) >> 4) | kDescLead;
      bool ok = true;
      // step j: O += P V of tile j, then S = Q K^T of tile j + 1, subtile by subtile (one copy
      // of the code for both)
#pragma unroll 1
      for (int j = -1; j < nt; ++j) {
        // both operands' stages first: the waits between a subtile's weights and its next scores
        // are on its critical path (chunks of 1000 behind 16411: 552 -> 538 us)
        if (j >= 0) ok = wait_for(sb + F::VF + 8 * (j % NS), (j / NS) & 1, abort_flag, DEV_ERR_MMA_WAIT);
        if (j + 1 < nt)
          ok = ok && wait_for(sb + F::KF + 8 * ((j + 1) % NS), ((j + 1) / NS) & 1, abort_flag, DEV_ERR_MMA_WAIT);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_after();
#pragma unroll 1
        for (int s = 0; s < 2 && ok; ++s) {
          const int my_nt = s ? nt1 : nt0;
          if (j >= 0 && j < my_nt) {
            const int st = j % NS;
            ok = __all_sync(0xffffffffu, wait_for(sb + F::PF + 8 * s, j & 1, abort_flag, DEV_ERR_MMA_WAIT));
            if (!ok) break;
            tc_after();
            const uint32_t va = v_lo + st * (F::VST >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < KT / 32; ++kk)
                mma_ts(256 + 128 * s, 128 * s + 8 * kk, va + ((kk * 2048) >> 4), id_pv, (j | kk) != 0);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, wait_for(sb + F::PG + 8 * s, j & 1, abort_flag, DEV_ERR_MMA_WAIT));
            if (!ok) break;
            tc_after();                                    // the weights' second half
            if (leader) {
#pragma unroll
              for (int kk = KT / 32; kk < KT / 16; ++kk)
                mma_ts(256 + 128 * s, 128 * s + 8 * kk, va + ((kk * 2048) >> 4), id_pv, 1);
              commit_pair(sb + F::OF + 8 * s);
              if (s == 1 || j >= nt1) commit_pair(sb + F::VE + 8 * st);
            }
            __syncwarp();
          }
          const int jn = j + 1;
          if (jn < my_nt) {
            const int st = jn % NS;
            if (jn == 0) {
              ok = __all_sync(0xffffffffu, wait_for(sb + F::QF + 8 * s, 0, abort_flag, DEV_ERR_MMA_WAIT));
              if (!ok) break;
              tc_after();
            }
            const uint32_t qa = q_lo + s * (F::QSUB >> 4), ka = k_lo + st * (F::KST >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(128 * s, qa + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                     ka + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), id_qk, kk != 0);
              commit_pair(sb + F::SF + 8 * s);
              if (s == 1 || jn >= nt1) commit_pair(sb + F::KE + 8 * st);
            }
            __syncwarp();
          }
        }
      }
      // every MMA issued above has completed once this commit arrives
      if (leader) commit_local(sb + F::DR);
      __syncwarp();
      const uint64_t t0 = now_ns();
      while (!bar_try(sb + F::DR, 0) && now_ns() - t0 < 2000000000ull) {
      }
    }
    __syncwarp();
    } else if (warp == 13) {
      // -------------------------------------------------------------- raw cells
      const int32_t* row_table = p.table + static_cast<int64_t>(b) * p.width;
      int fetched = 0, id = -1;
      uint32_t pg = 0;
      // lane i < 8 finds the page of cell i of tile j, a tile before its copy is issued
      auto look = [&](int j) {
        const int ci = key0 / kCell + j * 8 + lane;
        id = -1;
        if (lane < 8 && ci < n_cell) {
          pg = static_cast<uint32_t>(ci) / static_cast<uint32_t>(p.pool.cells);
          id = row_table[pg];
        }
      };
      bool ok = true;
      if (nt > 0) look(0);
      for (int j = 0; j < nt; ++j) {
        const int st = j % NR, ci = key0 / kCell + j * 8 + lane;
        if (j >= NR) ok = wait_for(sb + F::RE + 8 * st, (j / NR - 1) & 1, abort_flag, DEV_ERR_TMA_WAIT);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        // whole cells where this CTA expands K, the rest without their K codes
        const bool have = id >= 0 && id < p.pool.n_pages;
        const bool mine = (lane >> 2) == static_cast<int>(rank);
        const uint32_t all = __ballot_sync(0xffffffffu, have);
        const uint32_t own = __ballot_sync(0xffffffffu, have && mine);
        const uint32_t wanted = __ballot_sync(0xffffffffu, lane < 8 && ci < n_cell);
        if (lane == 0) {
          mask[st] = all;
          miss[j & 7] = wanted & ~all;
          bar_expect(sb + F::RF + 8 * st,
                     __popc(own) * C::BYTES + __popc(all & ~own) * (C::BYTES - C::V));
        }
        __syncwarp();
        if (have) {
          const uint8_t* src = p.pool.data +
                               ((static_cast<int64_t>(id) * p.pool.Hkv + kvh) * p.pool.cells +
                                (ci - static_cast<int>(pg) * p.pool.cells)) *
                                   static_cast<int64_t>(C::BYTES);
          const int skip = mine ? 0 : C::V;
          bulk_load(sb + F::RAW_OFF + st * F::RAW + lane * C::BYTES + skip, src + skip,
                    C::BYTES - skip, sb + F::RF + 8 * st);
        }
        ++fetched;
        look(j + 1);
      }
      if (!ok)                                             // copies in flight land before the end
        for (int i = fetched > NR ? fetched - NR : 0; i < fetched; ++i) {
          const uint64_t t0 = now_ns();
          while (!bar_try(sb + F::RF + 8 * (i % NR), (i / NR) & 1) && now_ns() - t0 < 2000000000ull) {
          }
        }
    } else if (warp < 12) {
      // -------------------------------------------------------------- expand
      const bool is_k = warp < 10;
      const int ct = (threadIdx.x - 256) & 63;             // thread of the two warps
      const float cq = p.scale * kLog2e;
      const int passes = is_k ? D / 32 : D == 128 || rank == 0 ? 4 : 0;
      const int piece_mask = is_k ? D / 32 - 1 : 1;
      const int code_off = is_k ? C::K : C::V + (D == 128 ? 32 * static_cast<int>(rank) : 0);
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        const int rs = j % NR, st = j % NS;
        const uint32_t raw = sb + F::RAW_OFF + rs * F::RAW;
        ok = wait_for(sb + F::RF + 8 * rs, (j / NR) & 1, abort_flag, DEV_ERR_TMA_WAIT);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const uint32_t cells = mask[rs];
        const int left = vis_max - key0 - j * KT;          // keys of the tile that anyone sees
        // Steps of key t's K or V row. A key that is not there gets zeros. A NaN step, or one whose
        // row has values that float16 rounds to infinity (a row's codes are 0 to 15), is kept out
        // of V, where it would meet the zero weights of rows that do not see the key, and a NaN put
        // into K instead, whose scores are masked row by row.
        auto steps = [&](int t, bool k) {
          const uint32_t a = raw + (t >> 4) * C::BYTES + C::KH + 4 * (t & 15);
          float h = 0.f, z = 0.f;
          if (((cells >> (t >> 4)) & 1u) && t < left) {
            const float kh = lds_f(a), vh = lds_f(a + 128);
            const float kz = static_cast<float>(lds_i(a + 64)), vz = static_cast<float>(lds_i(a + 192));
            const bool bad = !(kh == kh) || !(vh * fmaxf(fabsf(vz), fabsf(15.f - vz)) < 65520.f);
            h = k ? (bad ? NAN : kh * cq) : (bad ? 0.f : vh);
            z = k ? kz : vz;
          }
          return row_steps(h, z);
        };
        // K: this CTA's 64 keys, one a thread; V: its 64 columns (for D = 64 the first CTA's)
        // of keys ct and ct + 64. A pass expands 16 bytes of codes; which of the row's 16-byte
        // pieces it takes turns with the key, so loads and stores are free of bank conflicts.
        const int t0 = is_k ? 64 * static_cast<int>(rank) + ct : ct;
        const RowSteps r0 = steps(t0, is_k), r1 = is_k ? r0 : steps(ct + 64, false);
        if (j >= NS)
          ok = wait_for((is_k ? sb + F::KE : sb + F::VE) + 8 * st, (j / NS - 1) & 1, abort_flag,
                        DEV_ERR_TMA_WAIT);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int i = 0; i < passes; ++i) {
          const int t = is_k ? t0 : ct + 64 * (i >> 1);
          const int qd = (i + (ct >> 1)) & piece_mask;
          const uint32_t codes = raw + (t >> 4) * C::BYTES + (t & 15) * C::ROW + code_off + 16 * qd;
          const uint32_t out = (is_k ? sb + F::K_OFF + st * F::KST + ct * 128 + (qd >> 1) * 8192
                                     : sb + F::V_OFF + st * F::VST + t * 128);
          expand4(lds128(codes), is_k || i < 2 ? r0 : r1, out, 4 * (qd & 1), ct & 7);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          arrive_rank((is_k ? sb + F::KF : sb + F::VF) + 8 * st, 0);
          bar_arrive(sb + F::RE + 8 * rs);
        }
      }
    }
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  cluster_sync_all();
  tc_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// o of the rows of items whose keys were shared: sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M),
// M the largest m_i, in the parts' order. A block takes 64 rows of an item; a lane a row (the
// parts' loads are contiguous), a warp every fourth 8 columns.
template <int D>
__global__ void __launch_bounds__(256) kv_tiles_join_kernel(AttnParams p, int pieces, TilesSpace ws) {
  pdl_wait();
  pdl_launch();
  const int item = blockIdx.x / (ROWS / 64), g = blockIdx.x % (ROWS / 64);
  const int2 at = ws.desc[item];
  if (at.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = item % p.pool.Hkv, r = g * 64 + (warp & 1) * 32 + lane;
  const int first = p.cu[at.x];
  const int n_new = min(max(p.cu[at.x + 1] - first, 0), p.max_q);
  const int row = at.y * ROWS + r, tok = row / p.G, hq = kvh * p.G + row - tok * p.G;
  if (tok >= n_new || first + tok >= p.T) return;
  const float2* ml = ws.ml + static_cast<int64_t>(item) * pieces * ROWS + r;
  float M = -INFINITY;
  for (int i = 0; i < pieces; ++i) M = fmaxf(M, ml[static_cast<int64_t>(i) * ROWS].x);
  const float ref = M == -INFINITY ? 0.f : M;
  constexpr int CH = D / 32;                               // groups of 8 columns of a warp
  float l = 0.f, o[CH][8] = {};
  const float4* src = ws.o + static_cast<int64_t>(item) * pieces * (D / 4) * ROWS + r;
#pragma unroll 2
  for (int i = 0; i < pieces; ++i) {
    const float2 t = ml[static_cast<int64_t>(i) * ROWS];
    if (t.y == 0.f) continue;                              // no key (a NaN sum goes on)
    const float f = ex2((t.x == -INFINITY ? 0.f : t.x) - ref);
    l += t.y * f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 x = src[(static_cast<int64_t>(i) * (D / 4) + 2 * ((warp >> 1) + 4 * c) + k) * ROWS];
        o[c][4 * k] += x.x * f;
        o[c][4 * k + 1] += x.y * f;
        o[c][4 * k + 2] += x.z * f;
        o[c][4 * k + 3] += x.w * f;
      }
    }
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  const int64_t orow = static_cast<int64_t>(first + tok) * p.Hq + hq;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow * D);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[c][k] *= inv;
    dst[(warp >> 1) + 4 * c] = out_eight(o[c], p.out_dt);
  }
  if (p.lse && warp < 2) p.lse[orow] = none ? -INFINITY : 0.6931471805599453f * (ref + (__log2f(l) - UP));
}

// How a launch is laid out; the workspace depends on it.
struct TilesPlan {
  int64_t list;        // row tiles of all requests, at most
  int64_t items;       // the same of all kv heads
  int pieces;          // pairs that share an item's keys
  int64_t us;          // estimated time of requests of equal lengths
};
TilesPlan plan_tiles(const AttnParams& p, int min_rows) {
  TilesPlan r;
  const int64_t most = ceil_div(static_cast<int64_t>(p.max_q) * p.G, ROWS) * p.n_req;
  // the requests' rows are at most T G: so many full tiles, and one more of each request that
  // has enough rows
  const int64_t rows = p.T * p.G;
  const int64_t reqs = min_rows > 0 && rows / min_rows < p.n_req ? rows / min_rows : p.n_req;
  r.list = rows / ROWS + reqs < most ? rows / ROWS + reqs : most;
  r.items = r.list * p.pool.Hkv;
  const int64_t pairs = num_sms() / 2;
  const int64_t keys = ceil_div(static_cast<int64_t>(p.width) * p.pool.page, KT);
  // Estimated microseconds: 2 a tile of keys, 8 to begin and end a part, 6 for the join. One
  // request of 4096 tokens, 32 kv heads, 512 rows: 2 parts 54, whole 77; 2 requests of 8 kv heads,
  // 1024 rows: 2 parts 59, whole 82; 4 of 1024 tokens, 1024 rows: whole 36. Several requests may
  // be as long as each other or, as likely, spread evenly below the longest, when shares even
  // out the pairs: 33 requests of up to 53063 tokens, 2 kv heads, 33 x 4 rows: 3 parts 556, whole
  // 804 (of 20000 tokens each: 339, whole 309).
  int64_t best = 0;
  r.pieces = 1;
  for (int64_t n = 1; n <= 64 && (n == 1 || (n <= keys && n * r.items <= 3 * pairs)); ++n) {
    const int64_t part = ceil_div(keys, n), longest = 2 * part + 8;
    const int64_t equal = ceil_div(n * r.items, pairs) * longest;
    const int64_t mean = n * r.items * (part + 8) / pairs + longest / 2;
    const int64_t spread = p.n_req == 1 ? equal : mean > longest ? mean : longest;
    const int64_t us = equal + spread + (n > 1 ? 12 : 0);
    if (n == 1 || us < best) {
      best = us;
      r.pieces = static_cast<int>(n);
      r.us = equal + (n > 1 ? 6 : 0);
    }
  }
  return r;
}
template <int D>
size_t space_of(const TilesPlan& r, void* base, TilesSpace* ws) {
  if (r.pieces == 1) return 0;
  const size_t parts = static_cast<size_t>(r.items) * r.pieces;
  const size_t o = parts * ROWS * D * 4, ml = parts * ROWS * 8;
  if (ws) {
    ws->o = static_cast<float4*>(base);
    ws->ml = reinterpret_cast<float2*>(static_cast<char*>(base) + o);
    ws->desc = reinterpret_cast<int2*>(static_cast<char*>(base) + o + ml);
  }
  return o + ml + static_cast<size_t>(r.items) * sizeof(int2);
}

template <int D, bool SPLIT>
omq_status ready_on(int dev) {
  static thread_local int ready = -1;
  if (ready == dev) return OMQ_OK;
  cudaError_t e = cudaFuncSetAttribute(kv_tiles_kernel<D, SPLIT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, TilesCfg<D>::SMEM);
  cudaFuncAttributes fa = {};
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kv_tiles_kernel<D, SPLIT>);
  if (e != cudaSuccess) {
    set_cuda_error(e);
    return OMQ_ERR_CUDA;
  }
  // the softmax warps' larger share would wait for registers that were never allocated
  if (fa.numRegs < REGS) return OMQ_ERR_UNSUPPORTED;
  ready = dev;
  return OMQ_OK;
}

template <int D>
omq_status launch_tiles(const AttnParams& p, int min_rows, void* space, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  const TilesPlan r = plan_tiles(p, min_rows);
  TilesSpace ws = {};
  space_of<D>(r, space, &ws);
  const omq_status s = r.pieces > 1 ? ready_on<D, true>(dev) : ready_on<D, false>(dev);
  if (s != OMQ_OK) return s;
  const dim3 grid(static_cast<unsigned>(2 * r.items * r.pieces));
  if (r.pieces > 1) {
    launch_k(kv_tiles_kernel<D, true>, grid, THREADS, TilesCfg<D>::SMEM, st, p, r.pieces, min_rows, ws);
    launch_k(kv_tiles_join_kernel<D>, dim3(static_cast<unsigned>(r.items * (ROWS / 64))), 256, 0, st, p,
             r.pieces, ws);
  } else {
    launch_k(kv_tiles_kernel<D, false>, grid, THREADS, TilesCfg<D>::SMEM, st, p, 1, min_rows, ws);
  }
  return launch_status();
}

}  // namespace

int64_t attn_tiles_us(const AttnParams& p, int min_rows) { return plan_tiles(p, min_rows).us; }

size_t attn_tiles_space(const AttnParams& p, int64_t D, int min_rows) {
  const TilesPlan r = plan_tiles(p, min_rows);
  return D == 128 ? space_of<128>(r, nullptr, nullptr) : space_of<64>(r, nullptr, nullptr);
}

omq_status launch_attn_tiles(const AttnParams& p, int64_t D, int min_rows, void* space, cudaStream_t st) {
  return D == 128 ? launch_tiles<128>(p, min_rows, space, st) : launch_tiles<64>(p, min_rows, space, st);
}

}  // namespace kv
}  // namespace omq
