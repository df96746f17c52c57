// Attention of many query rows (prompts and their chunks) over the 4-bit paged cache on the
// 5th-generation tensor cores (tcgen05, sm_100a).
//
// The mathematics is that of kv_rows.cu, with the zero points taken out before the products:
//   x_ij = a_j (q_i . (c_j - z_j)) + log2 hv_j,  a_j = scale log2(e) hk_j
//   w_ij = 2^(x_ij - m_i),  o_i = sum_j w_ij (cv_j - zv_j) / sum_j (w_ij / hv_j)
// c - z is an integer: as the float16 operand (c - z) 2^-14 it is exact up to 2048 (beyond, its
// rounding is relative 2^-11: rows whose values are all 100 times further from zero than they
// spread). w_ij is rounded to float16; statistics, sums and accumulators are float32. The
// reference m_i follows the row's maximum only when that has grown by more than 2^8, so o is
// rescaled rarely; the result is the same in exact arithmetic.
//
// A pair of CTAs (cluster of 2, cta_group::2) takes 512 query rows of one (request, kv head),
// row r = new token r / G, query head r mod G of the group: two subtiles of 256 rows, whose
// products and softmax alternate (while one subtile's scores become weights, the other's
// products run). Per 128 keys: S = Q K^T (256 x 128 x D), O += P V (256 x D x 128), P straight
// from tensor memory, where it takes S's place. Each CTA expands the keys' codes it contributes
// to the pair's operands: K of 64 keys, V's 64 columns of all 128 keys (for D = 64 the second
// CTA's V half stays zero). Expanding costs an AND and a half-precision FMA per two codes; the
// order in which a word yields its 8 values (0 4 1 5 2 6 3 7) is kept in both operands (Q is
// staged in the same order) and undone where o is written.
// Warp roles (384 threads):
//   0-3, 4-7  softmax of subtile 0 / 1, a row a thread (32 TMEM lanes a warp); they also stage
//             Q and write o
//   8         MMA issue (one lane of the leader CTA); TMEM allocation
//   9-11      expand codes and steps; warp 9 issues the bulk copies of the raw cells
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
constexpr int NM = 2;                 // stages of the keys' steps
constexpr int CONV = 96;              // expanding threads
constexpr int THREADS = 384;
constexpr float GROW = 8.f;           // growth of a row's maximum (log2) that moves m_i

template <int D>
struct TilesCfg {
  using C = CellT<D>;
  static constexpr int QSUB = 128 * D * 2;               // one subtile's Q rows of a CTA
  static constexpr int KST = 64 * D * 2;                 // K stage: 64 keys
  static constexpr int VST = KT * 64 * 2;                // V stage: 64 columns of 128 keys
  static constexpr int RAW = (KT / kCell) * C::BYTES;
  static constexpr int Q_OFF = 0, K_OFF = 2 * QSUB, V_OFF = K_OFF + NS * KST,
                       RAW_OFF = V_OFF + NS * VST, META_OFF = RAW_OFF + NR * RAW,
                       CTL = META_OFF + NM * 3 * KT * 4;
  // barriers
  static constexpr int QF = CTL, KF = QF + 16, KE = KF + 8 * NS, VF = KE + 8 * NS,
                       VE = VF + 8 * NS, SF = VE + 8 * NS, PF = SF + 16, OF = PF + 16,
                       RF = OF + 16, RE = RF + 8 * NR, MF = RE + 8 * NR, ME = MF + 8 * NM, DR = ME + 8 * NM,
                       MASK = DR + 8, SLOT = MASK + 4 * NR, ABORT = SLOT + 4, END = ABORT + 4;
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
__device__ __forceinline__ void arrive_rank(uint32_t bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
               ::"r"(map_rank(bar, rank)) : "memory");
}
__device__ __forceinline__ bool try_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Bounded wait; also gives up once the CTA's abort flag is set.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         unsigned bit) {
  if (try_cluster(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  const uint64_t lim = *const_cast<const volatile uint64_t*>(&g_tiles_limit_ns);
  while (!try_cluster(bar, parity)) {
    if (*abort_flag) return false;
    if (now_ns() - t0 > lim) {
      atomicOr(&g_tiles_error, bit);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
// Operand descriptor, 128-byte swizzle (start, leading and stride byte offsets in 16-byte
// units, version 1, layout 2).
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46 |
         static_cast<uint64_t>(2) << 61;
}
// float16 operands, float32 accumulator: B K-major or MN-major, N / 8, M / 16.
constexpr uint32_t idesc(int m, int n, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(id), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
      "r"(id), "r"(acc));
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
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ldsf4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
               ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void stsf(uint32_t a, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
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
__device__ __forceinline__ float lg2a(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpa(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (c - z) 2^-14 of a word's eight codes, in the order 0 4 1 5 2 6 3 7; nz = (-z 2^-14) twice.
__device__ __forceinline__ void expand(uint32_t w, uint32_t nz, uint32_t addr) {
  const uint32_t w8 = w >> 8;
  // a code in the low nibble is c 2^-24 as it stands, in the next one 16 c 2^-24
  const uint32_t o0 = hfma2(w & 0x000F000Fu, 0x64006400u, nz);     // 2^10
  const uint32_t o1 = hfma2(w & 0x00F000F0u, 0x54005400u, nz);     // 2^6
  const uint32_t o2 = hfma2(w8 & 0x000F000Fu, 0x64006400u, nz);
  const uint32_t o3 = hfma2(w8 & 0x00F000F0u, 0x54005400u, nz);
  sts4(addr, o0, o1, o2, o3);
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    kv_tiles_kernel(AttnParams p, int tiles, int min_rows) {
  using F = TilesCfg<D>;
  using C = CellT<D>;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + F::ABORT);
  volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + F::MASK);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + F::SLOT);

  // the last tiles of the requests see the most keys: they go first
  const int item = blockIdx.x >> 1;
  const int per = p.n_req * p.pool.Hkv;
  const int tile = tiles - 1 - item / per;
  const int kvh = (item % per) % p.pool.Hkv;
  const int b = (item % per) / p.pool.Hkv;

  pdl_wait();
  pdl_launch();
  const int len = min(max(p.lens[b], 0), p.width * p.pool.page);
  const int first = p.cu[b];
  const int n_new = min(max(p.cu[b + 1] - first, 0), p.max_q);
  const int rows = n_new * p.G;
  const int row0 = tile * 512;
  if (row0 >= rows || rows < min_rows || first < 0) return;    // the same for both CTAs

  auto row_vis = [&](int r) {
    if (r >= rows || first + r / p.G >= p.T) return 0;
    return p.causal ? min(max(len - n_new + r / p.G + 1, 0), len) : len;
  };
  const int vis_max = row_vis(min(row0 + 511, rows - 1));
  const int nt = (vis_max + KT - 1) / KT;
  const int n_cell = (vis_max + kCell - 1) / kCell;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      bar_init(sb + F::QF + 8 * s, 8);        // leader's: four warps of either CTA
      bar_init(sb + F::SF + 8 * s, 1);
      bar_init(sb + F::PF + 8 * s, 8);        // leader's
      bar_init(sb + F::OF + 8 * s, 1);
    }
    for (int s = 0; s < NS; ++s) {
      bar_init(sb + F::KF + 8 * s, 6);        // leader's: three warps of either CTA
      bar_init(sb + F::KE + 8 * s, 1);
      bar_init(sb + F::VF + 8 * s, 6);        // leader's
      bar_init(sb + F::VE + 8 * s, 1);
    }
    for (int s = 0; s < NR; ++s) {
      bar_init(sb + F::RF + 8 * s, 1);
      bar_init(sb + F::RE + 8 * s, 3);
    }
    for (int s = 0; s < NM; ++s) {
      bar_init(sb + F::MF + 8 * s, 3);
      bar_init(sb + F::ME + 8 * s, 8);
    }
    bar_init(sb + F::DR, 1);
    *abort_flag = 0;
    bar_init_fence();
  }
  if (warp == 8) {
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
  const uint32_t tmem = *slot;
  // TMEM columns: S / P of subtile s at 128 s, O of subtile s at 256 + 128 s

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int s = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;                        // row of the CTA's half subtile
    const int row = row0 + 256 * s + 128 * static_cast<int>(rank) + r;
    const int vis = row_vis(row);
    const bool have_row = row < rows && first + row / p.G < p.T;
    const int tok = row / p.G, hq = kvh * p.G + row - tok * p.G;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = lane_base + 128 * s, tO = lane_base + 256 + 128 * s;
    float post = 1.f;                                      // 2^-e of a row staged as q 2^e
    bool any_post = false;
    {
      const bool f16 = p.dt == OMQ_F16;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) +
          (have_row ? static_cast<int64_t>(first + tok) * p.q_ld + static_cast<int64_t>(hq) * D : 0));
      float am = 0.f;
      if (!f16 && have_row) {
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 u = __ldg(src + i);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            am = fmaxf(am, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                 fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
        }
      }
      // float16 queries, and bfloat16 rows within its range, are exact as they stand; others
      // are moved by a power of two, taken back from the scores
      int e = 0;
      if (am > 0.f && am < INFINITY && (am >= 32768.f || am < 0.0009765625f)) e = 14 - ilogbf(am);
      e = min(max(e, -126), 126);
      const float up = __int_as_float((e + 127) << 23);
      post = __int_as_float((127 - e) << 23);
      any_post = __any_sync(0xffffffffu, e != 0);
      const uint32_t dst = sb + F::Q_OFF + s * F::QSUB + r * 128;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint4 u = have_row ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
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
    for (int j = 0; j < nt && ok; ++j) {
      const int ms = j % NM;
      ok = wait_for(sb + F::MF + 8 * ms, (j / NM) & 1, abort_flag, DEV_ERR_EPI_WAIT) &&
           wait_for(sb + F::SF + 8 * s, j & 1, abort_flag, DEV_ERR_EPI_WAIT);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_after();
      const uint32_t meta = sb + F::META_OFF + ms * 3 * KT * 4;
      float x[KT];
#pragma unroll
      for (int c = 0; c < KT; c += 32) tm_ld32(tS + c, reinterpret_cast<uint32_t*>(x + c));
      tm_ld_wait();
      if (any_post) {
#pragma unroll
        for (int c = 0; c < KT; ++c) x[c] *= post;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < KT; c += 4) {
        const float4 a = ldsf4(meta + 4 * c), lh = ldsf4(meta + 4 * (KT + c));
        const float2 u = __ffma2_rn(make_float2(x[c], x[c + 1]), make_float2(a.x, a.y),
                                    make_float2(lh.x, lh.y));
        const float2 v = __ffma2_rn(make_float2(x[c + 2], x[c + 3]), make_float2(a.z, a.w),
                                    make_float2(lh.z, lh.w));
        x[c] = u.x; x[c + 1] = u.y; x[c + 2] = v.x; x[c + 3] = v.y;
      }
      if (j * KT + KT > vis_warp) {
        const int lim = vis - j * KT;
#pragma unroll
        for (int c = 0; c < KT; ++c) x[c] = c < lim ? x[c] : -INFINITY;
      }
      {
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < KT; c += 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], x[c + k]);
        }
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
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tm_ld32(tO + c, o);
            tm_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tm_st32(tO + c, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const float2 nref = make_float2(-ref, -ref);
      float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const int cc = 64 * h + c;
          const float4 rh = ldsf4(meta + 4 * (2 * KT + cc));
          const float2 u = __fadd2_rn(make_float2(x[cc], x[cc + 1]), nref);
          const float2 v = __fadd2_rn(make_float2(x[cc + 2], x[cc + 3]), nref);
          const float2 wu = make_float2(ex2(u.x), ex2(u.y)), wv = make_float2(ex2(v.x), ex2(v.y));
          l2 = __ffma2_rn(wu, make_float2(rh.x, rh.y), l2);
          l2 = __ffma2_rn(wv, make_float2(rh.z, rh.w), l2);
          pk[c / 2] = pack_h2(wu.x, wu.y);
          pk[c / 2 + 1] = pack_h2(wv.x, wv.y);
        }
        tm_st32(tS + 32 * h, pk);
      }
      l += l2.x + l2.y;
      tm_st_wait();
      tc_before();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(sb + F::ME + 8 * ms);
        arrive_rank(sb + F::PF + 8 * s, 0);
      }
    }
    // ---- o
    if (ok && nt > 0)
      ok = wait_for(sb + F::OF + 8 * s, (nt - 1) & 1, abort_flag, DEV_ERR_EPI_WAIT);
    if (__all_sync(0xffffffffu, ok)) {
      tc_after();
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 16384.f / l;
      const int64_t orow = static_cast<int64_t>(first + tok) * p.Hq + hq;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (have_row ? orow * D : 0));
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (nt > 0) {
          tm_ld32(tO + c, o);
          tm_ld_wait();
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = none ? 0.f : __uint_as_float(o[i]) * inv;
        if (have_row) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            // elements 0 .. 7 stand at 0 2 4 6 1 3 5 7
            uint32_t w[4];
            if (p.out_dt == OMQ_F16) {
              w[0] = pack_h2(v[i], v[i + 2]);
              w[1] = pack_h2(v[i + 4], v[i + 6]);
              w[2] = pack_h2(v[i + 1], v[i + 3]);
              w[3] = pack_h2(v[i + 5], v[i + 7]);
            } else {
              const int e0[4] = {0, 4, 1, 5}, e1[4] = {2, 6, 3, 7};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 q = __floats2bfloat162_rn(v[i + e0[k]], v[i + e1[k]]);
                w[k] = *reinterpret_cast<const uint32_t*>(&q);
              }
            }
            dst[(c + i) / 8] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (p.lse && have_row)
        p.lse[orow] = none ? -INFINITY : 0.6931471805599453f * ((m == -INFINITY ? 0.f : m) + __log2f(l));
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0 && rank == 0 && nt > 0) {
      constexpr uint32_t id_qk = idesc(256, KT, false), id_pv = idesc(256, 128, true);
      bool ok = true;
      auto qk = [&](int s, int j) {
        const int st = j % NS;
        if (j == 0) ok = ok && wait_for(sb + F::QF + 8 * s, 0, abort_flag, DEV_ERR_MMA_WAIT);
        if (s == 0) ok = ok && wait_for(sb + F::KF + 8 * st, (j / NS) & 1, abort_flag, DEV_ERR_MMA_WAIT);
        if (!ok) return;
        tc_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + 128 * s,
                 sdesc(sb + F::Q_OFF + s * F::QSUB + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                 sdesc(sb + F::K_OFF + st * F::KST + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024),
                 id_qk, kk != 0);
        commit_pair(sb + F::SF + 8 * s);
        if (s == 1) commit_pair(sb + F::KE + 8 * st);
      };
      auto pv = [&](int s, int j) {
        const int st = j % NS;
        if (s == 0) ok = ok && wait_for(sb + F::VF + 8 * st, (j / NS) & 1, abort_flag, DEV_ERR_MMA_WAIT);
        ok = ok && wait_for(sb + F::PF + 8 * s, j & 1, abort_flag, DEV_ERR_MMA_WAIT);
        if (!ok) return;
        tc_after();
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_ts(tmem + 256 + 128 * s, tmem + 128 * s + 8 * kk,
                 sdesc(sb + F::V_OFF + st * F::VST + kk * 2048, 16384, 1024), id_pv,
                 (j | kk) != 0);
        commit_pair(sb + F::OF + 8 * s);
        if (s == 1) commit_pair(sb + F::VE + 8 * st);
      };
      qk(0, 0);
      qk(1, 0);
      for (int j = 0; j < nt && ok; ++j) {
        pv(0, j);
        if (j + 1 < nt) qk(0, j + 1);
        pv(1, j);
        if (j + 1 < nt) qk(1, j + 1);
      }
      // every MMA issued above has completed once this commit arrives
      commit_local(sb + F::DR);
      const uint64_t t0 = now_ns();
      while (!try_cluster(sb + F::DR, 0) && now_ns() - t0 < 2000000000ull) {
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- expand
    const int ct = threadIdx.x - 288;                      // 0 .. 95
    const int32_t* row_table = p.table + static_cast<int64_t>(b) * p.width;
    const float cq = p.scale * kLog2e * 16384.f;
    int fetched = 0;
    // warp 9: the copies of tile j's cells into raw stage j % NR: whole cells where this CTA
    // expands K, the rest without their K codes
    auto fetch = [&](int j) {
      const int st = j % NR, ci = j * 8 + lane;
      int id = -1;
      uint32_t pg = 0;
      if (lane < 8 && ci < n_cell) {
        pg = static_cast<uint32_t>(ci) / static_cast<uint32_t>(p.pool.cells);
        id = row_table[pg];
      }
      const bool have = id >= 0 && id < p.pool.n_pages;
      const bool mine = (lane >> 2) == static_cast<int>(rank);
      const uint32_t all = __ballot_sync(0xffffffffu, have);
      const uint32_t own = __ballot_sync(0xffffffffu, have && mine);
      if (lane == 0) {
        mask[st] = all;
        bar_expect(sb + F::RF + 8 * st,
                   __popc(own) * C::BYTES + __popc(all & ~own) * (C::BYTES - C::V));
      }
      __syncwarp();
      if (have) {
        const uint8_t* src = p.pool.data + ((static_cast<int64_t>(id) * p.pool.Hkv + kvh) * p.pool.cells +
                                            (ci - static_cast<int>(pg) * p.pool.cells)) *
                                               static_cast<int64_t>(C::BYTES);
        const int skip = mine ? 0 : C::V;
        bulk_load(sb + F::RAW_OFF + st * F::RAW + lane * C::BYTES + skip, src + skip, C::BYTES - skip,
                  sb + F::RF + 8 * st);
      }
      ++fetched;
    };
    if (warp == 9)
      for (int j = 0; j < NR && j < nt; ++j) fetch(j);
    bool ok = true;
    int j = 0;
    for (; j < nt; ++j) {
      const int rs = j % NR, st = j % NS, ms = j % NM;
      const uint32_t raw = sb + F::RAW_OFF + rs * F::RAW;
      ok = wait_for(sb + F::RF + 8 * rs, (j / NR) & 1, abort_flag, DEV_ERR_TMA_WAIT) &&
           (j < NM || wait_for(sb + F::ME + 8 * ms, (j / NM - 1) & 1, abort_flag, DEV_ERR_TMA_WAIT));
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint32_t cells = mask[rs];
      const int left = vis_max - j * KT;                   // keys of the tile that anyone sees
      auto key_ok = [&](int t) { return ((cells >> (t >> 4)) & 1u) && t < left; };
      for (int t = ct; t < KT; t += CONV) {
        const uint32_t a = raw + (t >> 4) * C::BYTES + C::KH + 4 * (t & 15);
        const uint32_t o = sb + F::META_OFF + ms * 3 * KT * 4 + 4 * t;
        const bool there = key_ok(t);
        const float kh = there ? lds_f(a) : 0.f, vh = there ? lds_f(a + 128) : 1.f;
        stsf(o, kh * cq);
        stsf(o + 4 * KT, there ? lg2a(vh) : -INFINITY);
        // a NaN step reaches the rows that see the key through log2 hv, and only those
        stsf(o + 8 * KT, there && vh == vh ? rcpa(vh) : 1.f);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(sb + F::MF + 8 * ms);
      // -z 2^-14 twice (0 for a key that is not there: finite operands everywhere)
      auto neg_z = [&](int t, int off) -> uint32_t {
        const float z = key_ok(t) ? static_cast<float>(lds_i(raw + (t >> 4) * C::BYTES + off + 4 * (t & 15)))
                                  : 0.f;
        const float v = fminf(fmaxf(z * -6.103515625e-05f, -65504.f), 65504.f);
        return pack_h2(v, v);
      };
      // K: 64 keys x D codes, 16 bytes (32 codes) a thread and pass; the quarter of the row
      // turns with the key, so loads and stores are free of bank conflicts
      if (j >= NS) ok = wait_for(sb + F::KE + 8 * st, (j / NS - 1) & 1, abort_flag, DEV_ERR_TMA_WAIT);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      {
        constexpr int QN = D / 32;
        const uint32_t out = sb + F::K_OFF + st * F::KST;
        for (int u = ct; u < 64 * QN; u += CONV) {
          const int key = u & 63, qd = ((u >> 6) + (key >> 1)) % QN;
          const int t = 64 * static_cast<int>(rank) + key;
          const uint4 w = lds128(raw + (t >> 4) * C::BYTES + C::K + (t & 15) * C::ROW + 16 * qd);
          const uint32_t nz = neg_z(t, C::KZ);
          const uint32_t base = out + (qd >> 1) * 8192 + key * 128;
          const int j0 = 4 * (qd & 1), sw = key & 7;
          expand(w.x, nz, base + (((j0 + 0) ^ sw) << 4));
          expand(w.y, nz, base + (((j0 + 1) ^ sw) << 4));
          expand(w.z, nz, base + (((j0 + 2) ^ sw) << 4));
          expand(w.w, nz, base + (((j0 + 3) ^ sw) << 4));
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) arrive_rank(sb + F::KF + 8 * st, 0);
      // V: 128 keys x 64 columns
      if (j >= NS) ok = wait_for(sb + F::VE + 8 * st, (j / NS - 1) & 1, abort_flag, DEV_ERR_TMA_WAIT);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (D == 128 || rank == 0) {
        const uint32_t out = sb + F::V_OFF + st * F::VST;
        const uint32_t half = D == 128 ? 32 * rank : 0;
        for (int u = ct; u < KT * 2; u += CONV) {
          const int key = u & 127, qd = ((u >> 7) + (key >> 1)) & 1;
          const uint4 w = lds128(raw + (key >> 4) * C::BYTES + C::V + (key & 15) * C::ROW + half + 16 * qd);
          const uint32_t nz = neg_z(key, C::VZ);
          const uint32_t base = out + key * 128;
          const int j0 = 4 * qd, sw = key & 7;
          expand(w.x, nz, base + (((j0 + 0) ^ sw) << 4));
          expand(w.y, nz, base + (((j0 + 1) ^ sw) << 4));
          expand(w.z, nz, base + (((j0 + 2) ^ sw) << 4));
          expand(w.w, nz, base + (((j0 + 3) ^ sw) << 4));
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) arrive_rank(sb + F::VF + 8 * st, 0);
      if (lane == 0) bar_arrive(sb + F::RE + 8 * rs);
      // once all three warps have read the raw stage it takes the tile NR further
      if (warp == 9 && j + NR < nt) {
        ok = wait_for(sb + F::RE + 8 * rs, (j / NR) & 1, abort_flag, DEV_ERR_TMA_WAIT);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          ++j;
          break;
        }
        fetch(j + NR);
      }
    }
    if (!ok && warp == 9)                                  // copies in flight land before the end
      for (int i = j; i < fetched; ++i) {
        const uint64_t t0 = now_ns();
        while (!try_cluster(sb + F::RF + 8 * (i % NR), (i / NR) & 1) && now_ns() - t0 < 2000000000ull) {
        }
      }
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  cluster_sync_all();
  tc_after();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <int D>
omq_status launch_tiles(const AttnParams& p, int min_rows, cudaStream_t st) {
  using F = TilesCfg<D>;
  static thread_local int ready = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (ready != dev) {
    const cudaError_t e = cudaFuncSetAttribute(kv_tiles_kernel<D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return OMQ_ERR_CUDA;
    }
    ready = dev;
  }
  const int64_t tiles = ceil_div(static_cast<int64_t>(p.max_q) * p.G, 512);
  const int64_t items = tiles * p.pool.Hkv * p.n_req;
  launch_k(kv_tiles_kernel<D>, dim3(static_cast<unsigned>(2 * items)), THREADS, F::SMEM, st, p,
           static_cast<int>(tiles), min_rows);
  return launch_status();
}

}  // namespace

omq_status launch_attn_tiles(const AttnParams& p, int64_t D, int min_rows, cudaStream_t st) {
  return D == 128 ? launch_tiles<128>(p, min_rows, st) : launch_tiles<64>(p, min_rows, st);
}

}  // namespace kv
}  // namespace omq
