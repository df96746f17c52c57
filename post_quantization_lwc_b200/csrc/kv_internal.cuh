// Internal declarations of the 4-bit paged key/value cache (kv_api.cu, kv_plan.cu, kv_store.cu,
// kv_rows.cu, kv_tiles.cu): the pool's layout, launch helpers with clusters, and the
// shared-memory barrier, bulk-copy and matrix-instruction wrappers of its kernels.
//
// Pool: uint8 [n_pages, Hkv, page / 16, cell]. A cell holds 16 consecutive tokens of one kv
// head, 16 D + 256 bytes back to back, so one bulk copy brings everything a kernel needs of
// those tokens:
//   K codes [16, D/2] | V codes [16, D/2] | K h f32[16] | K z i32[16] | V h f32[16] | V z i32[16]
// Element d of a row is the nibble d mod 2 (low first) of byte d / 2.
#pragma once

#include "omq_internal.cuh"

namespace omq {
namespace kv {

constexpr int kCell = 16;                     // tokens of a cell
constexpr int kMaxCluster = 8;                // portable cluster size

template <int D>
struct CellT {
  static constexpr int ROW = D / 2;                         // bytes of a token's codes
  static constexpr int K = 0, V = kCell * ROW;
  static constexpr int KH = 2 * kCell * ROW, KZ = KH + 64, VH = KH + 128, VZ = KH + 192;
  static constexpr int BYTES = KH + 256;
};
inline int64_t cell_bytes(int64_t D) { return kCell * D + 256; }

// The pool as a kernel sees it.
struct Pool {
  uint8_t* data;
  int64_t n_pages;
  int Hkv;
  int cells;        // cells per page (page / 16)
  int page;
  int shift;        // log2 of cells where it is a power of two, else -1
};

struct PlanParams {
  const int32_t* lens;
  const int32_t* new_tokens;
  int n_req;
  int32_t* table;
  int width, page;
  int32_t* free_pages;
  int n_pages;
  const int32_t* n_free;
  int32_t* lens_out;
  int32_t* n_free_out;
  int32_t* cu;
  int32_t* slots;
  int32_t* positions;
  int32_t* requests;
  int capacity;
};

struct AppendParams {
  Pool pool;
  int64_t T;
  int Hq;
  const void* q;          // NULL: no queries
  const void* k;
  const void* v;
  int64_t q_ld, k_ld, v_ld;   // elements between tokens
  omq_dtype dt;
  const int32_t* slots;
  const int32_t* positions;   // NULL: no rotation
  const float* rope;          // [2, n_pos, D/2] or NULL
  int64_t n_pos;
  const float* s_a;
  const float* s_o;
  const float* delta_o;
  int quant_q;
  float Qa;
  void* q_out;
  omq_dtype q_dt;
};

struct ReadParams {
  Pool pool;
  int64_t T;
  const int32_t* slots;
  void* k;
  void* v;
  omq_dtype dt;
};

struct AttnParams {
  Pool pool;
  int n_req;
  int64_t T;
  int Hq, G;
  const void* q;
  int64_t q_ld;
  omq_dtype dt;
  const int32_t* table;
  int width;
  const int32_t* lens;
  const int32_t* cu;
  int max_q;
  float scale;
  int causal;
  void* out;
  omq_dtype out_dt;
  float* lse;
};

omq_status launch_plan(const PlanParams& p, cudaStream_t st);
omq_status launch_append(const AppendParams& p, int64_t D, cudaStream_t st);
omq_status launch_read(const ReadParams& p, int64_t D, cudaStream_t st);
// Attention of the requests with at most max_rows query rows per kv head, 8 or 16 rows a block.
omq_status launch_attn_rows(const AttnParams& p, int64_t D, int max_rows, void* space,
                            cudaStream_t st);
size_t attn_rows_space(const AttnParams& p, int64_t D, int max_rows);   // bytes of `space`
// Attention of the requests with at least min_rows query rows per kv head, 512 rows a CTA pair.
omq_status launch_attn_tiles(const AttnParams& p, int64_t D, int min_rows, void* space,
                             cudaStream_t st);
int64_t attn_tiles_us(const AttnParams& p, int min_rows);   // estimate for full tables
size_t attn_tiles_space(const AttnParams& p, int64_t D, int min_rows);

// Per translation unit with barrier waits: read and clear its error flag, set its wait limit
// (the counterparts of take_device_error and set_wait_limit).
cudaError_t rows_take_error(unsigned* flag);
cudaError_t rows_set_limit(uint64_t ns);
cudaError_t tiles_take_error(unsigned* flag);
cudaError_t tiles_set_limit(uint64_t ns);

// kernel<<<grid, block, smem, stream>>> in clusters of `cluster` blocks along x, with
// programmatic stream serialization.
template <typename... KArgs, typename... Args>
cudaError_t launch_cl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                      cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---- device helpers ----------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cta_count() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// (the time hint lets the waiting warp sleep instead of taking issue slots from the others)
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Bounded wait for the phase with the given parity: false (and the error bit raised in *err)
// when it has not completed after *limit nanoseconds.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned* err,
                                         const uint64_t* limit, unsigned bit) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  const uint64_t lim = *const_cast<const volatile uint64_t*>(limit);
  while (!bar_try(bar, parity)) {
    if (now_ns() - t0 > lim) {
      atomicOr(err, bit);
      return false;
    }
  }
  return true;
}
// Asynchronous copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) from this
// GPU's global memory into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A B, A 16 x 16 and B 16 x 8 float16, D float32.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B of the same shapes.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int lds_i(uint32_t a) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

}  // namespace kv
}  // namespace omq
