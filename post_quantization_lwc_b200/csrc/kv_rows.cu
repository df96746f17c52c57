// Attention of a few query rows over the 4-bit paged cache (decoding, drafted tokens, chunks of
// up to 64 rows per kv head and, under short contexts, up to 512), a tile of 8 or 16 rows at a
// time.
//
// o = sum_j p_j v_j with p = softmax_j(scale q . k_j), k_j = (c - z) h and v_j alike. The codes
// themselves are the matrix instructions' operands and the steps stay outside, in binary32:
//   q . k_j       = h_j (sum_d q_d c_jd - z_j sum_d q_d)
//   x_j           = scale log2(e) q . k_j + log2 hv_j,   w_j = 2^(x_j - max x + 15)
//   o             = (sum_j w_j cv_jd - sum_j w_j zv_j) / sum_j (w_j / hv_j)
// so w_j = p_j hv_j up to the row's common factor lies in [0, 2^15] for any hv and its rounding to
// float16 (the operand; the same rounded value weighs zv_j) is relative to the largest
// contribution (zero points far from the codes: see kFarZ); the denominator sums the weights as
// they were, the largest exact in both. A code c < 16 is the float16 subnormal c 2^-24 as it stands, 16 c 2^-24 in the
// second nibble of a 16-bit lane: one AND makes two operands, exact, and the powers of two go
// into q (the odd nibbles' q times 1/16; the tile's q scaled by a power of two, so float16 is
// exact down to 2^-24 of the tile's largest, bfloat16 to 2^-27, and what is below to 2^-35 of it)
// and into the result.
//
// The floor is the cache's bytes: D + 16 per token and kv head. The work is a line of runs of
// 64 tokens, item after item (an item: request, tile of 8 NB rows, kv head), cut into equal parts,
// one a block, whatever the lengths, or into equal shares of each item (plan_rows says when): one
// block per item left the SMs 30% to 80% busy on 64 ragged contexts of up to 8192 tokens, and a
// cluster per item was slower for many items and reached only 128 SMs for few. Within a part each of the block's four warps takes every fourth
// run on its own: a ring of bulk copies (one per 16-token cell, which holds codes and steps
// together), K as the 16 x 16 operand straight from 16-byte shared loads, V transposed by
// ldmatrix, no barrier between warps. At the end of an item or part the warps join their (max,
// sum, o) in a fixed order; an item shared by up to eight blocks is joined by them, a cluster,
// through distributed shared memory, one cut otherwise leaves float32 partials in the workspace,
// which a second kernel joins; in the blocks' order either way.
//
// Measured: 64 decoding requests of up to 8192 tokens, 8 x 4 heads of 128: 80 us (4.0 TB/s), one
// of 131072 38 us (4.0 TB/s), 33 of up to 4001 with 5 drafted tokens, 4 x 2 heads of 64: 22 us, one
// of 2049, 32 heads 10.7 us. Neither DRAM (49%) nor issue (52%) is full: the registers (168 a
// thread) leave 12 warps an SM, each of which waits on its own chain of scores, weights and
// products; of the two, loads alone took 70 us and arithmetic alone 84 of then 92.
#include "kv_internal.cuh"

namespace omq {
namespace kv {

static __device__ unsigned g_rows_error = 0;
static __device__ uint64_t g_rows_limit_ns = 2000000000ull;

cudaError_t rows_take_error(unsigned* flag) {
  unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_rows_error, sizeof(unsigned));
  if (e == cudaSuccess && *flag) e = cudaMemcpyToSymbol(g_rows_error, &zero, sizeof(unsigned));
  return e;
}
cudaError_t rows_set_limit(uint64_t ns) {
  return cudaMemcpyToSymbol(g_rows_limit_ns, &ns, sizeof(ns));
}

namespace {

constexpr int STEP = 64;              // tokens of a run: four cells
constexpr int NCELL = STEP / kCell;
constexpr int STAGES = 2;
// Zero points beyond this are weighed by the float32 weight, not the float16 one: a constant row
// of 5 is 0 + 5e8 steps of 1e-8, and its weight, p 1e-8 beside another token's p 0.1, is below
// float16's numbers. The rounded weight then meets only codes (0 .. 15, less than |c - z|).
constexpr float kFarZ = 64.f;
// The largest weight of a row is 2^15, near the top of float16: what falls below its smallest
// number is then 2^-40 of the largest, and a long context's many small weights are kept.
constexpr float kUp = 15.f;
constexpr int W = 4;                  // warps of a block
constexpr int kCluster = 8;           // blocks that join their shares of an item by themselves

template <int D, int NB>
struct RowsCfg {
  // cells 16 bytes further apart than they are long: the eight token rows of an ldmatrix come
  // two from each of four cells and fall into eight different 16-byte bank groups (D = 128)
  static constexpr int PITCH = CellT<D>::BYTES + 16;
  static constexpr int STAGE = NCELL * PITCH;
  static constexpr int RING = W * STAGES * STAGE;
  static constexpr int R = 8 * NB;                      // query rows of a block
  static constexpr int LDO = D + 4;                     // row stride of the partial outputs
  static constexpr int PART = W * R * LDO * 4;          // the warps' partial outputs (ring reused)
  static constexpr int BODY = RING > PART ? RING : PART;
  static constexpr int STAT = BODY;                     // float [2][W][R]: max, sum
  static constexpr int JOIN = STAT + 2 * W * R * 4;     // float [R][2] the block's (max, sum)
  static constexpr int BARS = JOIN + R * 8;             // mbarriers [W][STAGES]
  static constexpr int SCAN = BARS + W * STAGES * 8;     // int64 [W], then the part's start
  static constexpr int SMEM = SCAN + W * 8 + 16;
};

// The workspace of a cut launch: per block its first and last item's partial o [2][R][D] and
// (max, sum) [2][R][2], and what of the item its first run continues the second kernel needs.
struct PartDesc {
  int joins;            // the item ends here: this block's number joins it
  int row0;             // its first query row: token row0 / G of the request
  int rows;             // its query rows that are stored
  int tok0;             // the request's first row of q and out
  int kvh;
  int first;            // the block it starts in
  int first_slot;       // that block's slot of it
  int pad;
};
struct RowsSpace {
  float* o;
  float2* ml;
  PartDesc* desc;
};

// The two 16-bit values of a word.
__device__ __forceinline__ float2 pair(uint32_t w, bool f16) {
  if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sts128(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
               ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Of a word of codes, per 16-bit lane: the low byte (16 c1 + c0) 2^-24 and c0 2^-24, and the same
// of the high byte. Four operations of the half-rate logic pipe (the masks and shifts are what
// this kernel issues most); 16 c1 is the difference, on the FMA pipe.
struct Nibbles {
  uint32_t u0, l0, u1, l1;
};
__device__ __forceinline__ Nibbles nibbles(uint32_t w) {
  Nibbles n;
  n.u0 = w & 0x00FF00FFu;
  n.l0 = w & 0x000F000Fu;
  n.u1 = __byte_perm(w, 0u, 0x4341);
  n.l1 = n.u1 & 0x000F000Fu;
  return n;
}
__device__ __forceinline__ uint32_t h2(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Two values of an output row from their unnormalised sums, its maximum m and sum l; the first
// column's thread also writes the row's log-sum-exp.
__device__ __forceinline__ void store_row(const AttnParams& p, int64_t orow, int D, int d, float2 o,
                                          float m, float l) {
  const bool none = l == 0.f;                            // a visible key adds 1 / hv, or NaN
  const float inv = none ? 0.f : 1.f / l;
  const float yx = none ? 0.f : o.x * inv, yy = none ? 0.f : o.y * inv;
  uint32_t packed;
  if (p.out_dt == OMQ_F16) {
    packed = h2(yx, yy);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(yx, yy);
    packed = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + orow * D + d) = packed;
  if (p.lse && d == 0) p.lse[orow] = none ? -INFINITY : 0.6931471805599453f * (m + (__log2f(l) - kUp));
}

// Query rows of a request, and its runs per item (one without keys still writes its zeros).
struct ReqWork {
  int len, first, n_new, rows, tiles, runs;
};
template <int R>
__device__ __forceinline__ ReqWork req_work(const AttnParams& p, int b, int max_rows) {
  ReqWork r;
  r.len = min(max(__ldg(p.lens + b), 0), p.width * p.pool.page);
  r.first = __ldg(p.cu + b);
  r.n_new = max(__ldg(p.cu + b + 1) - r.first, 0);
  r.rows = min(r.n_new, p.max_q) * p.G;
  r.tiles = r.rows > max_rows || r.first < 0 ? 0 : (r.rows + R - 1) / R;
  r.runs = max(1, (r.len + STEP - 1) / STEP);
  return r;
}
// Inclusive prefix sum over the block, and its total.
__device__ __forceinline__ int64_t scan_block(int64_t v, volatile int64_t* sm, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) sm[w] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    before += i < w ? sm[i] : 0;
    all += sm[i];
  }
  *total = all;
  return v + before;
}

// pieces == 0: the blocks share the line of runs evenly. pieces > 0: an item has that many
// blocks, each an equal share of its runs, at least one a warp (1: block i takes item i whole);
// together: they are one cluster, which joins them itself. tiles per request and head as the
// host bounds them.
template <int D, int NB>
__global__ void __launch_bounds__(32 * W, NB == 1 ? 3 : 2)
    kv_rows_kernel(AttnParams p, int tiles, int max_rows, int pieces, bool together, RowsSpace ws) {
  using F = RowsCfg<D, NB>;
  using C = CellT<D>;
  constexpr int KM = D / 16;            // K-side matrix steps
  constexpr int VM = D / 16;            // V-side row tiles
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const uint32_t bars = sb + F::BARS + warp * STAGES * 8;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) bar_init(bars + 8 * s, 1);
    bar_init_fence();
  }
  __syncwarp();
  pdl_wait();
  pdl_launch();

  // ---- this block's part of the line: [at, end) in request b, which starts at base
  int b = 0, bt = 0;
  int64_t base = 0, at = 0, end = 0, part = 0;
  const bool cut = pieces == 0;
  if (cut) {
    volatile int64_t* sm = reinterpret_cast<volatile int64_t*>(smem + F::SCAN);
    int64_t total = 0, sum;
    int64_t incl = 0, mine = 0;
    for (int c = 0; c < p.n_req; c += 32 * W) {
      mine = 0;
      if (c + static_cast<int>(threadIdx.x) < p.n_req) {
        const ReqWork r = req_work<F::R>(p, c + threadIdx.x, max_rows);
        mine = static_cast<int64_t>(r.tiles) * p.pool.Hkv * r.runs;
      }
      incl = total + scan_block(mine, sm, &sum);
      total += sum;
    }
    if (threadIdx.x == 0) ws.desc[blockIdx.x].joins = 0;
    // at least a run a warp
    part = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(W));
    at = part * blockIdx.x;
    end = min(at + part, total);
    if (at >= end) return;
    int64_t done = 0;
    for (int c = 0; c < p.n_req; c += 32 * W) {
      if (p.n_req > 32 * W) {                              // else the sums above are these
        mine = 0;
        if (c + static_cast<int>(threadIdx.x) < p.n_req) {
          const ReqWork r = req_work<F::R>(p, c + threadIdx.x, max_rows);
          mine = static_cast<int64_t>(r.tiles) * p.pool.Hkv * r.runs;
        }
        incl = done + scan_block(mine, sm, &sum);
        done += sum;
      }
      if (at < incl && at >= incl - mine) {
        sm[W] = incl - mine;
        reinterpret_cast<volatile int*>(sm + W + 1)[0] = c + threadIdx.x;
      }
      if (p.n_req > 32 * W && done > at) break;            // the same for the whole block
    }
    __syncthreads();
    base = sm[W];
    b = reinterpret_cast<volatile int*>(sm + W + 1)[0];
  } else {
    const int item = blockIdx.x / pieces;
    if (pieces > 1 && !together && threadIdx.x == 0) ws.desc[blockIdx.x].joins = 0;
    bt = item % tiles * p.pool.Hkv + (item / tiles) % p.pool.Hkv;
    b = item / tiles / p.pool.Hkv;
  }

  uint32_t it = 0;                       // runs this warp has taken: its ring position
  int seg = 0;
  bool ok = true;
  for (; cut ? at < end : seg == 0; ++seg) {
  const ReqWork rw = req_work<F::R>(p, b, max_rows);
  int run0 = 0, run1 = rw.runs;
  if (cut) {
    const int64_t off = at - base;
    if (off >= static_cast<int64_t>(rw.tiles) * p.pool.Hkv * rw.runs) {   // the next request
      base += static_cast<int64_t>(rw.tiles) * p.pool.Hkv * rw.runs;
      ++b;
      --seg;
      continue;
    }
    bt = static_cast<int>(off / rw.runs);
    run0 = static_cast<int>(off - static_cast<int64_t>(bt) * rw.runs);
    run1 = static_cast<int>(min(static_cast<int64_t>(rw.runs), run0 + (end - at)));
  } else if (pieces > 1) {
    const int share = max((rw.runs + pieces - 1) / pieces, W);
    run0 = min(static_cast<int>(blockIdx.x) % pieces * share, rw.runs);
    run1 = min(run0 + share, rw.runs);
    if (run0 >= rw.runs && !together) return;
  }
  const int tile = bt / p.pool.Hkv, kvh = bt - tile * p.pool.Hkv;
  const int len = rw.len, first = rw.first, n_new = rw.n_new, rows = rw.rows;
  const int row0 = tile * F::R;
  if (!cut && tile >= rw.tiles) return;

  // row r of the tile: new token (row0 + r) / G, query head kvh G + (row0 + r) mod G; it sees
  // the first vis(r) tokens
  auto row_ok = [&](int r) { return row0 + r < rows && first + (row0 + r) / p.G < p.T; };
  auto row_at = [&](int r) {
    const int i = (row0 + r) / p.G;
    return static_cast<int64_t>(first + i) * p.q_ld +
           static_cast<int64_t>(kvh * p.G + (row0 + r) - i * p.G) * D;
  };
  auto row_vis = [&](int r) {
    if (!row_ok(r)) return 0;
    return p.causal ? min(max(len - n_new + (row0 + r) / p.G + 1, 0), len) : len;
  };
  const int last_row = min(F::R, rows - row0) - 1;
  const int vis_max = row_vis(last_row);
  const int n_run = ok ? min(run1, (vis_max + STEP - 1) / STEP) : 0;

  const uint32_t ring = sb + warp * STAGES * F::STAGE;
  const int w0 = run0 + warp;
  const int32_t* row_table = p.table + static_cast<int64_t>(b) * p.width;
  const int n_cell = (vis_max + kCell - 1) / kCell;
  // The warp's runs are w0, w0 + W, ..; lane 4 n + i holds the source of cell i of the n-th of
  // eight of them (NULL: not there), looked up once for the eight.
  const uint8_t* src = nullptr;
  uint32_t there8 = 0;                   // the cells that are there, four bits a run
  auto look = [&](int run) {
    const int ci = (run + (lane >> 2) * W) * NCELL + (lane & 3);
    int id = -1;
    uint32_t pg = 0;
    if (ci < n_cell) {
      pg = p.pool.shift >= 0 ? static_cast<uint32_t>(ci) >> p.pool.shift
                             : static_cast<uint32_t>(ci) / static_cast<uint32_t>(p.pool.cells);
      id = row_table[pg];
    }
    src = id < 0 || id >= p.pool.n_pages
              ? nullptr
              : p.pool.data + ((static_cast<int64_t>(id) * p.pool.Hkv + kvh) * p.pool.cells +
                               (ci - static_cast<int>(pg) * p.pool.cells)) *
                                  static_cast<int64_t>(C::BYTES);
    there8 = __ballot_sync(0xffffffffu, src != nullptr);
  };
  // Copies the n-th run (of w0, w0 + W, ..) into stage s; returns which of its cells there are.
  auto fetch = [&](int n, uint32_t s) -> uint32_t {
    if ((n & 7) == 0) look(w0 + n * W);
    const uint32_t cells = (there8 >> (4 * (n & 7))) & 15u;
    if (lane == 0) bar_expect(bars + 8 * s, __popc(cells) * C::BYTES);
    __syncwarp();
    if ((lane >> 2) == (n & 7) && src)
      bulk_load(ring + s * F::STAGE + (lane & 3) * F::PITCH, src, C::BYTES, bars + 8 * s);
    return cells;
  };

  uint32_t have = 0;                     // four bits a stage: its cells that are there
  int fetched = 0;
#pragma unroll
  for (int n = 0; n < STAGES - 1; ++n)
    if (w0 + n * W < n_run) {
      const uint32_t st = (it + n) % STAGES;
      have |= fetch(n, st) << (4 * st);
      ++fetched;
    }

  // ---- q: this lane's operand values of query row 8 nb + g, its scale and its plain sum
  uint32_t qf[NB][KM][2];
  float sg[NB][2];                      // of the lane's accumulator columns 2 tq, 2 tq + 1
  int vis[NB][2];
  float cq;                             // what the products' powers of two and the scale come to
  {
    const bool f16 = p.dt == OMQ_F16;
    uint32_t raw[NB][D / 8];            // the lane's quarter of the row
    float am = 0.f;                     // the tile's largest magnitude
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = 8 * nb + g;
      const bool here = row_ok(r);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 u = here ? __ldg(reinterpret_cast<const uint4*>(
                                   static_cast<const uint16_t*>(p.q) + row_at(r) + tq * (D / 4)) + i)
                             : make_uint4(0u, 0u, 0u, 0u);
        raw[nb][4 * i] = u.x; raw[nb][4 * i + 1] = u.y;
        raw[nb][4 * i + 2] = u.z; raw[nb][4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 x = pair(raw[nb][i], f16);
        am = fmaxf(am, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (!(am < INFINITY)) {             // of the finite elements, for the sake of the other rows
      am = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 x = pair(raw[nb][i], f16);
          am = fmaxf(am, fmaxf(fabsf(x.x) < INFINITY ? fabsf(x.x) : 0.f,
                               fabsf(x.y) < INFINITY ? fabsf(x.y) : 0.f));
        }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    }
    int e = 0;
    if (am > 0.f) e = 14 - ilogbf(am);
    e = min(max(e, -100), 100);
    const float up = __int_as_float((e + 127) << 23), back = __int_as_float((127 - e) << 23);
    // x = h (acc cq + z sg) + log2 hv: codes and q carry 2^-24 and 2^e
    const float down = p.scale * kLog2e * back;
    cq = down * 16777216.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        // matrix step m: word m / 2 of the lane's codes, nibble pairs (0, 4), (1, 5) or (2, 6),
        // (3, 7): elements 8 (m / 2) + 2 (m & 1) and the next, and both four further
        const float2 lo = pair(raw[nb][4 * (m >> 1) + (m & 1)], f16);
        const float2 hi = pair(raw[nb][4 * (m >> 1) + 2 + (m & 1)], f16);
        // the odd nibbles' codes stand 16 times too high
        qf[nb][m][0] = h2(lo.x * up, hi.x * up);
        qf[nb][m][1] = h2(lo.y * up * 0.0625f, hi.y * up * 0.0625f);
        const float2 u = __half22float2(*reinterpret_cast<__half2*>(&qf[nb][m][0]));
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&qf[nb][m][1]));
        sum += (u.x + u.y) + 16.f * (v.x + v.y);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float my_sg = -down * sum;
      sg[nb][0] = __shfl_sync(0xffffffffu, my_sg, 8 * tq);       // lanes with g = 2 tq, 2 tq + 1
      sg[nb][1] = __shfl_sync(0xffffffffu, my_sg, 8 * tq + 4);
      vis[nb][0] = row_vis(8 * nb + 2 * tq);
      vis[nb][1] = row_vis(8 * nb + 2 * tq + 1);
    }
  }
  const int vis_min = row_vis(0);       // the rows' least (those past the end are not stored)

  float mx[NB][2];
  float ls[NB][2], zs[NB][2];
  float acc[NB][VM][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    mx[nb][0] = mx[nb][1] = -INFINITY;
    ls[nb][0] = ls[nb][1] = zs[nb][0] = zs[nb][1] = 0.f;
#pragma unroll
    for (int m = 0; m < VM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nb][m][i] = 0.f;
  }

  const int cell_i = g >> 1;                             // the lane's cell in K and P
  int taken = 0;
#pragma unroll 1
  for (int run = w0; run < n_run && ok; run += W) {
    {
      const uint32_t s = it % STAGES;
      const int ahead = run + (STAGES - 1) * W;
      if (ahead < n_run) {
        const uint32_t st = (it + STAGES - 1) % STAGES;
        have = (have & ~(15u << (4 * st))) | (fetch(fetched, st) << (4 * st));
        ++fetched;
      }
      // every lane observes the completed phase itself before it reads what the copies wrote
      const bool got = bar_wait(bars + 8 * s, (it / STAGES) & 1, &g_rows_error, &g_rows_limit_ns,
                                DEV_ERR_TMA_WAIT);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      ++it;
      ++taken;
      const uint32_t cells = (have >> (4 * s)) & 15u;
      const uint32_t st = ring + s * F::STAGE;
      const uint32_t cell = st + cell_i * F::PITCH;
      const int t0 = run * STEP + kCell * cell_i + (g & 1);    // + 4 s' + 2 a: the lane's tokens
      const bool cell_ok = (cells >> cell_i) & 1u;
      const bool edge = run * STEP + STEP > vis_min || cells != (1u << NCELL) - 1;

      // ---- the run's steps as the lanes need them: (kh cq, kh kz, log2 vh, vz) of token
      // (j, g) = 2 j + (g & 1) of cell g / 2, entry 8 j + g, in place of the cells' steps. A
      // token that is not there has no weight and finite steps; a NaN step of V is put into K's,
      // so that it reaches the rows that see the token, and only those.
      {
        float4 mt[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int en = lane + 32 * i, ce = (en & 7) >> 1, tok = 2 * (en >> 3) + (en & 1);
          const uint32_t a = st + ce * F::PITCH + C::KH + 4 * tok;
          const bool there = ((cells >> ce) & 1u) && run * STEP + kCell * ce + tok < vis_max;
          const float kh = there ? lds_f(a) : 0.f, kz = there ? static_cast<float>(lds_i(a + 64)) : 0.f;
          const float vh = there ? lds_f(a + 128) : 1.f;
          const bool bad = vh != vh;
          mt[i].x = bad ? NAN : kh * cq;
          mt[i].y = kh * kz;
          mt[i].z = bad ? 0.f : lg2(vh);
          mt[i].w = there ? static_cast<float>(lds_i(a + 192)) : 0.f;
        }
        __syncwarp();                    // a lane's entries lie over steps that others read
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int en = lane + 32 * i;
          sts128(st + (en >> 4) * F::PITCH + C::KH + (en & 15) * 16, mt[i].x, mt[i].y, mt[i].z,
                 mt[i].w);
        }
        __syncwarp();
      }
      // ---- scores of the lane's 8 tokens x 2 NB queries
      float2 x[NB][8];
#pragma unroll
      for (int ms = 0; ms < 4; ++ms) {
        float sacc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) sacc[nb][i] = 0.f;
        const int tok = 4 * ms + (g & 1);                 // and tok + 2
        const uint32_t ka = cell + C::K + tok * C::ROW + tq * (C::ROW / 4);
        uint32_t wa[D / 32], wb[D / 32];
        if constexpr (D == 128) {
          const uint4 u = lds128(ka), v = lds128(ka + 2 * C::ROW);
          wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
          wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
        } else {
          const uint2 u = lds64(ka), v = lds64(ka + 2 * C::ROW);
          wa[0] = u.x; wa[1] = u.y;
          wb[0] = v.x; wb[1] = v.y;
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const Nibbles a = nibbles(wa[w]), b2 = nibbles(wb[w]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816(sacc[nb], a.l0, b2.l0, hsub2(a.u0, a.l0), hsub2(b2.u0, b2.l0),
                     qf[nb][2 * w][0], qf[nb][2 * w][1]);
            mma16816(sacc[nb], a.l1, b2.l1, hsub2(a.u1, a.l1), hsub2(b2.u1, b2.l1),
                     qf[nb][2 * w + 1][0], qf[nb][2 * w + 1][1]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          x[nb][2 * ms] = make_float2(sacc[nb][0], sacc[nb][1]);
          x[nb][2 * ms + 1] = make_float2(sacc[nb][2], sacc[nb][3]);
        }
      }
      float lh[8], vz[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 mt = lds128f(st + (j >> 1) * F::PITCH + C::KH + (j & 1) * 128 + g * 16);
        lh[j] = mt.z;
        vz[j] = mt.w;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          x[nb][j].x = __fmaf_rn(x[nb][j].x, mt.x, __fmaf_rn(mt.y, sg[nb][0], mt.z));
          x[nb][j].y = __fmaf_rn(x[nb][j].y, mt.x, __fmaf_rn(mt.y, sg[nb][1], mt.z));
        }
        if (edge) {                                       // warp-uniform
          const int t = cell_ok ? t0 + 2 * j : 0x7fffffff;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if (t >= vis[nb][0]) x[nb][j].x = -INFINITY;
            if (t >= vis[nb][1]) x[nb][j].y = -INFINITY;
          }
        }
      }
      // ---- running maximum, weights, sums
      uint32_t pw[NB][4][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float m0 = max3(x[nb][0].x, x[nb][1].x, x[nb][2].x), m1 = max3(x[nb][0].y, x[nb][1].y, x[nb][2].y);
#pragma unroll
        for (int j = 3; j < 7; j += 2) {
          m0 = max3(m0, x[nb][j].x, x[nb][j + 1].x);
          m1 = max3(m1, x[nb][j].y, x[nb][j + 1].y);
        }
        m0 = fmaxf(m0, x[nb][7].x);
        m1 = fmaxf(m1, x[nb][7].y);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        m0 = fmaxf(m0, mx[nb][0]);
        m1 = fmaxf(m1, mx[nb][1]);
        const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
        const float up0 = ref0 - kUp, up1 = ref1 - kUp;
        const bool moved = m0 != mx[nb][0] || m1 != mx[nb][1];
        if (__any_sync(0xffffffffu, moved)) {
          const float al0 = ex2(mx[nb][0] - ref0), al1 = ex2(mx[nb][1] - ref1);
          mx[nb][0] = m0;
          mx[nb][1] = m1;
          ls[nb][0] *= al0;
          ls[nb][1] *= al1;
          zs[nb][0] *= al0;
          zs[nb][1] *= al1;
#pragma unroll
          for (int m = 0; m < VM; ++m) {
            acc[nb][m][0] *= al0;
            acc[nb][m][1] *= al1;
            acc[nb][m][2] *= al0;
            acc[nb][m][3] *= al1;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w0 = ex2(x[nb][j].x - up0), w1 = ex2(x[nb][j].y - up1);
          const float rh = ex2(-lh[j]);                    // 1 / vh
          ls[nb][0] = __fmaf_rn(w0, rh, ls[nb][0]);
          ls[nb][1] = __fmaf_rn(w1, rh, ls[nb][1]);
          // the weights as the matrix instruction takes them weigh the zero points, too
          const uint32_t wh = h2(w0, w1);
          const float2 wr = __half22float2(*reinterpret_cast<const __half2*>(&wh));
          zs[nb][0] = __fmaf_rn(wr.x, vz[j], zs[nb][0]);
          zs[nb][1] = __fmaf_rn(wr.y, vz[j], zs[nb][1]);
          pw[nb][j >> 1][j & 1] = movm_t(wh);
        }
        const float fz = max3(max3(fabsf(vz[0]), fabsf(vz[1]), fabsf(vz[2])),
                              max3(fabsf(vz[3]), fabsf(vz[4]), fabsf(vz[5])),
                              fmaxf(fabsf(vz[6]), fabsf(vz[7])));
        if (__any_sync(0xffffffffu, fz > kFarZ)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float w0 = ex2(x[nb][j].x - up0), w1 = ex2(x[nb][j].y - up1);
            const uint32_t wh = h2(w0, w1);
            const float2 wr = __half22float2(*reinterpret_cast<const __half2*>(&wh));
            const float z = fabsf(vz[j]) > kFarZ ? vz[j] : 0.f;
            zs[nb][0] = __fmaf_rn(w0 - wr.x, z, zs[nb][0]);
            zs[nb][1] = __fmaf_rn(w1 - wr.y, z, zs[nb][1]);
          }
        }
      }
      // ---- o^T += V^T w: V's 8 x 8 blocks transposed on their way to registers. A run's products
      // are summed by the matrix unit, from zero, and added to o here: the unit cuts its sums off
      // towards zero, and codes are never negative, so a whole context summed there lost 1e-4 of
      // sum w c (100000 tokens, 400 runs a warp), which is some 1e-3 of the result about the zero
      // point.
#pragma unroll
      for (int cg = 0; cg < D / 32; ++cg) {
        float run_acc[NB][2][4];
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          // matrices: (tokens a = 0, of step 2 mp), (a = 1, 2 mp), (0, 2 mp + 1), (1, 2 mp + 1)
          const int mi = lane >> 3, r = lane & 7;
          const uint32_t va = st + (r >> 1) * F::PITCH + C::V +
                              (4 * (2 * mp + (mi >> 1)) + 2 * (mi & 1) + (r & 1)) * C::ROW + 16 * cg;
          uint32_t v[4];
          ldsm4_t(va, v);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // the second row is the whole byte, 16 c' + c: c's sum comes off at the end
            const Nibbles lo = nibbles(v[2 * k]), hi = nibbles(v[2 * k + 1]);
            const int ms = 2 * mp + k;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if (ms == 0) {
                mma16816_first(run_acc[nb][0], lo.l0, lo.u0, hi.l0, hi.u0, pw[nb][0][0], pw[nb][0][1]);
                mma16816_first(run_acc[nb][1], lo.l1, lo.u1, hi.l1, hi.u1, pw[nb][0][0], pw[nb][0][1]);
              } else {
                mma16816(run_acc[nb][0], lo.l0, lo.u0, hi.l0, hi.u0, pw[nb][ms][0], pw[nb][ms][1]);
                mma16816(run_acc[nb][1], lo.l1, lo.u1, hi.l1, hi.u1, pw[nb][ms][0], pw[nb][ms][1]);
              }
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[nb][2 * cg][i] += run_acc[nb][0][i];
            acc[nb][2 * cg + 1][i] += run_acc[nb][1][i];
          }
      }
      // the stage may be written again: by the copy engine, after the stores above
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    }
  }
  if (!ok && lane == 0) {                                // copies in flight land before the end
    const uint32_t t0 = it - taken;
    for (uint32_t j = it; j < t0 + fetched; ++j)
      bar_wait(bars + 8 * (j % STAGES), (j / STAGES) & 1, &g_rows_error, &g_rows_limit_ns,
               DEV_ERR_TMA_WAIT);
  }
  __syncwarp();

  // ---- join the warps
  float* stat = reinterpret_cast<float*>(smem + F::STAT);
  float lsum[NB][2], zsum[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    lsum[nb][0] = ls[nb][0];
    lsum[nb][1] = ls[nb][1];
    zsum[nb][0] = zs[nb][0];
    zsum[nb][1] = zs[nb][1];
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        lsum[nb][c] += __shfl_xor_sync(0xffffffffu, lsum[nb][c], o);
        zsum[nb][c] += __shfl_xor_sync(0xffffffffu, zsum[nb][c], o);
      }
      if (g == 0) {
        const int r = 8 * nb + 2 * tq + c;
        stat[(0 * W + warp) * F::R + r] = mx[nb][c];
        stat[(1 * W + warp) * F::R + r] = lsum[nb][c];
      }
    }
  __syncthreads();                                       // the ring's last readers are done, too
  float* part_o = reinterpret_cast<float*>(smem);        // [W][R][LDO]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * nb + 2 * tq + c;
      float m = stat[r];
#pragma unroll
      for (int w = 1; w < W; ++w) m = fmaxf(m, stat[w * F::R + r]);
      const float f = mx[nb][c] == -INFINITY ? 0.f : ex2(mx[nb][c] - m);
#pragma unroll
      for (int q = 0; q < VM; ++q) {
        // row tile q: columns 32 (q / 2) + 4 g + e, e = 2 (q & 1) and the next (16 times high)
        const int d = 32 * (q >> 1) + 4 * g + 2 * (q & 1);
        float2 o;
        o.x = (acc[nb][q][c] * 16777216.f - zsum[nb][c]) * f;
        o.y = ((acc[nb][q][2 + c] - acc[nb][q][c]) * 1048576.f - zsum[nb][c]) * f;
        *reinterpret_cast<float2*>(part_o + (warp * F::R + r) * F::LDO + d) = o;
      }
    }
  __syncthreads();
  float* join = reinterpret_cast<float*>(smem + F::JOIN);
  if (threadIdx.x < F::R) {
    const int r = threadIdx.x;
    float m = stat[r];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, stat[w * F::R + r]);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float mw = stat[w * F::R + r];
      // without a key the sum is 0, or NaN where a key was NaN: both survive the product
      l += stat[(W + w) * F::R + r] * (mw == -INFINITY ? 0.f : ex2(mw - m));
    }
    join[2 * r] = m;
    join[2 * r + 1] = l;
  }
  for (int i = threadIdx.x; i < F::R * (D / 2); i += 32 * W) {
    const int r = i / (D / 2), d = 2 * (i % (D / 2));
    float2 s = *reinterpret_cast<float2*>(part_o + r * F::LDO + d);
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float2 u = *reinterpret_cast<float2*>(part_o + (w * F::R + r) * F::LDO + d);
      s.x += u.x;
      s.y += u.y;
    }
    *reinterpret_cast<float2*>(part_o + r * F::LDO + d) = s;
  }
  if (together) {
    // every block joins its part of the rows from all blocks' shared memory, in their order
    cluster_sync_all();
    const uint32_t n = static_cast<uint32_t>(pieces);
    for (int i = threadIdx.x + 32 * W * cta_rank(); i < F::R * (D / 2); i += 32 * W * n) {
      const int r = i / (D / 2), d = 2 * (i % (D / 2));
      if (!row_ok(r)) continue;
      float2 ml[kCluster], u[kCluster];
      float m = -INFINITY;
#pragma unroll
      for (uint32_t c = 0; c < kCluster; ++c) {
        if (c >= n) break;
        ml[c] = ld_cluster2(map_rank(sb + F::JOIN + 8 * r, c));
        u[c] = ld_cluster2(map_rank(sb + 4 * (r * F::LDO + d), c));
        m = fmaxf(m, ml[c].x);
      }
      float l = 0.f;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (uint32_t c = 0; c < kCluster; ++c) {
        if (c >= n) break;
        const float w = ml[c].x == -INFINITY ? 0.f : ex2(ml[c].x - m);
        l += ml[c].y * w;                                  // 0, or NaN where a key was NaN
        o.x = __fmaf_rn(u[c].x, w, o.x);
        o.y = __fmaf_rn(u[c].y, w, o.y);
      }
      const int tok = (row0 + r) / p.G;
      const int64_t orow = static_cast<int64_t>(first + tok) * p.Hq + kvh * p.G + (row0 + r) - tok * p.G;
      store_row(p, orow, D, d, o, m, l);
    }
    cluster_sync_all();                                    // the others have read this block's
    return;
  }
  __syncthreads();
  const bool whole = run0 == 0 && run1 == rw.runs;
  const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (seg > 0 ? 1 : 0);
  if (!whole) {
    if (threadIdx.x < F::R) ws.ml[slot * F::R + threadIdx.x] = make_float2(join[2 * threadIdx.x], join[2 * threadIdx.x + 1]);
    if (threadIdx.x == 0 && seg == 0 && run0 > 0 && run1 == rw.runs) {
      const int64_t start = at - run0;
      PartDesc d = {};
      d.joins = 1;
      d.row0 = row0;
      d.rows = min(F::R, rows - row0);
      d.tok0 = first;
      d.kvh = kvh;
      if (cut) {
        d.first = static_cast<int>(start / part);
        d.first_slot = start == d.first * part ? 0 : 1;
      } else {
        d.first = static_cast<int>(blockIdx.x) / pieces * pieces;
      }
      ws.desc[blockIdx.x] = d;
    }
  }
  for (int i = threadIdx.x; i < F::R * (D / 2); i += 32 * W) {
    const int r = i / (D / 2), d = 2 * (i % (D / 2));
    const float2 o = *reinterpret_cast<const float2*>(part_o + r * F::LDO + d);
    if (!whole) {
      *reinterpret_cast<float2*>(ws.o + (slot * F::R + r) * D + d) = o;
    } else if (row_ok(r)) {
      const int tok = (row0 + r) / p.G;
      const int64_t orow = static_cast<int64_t>(first + tok) * p.Hq + kvh * p.G + (row0 + r) - tok * p.G;
      store_row(p, orow, D, d, o, join[2 * r], join[2 * r + 1]);
    }
  }
  // the ring may be filled again: by the copy engine, after the stores above
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  at += run1 - run0;
  }
}

// One row of an item that was cut: blockIdx.x the block it ends in, blockIdx.y the row of the
// tile. The partials are joined in the blocks' order (interleaved halves or quarters, then their
// sum). Everything is latency here: a thread has its first four partials under way before it
// knows the maxima.
template <int D, int NB>
__global__ void __launch_bounds__(128) kv_rows_join_kernel(AttnParams p, RowsSpace ws) {
  constexpr int R = 8 * NB, TPR = D / 2, GRP = 128 / TPR, AHEAD = 4;
  __shared__ float2 grp_sum[GRP - 1][TPR];
  __shared__ float red[2][4];
  __shared__ float fac[128];
  pdl_wait();
  pdl_launch();
  const PartDesc d = ws.desc[blockIdx.x];
  const int r = blockIdx.y;
  if (!d.joins || r >= d.rows) return;
  const int row = d.row0 + r, tok = d.tok0 + row / p.G;
  if (tok >= p.T) return;
  const int n = static_cast<int>(blockIdx.x) - d.first + 1;
  auto slot_of = [&](int i) {
    return (2 * static_cast<int64_t>(d.first + i) + (i == 0 ? d.first_slot : 0)) * R + r;
  };
  const int h = threadIdx.x / TPR, v = threadIdx.x % TPR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (static_cast<int>(threadIdx.x) < n) ml = ws.ml[slot_of(threadIdx.x)];
  float2 u[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = h + k * GRP;
    u[k] = i < n ? *reinterpret_cast<const float2*>(ws.o + slot_of(i) * D + 2 * v) : make_float2(0.f, 0.f);
  }
  float m = ml.x;
  for (int i = threadIdx.x + 128; i < n; i += 128) m = fmaxf(m, ws.ml[slot_of(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  float l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  for (int c = 0; c < n; c += 128) {
    if (c) {
      __syncthreads();                                     // the last chunk's factors are read
      ml = make_float2(-INFINITY, 0.f);
      if (c + static_cast<int>(threadIdx.x) < n) ml = ws.ml[slot_of(c + threadIdx.x)];
    }
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
    fac[threadIdx.x] = f;
    float mine = ml.y * f;                                 // 0, or NaN where a key was NaN
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, k);
    if (lane == 0) red[1][warp] = mine;
    __syncthreads();
    l += (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    const int hi = min(n - c, 128);
    int i = h;
    if (c == 0) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k, i += GRP)
        if (i < hi) {
          o.x = __fmaf_rn(u[k].x, fac[i], o.x);
          o.y = __fmaf_rn(u[k].y, fac[i], o.y);
        }
    }
#pragma unroll 8
    for (; i < hi; i += GRP) {
      const float2 w = *reinterpret_cast<const float2*>(ws.o + slot_of(c + i) * D + 2 * v);
      o.x = __fmaf_rn(w.x, fac[i], o.x);
      o.y = __fmaf_rn(w.y, fac[i], o.y);
    }
  }
  if (h > 0) grp_sum[h - 1][v] = o;
  __syncthreads();
  if (h > 0) return;
#pragma unroll
  for (int k = 0; k < GRP - 1; ++k) {
    o.x += grp_sum[k][v].x;
    o.y += grp_sum[k][v].y;
  }
  const int64_t orow = static_cast<int64_t>(tok) * p.Hq + d.kvh * p.G + row - row / p.G * p.G;
  store_row(p, orow, D, 2 * v, o, m, l);
}

// How a launch is laid out; the workspace depends on it.
struct RowsPlan {
  int64_t tiles;
  int64_t blocks;
  int pieces;          // blocks of an item, 0: the line of runs is cut evenly
  bool together;       // an item's blocks are a cluster
};
template <int D, int NB>
RowsPlan plan_rows(const AttnParams& p, int max_rows) {
  const int64_t most = static_cast<int64_t>(p.max_q) * p.G;
  RowsPlan r;
  r.tiles = ceil_div(most < max_rows ? most : max_rows, 8 * NB);
  const int64_t items = r.tiles * p.pool.Hkv * p.n_req;
  const int64_t runs = ceil_div(static_cast<int64_t>(p.width) * p.pool.page, STEP);
  const int64_t room = (NB == 1 ? 3 : 2) * static_cast<int64_t>(num_sms());
  // Equal shares of each item while all blocks are resident at once, two up to 2.5 times that,
  // then whole items, if the requests are as long as each other (there is one), a share is at
  // most 16 runs a warp (the last case below lies on that limit), or the blocks are eight times
  // those resident (a request far longer than the others then ends alone). No block then handles two items, which costs it a second round of latencies: one
  // request of 2049 tokens and 32 heads took 10.8 us against 15.7 on the even line, 33 of up to
  // 4001 tokens 23.3 against 28.3, 64 of up to 8192 82.7 against 87.4. The even line else: it
  // does not depend on how the lengths, which the host does not know, are spread.
  int64_t pieces = items <= room ? room / items : 2 * items <= 5 * room ? 2 : 1;
  const int64_t useful = ceil_div(runs, W);
  if (pieces > useful) pieces = useful;
  if (p.n_req == 1 || ceil_div(runs, pieces) <= 16 * W || items >= 8 * room) {
    // Up to eight blocks join their shares through distributed shared memory, without a second
    // kernel and the workspace; more than eight are made eight where that leaves a warp no more
    // than two runs. 10 requests of 2417 tokens, 4 x 7 heads: 12.4 -> 11.2 us, 33 of up to 4001
    // with 5 drafted tokens 24.1 -> 21.2, one of 4096, 8 heads 10.2 -> 9.4, of 2049, 32 heads 10.6 ->
    // 10.5 (and one launch less for the host); one of 8192, 32 heads (four runs) 15.8 -> 16.7.
    if (pieces > kCluster && ceil_div(runs, kCluster) <= 2 * W) pieces = kCluster;
    r.together = pieces > 1 && pieces <= kCluster;
    r.pieces = static_cast<int>(pieces);
    r.blocks = items * pieces;
    return r;
  }
  const int64_t parts = ceil_div(items * runs, W);
  r.together = false;
  r.pieces = 0;
  r.blocks = parts < room ? parts : room;
  return r;
}
template <int D, int NB>
size_t space_of(const RowsPlan& r, void* base, RowsSpace* ws) {
  if (r.pieces == 1 || r.together) return 0;
  constexpr int R = 8 * NB;
  const size_t o = static_cast<size_t>(r.blocks) * 2 * R * D * 4, ml = static_cast<size_t>(r.blocks) * 2 * R * 8;
  if (ws) {
    ws->o = static_cast<float*>(base);
    ws->ml = reinterpret_cast<float2*>(static_cast<char*>(base) + o);
    ws->desc = reinterpret_cast<PartDesc*>(static_cast<char*>(base) + o + ml);
  }
  return o + ml + static_cast<size_t>(r.blocks) * sizeof(PartDesc);
}

template <int D, int NB>
omq_status launch_rows(const AttnParams& p, int max_rows, void* space, cudaStream_t st) {
  using F = RowsCfg<D, NB>;
  static thread_local int ready = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (ready != dev) {
    const cudaError_t e = cudaFuncSetAttribute(kv_rows_kernel<D, NB>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return OMQ_ERR_CUDA;
    }
    ready = dev;
  }
  const RowsPlan r = plan_rows<D, NB>(p, max_rows);
  RowsSpace ws = {};
  space_of<D, NB>(r, space, &ws);
  const dim3 grid(static_cast<unsigned>(r.blocks));
  if (r.together) {
    launch_cl(kv_rows_kernel<D, NB>, grid, 32 * W, F::SMEM, r.pieces, st, p, static_cast<int>(r.tiles),
              max_rows, r.pieces, true, ws);
    return launch_status();
  }
  launch_k(kv_rows_kernel<D, NB>, grid, 32 * W, F::SMEM, st, p, static_cast<int>(r.tiles), max_rows,
           r.pieces, false, ws);
  const omq_status s = launch_status();
  if (s != OMQ_OK || r.pieces == 1) return s;
  const int64_t most = static_cast<int64_t>(p.max_q) * p.G;
  launch_k(kv_rows_join_kernel<D, NB>,
           dim3(static_cast<unsigned>(r.blocks), static_cast<unsigned>(most < F::R ? most : F::R)),
           128, 0, st, p, ws);
  return launch_status();
}

bool one_tile(const AttnParams& p) { return static_cast<int64_t>(p.max_q) * p.G <= 8; }

}  // namespace

size_t attn_rows_space(const AttnParams& p, int64_t D, int max_rows) {
  if (D == 128)
    return one_tile(p) ? space_of<128, 1>(plan_rows<128, 1>(p, max_rows), nullptr, nullptr)
                       : space_of<128, 2>(plan_rows<128, 2>(p, max_rows), nullptr, nullptr);
  return one_tile(p) ? space_of<64, 1>(plan_rows<64, 1>(p, max_rows), nullptr, nullptr)
                     : space_of<64, 2>(plan_rows<64, 2>(p, max_rows), nullptr, nullptr);
}

omq_status launch_attn_rows(const AttnParams& p, int64_t D, int max_rows, void* space, cudaStream_t st) {
  if (D == 128)
    return one_tile(p) ? launch_rows<128, 1>(p, max_rows, space, st) : launch_rows<128, 2>(p, max_rows, space, st);
  return one_tile(p) ? launch_rows<64, 1>(p, max_rows, space, st) : launch_rows<64, 2>(p, max_rows, space, st);
}

}  // namespace kv
}  // namespace omq
