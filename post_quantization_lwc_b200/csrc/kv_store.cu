// Storing keys and values in the 4-bit paged cache, and reading them back.
//
// kv_append_kernel: per (token, head) row of D values, in binary32 with one rounding per
// operation (the order of the block's attention preparation, so the cache holds bit for bit
// what the calibration simulated):
//   r[i] = x[i] c - x[i + D/2] s,  r[i + D/2] = x[i + D/2] c + x[i] s       (q and k)
//   q~ = r / s_a,  k~ = r s_a,  v~ = (v - delta_o) / s_o
//   h = max((max - min) / 15, 1e-8), z = -rint(min / h), c = clamp(rint(x / h) + z, 0, 15)
// k~ and v~ go to the token's slot as codes with (h, z), q~ to q_out in 16 bits, quantized and
// dequantized at its own bit width when asked.
//
// Eight lanes hold a row (D / 8 values each, both halves of every rotate pair in one lane), a
// warp four rows: the row's reduction is three shuffle steps for four rows at once, and its
// scalar work (h, z, the reciprocal) is shared by four rows an instruction. Nothing is
// exchanged between warps.
#include "kv_internal.cuh"

namespace omq {
namespace kv {
namespace {

// 4 consecutive elements starting at a multiple of 4.
__device__ __forceinline__ void load4(const void* p, int64_t i, omq_dtype dt, float* v) {
  if (dt == OMQ_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    if (dt == OMQ_F16) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a.x));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&a.y));
      v[0] = x.x; v[1] = x.y; v[2] = y.x; v[3] = y.y;
    } else {
      v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
      v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void store4(void* p, int64_t i, omq_dtype dt, const float* v) {
  if (dt == OMQ_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
  uint2 o;
  if (dt == OMQ_F16) {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    o = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    o = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = o;
}

// The pool's address of a slot's cell for one head, or NULL for a slot outside the pool.
__device__ __forceinline__ uint8_t* slot_cell(const Pool& p, int slot, int head, int cell_bytes,
                                              int* row) {
  if (slot < 0) return nullptr;
  const uint32_t pg = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page);
  if (static_cast<int64_t>(pg) >= p.n_pages) return nullptr;
  const int off = slot - static_cast<int>(pg) * p.page;
  *row = off & (kCell - 1);
  return p.data + ((static_cast<int64_t>(pg) * p.Hkv + head) * p.cells + (off >> 4)) *
                      static_cast<int64_t>(cell_bytes);
}

template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendParams p) {
  pdl_wait();
  pdl_launch();
  constexpr int E = D / 16;               // values of a half a lane holds (8 or 4)
  using C = CellT<D>;
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int nq = p.q ? p.Hq : 0;
  const int rows = nq + 2 * p.pool.Hkv;   // q heads, then k heads, then v heads
  const int64_t total = p.T * rows;
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 4 +
                     (lane >> 3);
  if (id - (lane >> 3) >= total) return;              // warp-uniform
  const bool in = id < total;
  const int64_t t = in ? id / rows : 0;
  const int r = in ? static_cast<int>(id - t * rows) : 0;
  const int which = r < nq ? 0 : r < nq + p.pool.Hkv ? 1 : 2;
  const int head = which == 0 ? r : which == 1 ? r - nq : r - nq - p.pool.Hkv;
  const void* src = which == 0 ? p.q : which == 1 ? p.k : p.v;
  const int64_t ld = which == 0 ? p.q_ld : which == 1 ? p.k_ld : p.v_ld;
  const int64_t base = t * ld + static_cast<int64_t>(head) * D;
  float a[E], b[E];                       // elements E sub + e and D/2 + E sub + e
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    load4(src, base + E * sub + e, p.dt, a + e);
    load4(src, base + D / 2 + E * sub + e, p.dt, b + e);
  }
  const int slot = __ldg(p.slots + t);
  const int pos = p.positions ? __ldg(p.positions + t) : 0;
  const bool live = in && slot >= 0 && slot < p.pool.n_pages * p.pool.page && pos >= 0 && (!p.rope || pos < p.n_pos);
  if (which < 2 && p.rope && live) {
    const float* cp = p.rope + static_cast<int64_t>(pos) * (D / 2) + E * sub;
    const float* sp = cp + p.n_pos * (D / 2);
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      float c[4], s[4];
      load4(cp, e, OMQ_F32, c);
      load4(sp, e, OMQ_F32, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = a[e + i], y = b[e + i];
        a[e + i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
        b[e + i] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
      }
    }
  }
  // the learned scales are per kv head: q head j has those of kv head j / G
  const int hk = which == 0 ? head / (p.Hq / p.pool.Hkv) : head;
  const float* sc = which == 2 ? p.s_o : p.s_a;
  if (sc) {
    const int64_t o = static_cast<int64_t>(hk) * D + E * sub;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      float u[4], w[4];
      load4(sc, o + e, OMQ_F32, u);
      load4(sc, o + D / 2 + e, OMQ_F32, w);
      if (which == 2 && p.delta_o) {
        float du[4], dw[4];
        load4(p.delta_o, o + e, OMQ_F32, du);
        load4(p.delta_o, o + D / 2 + e, OMQ_F32, dw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[e + i] = __fsub_rn(a[e + i], du[i]);
          b[e + i] = __fsub_rn(b[e + i], dw[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[e + i] = which == 1 ? __fmul_rn(a[e + i], u[i]) : __fdiv_rn(a[e + i], u[i]);
        b[e + i] = which == 1 ? __fmul_rn(b[e + i], w[i]) : __fdiv_rn(b[e + i], w[i]);
      }
    }
  }
  const bool quant = which != 0 || p.quant_q;
  float vmax = -INFINITY, vmin = INFINITY;
  bool bad = false;                       // a NaN or an infinity in the row
#pragma unroll
  for (int e = 0; e < E; ++e) {
    vmax = fmaxf(vmax, fmaxf(a[e], b[e]));
    vmin = fminf(vmin, fminf(a[e], b[e]));
    bad |= !(fabsf(a[e]) < INFINITY) || !(fabsf(b[e]) < INFINITY);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
    vmin = fminf(vmin, __shfl_xor_sync(0xffffffffu, vmin, o));
  }
  bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 24)) & 0xffu;
  if (!live) return;
  if (quant) {
    const float Q = which == 0 ? p.Qa : 15.f;
    GroupQ g = group_params(1.f, 1.f, vmax, vmin, Q);
    // a row that is not finite, or whose range is not, reads back as NaN throughout
    if (bad || !(g.h < INFINITY)) {
      g.h = NAN;
      g.z = 0.f;
    }
    const float hinv = __frcp_rn(g.h);
    const float z = static_cast<float>(z_to_i32(g.z));
    uint32_t wa = 0, wb = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float ca = fminf(fmaxf(__fadd_rn(round_quotient(a[e], g.h, hinv), g.z), 0.f), Q);
      const float cb = fminf(fmaxf(__fadd_rn(round_quotient(b[e], g.h, hinv), g.z), 0.f), Q);
      if (which == 0) {
        a[e] = __fmul_rn(__fsub_rn(ca, z), g.h);
        b[e] = __fmul_rn(__fsub_rn(cb, z), g.h);
      } else {
        wa |= small_uint(ca) << (4 * e);
        wb |= small_uint(cb) << (4 * e);
      }
    }
    if (which != 0) {
      int row = 0;
      uint8_t* cell = slot_cell(p.pool, slot, head, C::BYTES, &row);
      if (!cell) return;
      uint8_t* codes = cell + (which == 1 ? C::K : C::V) + row * C::ROW + sub * (E / 2);
      if (E == 8) {
        *reinterpret_cast<uint32_t*>(codes) = wa;
        *reinterpret_cast<uint32_t*>(codes + C::ROW / 2) = wb;
      } else {
        *reinterpret_cast<uint16_t*>(codes) = static_cast<uint16_t>(wa);
        *reinterpret_cast<uint16_t*>(codes + C::ROW / 2) = static_cast<uint16_t>(wb);
      }
      if (sub == 0) {
        *reinterpret_cast<float*>(cell + (which == 1 ? C::KH : C::VH) + 4 * row) = g.h;
        *reinterpret_cast<int32_t*>(cell + (which == 1 ? C::KZ : C::VZ) + 4 * row) = z_to_i32(g.z);
      }
      return;
    }
  }
  const int64_t o = (t * p.Hq + head) * D + E * sub;
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    store4(p.q_out, o + e, p.q_dt, a + e);
    store4(p.q_out, o + D / 2 + e, p.q_dt, b + e);
  }
}

// Read-back: four values a lane, so a warp's stores are whole rows. v = (c - z) h, c - z exact
// for |z| < 2^24 - 16, one rounding of the product; slots outside the pool read as zero rows.
template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(ReadParams p) {
  pdl_wait();
  pdl_launch();
  using C = CellT<D>;
  constexpr int LPR = D / 4;              // lanes of a row
  const int64_t total = p.T * p.pool.Hkv * LPR;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i0 >= total) return;
  const int l = static_cast<int>(i0 % LPR);
  const int64_t row_id = i0 / LPR;
  const int64_t t = row_id / p.pool.Hkv;
  const int head = static_cast<int>(row_id - t * p.pool.Hkv);
  int row = 0;
  const uint8_t* cell = slot_cell(p.pool, __ldg(p.slots + t), head, C::BYTES, &row);
  float k[4] = {}, v[4] = {};
  if (cell) {
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(cell + C::K + row * C::ROW + 2 * l);
    const uint32_t vc = *reinterpret_cast<const uint16_t*>(cell + C::V + row * C::ROW + 2 * l);
    const float kh = *reinterpret_cast<const float*>(cell + C::KH + 4 * row);
    const float vh = *reinterpret_cast<const float*>(cell + C::VH + 4 * row);
    const float kz = static_cast<float>(*reinterpret_cast<const int32_t*>(cell + C::KZ + 4 * row));
    const float vz = static_cast<float>(*reinterpret_cast<const int32_t*>(cell + C::VZ + 4 * row));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      k[e] = __fmul_rn(__fsub_rn(static_cast<float>((kc >> (4 * e)) & 15u), kz), kh);
      v[e] = __fmul_rn(__fsub_rn(static_cast<float>((vc >> (4 * e)) & 15u), vz), vh);
    }
  }
  store4(p.k, row_id * D + 4 * l, p.dt, k);
  store4(p.v, row_id * D + 4 * l, p.dt, v);
}

}  // namespace

omq_status launch_append(const AppendParams& p, int64_t D, cudaStream_t st) {
  const int64_t rows = p.T * ((p.q ? p.Hq : 0) + 2 * p.pool.Hkv);
  // small calls spread over the SMs in blocks of one warp
  const int threads = ceil_div(rows, 4) <= 4 * num_sms() ? 32 : 256;
  const unsigned grid = static_cast<unsigned>(ceil_div(rows, 4 * (threads / 32)));
  if (D == 128) launch_k(kv_append_kernel<128>, grid, threads, 0, st, p);
  else launch_k(kv_append_kernel<64>, grid, threads, 0, st, p);
  return launch_status();
}

omq_status launch_read(const ReadParams& p, int64_t D, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(ceil_div(p.T * p.pool.Hkv * (D / 4), 256));
  if (D == 128) launch_k(kv_read_kernel<128>, grid, 256, 0, st, p);
  else launch_k(kv_read_kernel<64>, grid, 256, 0, st, p);
  return launch_status();
}

}  // namespace kv
}  // namespace omq
