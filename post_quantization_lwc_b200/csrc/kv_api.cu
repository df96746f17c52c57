// C entry points of the 4-bit paged key/value cache: validation on the host, then the launches.
#include "block_internal.cuh"
#include "kv_internal.cuh"

namespace omq {
namespace {

constexpr int64_t kMaxPage = 4096, kMaxHeads = 65536, kMaxReq = 65536, kMaxLd = int64_t{1} << 31;

bool any_float(omq_dtype d) { return d == OMQ_F32 || d == OMQ_BF16 || d == OMQ_F16; }
bool sixteen(omq_dtype d) { return d == OMQ_BF16 || d == OMQ_F16; }
int64_t esize(omq_dtype d) { return d == OMQ_F32 ? 4 : 2; }

omq_status check_pool(const omq_kv_pool& p) {
  if (!p.data) return OMQ_ERR_NULL;
  if (p.D != 64 && p.D != 128) return OMQ_ERR_SHAPE;
  if (p.page < 16 || p.page % 16 || p.page > kMaxPage) return OMQ_ERR_SHAPE;
  if (p.n_pages < 1 || p.n_pages > (int64_t{1} << 31) / p.page - 1) return OMQ_ERR_SHAPE;
  if (p.Hkv < 1 || p.Hkv > kMaxHeads) return OMQ_ERR_SHAPE;
  if (!aligned16(p.data)) return OMQ_ERR_ALIGN;
  return OMQ_OK;
}
kv::Pool view(const omq_kv_pool& p) {
  const int cells = static_cast<int>(p.page / 16);
  int shift = -1;
  if ((cells & (cells - 1)) == 0)
    for (shift = 0; (1 << shift) < cells; ++shift) {
    }
  return kv::Pool{static_cast<uint8_t*>(p.data), p.n_pages, static_cast<int>(p.Hkv), cells,
                  static_cast<int>(p.page), shift};
}
// Rows of `heads` heads, `ld` elements apart, each 16-byte aligned.
omq_status check_rows(const void* p, int64_t ld, int64_t heads, int64_t D, omq_dtype dt) {
  if (!p) return OMQ_ERR_NULL;
  if (ld < heads * D || ld > kMaxLd) return OMQ_ERR_SHAPE;
  if (!aligned16(p) || (ld * esize(dt)) % 16) return OMQ_ERR_ALIGN;
  return OMQ_OK;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uint64_t>(nb) && y < x + static_cast<uint64_t>(na);
}

#define KV_TRY(expr)                  \
  do {                                \
    omq_status _s = (expr);           \
    if (_s != OMQ_OK) return _s;      \
  } while (0)

omq_status check_attn(const omq_kv_attn_args* a) {
  if (!a) return OMQ_ERR_NULL;
  KV_TRY(check_pool(a->pool));
  if (!a->q || !a->table || !a->lens || !a->cu || !a->out) return OMQ_ERR_NULL;
  if (!sixteen(a->dt) || !sixteen(a->out_dt)) return OMQ_ERR_DTYPE;
  if (a->n_req < 1 || a->n_req > kMaxReq || a->T < 1 || a->T >= (int64_t{1} << 31)) return OMQ_ERR_SHAPE;
  if (a->Hq < 1 || a->Hq > kMaxHeads || a->Hq % a->pool.Hkv) return OMQ_ERR_SHAPE;
  if (a->width < 1 || a->width * a->pool.page >= (int64_t{1} << 31)) return OMQ_ERR_SHAPE;
  if (a->max_q < 1 || a->max_q > a->T) return OMQ_ERR_SHAPE;
  // a request's query rows per kv head, and the launch's blocks, stay 32-bit
  const int64_t rows = a->max_q * (a->Hq / a->pool.Hkv);
  if (rows >= (int64_t{1} << 30)) return OMQ_ERR_SHAPE;
  if ((rows / 8 + 1) * a->pool.Hkv >= (int64_t{1} << 27) / a->n_req) return OMQ_ERR_SHAPE;
  KV_TRY(check_rows(a->q, a->q_ld, a->Hq, a->pool.D, a->dt));
  if (!aligned16(a->out)) return OMQ_ERR_ALIGN;
  // q is read by several blocks, some after others have written out
  const int64_t row = a->Hq * a->pool.D * 2;
  if (overlap(a->q, 2 * (a->T - 1) * a->q_ld + row, a->out, a->T * row)) return OMQ_ERR_UNSUPPORTED;
  return OMQ_OK;
}

kv::AttnParams attn_params(const omq_kv_attn_args* a) {
  return kv::AttnParams{view(a->pool), static_cast<int>(a->n_req), a->T, static_cast<int>(a->Hq),
                        static_cast<int>(a->Hq / a->pool.Hkv), a->q, a->q_ld, a->dt, a->table,
                        static_cast<int>(a->width), a->lens, a->cu, static_cast<int>(a->max_q),
                        a->scale, a->causal ? 1 : 0, a->out, a->out_dt, a->lse};
}
// Query rows per kv head up to which a request goes to the row kernel, whose time grows with the
// rows (it expands the codes again for every 16), while the tile kernel's does not up to 512.
// 64 wherever the contexts are long. Row / tile kernel, us, at 64 rows and at 128: 8 requests of
// 4096 tokens and 8 kv heads 48 / 70 and 118 / 71; 32 of 2048 107 / 149 and 195 / 154; one of 65536
// 84 / 126 and 166 / 127; one of 4096 tokens and 32 kv heads 33 / 44 and 48 / 45; 8 kv heads of 64
// values 15 / 19 and 18 / 20. Under short contexts the tile kernel's fixed 8 us an item weigh more
// than the repeated codes, and all requests of up to 512 rows go to the row kernel where its
// estimate is below the other's: 10 us to begin and end and, while all blocks are resident, 3 for
// a run of 64 tokens a warp, else (half with D = 64) 5 a run and 1 a wave of blocks. One prompt of
// 512 tokens, 8 heads 20.4 -> 13.9 us; 39 of up to 124 tokens, 8 heads of 64 the same (42). Float16
// results may take half as long again there: its exact operands keep their last bit (error 2.2e-4
// of the result against 3.4e-4, where rounding the result alone gives 2.1e-4).
constexpr int kFew = 64, kFewShort = 512;

int64_t most_rows(const omq_kv_attn_args* a) { return a->max_q * (a->Hq / a->pool.Hkv); }
int few_rows(const omq_kv_attn_args* a, const kv::AttnParams& p) {
  const int64_t most = most_rows(a);
  if (most <= kFew || most > kFewShort) return kFew;
  const int64_t items = ceil_div(most, 16) * a->pool.Hkv * a->n_req;
  const int64_t runs = ceil_div(a->width * a->pool.page, 64), room = 2 * num_sms();
  const int64_t wave = (5 * ceil_div(runs, 4) + 1) * a->pool.D / 128;
  const int64_t rows_us = 10 + (items <= room ? 3 * ceil_div(items * runs, 4 * room)
                                              : ceil_div(items, room) * wave);
  const int64_t tiles_us = kv::attn_tiles_us(p, a->n_req == 1 ? 0 : kFew + 1);
  return (a->out_dt == OMQ_F16 ? 2 * rows_us <= 3 * tiles_us : rows_us <= tiles_us) ? kFewShort : kFew;
}
// What a call launches: the tile kernel for the requests of at least tiles_min rows (if any is),
// the row kernel for those of at most `few`, by the lengths on the device. They run one after
// the other and share the workspace.
struct AttnRoute {
  int few, tiles_min;
  bool rows, tiles;
  size_t space;
};
AttnRoute attn_route(const omq_kv_attn_args* a, const kv::AttnParams& p) {
  AttnRoute r;
  r.few = few_rows(a, p);
  r.tiles = most_rows(a) > r.few;
  r.rows = !r.tiles || a->n_req > 1;
  r.tiles_min = r.rows ? r.few + 1 : 0;
  const size_t rows = r.rows ? kv::attn_rows_space(p, a->pool.D, r.few) : 0;
  const size_t tiles = r.tiles ? kv::attn_tiles_space(p, a->pool.D, r.tiles_min) : 0;
  r.space = rows > tiles ? rows : tiles;
  return r;
}

}  // namespace
}  // namespace omq

using namespace omq;

extern "C" {

size_t omq_kv_cell_bytes(int64_t D) {
  return D == 64 || D == 128 ? static_cast<size_t>(kv::cell_bytes(D)) : 0;
}

omq_status omq_rope_table(int64_t n_pos, int64_t D, double base, float* table,
                          omq_stream_t stream) {
  if (!table) return OMQ_ERR_NULL;
  if (n_pos < 1 || n_pos > (int64_t{1} << 24) || (D != 64 && D != 128) || !(base > 1.0))
    return OMQ_ERR_SHAPE;
  if (!aligned16(table)) return OMQ_ERR_ALIGN;
  return launch_rope_table(n_pos, base, table, table + n_pos * (D / 2),
                           reinterpret_cast<cudaStream_t>(stream), static_cast<int>(D / 2));
}

omq_status omq_kv_plan(const omq_kv_plan_args* a, omq_stream_t stream) {
  if (!a || !a->lens || !a->new_tokens || !a->table || !a->free_pages || !a->n_free ||
      !a->lens_out || !a->n_free_out || !a->cu || !a->slots || !a->positions || !a->requests)
    return OMQ_ERR_NULL;
  if (a->n_req < 1 || a->n_req > kMaxReq || a->capacity < 1 || a->capacity >= (int64_t{1} << 31))
    return OMQ_ERR_SHAPE;
  if (a->page < 16 || a->page % 16 || a->page > kMaxPage) return OMQ_ERR_SHAPE;
  if (a->width < 1 || a->width >= (int64_t{1} << 31) / a->page) return OMQ_ERR_SHAPE;
  if (a->n_pages < 1 || a->n_pages > (int64_t{1} << 31) / a->page - 1) return OMQ_ERR_SHAPE;
  // the pages of a chunk of the kernel's 512 requests are counted in 32 bits
  if (a->width * (a->n_req < 512 ? a->n_req : 512) >= (int64_t{1} << 31)) return OMQ_ERR_SHAPE;
  kv::PlanParams p{a->lens, a->new_tokens, static_cast<int>(a->n_req), a->table,
                   static_cast<int>(a->width), static_cast<int>(a->page), a->free_pages,
                   static_cast<int>(a->n_pages), a->n_free, a->lens_out, a->n_free_out, a->cu,
                   a->slots, a->positions, a->requests, static_cast<int>(a->capacity)};
  return kv::launch_plan(p, reinterpret_cast<cudaStream_t>(stream));
}

omq_status omq_kv_append(const omq_kv_append_args* a, omq_stream_t stream) {
  if (!a) return OMQ_ERR_NULL;
  KV_TRY(check_pool(a->pool));
  if (!a->slots || !a->k || !a->v) return OMQ_ERR_NULL;
  if (!any_float(a->dt)) return OMQ_ERR_DTYPE;
  if (a->T < 1 || a->T >= (int64_t{1} << 31)) return OMQ_ERR_SHAPE;
  const bool rot = a->rope && a->positions;
  if (a->rope && (a->n_pos < 1 || a->n_pos >= (int64_t{1} << 31))) return OMQ_ERR_SHAPE;
  if (!aligned16(a->rope) || !aligned16(a->s_a) || !aligned16(a->s_o) || !aligned16(a->delta_o))
    return OMQ_ERR_ALIGN;
  if (a->delta_o && !a->s_o) return OMQ_ERR_NULL;
  KV_TRY(check_rows(a->k, a->k_ld, a->pool.Hkv, a->pool.D, a->dt));
  KV_TRY(check_rows(a->v, a->v_ld, a->pool.Hkv, a->pool.D, a->dt));
  const int ab = a->abits;
  if (a->q) {
    if (!a->q_out) return OMQ_ERR_NULL;
    if (!any_float(a->q_dt)) return OMQ_ERR_DTYPE;
    if (ab != 2 && ab != 3 && ab != 4 && ab != 6 && ab != 8 && ab != 16) return OMQ_ERR_BITS;
    if (a->Hq < 1 || a->Hq > kMaxHeads || a->Hq % a->pool.Hkv) return OMQ_ERR_SHAPE;
    KV_TRY(check_rows(a->q, a->q_ld, a->Hq, a->pool.D, a->dt));
    if (!aligned16(a->q_out)) return OMQ_ERR_ALIGN;
  }
  const int64_t rows = (a->q ? a->Hq : 0) + 2 * a->pool.Hkv;
  if (a->T > (int64_t{1} << 31) / rows) return OMQ_ERR_SHAPE;
  if (a->q) {                                              // other blocks still read these
    const int64_t es = esize(a->dt), kv = a->pool.Hkv * a->pool.D, qw = a->Hq * a->pool.D;
    const int64_t n = a->T * qw * esize(a->q_dt), last = a->T - 1;
    if (overlap(a->q, es * (last * a->q_ld + qw), a->q_out, n) ||
        overlap(a->k, es * (last * a->k_ld + kv), a->q_out, n) ||
        overlap(a->v, es * (last * a->v_ld + kv), a->q_out, n))
      return OMQ_ERR_UNSUPPORTED;
  }
  kv::AppendParams p{};
  p.pool = view(a->pool);
  p.T = a->T;
  p.Hq = a->q ? static_cast<int>(a->Hq) : 0;
  p.q = a->q; p.k = a->k; p.v = a->v;
  p.q_ld = a->q_ld; p.k_ld = a->k_ld; p.v_ld = a->v_ld;
  p.dt = a->dt;
  p.slots = a->slots;
  p.positions = rot ? a->positions : nullptr;
  p.rope = rot ? a->rope : nullptr;
  p.n_pos = a->n_pos;
  p.s_a = a->s_a; p.s_o = a->s_o; p.delta_o = a->delta_o;
  p.quant_q = a->q && ab < 16;
  p.Qa = static_cast<float>((1 << (p.quant_q ? ab : 1)) - 1);
  p.q_out = a->q_out;
  p.q_dt = a->q_dt;
  return kv::launch_append(p, a->pool.D, reinterpret_cast<cudaStream_t>(stream));
}

omq_status omq_kv_read(const omq_kv_pool* pool, int64_t T, const int32_t* slots, void* k, void* v,
                       omq_dtype dt, omq_stream_t stream) {
  if (!pool) return OMQ_ERR_NULL;
  KV_TRY(check_pool(*pool));
  if (!slots || !k || !v) return OMQ_ERR_NULL;
  if (!any_float(dt)) return OMQ_ERR_DTYPE;
  if (T < 1 || T > (int64_t{1} << 31) / pool->Hkv) return OMQ_ERR_SHAPE;
  if (!aligned16(k) || !aligned16(v)) return OMQ_ERR_ALIGN;
  kv::ReadParams p{view(*pool), T, slots, k, v, dt};
  return kv::launch_read(p, pool->D, reinterpret_cast<cudaStream_t>(stream));
}

size_t omq_kv_attn_workspace_bytes(const omq_kv_attn_args* a) {
  if (check_attn(a) != OMQ_OK) return 0;
  const kv::AttnParams p = attn_params(a);
  return attn_route(a, p).space;
}

omq_status omq_kv_attn(const omq_kv_attn_args* a, void* workspace, size_t ws_bytes,
                       omq_stream_t stream) {
  KV_TRY(check_attn(a));
  const kv::AttnParams p = attn_params(a);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const AttnRoute r = attn_route(a, p);
  if (r.space && (!workspace || ws_bytes < r.space)) return OMQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return OMQ_ERR_ALIGN;
  if (r.tiles) KV_TRY(kv::launch_attn_tiles(p, a->pool.D, r.tiles_min, workspace, st));
  return r.rows ? kv::launch_attn_rows(p, a->pool.D, r.few, workspace, st) : OMQ_OK;
}

}  // extern "C"
