// attn_paged.cu — the C ABI of the position rotation, the paged cache and the
// decode (include/attn.h): argument checks, the rates' fixed-point form, the
// decode workspace and the launches.  Host code; the arithmetic is in
// attn_rope.cu and attn_decode.cu.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "attn_paged.h"
#include "attn_prefill.h"
#include "tmap.h"

using namespace attn;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool head_size(int d) { return d == 64 || d == 128 || d == 192; }
int cuda_err(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// Distance between rows of H heads of d columns: 0 stands for dense.
bool row_stride(long long* row, int H, int d) {
  const long long dense = (long long)H * d;
  if (*row == 0) *row = dense;
  return *row >= dense && *row % 8 == 0;
}

int check_rotation(const attn_rotation* r, int d, Rotation* out) {
  std::memset(out, 0, sizeof(*out));
  if (r == nullptr) return ATTN_OK;
  if (r->rates == nullptr || !aligned(r->rates, 8)) return ATTN_ERR_INVALID_ARG;
  if (r->style != ATTN_ROPE_HALVES && r->style != ATTN_ROPE_PAIRS) return ATTN_ERR_INVALID_ARG;
  if (r->begin < 0 || r->dim <= 0 || r->begin % 16 || r->dim % 16 || r->begin > d ||
      r->dim > d - r->begin)
    return ATTN_ERR_INVALID_ARG;
  out->rates = r->rates;
  out->begin = r->begin;
  out->dim = r->dim;
  out->pairs = r->style == ATTN_ROPE_PAIRS;
  return ATTN_OK;
}

int check_norm(const attn_head_norm* n, HeadNorm* out) {
  if (n == nullptr || !aligned(n->q_weight, 4) || !aligned(n->k_weight, 4)) return ATTN_ERR_INVALID_ARG;
  // (eps keeps the root of a row of zeros finite)
  if (!(n->eps >= std::numeric_limits<float>::min()) || !std::isfinite(n->eps))
    return ATTN_ERR_INVALID_ARG;
  *out = HeadNorm{n->q_weight, n->k_weight, n->eps};
  return ATTN_OK;
}

// Host offsets of nseq sequences over `total` rows, into a by-value table.
int check_offsets(const int* cu, int nseq, int total, RowOffsets* out) {
  if (nseq > ATTN_MAX_VARLEN_SEQS) return ATTN_ERR_UNSUPPORTED;
  if (cu[0] != 0 || cu[nseq] != total) return ATTN_ERR_INVALID_ARG;
  for (int b = 0; b < nseq; ++b)
    if (cu[b + 1] < cu[b]) return ATTN_ERR_INVALID_ARG;
  std::memcpy(out->cu, cu, (nseq + 1) * sizeof(int));
  return ATTN_OK;
}

bool cache_side(const void* base, const float* scale, long long page, long long token,
                long long head, int elt, CacheSide* out) {
  const long long unit = 16 / elt;
  if (base == nullptr || !aligned(base, 16) || !aligned(scale, 4)) return false;
  if (page < 0 || token < 0 || head < 0 || page % unit || token % unit || head % unit) return false;
  if (page / unit > UINT32_MAX || token / unit > UINT32_MAX) return false;
  out->base = static_cast<char*>(const_cast<void*>(base));
  out->scale = scale;
  out->page = (uint32_t)(page / unit);
  out->token = (uint32_t)(token / unit);
  out->head = head * elt;
  return true;
}

int check_cache(const attn_paged_cache* c, const int* table, int max_pages, long long table_stride,
                const int* lens, int B, CacheView* out) {
  std::memset(out, 0, sizeof(*out));
  if (c == nullptr || table == nullptr || lens == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4)) return ATTN_ERR_INVALID_ARG;
  if (c->type != ATTN_CACHE_BF16 && c->type != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || c->num_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || max_pages <= 0 ||
      table_stride < max_pages)
    return ATTN_ERR_INVALID_ARG;
  if (!((c->dqk == 64 && c->dv == 64) || (c->dqk == 128 && c->dv == 128) ||
        (c->dqk == 192 && c->dv == 128)))
    return ATTN_ERR_UNSUPPORTED;
  const int elt = c->type == ATTN_CACHE_E4M3 ? 1 : 2;
  const bool e4m3 = c->type == ATTN_CACHE_E4M3;
  if (!e4m3 && (c->k_scale || c->v_scale)) return ATTN_ERR_INVALID_ARG;
  if (!cache_side(c->k, c->k_scale, c->k_page_stride, c->k_token_stride, c->k_head_stride, elt,
                  &out->k) ||
      !cache_side(c->v, c->v_scale, c->v_page_stride, c->v_token_stride, c->v_head_stride, elt,
                  &out->v))
    return ATTN_ERR_INVALID_ARG;
  out->table = table;
  out->table_stride = table_stride;
  out->lens = lens;
  out->max_pages = max_pages;
  out->num_pages = c->num_pages;
  out->heads = c->heads;
  out->e4m3 = e4m3;
  set_page_size(out, c->page_size);
  return ATTN_OK;
}

// Whether no two rows of d columns of a cache side share memory: each dimension steps over
// all that the narrower ones cover.  Tokens written to rows that do share it would race.
bool rows_apart(const attn_paged_cache* c, long long page, long long token, long long head,
                int d) {
  struct {
    long long stride;
    int size;
  } dims[3] = {{page, c->num_pages}, {token, c->page_size}, {head, c->heads}};
  std::sort(dims, dims + 3, [](const auto& a, const auto& b) { return a.stride < b.stride; });
  __int128 extent = d;
  for (const auto& dim : dims) {
    if (dim.size == 1) continue;
    if (dim.stride < extent) return false;
    extent += (__int128)dim.stride * (dim.size - 1);
  }
  return true;
}

// Map of one side of a cache over (columns, heads and tokens, pages), boxes of `box` tokens of one
// page and head: 64 columns swizzled as the products read them, or all bytes of an e4m3 row.  False
// where it cannot be described so (broadcast dimensions, strides beyond a map's).
bool page_map(CUtensorMap* map, const attn_paged_cache* c, bool values, int box, bool heads_inner) {
  const bool e4m3 = c->type == ATTN_CACHE_E4M3;
  const int d = values ? c->dv : c->dqk, elt = e4m3 ? 1 : 2;
  const long long page = (values ? c->v_page_stride : c->k_page_stride) * elt;
  const long long token = (values ? c->v_token_stride : c->k_token_stride) * elt;
  const long long head = (values ? c->v_head_stride : c->k_head_stride) * elt;
  for (long long s : {page, token, head})
    if (s <= 0 || s >= (1ll << 40)) return false;
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  const cuuint64_t tokens = (cuuint64_t)c->page_size, heads = (cuuint64_t)c->heads;
  const cuuint64_t dims[4] = {(cuuint64_t)d, heads_inner ? heads : tokens,
                              heads_inner ? tokens : heads, (cuuint64_t)c->num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)(heads_inner ? head : token),
                                 (cuuint64_t)(heads_inner ? token : head), (cuuint64_t)page};
  const cuuint32_t boxes[4] = {(cuuint32_t)(e4m3 ? d : 64), heads_inner ? 1u : (cuuint32_t)box,
                               heads_inner ? (cuuint32_t)box : 1u, 1u};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             values ? c->v : c->k, dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device (asked once for each).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// The norm with the rotation (dy == null), and its backward: queries and keys, each x, dy, y
// and their rows' distances.
int norm_impl(const void* const* x, const void* const* dy, void* const* y, float* const* dw, int B,
              int Hq, int Hk, int Tq, int Tk, int d, const long long (*given)[3],
              const attn_head_norm* norm, const attn_rotation* rotation, int pos0,
              const int* cu_seqlens_q, const int* cu_seqlens_k, void* workspace,
              size_t workspace_bytes, void* stream) {
  (void)workspace_bytes;
  const int H[2] = {Hq, Hk}, T[2] = {Tq, Tk};
  if (x[0] == nullptr && x[1] == nullptr) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Tq < 0 || Tk < 0 || pos0 < 0) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    if ((x[i] == nullptr) != (y[i] == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (x[i] != nullptr && (H[i] <= 0 || T[i] == 0)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(x[i], 16) || !aligned(y[i], 16) || (dy && !aligned(dy[i], 16)))
      return ATTN_ERR_INVALID_ARG;
  }
  if (!head_size(d)) return ATTN_ERR_UNSUPPORTED;
  NormLaunch L;
  std::memset(&L, 0, sizeof(L));
  HeadNorm n;
  int rc = check_norm(norm, &n);
  if (rc) return rc;
  if ((rc = check_rotation(rotation, d, &L.rot)) != 0) return rc;
  static thread_local RowOffsets cu[2];
  const bool varlen = cu_seqlens_q != nullptr;
  if (!varlen && cu_seqlens_k != nullptr) return ATTN_ERR_INVALID_ARG;
  const int* cuk = cu_seqlens_k != nullptr ? cu_seqlens_k : cu_seqlens_q;
  if (varlen) {
    if ((rc = check_offsets(cu_seqlens_q, B, Tq, &cu[0])) != 0) return rc;
    if ((rc = check_offsets(cuk, B, Tk, &cu[1])) != 0) return rc;
    L.cu[0] = &cu[0];
    L.cu[1] = &cu[1];
  }
  if ((int64_t)pos0 + std::max(Tq, Tk) > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i) {
    if (x[i] == nullptr) continue;
    long long row[3] = {given[i][0], given[i][1], given[i][2]};
    for (long long& r : row)
      if (!row_stride(&r, H[i], d)) return ATTN_ERR_INVALID_ARG;
    const int64_t rows = varlen ? T[i] : (int64_t)B * T[i];
    if (rows > INT32_MAX - 1024 || (int64_t)H[i] * d > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
    NormTensor& t = L.t[i];
    t.x = x[i];
    t.dy = dy ? dy[i] : nullptr;
    t.y = y[i];
    t.x_row = row[0];
    t.dy_row = row[1];
    t.y_row = row[2];
    t.rows = (int)rows;
    t.H = H[i];
    t.T = T[i];
    t.shift = !varlen && i == 0 ? Tk - Tq : 0;
    t.weight = i ? n.k_weight : n.q_weight;
    t.dw = dw ? dw[i] : nullptr;
  }
  L.eps = n.eps;
  L.nseq = B;
  L.pos0 = pos0;
  L.d = d;
  L.workspace = static_cast<float*>(workspace);
  L.num_sms = sm_count();
  if (L.num_sms <= 0) return ATTN_ERR_CUDA;
  L.stream = static_cast<cudaStream_t>(stream);
  return cuda_err(dy ? launch_norm_bwd(L) : launch_norm(L));
}

}  // namespace

extern "C" {

int attn_rope_rates(const double* rates_rad, int n, unsigned long long* out) {
  if (rates_rad == nullptr || out == nullptr || n <= 0) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(rates_rad[i])) return ATTN_ERR_INVALID_ARG;
  // 1 / (2 pi) in two doubles; the product is then exact to about 2^-105
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int i = 0; i < n; ++i) {
    const double w = rates_rad[i];
    const double t = w * hi;
    const double rest = std::fma(w, hi, -t) + w * lo;
    // each part's fraction in [-0.5, 0.5), where the subtraction is exact
    auto turns = [](double f) {
      f -= std::floor(f + 0.5);
      if (f < -0.5) f += 1.0;  // (f + 0.5 had rounded up to a whole number)
      return (unsigned long long)(long long)std::ldexp(f, 64);
    };
    out[i] = turns(t) + turns(rest);
  }
  return ATTN_OK;
}

int attn_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int Hq, int Hk,
              int Tq, int Tk, int d, long long q_row, long long k_row, long long q_out_row,
              long long k_out_row, const attn_rotation* rotation, int inverse, int pos0,
              const int* cu_seqlens_q, const int* cu_seqlens_k, void* stream) {
  if ((q == nullptr && k == nullptr) || (q == nullptr) != (q_out == nullptr) ||
      (k == nullptr) != (k_out == nullptr) || rotation == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Tq < 0 || Tk < 0 || pos0 < 0 || (q && (Hq <= 0 || Tq == 0)) ||
      (k && (Hk <= 0 || Tk == 0)))
    return ATTN_ERR_INVALID_ARG;
  if (!head_size(d)) return ATTN_ERR_UNSUPPORTED;
  if ((q && (!row_stride(&q_row, Hq, d) || !row_stride(&q_out_row, Hq, d))) ||
      (k && (!row_stride(&k_row, Hk, d) || !row_stride(&k_out_row, Hk, d))))
    return ATTN_ERR_INVALID_ARG;
  RopeLaunch L;
  std::memset(&L, 0, sizeof(L));
  int rc = check_rotation(rotation, d, &L.rot);
  if (rc) return rc;
  static thread_local RowOffsets cu[2];
  const bool varlen = cu_seqlens_q != nullptr;
  if (!varlen && cu_seqlens_k != nullptr) return ATTN_ERR_INVALID_ARG;
  const int* cuk = cu_seqlens_k != nullptr ? cu_seqlens_k : cu_seqlens_q;
  if (varlen) {
    if ((rc = check_offsets(cu_seqlens_q, B, Tq, &cu[0])) != 0) return rc;
    if ((rc = check_offsets(cuk, B, Tk, &cu[1])) != 0) return rc;
    L.cu[0] = &cu[0];
    L.cu[1] = &cu[1];
  }
  // the largest position is that of the last key, or of a query beside it
  if ((int64_t)pos0 + std::max(Tq, Tk) > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  const int64_t rows_q = varlen ? Tq : (int64_t)B * Tq, rows_k = varlen ? Tk : (int64_t)B * Tk;
  // (a block's last row may lie past the end: keep its index in range too)
  if (std::max(rows_q, rows_k) > INT32_MAX - 1024) return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)std::max(Hq, Hk) * d > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  auto put = [&](int i, const void* x, void* y, int64_t rows, int H, int T, long long xr,
                 long long yr, int shift) {
    if (x == nullptr) return;
    RopeTensor& t = L.t[i];
    t.x = x;
    t.y = y;
    t.x_row = xr;
    t.y_row = yr;
    t.rows = (int)rows;
    t.H = H;
    t.T = T;
    t.shift = shift;
  };
  put(0, q, q_out, rows_q, Hq, Tq, q_row, q_out_row, varlen ? 0 : Tk - Tq);
  put(1, k, k_out, rows_k, Hk, Tk, k_row, k_out_row, 0);
  L.inverse = inverse ? 1 : 0;
  L.nseq = B;
  L.pos0 = pos0;
  L.d = d;
  L.num_sms = sm_count();
  if (L.num_sms <= 0) return ATTN_ERR_CUDA;
  L.stream = static_cast<cudaStream_t>(stream);
  return cuda_err(launch_rope(L));
}

int attn_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int Hq, int Hk,
                   int Tq, int Tk, int d, long long q_row, long long k_row, long long q_out_row,
                   long long k_out_row, const attn_head_norm* norm, const attn_rotation* rotation,
                   int pos0, const int* cu_seqlens_q, const int* cu_seqlens_k, void* stream) {
  const void* x[2] = {q, k};
  void* y[2] = {q_out, k_out};
  const long long rows[2][3] = {{q_row, 0, q_out_row}, {k_row, 0, k_out_row}};
  return norm_impl(x, nullptr, y, nullptr, B, Hq, Hk, Tq, Tk, d, rows, norm, rotation, pos0,
                   cu_seqlens_q, cu_seqlens_k, nullptr, 0, stream);
}

size_t attn_norm_rope_bwd_workspace_size(int d) { return head_size(d) ? norm_workspace_bytes(d) : 0; }

int attn_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                       void* dq, void* dk, float* dq_weight, float* dk_weight, int B, int Hq,
                       int Hk, int Tq, int Tk, int d, const attn_norm_rows* rows,
                       const attn_head_norm* norm, const attn_rotation* rotation, int pos0,
                       const int* cu_seqlens_q, const int* cu_seqlens_k, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const void* x[2] = {q, k};
  const void* dy[2] = {dq_out, dk_out};
  void* y[2] = {dq, dk};
  float* dw[2] = {dq_weight, dk_weight};
  const attn_norm_rows none = {}, &r = rows != nullptr ? *rows : none;
  const long long given[2][3] = {{r.q, r.dq_out, r.dq}, {r.k, r.dk_out, r.dk}};
  if (workspace == nullptr || !aligned(workspace, 256)) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    if ((x[i] == nullptr) != (dy[i] == nullptr) || (x[i] == nullptr && dw[i] != nullptr) ||
        !aligned(dw[i], 4))
      return ATTN_ERR_INVALID_ARG;
  if (head_size(d) && workspace_bytes < norm_workspace_bytes(d)) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  return norm_impl(x, dy, y, dw, B, Hq, Hk, Tq, Tk, d, given, norm, rotation, pos0, cu_seqlens_q,
                   cu_seqlens_k, workspace, workspace_bytes, stream);
}

int attn_cache_append(const attn_paged_cache* cache, const int* block_table, int max_pages,
                      long long table_stride, const int* lens, int B, int T,
                      const int* cu_seqlens, const void* k, long long k_row, const void* v,
                      long long v_row, const void* q, long long q_row, void* q_out,
                      long long q_out_row, int Hq, const attn_rotation* rotation, void* stream) {
  return attn_cache_append_norm(cache, block_table, max_pages, table_stride, lens, B, T, cu_seqlens,
                                k, k_row, v, v_row, q, q_row, q_out, q_out_row, Hq, nullptr,
                                rotation, stream);
}

int attn_cache_append_norm(const attn_paged_cache* cache, const int* block_table, int max_pages,
                           long long table_stride, const int* lens, int B, int T,
                           const int* cu_seqlens, const void* k, long long k_row, const void* v,
                           long long v_row, const void* q, long long q_row, void* q_out,
                           long long q_out_row, int Hq, const attn_head_norm* norm,
                           const attn_rotation* rotation, void* stream) {
  AppendLaunch L;
  std::memset(&L, 0, sizeof(L));
  int rc = check_cache(cache, block_table, max_pages, table_stride, lens, B, &L.cache);
  if (rc) return rc;
  if (k == nullptr || v == nullptr || (q == nullptr) != (q_out == nullptr) || T < 0 ||
      (q && Hq <= 0))
    return ATTN_ERR_INVALID_ARG;
  if (!rows_apart(cache, cache->k_page_stride, cache->k_token_stride, cache->k_head_stride,
                  cache->dqk) ||
      !rows_apart(cache, cache->v_page_stride, cache->v_token_stride, cache->v_head_stride,
                  cache->dv))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16))
    return ATTN_ERR_INVALID_ARG;
  if (!row_stride(&k_row, cache->heads, cache->dqk) || !row_stride(&v_row, cache->heads, cache->dv) ||
      (q && (!row_stride(&q_row, Hq, cache->dqk) || !row_stride(&q_out_row, Hq, cache->dqk))))
    return ATTN_ERR_INVALID_ARG;
  if ((int64_t)std::max(q ? Hq : 0, cache->heads) * cache->dqk > (1 << 20) ||
      T > INT32_MAX - (1 << 20))
    return ATTN_ERR_UNSUPPORTED;
  rc = check_rotation(rotation, cache->dqk, &L.rot);
  if (rc) return rc;
  HeadNorm head_norm;
  if (norm != nullptr) {
    if ((rc = check_norm(norm, &head_norm)) != 0) return rc;
    L.norm = &head_norm;
  }
  static thread_local RowOffsets offsets;
  if (cu_seqlens != nullptr) {
    if ((rc = check_offsets(cu_seqlens, B, T, &offsets)) != 0) return rc;
    L.offsets = &offsets;
  } else if (T % B != 0) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (T == 0) return ATTN_OK;
  L.k = k;
  L.v = v;
  L.q = q;
  L.q_out = q_out;
  L.k_row = k_row;
  L.v_row = v_row;
  L.q_row = q_row;
  L.q_out_row = q_out_row;
  L.B = B;
  L.T = T;
  L.Hq = q ? Hq : 0;
  L.per_seq = T / B;
  L.dqk = cache->dqk;
  L.dv = cache->dv;
  L.num_sms = sm_count();
  if (L.num_sms <= 0) return ATTN_ERR_CUDA;
  L.status = cache_status_ptr();
  if (!L.status) return ATTN_ERR_CUDA;
  L.stream = static_cast<cudaStream_t>(stream);
  return cuda_err(norm != nullptr ? launch_append_norm(L) : launch_append(L));
}

size_t attn_decode_workspace_size(void) { return kDecodeWorkspaceBytes; }

int attn_decode_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
  if (workspace == nullptr || !aligned(workspace, 256)) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < kDecodeWorkspaceBytes) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the counters at zero, then the header's mark
  if (cudaMemsetAsync(workspace, 0, 256 + kDecodeCounterBytes, s) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return cuda_err(cudaMemsetAsync(workspace, kDecodeReady & 0xFF, sizeof(uint32_t), s));
}

int attn_decode(const attn_paged_cache* cache, const int* block_table, int max_pages,
                long long table_stride, const int* lens, int B, const void* q, long long q_row,
                void* o, float* lse, int Hq, int window_left, float scale, void* workspace,
                size_t workspace_bytes, void* stream) {
  DecodeLaunch L;
  std::memset(&L, 0, sizeof(L));
  int rc = check_cache(cache, block_table, max_pages, table_stride, lens, B, &L.cache);
  if (rc) return rc;
  if (q == nullptr || o == nullptr || workspace == nullptr || Hq <= 0 || window_left < -1)
    return ATTN_ERR_INVALID_ARG;
  // (a factor that is 0 or inf would make a hidden key's -inf, or a score of 0, NaN)
  if (!(scale >= std::numeric_limits<float>::min()) || !std::isfinite(scale * kLog2e))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
    return ATTN_ERR_INVALID_ARG;
  if (!row_stride(&q_row, Hq, cache->dqk)) return ATTN_ERR_INVALID_ARG;
  if (Hq % cache->heads != 0) return ATTN_ERR_INVALID_ARG;
  if ((int64_t)Hq * cache->dqk > (1 << 20) || B > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < kDecodeWorkspaceBytes) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  L.q = q;
  L.q_row = q_row;
  L.o = o;
  L.lse = lse;
  L.B = B;
  L.Hq = Hq;
  L.group = Hq / cache->heads;
  // large groups are cut into tiles of equal size
  L.row_tiles = cdiv(L.group, most_tile_rows(cache->dqk, L.cache.e4m3 != 0));
  L.tile_rows = cdiv(L.group, L.row_tiles);
  L.row_tiles = cdiv(L.group, L.tile_rows);
  L.window = window_left;
  L.scale_log2 = scale * kLog2e;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  L.header = reinterpret_cast<DecodeHeader*>(base);
  L.counters = reinterpret_cast<int*>(base + 256);
  base += 256 + ((kDecodeCounterBytes + 255) & ~size_t(255));
  L.ml = reinterpret_cast<float*>(base);
  L.acc = reinterpret_cast<float*>(base + kDecodeMlBytes);
  L.dqk = cache->dqk;
  L.dv = cache->dv;
  L.num_sms = sm_count();
  if (L.num_sms <= 0) return ATTN_ERR_CUDA;
  L.status = cache_status_ptr();
  if (!L.status) return ATTN_ERR_CUDA;
  L.stream = static_cast<cudaStream_t>(stream);
  return cuda_err(launch_decode(L));
}

size_t attn_prefill_workspace_size(void) { return kPrefillWorkspaceBytes; }

int attn_prefill(const attn_paged_cache* cache, const int* block_table, int max_pages,
                 long long table_stride, const int* lens, int B, int T, const int* cu_seqlens,
                 const void* q, long long q_row, void* o, float* lse, int Hq, int window_left,
                 float scale, void* workspace, size_t workspace_bytes, void* stream) {
  PrefillLaunch L;
  std::memset(&L, 0, sizeof(L));
  int rc = check_cache(cache, block_table, max_pages, table_stride, lens, B, &L.cache);
  if (rc) return rc;
  if (q == nullptr || o == nullptr || workspace == nullptr || Hq <= 0 || T < 0 ||
      window_left < -1)
    return ATTN_ERR_INVALID_ARG;
  // (a factor that is 0 or inf would make a hidden key's -inf, or a score of 0, NaN)
  if (!(scale >= std::numeric_limits<float>::min()) || !std::isfinite(scale * kLog2e))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
    return ATTN_ERR_INVALID_ARG;
  if (!row_stride(&q_row, Hq, cache->dqk) || q_row >= (1ll << 38)) return ATTN_ERR_INVALID_ARG;
  if (Hq % cache->heads != 0) return ATTN_ERR_INVALID_ARG;
  const int group = Hq / cache->heads;
  if (group > kTile || (int64_t)Hq * cache->dqk > (1 << 20) || T > INT32_MAX - (1 << 20) ||
      B > (1 << 20))
    return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < kPrefillWorkspaceBytes) return ATTN_ERR_WORKSPACE_TOO_SMALL;
  PrefillShape& sh = L.sh;
  sh.B = B;
  sh.group = group;
  sh.per_tile = kTile / group;
  // (a window as long as the table's room is none; shorter ones leave sums with it in range)
  sh.window = window_left >= std::min<int64_t>((int64_t)max_pages * cache->page_size,
                                               INT32_MAX - (1 << 20))
                  ? -1
                  : window_left;
  static thread_local PrefillOffsets offsets;
  int64_t units = 0;
  if (cu_seqlens != nullptr) {
    if (B > ATTN_MAX_VARLEN_SEQS) return ATTN_ERR_UNSUPPORTED;
    if (cu_seqlens[0] != 0 || cu_seqlens[B] != T) return ATTN_ERR_INVALID_ARG;
    for (int b = 0; b < B; ++b) {
      if (cu_seqlens[b + 1] < cu_seqlens[b]) return ATTN_ERR_INVALID_ARG;
      offsets.cu[b] = cu_seqlens[b];
      offsets.unit0[b] = (int)units;
      units += prefill_units(cu_seqlens[b + 1] - cu_seqlens[b], sh.per_tile);
    }
    offsets.cu[B] = T;
    offsets.unit0[B] = (int)units;
    L.offsets = &offsets;
  } else {
    if (T % B != 0) return ATTN_ERR_INVALID_ARG;
    sh.per_seq = T / B;
    sh.units_per_seq = prefill_units(sh.per_seq, sh.per_tile);
    units = (int64_t)B * sh.units_per_seq;
  }
  if (T == 0) return ATTN_OK;
  sh.units = (int)units;  // (at most T)
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return ATTN_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)cache->dqk, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)cache->dqk * 2, (cuuint64_t)q_row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)sh.per_tile}, one[3] = {1, 1, 1};
  if (enc(&L.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
          one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return ATTN_ERR_CUDA;
  // Boxes of rows of one page for whole tiles, where pages are multiples of 8 tokens (the
  // swizzle's period) and the strides are what a map takes; else those tiles come by rows too.
  L.box = cache->page_size % 32 == 0 ? 32 : cache->page_size % 16 == 0 ? 16
                                        : cache->page_size % 8 == 0 ? 8 : 0;
  L.heads_inner = cache->k_head_stride < cache->k_token_stride;
  if (L.box > 0 && (!page_map(&L.tm_k, cache, false, L.box, L.heads_inner) ||
                    !page_map(&L.tm_v, cache, true, L.box, L.heads_inner)))
    L.box = 0;
  L.T = T;
  L.Hq = Hq;
  L.o = o;
  L.lse = lse;
  L.scale_log2 = scale * kLog2e;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  L.desc = reinterpret_cast<PrefillDesc*>(base);
  L.ml = reinterpret_cast<float2*>(base + kPrefillDescBytes);
  L.acc = reinterpret_cast<float*>(base + kPrefillDescBytes + kPrefillMlBytes);
  L.dqk = cache->dqk;
  L.dv = cache->dv;
  L.num_sms = sm_count();
  if (L.num_sms <= 0) return ATTN_ERR_CUDA;
  L.status = cache_status_ptr();
  if (!L.status) return ATTN_ERR_CUDA;
  L.stream = static_cast<cudaStream_t>(stream);
  return cuda_err(launch_prefill(L));
}

int attn_cache_status(void* stream) {
  return take_status(cache_status_ptr(), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
