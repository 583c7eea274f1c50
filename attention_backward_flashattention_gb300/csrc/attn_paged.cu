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

int attn_cache_append(const attn_paged_cache* cache, const int* block_table, int max_pages,
                      long long table_stride, const int* lens, int B, int T,
                      const int* cu_seqlens, const void* k, long long k_row, const void* v,
                      long long v_row, const void* q, long long q_row, void* q_out,
                      long long q_out_row, int Hq, const attn_rotation* rotation, void* stream) {
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
  return cuda_err(launch_append(L));
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

int attn_cache_status(void* stream) {
  return take_status(cache_status_ptr(), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
