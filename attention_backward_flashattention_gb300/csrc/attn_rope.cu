// attn_rope.cu — position rotation of queries and keys, and the append of new
// tokens to a paged cache with that rotation applied on the way.
//
// Mathematics.  Pair i of a head at position p turns by p * w_i.  The rate w_i
// is stored as a fraction of a turn times 2^64, so p * rate modulo 2^64 is the
// angle modulo one turn with no loss at far positions (in fp32 the product
// p * w_i at p = 10^6 is off by 0.03 rad).  Its top 32 bits, as a signed
// fraction, go to sincospif, whose argument is then in [-1, 1): the angle
// handed over is off by at most pi * 2^-24, of the order of sincospif's own
// rounding.  Negative positions (the inverse rotation negates p) work by two's
// complement.  The rotation is two products and a sum in fp32, rounded to the
// output's type once.
//
// Bound: memory.  Each element is read once and written once (2 + 2 bytes; 2 + 1
// into an e4m3 cache), against three flops.  So a block takes a few whole token rows,
// computes each (position, pair) angle once for all heads into shared memory,
// and every thread moves units of 16 columns — two 16-byte loads and stores — two
// units at a time, the first loads issued before the angles are computed.
#include <algorithm>
#include <cstring>

#include "attn_paged.h"
#include "ptx.cuh"

namespace attn {

__device__ int g_cache_status = 0;

int* cache_status_ptr() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_cache_status) != cudaSuccess) return nullptr;
  return static_cast<int*>(p);
}

namespace {

constexpr int kThreads = 256;
constexpr int kUnitsInFlight = 2;     // units a thread loads before it uses the first
constexpr int kMaxTokens = 32;        // token rows of one block at most
constexpr int kMaxAngles = 2048;      // (token, pair) angles of one block at most

// Token rows of a block: enough units that each thread has kUnitsInFlight.
int tokens_per_block(int units_per_token, int dim) {
  int n = kThreads * kUnitsInFlight / std::max(units_per_token, 1);
  if (dim > 0) n = std::min(n, kMaxAngles / (dim / 2));
  return std::max(1, std::min(n, kMaxTokens));
}

// Sixteen columns of a head, in two chunks of eight: columns ca .. ca + 7 and
// cb .. cb + 7.  Units 0 .. dim/16 - 1 hold eight pairs each; the others the
// columns that pass unchanged.
struct Unit {
  uint4 a, b;
};

__device__ __forceinline__ void unit_columns(const Rotation& rot, int u, int& ca, int& cb) {
  const int turning = rot.dim >> 4;
  if (u >= turning) {
    const int e = (u - turning) << 4;
    ca = e < rot.begin ? e : e + rot.dim;
    cb = ca + 8;
  } else if (rot.pairs) {
    ca = rot.begin + (u << 4);
    cb = ca + 8;
  } else {
    ca = rot.begin + (u << 3);
    cb = ca + (rot.dim >> 1);
  }
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r[i] << 16);
    x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// Angles of one block: (cos, sin) of token t's pair 8u + e is the float2
// ((t*4 + e/2) * units + u) * 2 + e%2, so that the threads of consecutive
// units read consecutive 16 bytes.
__device__ __forceinline__ void fill_angles(float2* sc, const int* pos, int tokens,
                                            const Rotation& rot, bool inverse) {
  const int pairs = rot.dim >> 1, units = rot.dim >> 4;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, pair = i - t * pairs;
    const long long p = inverse ? -(long long)pos[t] : (long long)pos[t];
    const unsigned long long turn = (unsigned long long)p * __ldg(rot.rates + pair);
    float s, c;
    sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f /* 2^-31 */, &s, &c);
    sc[((t * 4 + ((pair & 7) >> 1)) * units + (pair >> 3)) * 2 + (pair & 1)] = make_float2(c, s);
  }
}

// Rotates the eight pairs of unit u; x and y: the unit's chunks, in and out.
__device__ __forceinline__ void turn_unit(const float2* sc, int t, int u, const Rotation& rot,
                                          float (&x)[8], float (&y)[8]) {
  const int units = rot.dim >> 4;
  const float4* at = reinterpret_cast<const float4*>(sc) + t * 4 * units + u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 w = at[k * units];  // cos, sin of pairs 2k and 2k + 1
    if (rot.pairs) {
      float* z = k < 2 ? x + 4 * k : y + 4 * (k - 2);
      const float a0 = z[0], b0 = z[1], a1 = z[2], b1 = z[3];
      z[0] = a0 * w.x - b0 * w.y;
      z[1] = a0 * w.y + b0 * w.x;
      z[2] = a1 * w.z - b1 * w.w;
      z[3] = a1 * w.w + b1 * w.z;
    } else {
      const float a0 = x[2 * k], b0 = y[2 * k], a1 = x[2 * k + 1], b1 = y[2 * k + 1];
      x[2 * k] = a0 * w.x - b0 * w.y;
      y[2 * k] = a0 * w.y + b0 * w.x;
      x[2 * k + 1] = a1 * w.z - b1 * w.w;
      y[2 * k + 1] = a1 * w.w + b1 * w.z;
    }
  }
}

// Sequence of row r: the last s with cu[s] <= r (r < cu[nseq]; empty sequences
// are passed over).
__device__ __forceinline__ int sequence_of(const int* cu, int nseq, int r) {
  int lo = 0, hi = nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct NoOffsets {};
struct PairOffsets {
  RowOffsets q, k;
};

struct RopeParams {
  RopeTensor t[2];
  Rotation rot;
  int inverse, nseq, pos0;
};

// ----------------------------------------------------------------------------
// attn_rope: blocks 0 .. t[0].blocks - 1 take the queries, the others the keys.
//
// Measured (GB300): see the rates at the launch below.
// ----------------------------------------------------------------------------
template <int D, typename Offsets>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeParams P, const __grid_constant__ Offsets off) {
  __shared__ int pos[kMaxTokens];
  __shared__ __align__(16) float2 sc[kMaxAngles];
  constexpr int kUnits = D / 16;
  const int which = blockIdx.x < P.t[0].blocks ? 0 : 1;
  const RopeTensor& X = P.t[which];
  const int row0 = (blockIdx.x - (which ? P.t[0].blocks : 0)) * X.tokens_per_block;
  const int tokens = min(X.tokens_per_block, X.rows - row0);
  const int per_token = X.H * kUnits;
  const int n = tokens * per_token;
  const uint16_t* x = static_cast<const uint16_t*>(X.x);
  uint16_t* y = static_cast<uint16_t*>(X.y);

  if (threadIdx.x < tokens) {
    const int r = row0 + threadIdx.x;
    if constexpr (sizeof(Offsets) > sizeof(RowOffsets)) {
      const int s = sequence_of(which ? off.k.cu : off.q.cu, P.nseq, r);
      // the queries are the last positions of the sequence's keys
      const int shift = which ? 0
                              : (off.k.cu[s + 1] - off.k.cu[s]) - (off.q.cu[s + 1] - off.q.cu[s]);
      pos[threadIdx.x] = P.pos0 + shift + r - (which ? off.k.cu[s] : off.q.cu[s]);
    } else {
      pos[threadIdx.x] = P.pos0 + X.shift + r % X.T;
    }
  }
  bool ready = false;
  for (int base = threadIdx.x; base - (int)threadIdx.x < n; base += kThreads * kUnitsInFlight) {
    Unit w[kUnitsInFlight];
    int64_t ya[kUnitsInFlight], yb[kUnitsInFlight];
    int tok[kUnitsInFlight], unit[kUnitsInFlight];
#pragma unroll
    for (int j = 0; j < kUnitsInFlight; ++j) {
      const int item = base + j * kThreads;
      tok[j] = -1;
      if (item < n) {
        tok[j] = item / per_token;
        const int rem = item - tok[j] * per_token;
        const int head = rem / kUnits;
        unit[j] = rem - head * kUnits;
        int ca, cb;
        unit_columns(P.rot, unit[j], ca, cb);
        const int64_t xr = (int64_t)(row0 + tok[j]) * X.x_row + head * D;
        const int64_t yr = (int64_t)(row0 + tok[j]) * X.y_row + head * D;
        ya[j] = yr + ca;
        yb[j] = yr + cb;
        w[j].a = *reinterpret_cast<const uint4*>(x + xr + ca);
        w[j].b = *reinterpret_cast<const uint4*>(x + xr + cb);
      }
    }
    if (!ready) {  // the same in every thread: the first loads are on their way
      __syncthreads();
      fill_angles(sc, pos, tokens, P.rot, P.inverse != 0);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int j = 0; j < kUnitsInFlight; ++j) {
      if (tok[j] < 0) continue;
      if (unit[j] < (P.rot.dim >> 4)) {
        float a[8], b[8];
        unpack8(w[j].a, a);
        unpack8(w[j].b, b);
        turn_unit(sc, tok[j], unit[j], P.rot, a, b);
        w[j].a = pack8(a);
        w[j].b = pack8(b);
      }
      *reinterpret_cast<uint4*>(y + ya[j]) = w[j].a;
      *reinterpret_cast<uint4*>(y + yb[j]) = w[j].b;
    }
  }
}

// ----------------------------------------------------------------------------
// attn_cache_append
// ----------------------------------------------------------------------------
struct AppendParams {
  CacheView cache;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_row, v_row, q_row, q_out_row;
  int B, T, Hq, per_seq, tokens_per_block;
  Rotation rot;
  int* status;
};

// Eight values as e4m3 of x / scale, saturated (one rounding: the division is
// correctly rounded to fp32 first, which moves a value across a border between two e4m3
// neighbours only where it lies within 2^-24 of it).
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r)
        : "f"(__fdiv_rn(x[2 * i + 1], scale)), "f"(__fdiv_rn(x[2 * i], scale)));
    h[i] = r;
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <int DQK, int DV, bool E4M3, typename Offsets>
__global__ void __launch_bounds__(kThreads)
append_kernel(const __grid_constant__ AppendParams P, const __grid_constant__ Offsets off) {
  __shared__ int pos[kMaxTokens];
  __shared__ int64_t koff[kMaxTokens], voff[kMaxTokens];  // byte offset of the slot; -1: none
  __shared__ __align__(16) float2 sc[kMaxAngles];
  constexpr int kUnits = DQK / 16, kUnitsV = DV / 16;
  constexpr int kBytes = E4M3 ? 1 : 2;
  const int row0 = blockIdx.x * P.tokens_per_block;
  const int tokens = min(P.tokens_per_block, P.T - row0);
  const int n_q = P.Hq * kUnits, n_k = P.cache.heads * kUnits, n_v = P.cache.heads * kUnitsV;
  const int per_token = n_q + n_k + n_v;
  const int n = tokens * per_token;

  if (threadIdx.x < tokens) {
    const int r = row0 + threadIdx.x;
    int s, from_end;  // the row's sequence, and its distance from the sequence's end
    if constexpr (sizeof(Offsets) >= sizeof(RowOffsets)) {
      s = sequence_of(off.cu, P.B, r);
      from_end = off.cu[s + 1] - r;
    } else {
      s = r / P.per_seq;
      from_end = P.per_seq - (r - s * P.per_seq);
    }
    const int p = max(P.cache.lens[s], 0) - from_end;
    int64_t ko = -1, vo = -1;
    if (p >= 0) {
      const int slot = div_page(P.cache, p);
      int page = -1;
      if (slot < P.cache.max_pages) page = P.cache.table[s * P.cache.table_stride + slot];
      if (page_in(P.cache, page)) {
        ko = token_at(P.cache, P.cache.k, page, p);
        vo = token_at(P.cache, P.cache.v, page, p);
      } else {
        atomicCAS(P.status, 0, kStatusBadPage);
      }
    }
    pos[threadIdx.x] = p;
    koff[threadIdx.x] = ko;
    voff[threadIdx.x] = vo;
  }
  bool ready = false;
  for (int base = threadIdx.x; base - (int)threadIdx.x < n; base += kThreads * kUnitsInFlight) {
    Unit w[kUnitsInFlight];
    int tok[kUnitsInFlight], head[kUnitsInFlight], unit[kUnitsInFlight], what[kUnitsInFlight];
    int ca[kUnitsInFlight], cb[kUnitsInFlight];
#pragma unroll
    for (int j = 0; j < kUnitsInFlight; ++j) {
      const int item = base + j * kThreads;
      tok[j] = -1;
      if (item < n) {
        tok[j] = item / per_token;
        int rem = item - tok[j] * per_token;
        const uint16_t* x;
        if (rem < n_q + n_k) {
          what[j] = rem < n_q ? 0 : 1;
          if (what[j]) rem -= n_q;
          head[j] = rem / kUnits;
          unit[j] = rem - head[j] * kUnits;
          unit_columns(P.rot, unit[j], ca[j], cb[j]);
          x = (what[j] ? P.k + (row0 + tok[j]) * P.k_row : P.q + (row0 + tok[j]) * P.q_row) +
              head[j] * DQK;
        } else {
          what[j] = 2;
          rem -= n_q + n_k;
          head[j] = rem / kUnitsV;
          unit[j] = rem - head[j] * kUnitsV;
          ca[j] = unit[j] * 16;
          cb[j] = ca[j] + 8;
          x = P.v + (row0 + tok[j]) * P.v_row + head[j] * DV;
        }
        w[j].a = *reinterpret_cast<const uint4*>(x + ca[j]);
        w[j].b = *reinterpret_cast<const uint4*>(x + cb[j]);
      }
    }
    if (!ready) {  // the same in every thread: the first loads are on their way
      __syncthreads();
      fill_angles(sc, pos, tokens, P.rot, false);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int j = 0; j < kUnitsInFlight; ++j) {
      if (tok[j] < 0 || pos[tok[j]] < 0) continue;
      const bool turns = what[j] < 2 && unit[j] < (P.rot.dim >> 4);
      float a[8], b[8];
      if (turns || (E4M3 && what[j] > 0)) {
        unpack8(w[j].a, a);
        unpack8(w[j].b, b);
      }
      if (turns) turn_unit(sc, tok[j], unit[j], P.rot, a, b);
      if (what[j] == 0) {
        uint16_t* y = P.q_out + (row0 + tok[j]) * P.q_out_row + head[j] * DQK;
        if (turns) {
          w[j].a = pack8(a);
          w[j].b = pack8(b);
        }
        *reinterpret_cast<uint4*>(y + ca[j]) = w[j].a;
        *reinterpret_cast<uint4*>(y + cb[j]) = w[j].b;
      } else {
        const CacheSide& side = what[j] == 1 ? P.cache.k : P.cache.v;
        const int64_t at = what[j] == 1 ? koff[tok[j]] : voff[tok[j]];
        if (at < 0) continue;
        char* y = side.base + at + head[j] * side.head;
        if constexpr (E4M3) {
          const float scale = side.scale ? __ldg(side.scale + head[j]) : 1.f;
          *reinterpret_cast<uint2*>(y + ca[j] * kBytes) = quantise8(a, scale);
          *reinterpret_cast<uint2*>(y + cb[j] * kBytes) = quantise8(b, scale);
        } else {
          if (turns) {
            w[j].a = pack8(a);
            w[j].b = pack8(b);
          }
          *reinterpret_cast<uint4*>(y + ca[j] * kBytes) = w[j].a;
          *reinterpret_cast<uint4*>(y + cb[j] * kBytes) = w[j].b;
        }
      }
    }
  }
}

template <int D>
cudaError_t rope_typed(const RopeLaunch& L, const RopeParams& P, int blocks) {
  if (L.cu[0] != nullptr) {
    PairOffsets off;
    std::memcpy(&off.q, L.cu[0], sizeof(RowOffsets));
    std::memcpy(&off.k, L.cu[1], sizeof(RowOffsets));
    rope_kernel<D><<<blocks, kThreads, 0, L.stream>>>(P, off);
  } else {
    rope_kernel<D><<<blocks, kThreads, 0, L.stream>>>(P, NoOffsets{});
  }
  return cudaGetLastError();
}

template <int DQK, int DV, bool E4M3>
cudaError_t append_typed(const AppendLaunch& L, const AppendParams& P, int blocks) {
  if (L.offsets != nullptr)
    append_kernel<DQK, DV, E4M3><<<blocks, kThreads, 0, L.stream>>>(P, *L.offsets);
  else
    append_kernel<DQK, DV, E4M3><<<blocks, kThreads, 0, L.stream>>>(P, NoOffsets{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L) {
  RopeParams P;
  std::memset(&P, 0, sizeof(P));
  int blocks = 0;
  for (int i = 0; i < 2; ++i) {
    P.t[i] = L.t[i];
    if (P.t[i].rows == 0) continue;
    P.t[i].tokens_per_block = tokens_per_block(P.t[i].H * (L.d / 16), L.rot.dim);
    P.t[i].blocks = cdiv(P.t[i].rows, P.t[i].tokens_per_block);
    blocks += P.t[i].blocks;
  }
  if (blocks == 0) return cudaSuccess;
  P.rot = L.rot;
  P.inverse = L.inverse;
  P.nseq = L.nseq;
  P.pos0 = L.pos0;
  switch (L.d) {
    case 64: return rope_typed<64>(L, P, blocks);
    case 128: return rope_typed<128>(L, P, blocks);
    case 192: return rope_typed<192>(L, P, blocks);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_append(const AppendLaunch& L) {
  AppendParams P;
  std::memset(&P, 0, sizeof(P));
  P.cache = L.cache;
  P.k = static_cast<const uint16_t*>(L.k);
  P.v = static_cast<const uint16_t*>(L.v);
  P.q = static_cast<const uint16_t*>(L.q);
  P.q_out = static_cast<uint16_t*>(L.q_out);
  P.k_row = L.k_row;
  P.v_row = L.v_row;
  P.q_row = L.q_row;
  P.q_out_row = L.q_out_row;
  P.B = L.B;
  P.T = L.T;
  P.Hq = L.Hq;
  P.per_seq = L.per_seq;
  P.rot = L.rot;
  P.status = L.status;
  const int units = (L.Hq + L.cache.heads) * (L.dqk / 16) + L.cache.heads * (L.dv / 16);
  P.tokens_per_block = tokens_per_block(units, L.rot.dim);
  const int blocks = cdiv(L.T, P.tokens_per_block);
  const bool e = L.cache.e4m3 != 0;
  if (L.dqk == 64) return e ? append_typed<64, 64, true>(L, P, blocks) : append_typed<64, 64, false>(L, P, blocks);
  if (L.dqk == 128) return e ? append_typed<128, 128, true>(L, P, blocks) : append_typed<128, 128, false>(L, P, blocks);
  if (L.dqk == 192) return e ? append_typed<192, 128, true>(L, P, blocks) : append_typed<192, 128, false>(L, P, blocks);
  return cudaErrorInvalidValue;
}

}  // namespace attn
