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
// into an e4m3 cache), against three flops.  What is left to do is to keep the
// index work and the angles off the path:
//   * a thread moves units of 16 columns, two 16-byte loads and stores each, and
//     keeps its unit (head, columns, destination) from token to token of its
//     block, so the divisions that find it are paid once;
//   * a block takes several token rows where there are many, computes each
//     (position, pair) angle once for all heads into shared memory, and has its
//     first loads, two units a thread, on their way meanwhile.
// Measured on a GB300 (a plain copy there: 6.78 TB/s): rotation of 537 MB (B 1, T
// 32768, 16 + 16 heads of 128) 81.6 us, 6.58 TB/s; of 458 MB of ragged (192, 64 of it
// turned) heads 70.2 us, 6.52 TB/s; append of 16.8 K prompt tokens, 32 query and 8 key
// heads of 128, into e4m3: 378 MB in 77.9 us, 4.86 TB/s (the conversions' registers
// leave a third of the warps: 85 registers, 21 warps of 64 on an SM; with 64 registers
// they spill, 82 us); (192, 128) heads, 336 MB in 59.3 us, 5.66 TB/s.
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

// Threads of a block at most, and blocks on an SM that the registers are to leave
// room for: many loads on their way (bf16: 59.5 us where 512 threads and two
// blocks take 63.7), or the registers that eight-bit conversions need (76.5 us, and
// 82 to 104 us with others; the (192, 128) append and the e4m3 append above).
template <bool E4M3>
struct Bounds {
  static constexpr int kThreads = E4M3 ? 384 : 256, kBlocks = E4M3 ? 2 : 5;
};
constexpr int kMaxTokens = 32;        // token rows of one block at most
constexpr int kMaxAngles = 2048;      // (token, pair) angles of one block at most
constexpr int kRounds = 4;            // tokens a thread walks over, where there are many

// Shape of the blocks over `rows` token rows of `units` units each: `side`
// token rows side by side (about 256 threads, or one row), and up to kRounds of
// them one after the other as long as every SM has some blocks (4 and 8 measure
// alike, 16 loses 4 to 10 %: a block's angles come before its first store).
struct BlockShape {
  int threads, side, tokens, blocks;
};
BlockShape block_shape(int rows, int units, int dim, int sms, int most_threads) {
  BlockShape s;
  const int most = dim > 0 ? std::min(kMaxTokens, kMaxAngles / (dim / 2)) : kMaxTokens;
  s.side = std::min(std::max(1, std::min(256, most_threads) / units), most);
  s.threads = std::min(most_threads, cdiv(s.side * units, 32) * 32);
  const int rounds = std::max(1, std::min(kRounds, rows / (s.side * sms * 8)));
  s.tokens = std::min(s.side * rounds, most);
  s.blocks = cdiv(rows, s.tokens);
  return s;
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
  for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
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
// ----------------------------------------------------------------------------
template <int D, typename Offsets>
__global__ void __launch_bounds__(Bounds<false>::kThreads, Bounds<false>::kBlocks)
rope_kernel(const __grid_constant__ RopeParams P, const __grid_constant__ Offsets off) {
  __shared__ int pos[kMaxTokens];
  __shared__ __align__(16) float2 sc[kMaxAngles];
  constexpr int kUnits = D / 16;
  const int which = blockIdx.x < P.t[0].blocks ? 0 : 1;
  const RopeTensor& X = P.t[which];
  const int row0 = (blockIdx.x - (which ? P.t[0].blocks : 0)) * X.tokens;
  const int tokens = min(X.tokens, X.rows - row0);
  const int units = X.H * kUnits;  // of a token row
  const int side = X.side;
  const uint16_t* x = static_cast<const uint16_t*>(X.x) + row0 * X.x_row;
  uint16_t* y = static_cast<uint16_t*>(X.y) + row0 * X.y_row;

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

  // this thread's unit, and the token rows t0, t0 + side, ... of it
  const int t0 = threadIdx.x / units;
  int at = threadIdx.x - t0 * units;
  int unit = 0, ca = 0, cb = 0;  // columns within a row
  auto take = [&]() {
    const int head = at / kUnits;
    unit = at - head * kUnits;
    unit_columns(P.rot, unit, ca, cb);
    ca += head * D;
    cb += head * D;
  };
  Unit w[2];
  auto load = [&](int t, Unit& w) {
    if (t >= tokens) return;
    const uint16_t* row = x + t * X.x_row;
    w.a = *reinterpret_cast<const uint4*>(row + ca);
    w.b = *reinterpret_cast<const uint4*>(row + cb);
  };
  bool busy = t0 < min(side, tokens) && at < units;
  int t = t0;
  if (busy) {
    take();
    load(t, w[0]);
    load(t + side, w[1]);
  }
  __syncthreads();
  fill_angles(sc, pos, tokens, P.rot, P.inverse != 0);
  __syncthreads();
  while (busy) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tj = t + j * side;
      if (tj >= tokens) break;
      if (unit < (P.rot.dim >> 4)) {
        float a[8], b[8];
        unpack8(w[j].a, a);
        unpack8(w[j].b, b);
        turn_unit(sc, tj, unit, P.rot, a, b);
        w[j].a = pack8(a);
        w[j].b = pack8(b);
      }
      uint16_t* row = y + tj * X.y_row;
      *reinterpret_cast<uint4*>(row + ca) = w[j].a;
      *reinterpret_cast<uint4*>(row + cb) = w[j].b;
      load(tj + 2 * side, w[j]);
    }
    t += 2 * side;
    const bool fresh = t >= tokens;
    if (fresh) {  // the next unit, in rows of more units than threads
      at += blockDim.x;
      busy = at < units && units > (int)blockDim.x;
      t = t0;
      if (busy) take();
    }
    if (fresh && busy) {
      load(t, w[0]);
      load(t + side, w[1]);
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
  int B, T, Hq, per_seq, tokens, side;
  Rotation rot;
  int* status;
};

// Division by a scale s as a product with 1 / s in two terms.  With hi = 1 / s
// rounded and lo = (1 - s hi) hi, x (hi + lo) is x / s to 2^-47; the error-free
// product x hi = p + e (Dekker's, by fma) keeps that up to one rounding to fp32, as a
// division has: a quotient on the border between two e4m3 neighbours stays there.
struct Scale {
  float hi = 1.f, lo = 0.f;
  __device__ __forceinline__ void set(float s) {
    hi = __fdiv_rn(1.f, s);
    lo = fmaf(-s, hi, 1.f) * hi;
  }
  __device__ __forceinline__ float divide(float x) const {
    const float p = x * hi;
    const float q = p + fmaf(x, lo, fmaf(x, hi, -p));
    return fabsf(p) <= 3.402823466e38f ? q : p;  // (infinite: no rest to add)
  }
};

// Eight values as e4m3 of x / scale, saturated.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], const Scale& scale) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r)
        : "f"(scale.divide(x[2 * i + 1])), "f"(scale.divide(x[2 * i])));
    h[i] = r;
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <int DQK, int DV, bool E4M3, typename Offsets>
__global__ void __launch_bounds__(Bounds<E4M3>::kThreads, Bounds<E4M3>::kBlocks)
append_kernel(const __grid_constant__ AppendParams P, const __grid_constant__ Offsets off) {
  __shared__ int pos[kMaxTokens];
  __shared__ int64_t koff[kMaxTokens], voff[kMaxTokens];  // byte offset of the slot; -1: none
  __shared__ __align__(16) float2 sc[kMaxAngles];
  constexpr int kUnits = DQK / 16, kUnitsV = DV / 16;
  const int row0 = blockIdx.x * P.tokens;
  const int tokens = min(P.tokens, P.T - row0);
  const int n_q = P.Hq * kUnits, n_k = P.cache.heads * kUnits, n_v = P.cache.heads * kUnitsV;
  const int units = n_q + n_k + n_v;  // of a token
  const int side = P.side;

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
        const int in = p - slot * P.cache.page_size;
        ko = token_at(P.cache.k, page, in);
        vo = token_at(P.cache.v, page, in);
      } else {
        atomicCAS(P.status, 0, kStatusBadPage);
      }
    }
    pos[threadIdx.x] = p;
    koff[threadIdx.x] = ko;
    voff[threadIdx.x] = vo;
  }
  // this thread's unit: where it is read, where it goes, whether it turns
  const int t0 = threadIdx.x / units;
  int at = threadIdx.x - t0 * units;
  int unit = 0, ca = 0, cb = 0;
  bool turns = false;
  const uint16_t* x = nullptr;
  int64_t x_row = 0;
  char* y = nullptr;                    // q_out (rows y_row bytes apart) or one side of the cache
  const int64_t* slots = nullptr;       // null: q_out
  Scale scale;
  auto take = [&]() {
    int rem = at;
    if (rem < n_q + n_k) {
      const bool key = rem >= n_q;
      if (key) rem -= n_q;
      const int head = rem / kUnits;
      unit = rem - head * kUnits;
      turns = unit < (P.rot.dim >> 4);
      unit_columns(P.rot, unit, ca, cb);
      x_row = key ? P.k_row : P.q_row;
      x = (key ? P.k : P.q) + row0 * x_row + head * DQK;
      if (key) {
        y = P.cache.k.base + head * P.cache.k.head;
        slots = koff;
        if (E4M3 && P.cache.k.scale) scale.set(__ldg(P.cache.k.scale + head));
      } else {
        y = reinterpret_cast<char*>(P.q_out + row0 * P.q_out_row + head * DQK);
        slots = nullptr;
      }
    } else {
      rem -= n_q + n_k;
      const int head = rem / kUnitsV;
      unit = rem - head * kUnitsV;
      turns = false;
      ca = unit * 16;
      cb = ca + 8;
      x_row = P.v_row;
      x = P.v + row0 * x_row + head * DV;
      y = P.cache.v.base + head * P.cache.v.head;
      slots = voff;
      if constexpr (E4M3) scale.set(P.cache.v.scale ? __ldg(P.cache.v.scale + head) : 1.f);
    }
  };
  Unit w[2];
  auto load = [&](int t, Unit& w) {
    if (t >= tokens) return;
    const uint16_t* row = x + t * x_row;
    w.a = *reinterpret_cast<const uint4*>(row + ca);
    w.b = *reinterpret_cast<const uint4*>(row + cb);
  };
  bool busy = t0 < min(side, tokens) && at < units;
  int t = t0;
  if (busy) {
    take();
    load(t, w[0]);
    load(t + side, w[1]);
  }
  __syncthreads();
  fill_angles(sc, pos, tokens, P.rot, false);
  __syncthreads();
  while (busy) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tj = t + j * side;
      if (tj >= tokens) break;
      const bool eight = E4M3 && slots != nullptr;
      char* row;
      bool put = pos[tj] >= 0;
      if (slots != nullptr) {
        put = put && slots[tj] >= 0;
        row = y + slots[tj];
      } else {
        row = y + tj * P.q_out_row * 2;
      }
      if (put) {
        float a[8], b[8];
        if (turns || eight) {
          unpack8(w[j].a, a);
          unpack8(w[j].b, b);
        }
        if (turns) turn_unit(sc, tj, unit, P.rot, a, b);
        if (eight) {
          *reinterpret_cast<uint2*>(row + ca) = quantise8(a, scale);
          *reinterpret_cast<uint2*>(row + cb) = quantise8(b, scale);
        } else {
          if (turns) {
            w[j].a = pack8(a);
            w[j].b = pack8(b);
          }
          *reinterpret_cast<uint4*>(row + ca * 2) = w[j].a;
          *reinterpret_cast<uint4*>(row + cb * 2) = w[j].b;
        }
      }
      load(tj + 2 * side, w[j]);
    }
    t += 2 * side;
    const bool fresh = t >= tokens;
    if (fresh) {  // the next unit, where a token has more units than there are threads
      at += blockDim.x;
      busy = at < units && units > (int)blockDim.x;
      t = t0;
      if (busy) take();
    }
    if (fresh && busy) {
      load(t, w[0]);
      load(t + side, w[1]);
    }
  }
}

template <int D>
cudaError_t rope_typed(const RopeLaunch& L, const RopeParams& P, int blocks, int threads) {
  if (L.cu[0] != nullptr) {
    PairOffsets off;
    std::memcpy(&off.q, L.cu[0], sizeof(RowOffsets));
    std::memcpy(&off.k, L.cu[1], sizeof(RowOffsets));
    rope_kernel<D><<<blocks, threads, 0, L.stream>>>(P, off);
  } else {
    rope_kernel<D><<<blocks, threads, 0, L.stream>>>(P, NoOffsets{});
  }
  return cudaGetLastError();
}

template <int DQK, int DV, bool E4M3>
cudaError_t append_typed(const AppendLaunch& L, const AppendParams& P, const BlockShape& s) {
  if (L.offsets != nullptr)
    append_kernel<DQK, DV, E4M3><<<s.blocks, s.threads, 0, L.stream>>>(P, *L.offsets);
  else
    append_kernel<DQK, DV, E4M3><<<s.blocks, s.threads, 0, L.stream>>>(P, NoOffsets{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L) {
  RopeParams P;
  std::memset(&P, 0, sizeof(P));
  int blocks = 0, threads = 0;
  for (int i = 0; i < 2; ++i) {
    P.t[i] = L.t[i];
    if (P.t[i].rows == 0) continue;
    const BlockShape s = block_shape(P.t[i].rows, P.t[i].H * (L.d / 16), L.rot.dim, L.num_sms,
                                     Bounds<false>::kThreads);
    P.t[i].tokens = s.tokens;
    P.t[i].side = s.side;
    P.t[i].blocks = s.blocks;
    blocks += s.blocks;
    threads = std::max(threads, s.threads);  // (a wider block serves the narrower tensor too)
  }
  if (blocks == 0) return cudaSuccess;
  P.rot = L.rot;
  P.inverse = L.inverse;
  P.nseq = L.nseq;
  P.pos0 = L.pos0;
  switch (L.d) {
    case 64: return rope_typed<64>(L, P, blocks, threads);
    case 128: return rope_typed<128>(L, P, blocks, threads);
    case 192: return rope_typed<192>(L, P, blocks, threads);
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
  const bool e = L.cache.e4m3 != 0;
  const int units = (L.Hq + L.cache.heads) * (L.dqk / 16) + L.cache.heads * (L.dv / 16);
  const BlockShape s = block_shape(L.T, units, L.rot.dim, L.num_sms,
                                   e ? Bounds<true>::kThreads : Bounds<false>::kThreads);
  P.tokens = s.tokens;
  P.side = s.side;
  if (L.dqk == 64)
    return e ? append_typed<64, 64, true>(L, P, s) : append_typed<64, 64, false>(L, P, s);
  if (L.dqk == 128)
    return e ? append_typed<128, 128, true>(L, P, s) : append_typed<128, 128, false>(L, P, s);
  if (L.dqk == 192)
    return e ? append_typed<192, 128, true>(L, P, s) : append_typed<192, 128, false>(L, P, s);
  return cudaErrorInvalidValue;
}

}  // namespace attn
