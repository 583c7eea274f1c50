// attn_norm.cu — norm of each query and key head with the position rotation in the same pass,
// its gradient, and the append of new tokens to a paged cache with both on the way.
//
// Mathematics.  A head x of d columns becomes y = R(p) (r x * w) with r = 1 / sqrt(mean x^2 +
// eps), w a weight per column, R(p) the rotation of attn_rope.cu at the row's position.  With
// g = w * (R(p)^T dy) the gradients are dx = r (g - x r^2 mean(g x)) and, over all rows and
// heads, dw = sum (R(p)^T dy) * r x.
//
// Bound: memory (2 + 2 bytes an element, 4 + 2 in the backward).  A head lies on d / 16 lanes
// (of 4, 8 or 16), a unit of 16 columns each: both of its sums are shuffles, a pair of columns is
// always in one lane, and a lane keeps its columns' weights, and the sums of their gradients, from
// head to head.  The sums over rows are taken in a fixed order: by lane, block, and then over the
// blocks in a second launch.  Measured, 16384 tokens, 32 + 8 heads of 128 (device time): forward 57 us
// (5.9 TB/s, 88 % of a copy), backward 90 us (5.6 TB/s, 83 %).
#include <algorithm>
#include <cstring>

#include "attn_rotate.cuh"

namespace attn {
namespace {

constexpr int kNormThreads = 256;
// Heads of a group in a chunk, where there are enough (16384 tokens, 32 + 8 heads of 128, forward and
// backward: 60.7 and 107 us with 4, 57.3 and 104 with 8, 56.9 and 103 with 16).
constexpr int kNormRounds = 16;

// Lanes of a head, and whether they are all used.
template <int D>
struct HeadLanes {
  static constexpr int kUnits = D / 16;
  static constexpr int kLanes = D == 192 ? 16 : kUnits;
  static constexpr int kGroups = kNormThreads / kLanes;  // heads side by side in a block
};

// Sum over the lanes of a head.
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int k = 1; k < LANES; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
  return x;
}

__device__ __forceinline__ void unpack(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_of(w[i]);
    f[2 * i + 1] = hi_of(w[i]);
  }
}
__device__ __forceinline__ uint4 packed(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// The eight pairs of unit u of token t, turned (angles as fill_angles leaves them).
template <bool PAIRS>
__device__ __forceinline__ void turn_unit(const float2* sc, int t, int u, int units,
                                          float (&f)[16]) {
  const float4* at = reinterpret_cast<const float4*>(sc) + t * 4 * units + u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 c = at[k * units];  // cos, sin of pairs 2k and 2k + 1
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = 2 * k + h, i = PAIRS ? 2 * e : e, j = PAIRS ? 2 * e + 1 : e + 8;
      const float cs = h ? c.z : c.x, sn = h ? c.w : c.y;
      const float a = f[i], b = f[j];
      f[i] = a * cs - b * sn;
      f[j] = a * sn + b * cs;
    }
  }
}
__device__ __forceinline__ void turn_unit(const float2* sc, int t, int u, const Rotation& rot,
                                          float (&f)[16]) {
  if (rot.pairs) turn_unit<true>(sc, t, u, rot.dim >> 4, f);
  else turn_unit<false>(sc, t, u, rot.dim >> 4, f);
}

struct NormParams {
  NormTensor t[2];
  Rotation rot;
  float eps;
  int nseq, pos0;
  int tokens[2];   // token rows of a chunk, by tensor
  int blocks[2];   // of each tensor; a block takes a chunk, and then the one `blocks` behind it
};

// Blocks 0 .. blocks[0] - 1 take the queries, the others the keys.
template <int D, bool GRAD, typename Offsets>
__global__ void __launch_bounds__(kNormThreads, GRAD ? 2 : 3)
norm_kernel(const __grid_constant__ NormParams P, const __grid_constant__ Offsets off) {
  using L = HeadLanes<D>;
  __shared__ int pos[kMaxTokens];
  __shared__ __align__(16) float2 sc[kMaxAngles];
  const int which = blockIdx.x < P.blocks[0] ? 0 : 1;
  const NormTensor& X = P.t[which];
  const int block = blockIdx.x - (which ? P.blocks[0] : 0);
  const int group = threadIdx.x / L::kLanes, unit = threadIdx.x % L::kLanes;
  const bool lane_on = L::kUnits == L::kLanes || unit < L::kUnits;
  int ca = 0, cb = 8;
  unit_columns(P.rot, lane_on ? unit : 0, ca, cb);
  const bool turns = unit < (P.rot.dim >> 4);
  const uint16_t* x = static_cast<const uint16_t*>(X.x);
  const uint16_t* dy = static_cast<const uint16_t*>(X.dy);
  uint16_t* y = static_cast<uint16_t*>(X.y);
  float w[16], dw[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int c = e < 8 ? ca + e : cb + e - 8;
    w[e] = X.weight != nullptr ? __ldg(X.weight + c) : 1.f;
    dw[e] = 0.f;
  }
  const int dt = L::kGroups / X.H, dh = L::kGroups - dt * X.H;  // from one head to the next

  const int per_chunk = P.tokens[which];
  for (int64_t first = (int64_t)block * per_chunk; first < X.rows;
       first += (int64_t)P.blocks[which] * per_chunk) {
    const int row0 = (int)first;
    const int tokens = min(per_chunk, X.rows - row0);
    if (threadIdx.x < tokens) {
      const int r = row0 + threadIdx.x;
      if constexpr (sizeof(Offsets) > sizeof(RowOffsets)) {
        const int s = sequence_of(which ? off.k.cu : off.q.cu, P.nseq, r);
        // the queries are the last positions of the sequence's keys
        const int shift =
            which ? 0 : (off.k.cu[s + 1] - off.k.cu[s]) - (off.q.cu[s + 1] - off.q.cu[s]);
        pos[threadIdx.x] = P.pos0 + shift + r - (which ? off.k.cu[s] : off.q.cu[s]);
      } else {
        pos[threadIdx.x] = P.pos0 + X.shift + r % X.T;
      }
    }
    // heads group, group + kGroups, ... of the chunk's
    const int rounds = (tokens * X.H + L::kGroups - 1) / L::kGroups;
    int t = group / X.H, head = group - t * X.H;        // of the head worked on
    int tl = t, hl = head;                               // of the head loaded
    uint4 v[2][GRAD ? 4 : 2];
    auto load = [&](uint4 (&d)[GRAD ? 4 : 2]) {
      if (lane_on && tl < tokens) {
        const uint16_t* p = x + (row0 + tl) * X.x_row + hl * D;
        d[0] = *reinterpret_cast<const uint4*>(p + ca);
        d[1] = *reinterpret_cast<const uint4*>(p + cb);
        if constexpr (GRAD) {
          const uint16_t* q = dy + (row0 + tl) * X.dy_row + hl * D;
          d[2] = *reinterpret_cast<const uint4*>(q + ca);
          d[3] = *reinterpret_cast<const uint4*>(q + cb);
        }
      } else {
#pragma unroll
        for (int i = 0; i < (GRAD ? 4 : 2); ++i) d[i] = make_uint4(0, 0, 0, 0);
      }
      tl += dt;
      hl += dh;
      if (hl >= X.H) hl -= X.H, ++tl;
    };
    load(v[0]);
    load(v[1]);
    __syncthreads();
    if (P.rot.dim > 0) fill_angles(sc, pos, tokens, P.rot, GRAD);
    __syncthreads();
    for (int i = 0; i < rounds; i += 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (i + j >= rounds) break;
        float f[16], g[16];
        unpack(v[j][0], f);
        unpack(v[j][1], f + 8);
        if constexpr (GRAD) {
          unpack(v[j][2], g);
          unpack(v[j][3], g + 8);
        }
        load(v[j]);
        const bool there = lane_on && t < tokens;
        float ss = 0.f, gx = 0.f;
        if constexpr (GRAD)
          if (turns && there) turn_unit(sc, t, unit, P.rot, g);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          ss = fmaf(f[e], f[e], ss);
          if constexpr (GRAD) gx = fmaf(g[e] * w[e], f[e], gx);
        }
        ss = head_sum<L::kLanes>(ss);
        if constexpr (GRAD) gx = head_sum<L::kLanes>(gx);
        const float r = rsqrtf(ss * (1.f / D) + P.eps);
        if constexpr (GRAD) {
          const float back = r * r * gx * (1.f / D);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float n = f[e] * r;
            dw[e] = fmaf(g[e], n, dw[e]);
            f[e] = r * fmaf(g[e], w[e], -f[e] * back);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = f[e] * r * w[e];
          if (turns && there) turn_unit(sc, t, unit, P.rot, f);
        }
        if (there) {
          uint16_t* p = y + (row0 + t) * X.y_row + head * D;
          *reinterpret_cast<uint4*>(p + ca) = packed(f);
          *reinterpret_cast<uint4*>(p + cb) = packed(f + 8);
        }
        t += dt;
        head += dh;
        if (head >= X.H) head -= X.H, ++t;
      }
    }
    __syncthreads();  // (the next chunk's positions and angles take this one's place)
  }

  if constexpr (GRAD) {
    if (X.dw == nullptr) return;
    // the block's sums: over the heads of a warp by shuffles, then over its warps in order
    float* sums = reinterpret_cast<float*>(sc);  // [warp][D]
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = dw[e];
#pragma unroll
      for (int k = L::kLanes; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      if ((threadIdx.x & 31) < L::kLanes && lane_on)
        sums[warp * D + (e < 8 ? ca + e : cb + e - 8)] = s;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kNormThreads / 32; ++i) s += sums[i * D + threadIdx.x];
      // (dw points to the tensor's rows of sums here)
      X.dw[(int64_t)block * D + threadIdx.x] = s;
    }
  }
}

// The weights' gradients from the blocks' rows of sums: a cluster of eight blocks takes 32 columns of
// one tensor, each block an eighth of the rows, whose sums meet in the first one, in order (one
// block of each 32 columns took 17 us of 103).
struct NormSums {
  const float* rows[2];
  float* dw[2];
  int blocks[2];
  int d;
};
constexpr int kSumSlices = 8, kSumThreads = 512;
__global__ void __cluster_dims__(kSumSlices, 1, 1) __launch_bounds__(kSumThreads)
norm_sums_kernel(const NormSums P) {
  __shared__ float part[kSumThreads / 32][32];
  __shared__ float met[kSumSlices][32];
  const int per = P.d / 32, which = blockIdx.y / per, slice = blockIdx.x;
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = (blockIdx.y - which * per) * 32 + lane;
  // (every thread: this kernel may not end in front of the one that it is launched behind)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (P.dw[which] != nullptr) {
    const float* rows = P.rows[which];
    const int n = P.blocks[which], each = (n + kSumSlices - 1) / kSumSlices;
    const int end = min(n, (slice + 1) * each);
#pragma unroll 8
    for (int i = slice * each + y; i < end; i += kSumThreads / 32) s += rows[(int64_t)i * P.d + c];
  }
  part[y][lane] = s;
  __syncthreads();
  if (y == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumThreads / 32; ++i) s += part[i][lane];
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                     mapa_shared(smem_u32(&met[slice][lane]), 0)),
                 "f"(s)
                 : "memory");
  }
  cluster_sync();
  if (slice == 0 && y == 0 && P.dw[which] != nullptr) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumSlices; ++i) s += met[i][lane];
    P.dw[which][c] = s;
  }
}

// ----------------------------------------------------------------------------
// Append with the norm: a block takes a chunk of token rows, the heads of their queries and
// keys as above, the values unit by unit.
// ----------------------------------------------------------------------------
struct AppendNormParams {
  CacheView cache;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_row, v_row, q_row, q_out_row;
  int B, T, Hq, per_seq, tokens;
  Rotation rot;
  HeadNorm norm;
  int* status;
};

template <int DQK, int DV, bool E4M3, typename Offsets>
__global__ void __launch_bounds__(kNormThreads, 3)
append_norm_kernel(const __grid_constant__ AppendNormParams P, const __grid_constant__ Offsets off) {
  using L = HeadLanes<DQK>;
  __shared__ int pos[kMaxTokens];
  __shared__ int64_t places[2][kMaxTokens];  // byte offsets in the cache (-1: nowhere)
  __shared__ __align__(16) float weight[2][DQK];
  __shared__ __align__(16) float2 sc[kMaxAngles];
  const int row0 = blockIdx.x * P.tokens, tokens = min(P.tokens, P.T - row0);
  const int heads = P.Hq + P.cache.heads;
  const int group = threadIdx.x / L::kLanes, unit = threadIdx.x % L::kLanes;
  const bool lane_on = L::kUnits == L::kLanes || unit < L::kUnits;
  int ca = 0, cb = 8;
  unit_columns(P.rot, lane_on ? unit : 0, ca, cb);
  const bool turns = unit < (P.rot.dim >> 4);
  const int dt = L::kGroups / heads, dh = L::kGroups - dt * heads;
  int t = group / heads, head = group - t * heads, tl = t, hl = head;
  uint4 v[2][2];
  auto load = [&](uint4 (&d)[2]) {
    if (lane_on && tl < tokens) {
      const uint16_t* p = hl < P.Hq ? P.q + (row0 + tl) * P.q_row + hl * DQK
                                    : P.k + (row0 + tl) * P.k_row + (hl - P.Hq) * DQK;
      d[0] = *reinterpret_cast<const uint4*>(p + ca);
      d[1] = *reinterpret_cast<const uint4*>(p + cb);
    } else {
      d[0] = d[1] = make_uint4(0, 0, 0, 0);
    }
    tl += dt;
    hl += dh;
    if (hl >= heads) hl -= heads, ++tl;
  };
  load(v[0]);
  load(v[1]);

  // where the chunk's tokens go
  if (threadIdx.x < tokens) {
    const int r = row0 + threadIdx.x;
    int s, from_end;
    if constexpr (sizeof(Offsets) >= sizeof(RowOffsets)) {
      s = sequence_of(off.cu, P.B, r);
      from_end = off.cu[s + 1] - r;
    } else {
      s = r / P.per_seq;
      from_end = P.per_seq - (r - s * P.per_seq);
    }
    const int p = max(__ldg(P.cache.lens + s), 0) - from_end;
    int64_t ko = -1, vo = -1;
    if (p >= 0) {
      const int slot = div_page(P.cache, p);
      const int page = slot < P.cache.max_pages
                           ? __ldg(P.cache.table + s * P.cache.table_stride + slot)
                           : -1;
      if (page_in(P.cache, page)) {
        const int in = p - slot * P.cache.page_size;
        ko = token_at(P.cache.k, page, in);
        vo = token_at(P.cache.v, page, in);
      } else {
        atomicCAS(P.status, 0, kStatusBadPage);
      }
    }
    pos[threadIdx.x] = p;
    places[0][threadIdx.x] = ko;
    places[1][threadIdx.x] = vo;
  }
  for (int i = threadIdx.x; i < 2 * DQK; i += kNormThreads) {
    const float* w = i < DQK ? P.norm.q_weight : P.norm.k_weight;
    weight[i / DQK][i % DQK] = w != nullptr ? __ldg(w + i % DQK) : 1.f;
  }
  __syncthreads();
  if (P.rot.dim > 0) fill_angles(sc, pos, tokens, P.rot, false);
  __syncthreads();

  const int rounds = (tokens * heads + L::kGroups - 1) / L::kGroups;
  for (int i = 0; i < rounds; i += 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (i + j >= rounds) break;
      float f[16];
      unpack(v[j][0], f);
      unpack(v[j][1], f + 8);
      load(v[j]);
      bool there = lane_on && t < tokens;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
      ss = head_sum<L::kLanes>(ss);
      const float r = rsqrtf(ss * (1.f / DQK) + P.norm.eps);
      const bool key = head >= P.Hq;
      const float* w = weight[key];
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 q = *reinterpret_cast<const float4*>(w + (e < 8 ? ca + e : cb + e - 8));
        // (in norm_kernel's order: the cache holds the bits that attn_norm_rope gives)
        f[e] = f[e] * r * q.x, f[e + 1] = f[e + 1] * r * q.y;
        f[e + 2] = f[e + 2] * r * q.z, f[e + 3] = f[e + 3] * r * q.w;
      }
      there = there && pos[min(t, tokens - 1)] >= 0;
      if (there) {
        if (turns) turn_unit(sc, t, unit, P.rot, f);
        if (!key) {
          uint16_t* p = P.q_out + (row0 + t) * P.q_out_row + head * DQK;
          *reinterpret_cast<uint4*>(p + ca) = packed(f);
          *reinterpret_cast<uint4*>(p + cb) = packed(f + 8);
        } else if (places[0][t] >= 0) {
          const int h = head - P.Hq;
          char* p = P.cache.k.base + places[0][t] + h * P.cache.k.head;
          if constexpr (E4M3) {
            Scale s;
            if (P.cache.k.scale) s.set(__ldg(P.cache.k.scale + h));
            uint32_t b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = quantise2(f[2 * e], f[2 * e + 1], s);
            *reinterpret_cast<uint2*>(p + ca) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            *reinterpret_cast<uint2*>(p + cb) = make_uint2(b[4] | b[5] << 16, b[6] | b[7] << 16);
          } else {
            *reinterpret_cast<uint4*>(p + 2 * ca) = packed(f);
            *reinterpret_cast<uint4*>(p + 2 * cb) = packed(f + 8);
          }
        }
      }
      t += dt;
      head += dh;
      if (head >= heads) head -= heads, ++t;
    }
  }
  // values
  constexpr int kUnitsV = DV / 16;
  const int n = P.cache.heads * kUnitsV;
  for (int i = threadIdx.x; i < tokens * n; i += kNormThreads) {
    const int tv = i / n, h = (i - tv * n) / kUnitsV, u = i % kUnitsV;
    const int64_t o = places[1][tv];
    if (o < 0) continue;
    const uint16_t* src = P.v + (row0 + tv) * P.v_row + h * DV + u * 16;
    const uint4 a = *reinterpret_cast<const uint4*>(src);
    const uint4 b = *reinterpret_cast<const uint4*>(src + 8);
    char* p = P.cache.v.base + o + h * P.cache.v.head + u * (E4M3 ? 16 : 32);
    if constexpr (E4M3) {
      Scale s;
      if (P.cache.v.scale) s.set(__ldg(P.cache.v.scale + h));
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = quantise2(lo_of(w[e]), hi_of(w[e]), s);
      *reinterpret_cast<uint4*>(p) = make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16,
                                                q[4] | q[5] << 16, q[6] | q[7] << 16);
    } else {
      *reinterpret_cast<uint4*>(p) = a;
      *reinterpret_cast<uint4*>(p + 16) = b;
    }
  }
}

template <int D, bool GRAD>
cudaError_t norm_typed(const NormLaunch& L) {
  NormParams P;
  std::memset(&P, 0, sizeof(P));
  // Token rows of a chunk: about kNormRounds heads a group, as far as the angles' memory goes,
  // fewer where that left SMs without a block.
  int blocks = 0;
  for (int i = 0; i < 2; ++i) {
    const NormTensor& t = L.t[i];
    P.t[i] = t;
    P.tokens[i] = 1;
    if (t.rows == 0) continue;
    int tokens = std::max(1, kNormRounds * HeadLanes<D>::kGroups / t.H);
    tokens = std::min(tokens, most_tokens(L.rot.dim));
    while (tokens > 1 && cdiv(t.rows, tokens) < 4 * L.num_sms) tokens /= 2;
    P.tokens[i] = tokens;
    P.blocks[i] = cdiv(t.rows, tokens);
    if (GRAD) P.blocks[i] = std::min(P.blocks[i], kMaxNormBlocks);
    if (GRAD && t.dw != nullptr) P.t[i].dw = L.workspace + (int64_t)i * kMaxNormBlocks * D;
    blocks += P.blocks[i];
  }
  P.rot = L.rot;
  P.eps = L.eps;
  P.nseq = L.nseq;
  P.pos0 = L.pos0;
  if (blocks == 0) return cudaSuccess;
  if (L.cu[0] != nullptr) {
    PairOffsets off;
    std::memcpy(&off.q, L.cu[0], sizeof(RowOffsets));
    std::memcpy(&off.k, L.cu[1], sizeof(RowOffsets));
    norm_kernel<D, GRAD><<<blocks, kNormThreads, 0, L.stream>>>(P, off);
  } else {
    norm_kernel<D, GRAD><<<blocks, kNormThreads, 0, L.stream>>>(P, NoOffsets{});
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !GRAD || (L.t[0].dw == nullptr && L.t[1].dw == nullptr)) return e;
  NormSums S;
  for (int i = 0; i < 2; ++i) {
    S.rows[i] = P.t[i].dw;
    S.dw[i] = L.t[i].dw;
    S.blocks[i] = P.blocks[i];
  }
  S.d = D;
  // on its way while the main kernel runs; it waits for that one's end before it reads
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSumSlices, 2 * (D / 32));
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_sums_kernel, S);
}

template <int DQK, int DV, bool E4M3>
cudaError_t append_norm_typed(const AppendLaunch& L, AppendNormParams& P) {
  const int heads = L.Hq + L.cache.heads;
  int tokens = std::max(1, 8 * HeadLanes<DQK>::kGroups / heads);
  while (tokens > 1 && L.T / tokens < 4 * L.num_sms) tokens /= 2;
  P.tokens = std::min(tokens, most_tokens(P.rot.dim));
  const int blocks = cdiv(L.T, P.tokens);
  if (L.offsets != nullptr)
    append_norm_kernel<DQK, DV, E4M3><<<blocks, kNormThreads, 0, L.stream>>>(P, *L.offsets);
  else
    append_norm_kernel<DQK, DV, E4M3><<<blocks, kNormThreads, 0, L.stream>>>(P, NoOffsets{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormLaunch& L) {
  switch (L.d) {
    case 64: return norm_typed<64, false>(L);
    case 128: return norm_typed<128, false>(L);
    case 192: return norm_typed<192, false>(L);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_bwd(const NormLaunch& L) {
  switch (L.d) {
    case 64: return norm_typed<64, true>(L);
    case 128: return norm_typed<128, true>(L);
    case 192: return norm_typed<192, true>(L);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_append_norm(const AppendLaunch& L) {
  AppendNormParams P;
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
  P.norm = *L.norm;
  P.status = L.status;
  const bool e = L.cache.e4m3 != 0;
  if (L.dqk == 64)
    return e ? append_norm_typed<64, 64, true>(L, P) : append_norm_typed<64, 64, false>(L, P);
  if (L.dqk == 128)
    return e ? append_norm_typed<128, 128, true>(L, P) : append_norm_typed<128, 128, false>(L, P);
  if (L.dqk == 192)
    return e ? append_norm_typed<192, 128, true>(L, P) : append_norm_typed<192, 128, false>(L, P);
  return cudaErrorInvalidValue;
}

}  // namespace attn
