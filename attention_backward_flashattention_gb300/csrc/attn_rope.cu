// attn_rope.cu — position rotation of queries and keys, and the append of new
// tokens to a paged cache with that rotation applied on the way.
//
// Mathematics.  Pair i of a head at position p turns by p * w_i.  The rate w_i
// is stored as a fraction of a turn times 2^64, so p * rate modulo 2^64 is the
// angle modulo one turn with no loss at far positions (in fp32 the product
// p * w_i at p = 10^6 is off by 0.03 rad).  The nearest quarter turn is taken off
// in whole numbers, and what is left, to 2^-33 of a half turn, goes to sincospif
// as an argument in [-1/4, 1/4), rounded to 2^-24 of itself: next to a zero of the
// sine or the cosine the small one of the two has as many right bits as the large
// one.  Negative positions (the inverse rotation negates p) work by two's
// complement.  The rotation is two products and a sum in fp32, rounded to the
// output's type once.
//
// Bound: memory.  Each element is read once and written once (2 + 2 bytes; 2 + 1
// into an e4m3 cache), against three flops.  What is left to do is to keep the
// index work and the angles off the path:
//   * a thread moves units of 16 columns, two 16-byte loads and stores each, and
//     keeps its unit (head, columns, destination) from token to token, so the
//     divisions that find it are paid once;
//   * a block takes several token rows where there are many, computes each
//     (position, pair) angle once for all heads into shared memory, and has its
//     next loads on their way meanwhile.
// Measured on a GB300 (a plain copy there: 6.78 TB/s): rotation of 537 MB (B 1, T
// 32768, 16 + 16 heads of 128) 81.6 us, 6.58 TB/s; of 458 MB of ragged (192, 64 of it
// turned) heads 70.2 us, 6.52 TB/s; append of 16.8 K prompt tokens, 32 query and 8 key
// heads of 128, into e4m3: 378 MB in 63 us, 6.0 TB/s; of 10.2 K tokens, 16 + 16
// (192, 128) heads, into bf16: 336 MB in 56.5 us, 5.95 TB/s.
#include <algorithm>
#include <cstring>

#include "attn_rotate.cuh"

namespace attn {

__device__ int g_cache_status = 0;

int* cache_status_ptr() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_cache_status) != cudaSuccess) return nullptr;
  return static_cast<int*>(p);
}

namespace {


// Rotation: many small blocks, their registers held down to five on an SM.
constexpr int kRopeThreads = 256, kRopeBlocks = 5;
constexpr int kRounds = 4;            // tokens a thread walks over, where there are many

// Append: as many threads as an SM has room for at 64 registers, in blocks of about
// kBlockThreads or of one token's units.  Units of a thread on their way (kDepth), and
// its rows of a chunk (kRounds), by the cache's type: prompts of 10 to 26 K tokens, in us,
//                       2 and 2   2 and 4   3 and 4   4 and 4
//   bf16, (192, 128)        57        59        62        62
//   bf16, 128               68        68        72        76
//   bf16, 64                43        43        44        44
//   e4m3, (192, 128)        55        55        55        57
//   e4m3, 128               68        65        63        64
//   e4m3, 64                51        45        45        47
// (2 and 1: 49 to 89.)  More in flight costs a memory that reads and writes at once.
constexpr int kAppendThreads = 1024, kBlockThreads = 256;
template <bool E4M3>
struct Append {
  static constexpr int kDepth = E4M3 ? 3 : 2, kRounds = E4M3 ? 4 : 2;
};

// Shape of the rotation's blocks over `rows` token rows of `units` units each: `side`
// token rows side by side (about 256 threads, or one row), and up to kRounds of
// them one after the other as long as every SM has some blocks (4 and 8 measure
// alike, 16 loses 4 to 10 %: a block's angles come before its first store).
struct BlockShape {
  int threads, side, tokens, blocks;
};
BlockShape block_shape(int rows, int units, int dim, int sms) {
  BlockShape s;
  const int most = most_tokens(dim);
  s.side = std::min(std::max(1, kRopeThreads / units), most);
  s.threads = std::min(kRopeThreads, cdiv(s.side * units, 32) * 32);
  const int rounds = std::max(1, std::min(kRounds, rows / (s.side * sms * 8)));
  s.tokens = std::min(s.side * rounds, most);
  s.blocks = cdiv(rows, s.tokens);
  return s;
}

// The eight pairs of unit u of token t, from and to the words of its two chunks (w[0 .. 3]
// and w[4 .. 7]); out(x, y): the word for two neighbours.
template <bool PAIRS, typename Out>
__device__ __forceinline__ void turn_words(const float2* sc, int t, int u, int units,
                                           uint32_t (&w)[8], Out out) {
  const float4* at = reinterpret_cast<const float4*>(sc) + t * 4 * units + u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 c = at[k * units];  // cos, sin of pairs 2k and 2k + 1
    const int i = PAIRS ? 2 * k : k, j = PAIRS ? 2 * k + 1 : k + 4;
    const float a0 = lo_of(w[i]), b0 = PAIRS ? hi_of(w[i]) : lo_of(w[j]);
    const float a1 = PAIRS ? lo_of(w[j]) : hi_of(w[i]), b1 = hi_of(w[j]);
    const float c0 = a0 * c.x - b0 * c.y, d0 = a0 * c.y + b0 * c.x;
    const float c1 = a1 * c.z - b1 * c.w, d1 = a1 * c.w + b1 * c.z;
    w[i] = out(c0, PAIRS ? d0 : c1);
    w[j] = out(PAIRS ? c1 : d0, d1);
  }
}
template <typename Out>
__device__ __forceinline__ void turn_words(const float2* sc, int t, int u, const Rotation& rot,
                                           uint32_t (&w)[8], Out out) {
  if (rot.pairs)
    turn_words<true>(sc, t, u, rot.dim >> 4, w, out);
  else
    turn_words<false>(sc, t, u, rot.dim >> 4, w, out);
}

struct RopeParams {
  RopeTensor t[2];
  Rotation rot;
  int inverse, nseq, pos0;
};

// ----------------------------------------------------------------------------
// attn_rope: blocks 0 .. t[0].blocks - 1 take the queries, the others the keys.
// ----------------------------------------------------------------------------
template <int D, typename Offsets>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
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
        uint32_t v[8] = {w[j].a.x, w[j].a.y, w[j].a.z, w[j].a.w,
                         w[j].b.x, w[j].b.y, w[j].b.z, w[j].b.w};
        turn_words(sc, tj, unit, P.rot, v, [](float a, float b) { return pack_bf16(a, b); });
        w[j].a = make_uint4(v[0], v[1], v[2], v[3]);
        w[j].b = make_uint4(v[4], v[5], v[6], v[7]);
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
// attn_cache_append: a grid that fits the SMs once walks over the token rows in
// chunks.  A thread keeps its unit and takes the rows of it one after the other
// through a ring in shared memory that only it uses, filled by asynchronous copies
// (loads into registers: 78 us into e4m3 where this takes 63, with a third fewer
// warps).  Where the next chunks go, and the next one's angles, is found meanwhile.
// ----------------------------------------------------------------------------
struct AppendParams {
  CacheView cache;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_row, v_row, q_row, q_out_row;
  int B, T, Hq, per_seq;
  int side, tokens;  // token rows side by side, of a chunk
  int parts;         // blocks that share the units of a token
  Rotation rot;
  int* status;
};

template <int DQK, int DV, bool E4M3, typename Offsets>
__global__ void __launch_bounds__(kAppendThreads, 1)
append_kernel(const __grid_constant__ AppendParams P, const __grid_constant__ Offsets off) {
  // of the chunks i, i + 1 and i + 2 of this block: positions, and the byte offsets of the
  // cache slots (-1: none)
  __shared__ int pos[3][kMaxTokens];
  __shared__ int64_t places[2][3][kMaxTokens];  // of keys, of values
  __shared__ int seq[kMaxTokens], from_end[kMaxTokens];  // (each thread's own)
  // the ring: kDepth units of each thread, as [step][chunk a, b][thread]; then the angles
  // of two chunks
  constexpr int kDepth = Append<E4M3>::kDepth;
  extern __shared__ __align__(16) uint4 ring[];
  float2* const sc0 = reinterpret_cast<float2*>(ring + kDepth * 2 * blockDim.x);
  const int sc_size = P.tokens * (P.rot.dim >> 1);
  constexpr int kUnits = DQK / 16, kUnitsV = DV / 16;
  const int n_q = P.Hq * kUnits, n_k = P.cache.heads * kUnits, n_v = P.cache.heads * kUnitsV;
  const int part = blockIdx.x % P.parts;
  const int all = n_q + n_k + n_v, share = (all + P.parts - 1) / P.parts;
  const int first = part * share, units = min(share, all - first);  // of a token, here
  const int side = P.side, tid = threadIdx.x;

  // this block's chunks of token rows: each gridDim.x / parts chunks behind the last
  int row0 = blockIdx.x / P.parts * P.tokens;
  const int stride = gridDim.x / P.parts * P.tokens;

  // Where a chunk's tokens go takes two loads, one after the other: a thread per token
  // has the first on its way for the chunk after next but one, the second for the one
  // before that.
  int len = 0, page = -1;
  auto find = [&](int at) {  // the row's sequence, its distance from that one's end, its length
    const int r = at + tid;
    if (tid >= P.tokens || r >= P.T) return;
    int s;
    if constexpr (sizeof(Offsets) >= sizeof(RowOffsets)) {
      s = sequence_of(off.cu, P.B, r);
      from_end[tid] = off.cu[s + 1] - r;
    } else {
      s = r / P.per_seq;
      from_end[tid] = P.per_seq - (r - s * P.per_seq);
    }
    seq[tid] = s;
    len = __ldg(P.cache.lens + s);
  };
  auto look_up = [&](int at, int buf) {  // the position and the page of the token found
    if (tid >= P.tokens) return;
    page = -1;
    const int p = at + tid < P.T ? max(len, 0) - from_end[tid] : -1;
    pos[buf][tid] = p;
    const int slot = div_page(P.cache, max(p, 0));
    if (p >= 0 && slot < P.cache.max_pages)
      page = __ldg(P.cache.table + seq[tid] * P.cache.table_stride + slot);
  };
  auto put_down = [&](int buf) {
    if (tid >= P.tokens) return;
    const int p = pos[buf][tid];
    int64_t ko = -1, vo = -1;
    if (p >= 0) {
      if (page_in(P.cache, page)) {
        const int in = p - div_page(P.cache, p) * P.cache.page_size;
        ko = token_at(P.cache.k, page, in);
        vo = token_at(P.cache.v, page, in);
      } else {
        atomicCAS(P.status, 0, kStatusBadPage);
      }
    }
    places[0][buf][tid] = ko;
    places[1][buf][tid] = vo;
  };

  // this thread's unit: where it is read, where it goes, whether it turns
  const int t0 = tid / units;
  const bool busy = t0 < side;
  int unit = 0, apart = 8;  // columns from its first chunk of eight to its second
  bool turns = false;
  int kind = 0;             // query, key, value
  const uint16_t* x = P.k;
  int64_t x_row = 0;
  char* y = nullptr;        // q_out or one side of the cache
  Scale scale;
  if (busy) {
    int rem = first + tid - t0 * units;
    if (rem < n_q + n_k) {
      const bool key = rem >= n_q;
      if (key) rem -= n_q;
      const int head = rem / kUnits;
      unit = rem - head * kUnits;
      turns = unit < (P.rot.dim >> 4);
      int ca, cb;
      unit_columns(P.rot, unit, ca, cb);
      apart = cb - ca;
      x_row = key ? P.k_row : P.q_row;
      x = (key ? P.k : P.q) + head * DQK + ca;
      if (key) {
        y = P.cache.k.base + head * P.cache.k.head + ca * (E4M3 ? 1 : 2);
        kind = 1;
        if (E4M3 && P.cache.k.scale) scale.set(__ldg(P.cache.k.scale + head));
      } else {
        y = reinterpret_cast<char*>(P.q_out + head * DQK + ca);
      }
    } else {
      rem -= n_q + n_k;
      const int head = rem / kUnitsV;
      unit = rem - head * kUnitsV;
      x_row = P.v_row;
      x = P.v + head * DV + unit * 16;
      y = P.cache.v.base + head * P.cache.v.head + unit * (E4M3 ? 16 : 32);
      kind = 2;
      if (E4M3 && P.cache.v.scale) scale.set(__ldg(P.cache.v.scale + head));
    }
  }

  // Rows of this thread, one after the other through its chunks, on their way to the ring.
  int load_row0 = row0, load_t = t0;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring + tid);
  auto load = [&](int step) {
    if (busy && load_row0 + load_t < P.T) {
      const uint16_t* p = x + (load_row0 + load_t) * x_row;
      const uint32_t at = mine + step * 32 * blockDim.x;
      // (through L1: the two chunks may be the halves of one sector)
      cp_async16_l1(at, p);
      cp_async16_l1(at + 16 * blockDim.x, p + apart);
    }
    cp_commit();
    load_t += side;
    if (load_t >= P.tokens) load_t = t0, load_row0 = min(load_row0 + stride, P.T);
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(i);
  int step = 0;

  find(row0);
  look_up(row0, 0);
  find(row0 + stride);
  put_down(0);
  look_up(row0 + stride, 1);
  find(row0 + 2 * stride);
  put_down(1);
  __syncthreads();
  fill_angles(sc0, pos[0], min(P.tokens, P.T - row0), P.rot, false);
  for (int buf = 0, odd = 0; row0 < P.T; row0 += stride, odd ^= 1) {
    const int next = buf == 2 ? 0 : buf + 1, after = next == 2 ? 0 : next + 1;
    __syncthreads();
    look_up(row0 + 2 * stride, after);
    find(row0 + 3 * stride);
    const int next0 = row0 + stride;
    if (next0 < P.T)
      fill_angles(sc0 + (odd ^ 1) * sc_size, pos[next], min(P.tokens, P.T - next0), P.rot,
                  false);
    const int tokens = busy ? min(P.tokens, P.T - row0) : 0;
    for (int t = t0; t < tokens; t += side) {
      cp_wait<kDepth - 1>();
      const uint32_t at = mine + step * 32 * blockDim.x;
      const uint4 wa = lds128(at), wb = lds128(at + 16 * blockDim.x);
      bool there = pos[buf][t] >= 0;
      char* row = y;
      if (kind != 0) {
        const int64_t o = places[kind - 1][buf][t];
        there = there && o >= 0;
        row += o;
      } else {
        row += (row0 + t) * P.q_out_row * 2;
      }
      if (there) {
        uint32_t w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
        const float2* angles = sc0 + odd * sc_size;
        if (E4M3 && kind != 0) {
          auto small = [&](float a, float b) { return quantise2(a, b, scale); };
          if (turns) {
            turn_words(angles, t, unit, P.rot, w, small);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = small(lo_of(w[i]), hi_of(w[i]));
          }
          *reinterpret_cast<uint2*>(row) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
          *reinterpret_cast<uint2*>(row + apart) = make_uint2(w[4] | w[5] << 16, w[6] | w[7] << 16);
        } else {
          if (turns)
            turn_words(angles, t, unit, P.rot, w, [](float a, float b) { return pack_bf16(a, b); });
          *reinterpret_cast<uint4*>(row) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(row + apart * 2) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      load(step);
      step = step + 1 == kDepth ? 0 : step + 1;
    }
    put_down(after);
    buf = next;
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
cudaError_t append_typed(const AppendLaunch& L, AppendParams& P) {
  constexpr int kDepth = Append<E4M3>::kDepth;
  const int all = (L.Hq + L.cache.heads) * (DQK / 16) + L.cache.heads * (DV / 16);
  P.parts = cdiv(all, kAppendThreads);
  const int units = cdiv(all, P.parts), most = most_tokens(P.rot.dim);
  P.side = std::min(std::max(1, kBlockThreads / units), most);
  const int threads = cdiv(P.side * units, 32) * 32;
  const int blocks = std::max(1, L.num_sms * (kAppendThreads / threads) / P.parts);
  int rounds = 1;  // (more of them as long as each block has two chunks)
  while (rounds < Append<E4M3>::kRounds && 2 * rounds * P.side <= most &&
         L.T >= (int64_t)blocks * 2 * rounds * P.side * 2)
    rounds *= 2;
  P.tokens = P.side * rounds;
  const int walkers = std::min(cdiv(L.T, P.tokens), blocks);
  const int smem = kDepth * 32 * threads + 2 * P.tokens * (P.rot.dim / 2) * (int)sizeof(float2);
  constexpr int most_smem = kDepth * 32 * kAppendThreads + 2 * kMaxAngles * (int)sizeof(float2);
  auto launch = [&](auto* kernel, const auto& off) {
    if (smem > 40 * 1024) {  // (48 KB, the static part among them, need no leave)
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
      if (e != cudaSuccess) return e;
    }
    kernel<<<walkers * P.parts, threads, smem, L.stream>>>(P, off);
    return cudaGetLastError();
  };
  if (L.offsets != nullptr) return launch(append_kernel<DQK, DV, E4M3, RowOffsets>, *L.offsets);
  return launch(append_kernel<DQK, DV, E4M3, NoOffsets>, NoOffsets{});
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L) {
  RopeParams P;
  std::memset(&P, 0, sizeof(P));
  int blocks = 0, threads = 0;
  for (int i = 0; i < 2; ++i) {
    P.t[i] = L.t[i];
    if (P.t[i].rows == 0) continue;
    const BlockShape s = block_shape(P.t[i].rows, P.t[i].H * (L.d / 16), L.rot.dim, L.num_sms);
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
  if (L.dqk == 64)
    return e ? append_typed<64, 64, true>(L, P) : append_typed<64, 64, false>(L, P);
  if (L.dqk == 128)
    return e ? append_typed<128, 128, true>(L, P) : append_typed<128, 128, false>(L, P);
  if (L.dqk == 192)
    return e ? append_typed<192, 128, true>(L, P) : append_typed<192, 128, false>(L, P);
  return cudaErrorInvalidValue;
}

}  // namespace attn
