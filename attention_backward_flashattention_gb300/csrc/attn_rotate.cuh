// attn_rotate.cuh — what the kernels that turn heads to their positions share (attn_rope.cu,
// attn_norm.cu): units of sixteen columns, angles, sequences of rows, rounding to e4m3.
#pragma once

#include <algorithm>

#include "attn_paged.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kMaxTokens = 32;        // token rows of a block (of a chunk) at most
constexpr int kMaxAngles = 2048;      // (token, pair) angles of these at most

int most_tokens(int dim) {
  return dim > 0 ? std::min(kMaxTokens, kMaxAngles / (dim / 2)) : kMaxTokens;
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

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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
    // turn = quarter * 2^62 + rest, -2^61 <= rest < 2^61: bits 30 .. 61 are rest / 2^30
    const uint32_t quarter = ((uint32_t)(turn >> 61) + 1) >> 1;
    const float rest = (float)(int)(uint32_t)(turn >> 30);
    float s, c;
    sincospif(rest * 0x1p-33f, &s, &c);
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    sc[((t * 4 + ((pair & 7) >> 1)) * units + (pair >> 3)) * 2 + (pair & 1)] =
        quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
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

// Two values as e4m3 of x / scale, saturated.
__device__ __forceinline__ uint32_t quantise2(float x, float y, const Scale& scale) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(r)
      : "f"(scale.divide(y)), "f"(scale.divide(x)));
  return r;
}

}  // namespace
}  // namespace attn
