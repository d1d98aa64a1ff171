// mx_device.cuh -- packed rows (include/a2av_mx.h): their layout, and a block's
// way to codes and a scale and back.
#pragma once

#include "a2av_mx.h"
#include "moe_device.cuh"

#include <type_traits>

namespace {

constexpr int kMxBlock = 32;  // values a scale

// Where the parts of a packed row lie.
struct MxRow {
  int values, scales, bytes;  // bytes of the values, of the scales, of the row
};

__host__ __device__ __forceinline__ MxRow mx_row(long long features, int format) {
  MxRow r;
  r.scales = (int)((features + kMxBlock - 1) / kMxBlock);
  r.values = r.scales * (format == A2AV_MXFP8 ? kMxBlock : kMxBlock / 2);
  r.bytes = (r.values + r.scales + 31) / 32 * 32;
  return r;
}

// The scale byte of a block whose largest magnitude has these bits (as integers
// magnitudes keep their order, NaN above infinity above the rest).  The largest
// code is 1.75 * 2^8 (e4m3), 1.5 * 2^2 (e2m1): a significand above 1.75, 1.5
// takes the next power of two, to which the addition carries.
template <int kFormat>
__device__ __forceinline__ unsigned mx_scale(unsigned bits) {
  constexpr unsigned kCarry = kFormat == A2AV_MXFP8 ? 0x1fffffu : 0x3fffffu;
  constexpr int kTop = kFormat == A2AV_MXFP8 ? 8 : 2;
  return bits >= 0x7f800000u ? 255u : (unsigned)max((int)((bits + kCarry) >> 23) - kTop, 0);
}

// 1 / scale (s < 255: at most 253), a power of two.
__device__ __forceinline__ float mx_inverse(unsigned s) { return __uint_as_float((254u - s) << 23); }  // (255: of no use)

// 2^(s - 127), NaN for 255 (2^-127 has no exponent of its own in 32 bits).
__device__ __forceinline__ float mx_scale_value(unsigned s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255u ? 0x7fffffffu : s << 23);
}

// The largest of a value over the lanes that differ in the low kLanes - 1 bits.
template <int kLanes>
__device__ __forceinline__ unsigned lanes_max(unsigned x) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x = max(x, __shfl_xor_sync(kAll, x, o));
  return x;
}

// Two codes (in the low bits) as the values they stand for.
__device__ __forceinline__ float2 e4m3_values(unsigned pair) {
  unsigned r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)pair));
  return unpack2(r, __half());
}

__device__ __forceinline__ float2 e2m1_values(unsigned pair) {
  unsigned r;
  asm("{\n\t.reg .b8 b, z;\n\t"
      "mov.b16 {b, z}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(r)
      : "h"((unsigned short)pair));
  return unpack2(r, __half());
}

// Values are held in pairs: products of pairs are one instruction on this architecture.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return r;
}
__device__ __forceinline__ float2 minus(float2 x) { return make_float2(-x.x, -x.y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// Value i of some pairs.
template <int M>
__device__ __forceinline__ float value_of(const float2 (&f)[M], int i) { return i % 2 == 0 ? f[i / 2].x : f[i / 2].y; }

// A vector of 16 bytes, N elements of a row, between memory's words and pairs.
template <typename T>
struct Pairs {
  static constexpr int N = 16 / sizeof(T);
  using Raw = typename Piece<T, N>::Raw;
  static __device__ __forceinline__ void unpack(const Raw& r, float2 (&f)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (sizeof(T) == 4)
        f[i] = make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
      else if constexpr (__is_same(T, __nv_bfloat16))
        f[i] = make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
      else
        f[i] = unpack2(r.w[i], T());
    }
  }
  static __device__ __forceinline__ Raw pack(const float2 (&f)[N / 2]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (sizeof(T) == 4) {
        r.w[2 * i] = __float_as_uint(f[i].x);
        r.w[2 * i + 1] = __float_as_uint(f[i].y);
      } else {
        r.w[i] = pack2(f[i].x, f[i].y, T());
      }
    }
    return r;
  }
};

// Rows that take no vectors (of any alignment).  A warp moves what are 32 vectors
// elsewhere element by element, neighbouring lanes on neighbouring elements: lane l has the
// elements 32 k + l of them.  That serves where a value does not depend on its
// neighbours; for codes (whose blocks would have an element a lane: two to three times as
// long) they go through 512 bytes of the warp's own to the lanes that have them as vectors.
template <typename T>
struct Loose {
  static constexpr int N = 16 / sizeof(T);
  using Raw = typename Pairs<T>::Raw;
  using Bits = std::conditional_t<sizeof(T) == 4, unsigned, unsigned short>;

  static __device__ __forceinline__ int element(int first, int k) { return first * N + 32 * k + threadIdx.x % 32; }

  // Of the 32 vectors from `first` on of a row of n elements, U times, `step` vectors further
  // each: the lane's elements, zeros past the row.
  template <int U>
  static __device__ __forceinline__ void load(Raw (&to)[U], const void* row, int first, int step, int n) {
    Bits e[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = element(first + u * step, k);
        e[u][k] = i < n ? static_cast<const Bits*>(row)[i] : Bits(0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4)
          to[u].w[j] = e[u][j];
        else
          to[u].w[j] = e[u][2 * j] | (unsigned)e[u][2 * j + 1] << 16;
      }
  }
  static __device__ __forceinline__ Bits of(const Raw& r, int k) {
    if constexpr (sizeof(T) == 4)
      return r.w[k];
    else
      return (Bits)(r.w[k / 2] >> (k % 2 * 16));
  }
  template <int U>
  static __device__ __forceinline__ void store(void* row, const Raw (&from)[U], int first, int step, int n) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = element(first + u * step, k);
        if (i < n) static_cast<Bits*>(row)[i] = of(from[u], k);
      }
  }

  // From the lanes that have the elements to those that have the vectors, and back.
  template <int U>
  static __device__ __forceinline__ void spread(Raw (&x)[U], uint4 (*place)[32]) {
    const int lane = threadIdx.x % 32;
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) reinterpret_cast<Bits*>(place[u])[32 * k + lane] = of(x[u], k);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u) reinterpret_cast<uint4&>(x[u]) = place[u][lane];
  }
  template <int U>
  static __device__ __forceinline__ void gather(Raw (&x)[U], uint4 (*place)[32]) {
    const int lane = threadIdx.x % 32;
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u) place[u][lane] = reinterpret_cast<const uint4&>(x[u]);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4)
          x[u].w[j] = reinterpret_cast<const Bits*>(place[u])[32 * j + lane];
        else
          x[u].w[j] = reinterpret_cast<const Bits*>(place[u])[64 * j + lane] |
                      (unsigned)reinterpret_cast<const Bits*>(place[u])[64 * j + 32 + lane] << 16;
      }
  }
};

// The largest magnitude of some values, NaN where one is NaN.
template <int M>
__device__ __forceinline__ float largest(const float2 (&f)[M]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < M; ++i)
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(f[i].x)), "f"(fabsf(f[i].y)));
  return m;
}

// The codes of N neighbouring values (already divided by their scale), the first
// lowest.
template <int kFormat, int N>
struct MxCodes {
  static constexpr int kBits = kFormat == A2AV_MXFP8 ? 8 : 4;
  static constexpr int kWords = N * kBits >= 32 ? N * kBits / 32 : 1;
  unsigned w[kWords];

  __device__ __forceinline__ void encode(const float2 (&f)[N / 2]) {
    if constexpr (kFormat == A2AV_MXFP8) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        asm("{\n\t.reg .b16 l, h;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(w[i])
            : "f"(f[2 * i].x), "f"(f[2 * i].y), "f"(f[2 * i + 1].x), "f"(f[2 * i + 1].y));
    } else {
      static_assert(N == 4 || N == 8, "vectors of 16 bytes");
      unsigned part[N / 4];  // (four .b8 in one mov.b32 came out wrong)
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        unsigned short r;
        asm("{\n\t.reg .b8 a, b;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "mov.b16 %0, {a, b};\n\t}"
            : "=h"(r)
            : "f"(f[2 * i].x), "f"(f[2 * i].y), "f"(f[2 * i + 1].x), "f"(f[2 * i + 1].y));
        part[i] = r;
      }
      w[0] = N == 8 ? part[0] | part[N / 4 - 1] << 16 : part[0];
    }
  }

  // To the values' place of a row, v being the number of these N in it.
  __device__ __forceinline__ void store(unsigned char* row, int v) const {
    if constexpr (N * kBits == 64) {
      reinterpret_cast<uint2*>(row)[v] = make_uint2(w[0], w[1]);
    } else if constexpr (N * kBits == 32) {
      reinterpret_cast<unsigned*>(row)[v] = w[0];
    } else {
      static_assert(N * kBits == 16, "four 4-bit codes");
      reinterpret_cast<unsigned short*>(row)[v] = (unsigned short)w[0];
    }
  }
};

// Values that are what they are: none lies above its bits.
struct Exact {
  __device__ __forceinline__ bool operator()(unsigned) const { return false; }
};

// N values of a row, the number v of such, to codes and (by the block's first
// lane) their scale: by whole warps, 32 / N neighbouring lanes a block; `top` has
// the bits of the lane's largest magnitude, and `write` says whether the lane's block
// is in the row (values past the row's end are 0).  above(bits): whether one of the lane's
// values of that magnitude was rounded down to it, asked where it is the largest that a scale
// takes (one block in some 10^7 would otherwise get the scale below).
template <int kFormat, int N, typename Above>
__device__ __forceinline__ void mx_store(unsigned char* row, int scales_at, int v, float2 (&f)[N / 2],
                                         unsigned top, bool write, Above above) {
  constexpr int kLanes = kMxBlock / N;
  const unsigned bits = lanes_max<kLanes>(top);
  unsigned s = mx_scale<kFormat>(bits);
  if constexpr (!std::is_same_v<Above, Exact>) {
    const bool full = (bits & 0x7fffffu) == (kFormat == A2AV_MXFP8 ? 0x600000u : 0x400000u);
    if (__any_sync(kAll, full)) s += lanes_max<kLanes>(full && s > 0 && s < 255u && above(bits) ? 1u : 0u);
  }
  const float2 by = both(mx_inverse(s));
#pragma unroll
  for (int i = 0; i < N / 2; ++i) f[i] = mul2(f[i], by);
  MxCodes<kFormat, N> c;
  c.encode(f);
#pragma unroll
  for (int i = 0; i < c.kWords; ++i) c.w[i] = s == 255u ? 0u : c.w[i];
  if (write) {
    c.store(row, v);
    if (threadIdx.x % kLanes == 0) row[scales_at + v / kLanes] = (unsigned char)s;
  }
}

}  // namespace
