// mx_device.cuh -- packed rows (include/a2av_mx.h): their layout, and a block's
// way to codes and a scale and back.
#pragma once

#include "a2av_mx.h"
#include "moe_device.cuh"

namespace {

constexpr int kMxBlock = 32;  // values a scale

// Where the parts of a packed row lie.
struct MxRow {
  long long values, scales, bytes;  // bytes of the values, of the scales, of the row
};

__host__ __device__ __forceinline__ MxRow mx_row(long long features, int format) {
  MxRow r;
  r.scales = (features + kMxBlock - 1) / kMxBlock;
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
__device__ __forceinline__ float mx_inverse(unsigned s) { return __uint_as_float((254u - s) << 23); }

// 2^(s - 127), NaN for 255 (2^-127 has no exponent of its own in 32 bits).
__device__ __forceinline__ float mx_scale_value(unsigned s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255u ? 0x7fffffffu : s << 23);
}

// The largest of a value over the lanes that differ in the low kLanes - 1 bits.
template <int kLanes>
__device__ __forceinline__ unsigned lanes_max(unsigned x) {
  if constexpr (kLanes == 32) {
    return __reduce_max_sync(kAll, x);
  } else {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) x = max(x, __shfl_xor_sync(kAll, x, o));
    return x;
  }
}

__device__ __forceinline__ unsigned e4m3_pair(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ unsigned e2m1_pair(float lo, float hi) {
  unsigned short r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b16 %0, {b, b};\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r & 0xffu;
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

// The codes of N neighbouring values (already divided by their scale), the first
// lowest.
template <int kFormat, int N>
struct MxCodes {
  static constexpr int kBits = kFormat == A2AV_MXFP8 ? 8 : 4;
  static constexpr int kWords = N * kBits >= 32 ? N * kBits / 32 : 1;
  unsigned w[kWords];

  __device__ __forceinline__ void encode(const float (&f)[N]) {
    if constexpr (N == 1) {
      w[0] = kFormat == A2AV_MXFP8 ? e4m3_pair(f[0], 0.0f) & 0xffu : e2m1_pair(f[0], 0.0f) & 0xfu;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const unsigned p = kFormat == A2AV_MXFP8 ? e4m3_pair(f[2 * i], f[2 * i + 1])
                                                 : e2m1_pair(f[2 * i], f[2 * i + 1]);
        w[2 * i * kBits / 32] |= p << (2 * i * kBits % 32);
      }
    }
  }

  // To the values' place of a row, v being the number of these N in it.  With N = 1
  // (by a whole warp) two lanes share a byte of 4-bit codes.
  __device__ __forceinline__ void store(unsigned char* row, long long v) const {
    if constexpr (N == 1 && kFormat == A2AV_MXFP8) {
      row[v] = (unsigned char)w[0];
    } else if constexpr (N == 1) {
      const unsigned next = __shfl_down_sync(kAll, w[0], 1);
      if (v % 2 == 0) row[v / 2] = (unsigned char)(w[0] | next << 4);
    } else if constexpr (N * kBits == 64) {
      reinterpret_cast<uint2*>(row)[v] = make_uint2(w[0], w[1]);
    } else if constexpr (N * kBits == 32) {
      reinterpret_cast<unsigned*>(row)[v] = w[0];
    } else {
      static_assert(N * kBits == 16, "four 4-bit codes");
      reinterpret_cast<unsigned short*>(row)[v] = (unsigned short)w[0];
    }
  }
};

// N values of a row, the number v of such, to codes and (by the block's first
// lane) their scale: by whole warps, 32 / N neighbouring lanes a block; `write`
// says whether the lane's block is in the row (values past the row's end are 0).
template <int kFormat, int N>
__device__ __forceinline__ void mx_store(unsigned char* row, long long scales_at, long long v,
                                         float (&f)[N], bool write) {
  constexpr int kLanes = kMxBlock / N;
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  const unsigned s = mx_scale<kFormat>(lanes_max<kLanes>(top));
  const float by = mx_inverse(s);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = s == 255u ? 0.0f : f[i] * by;
  MxCodes<kFormat, N> c;
  c.encode(f);
  if (write) {  // (N = 1: the whole warp or none of it)
    c.store(row, v);
    if (threadIdx.x % kLanes == 0) row[scales_at + v / kLanes] = (unsigned char)s;
  }
}

}  // namespace
