// experts_mx.cu -- the experts' products on packed rows and weights
// (a2av_expert_matmul_mx); the interface is in include/a2av_mx.h.
#include "experts.cuh"
#include "mx_device.cuh"

namespace {

constexpr int kTile = 64, kPlainThreads = 256;

// Eight values of a packed row, 8 i .. 8 i + 7.
template <int kFormat>
__device__ __forceinline__ void eight(const unsigned char* row, const MxRow& at, long long i, float (&f)[8]) {
  const float by = mx_scale_value(row[at.values + i / 4]);
  unsigned w[2];
  if constexpr (kFormat == A2AV_MXFP8) {
    const uint2 c = reinterpret_cast<const uint2*>(row)[i];
    w[0] = c.x;
    w[1] = c.y;
  } else {
    w[0] = reinterpret_cast<const unsigned*>(row)[i];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = kFormat == A2AV_MXFP8 ? e4m3_values(w[j / 2] >> (j % 2 * 16)) : e2m1_values(w[0] >> (8 * j));
    f[2 * j] = by * p.x;
    f[2 * j + 1] = by * p.y;
  }
}

// 64 x 64 tiles of the result, a block of the contraction in shared memory at a
// time, 4 x 4 results a thread.
template <typename T, int kFormat, bool kGated>
__global__ void __launch_bounds__(kPlainThreads)
    expert_mx_plain_kernel(const __grid_constant__ ExpertParams P, MxRow at) {
  chain();
  __shared__ GroupTable g;
  __shared__ GroupTiles tiles;
  __shared__ float xs[kMxBlock][kTile + 1], ws[kGated ? 2 : 1][kMxBlock][kTile + 1];
  const long long F = P.N;
  const int nf = (int)((F + kTile - 1) / kTile);
  if (!build_groups(P.g, g, &tiles, kTile, nf)) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (long long tile = blockIdx.x; tile < tiles.first[g.entries]; tile += gridDim.x) {
    const GroupTile gt = find_tile(P.g, g, tiles, tile, kTile, nf);
    const long long f0 = gt.local % nf * kTile, m0 = gt.local / nf * kTile;
    const unsigned char* x = static_cast<const unsigned char*>(P.x[gt.p]) + (gt.first + m0) * at.bytes;
    const unsigned char* w = static_cast<const unsigned char*>(P.w[gt.p]) + (long long)gt.e * P.Z * at.bytes;
    const int rows = (int)min((long long)kTile, gt.rows - m0);
    float acc[kGated ? 2 : 1][4][4] = {};
    const int m = tid / 4, part = tid % 4;
    for (long long b = 0; b < at.scales; ++b) {
      float f[8];
      if (m < rows) eight<kFormat>(x + m * at.bytes, at, 4 * b + part, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) xs[8 * part + i][m] = m < rows ? f[i] : 0.0f;
#pragma unroll
      for (int h = 0; h < (kGated ? 2 : 1); ++h) {
        if (f0 + m < F) eight<kFormat>(w + (h * F + f0 + m) * at.bytes, at, 4 * b + part, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ws[h][8 * part + i][m] = f0 + m < F ? f[i] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kMxBlock; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < (kGated ? 2 : 1); ++h)
              acc[h][i][j] += xs[c][ty + 16 * i] * ws[h][c][tx + 16 * j];
      __syncthreads();
    }
    const T* bias = P.bias[gt.p] != nullptr
                        ? static_cast<const T*>(P.bias[gt.p]) + gt.e * P.Z : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ty + 16 * i >= rows) continue;
      const long long row = gt.first + m0 + ty + 16 * i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long f = f0 + tx + 16 * j;
        if (f >= F) continue;
        float y = act_fn(P.act, acc[0][i][j] + (bias != nullptr ? to_float(bias[f]) : 0.0f));
        if (kGated) y *= acc[kGated ? 1 : 0][i][j] + (bias != nullptr ? to_float(bias[F + f]) : 0.0f);
        if (P.residual[gt.p] != nullptr)
          y += to_float(static_cast<const T*>(P.residual[gt.p])[row * F + f]);
        static_cast<T*>(P.out[gt.p])[row * F + f] = from_float<T>(y);
      }
    }
  }
}

template <typename T, int kFormat>
cudaError_t launch_plain(a2av_handle* h, const ExpertParams& P, const MxRow& at, cudaStream_t s) {
  return launch_chained(P.gated ? expert_mx_plain_kernel<T, kFormat, true> : expert_mx_plain_kernel<T, kFormat, false>,
                        dim3(4 * h->sms), kPlainThreads, 0, s, h->pdl, P, at);
}

template <typename T>
cudaError_t launch_mx(a2av_handle* h, const ExpertParams& P, int format, cudaStream_t s) {
  const MxRow at = mx_row(P.D, format);
  return format == A2AV_MXFP8 ? launch_plain<T, A2AV_MXFP8>(h, P, at, s)
                              : launch_plain<T, A2AV_MXFP4>(h, P, at, s);
}

}  // namespace

extern "C" int a2av_expert_matmul_mx(a2av_handle* h, const a2av_expert_t* shape, int format,
                                     const void* const* rows_ptrs, const int64_t* rows_per_peer,
                                     const int64_t* counts_dev, const void* const* weight_ptrs,
                                     const void* const* bias_ptrs, const void* const* residual_ptrs,
                                     void* const* out_ptrs, void* stream) {
  if (rows_ptrs == nullptr || weight_ptrs == nullptr || out_ptrs == nullptr ||
      (format != A2AV_MXFP8 && format != A2AV_MXFP4))
    return A2AV_ERR_INVALID_ARG;
  ExpertParams P;
  const int rc = a2av_expert_params(h, shape, rows_per_peer, counts_dev, &P);
  if (rc != A2AV_OK) return rc;
  const int W = h->W, size = dtype_bytes(shape->dtype);
  if (!take(P.x, rows_ptrs, W, rows_per_peer, 16) || !take(P.w, weight_ptrs, W, nullptr, 16) ||
      !take(P.bias, bias_ptrs, W, nullptr, size) ||
      !take(P.residual, residual_ptrs, W, rows_per_peer, size) ||
      !take(P.out, out_ptrs, W, rows_per_peer, size))
    return A2AV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = shape->dtype == A2AV_BF16 ? launch_mx<__nv_bfloat16>(h, P, format, s)
                                                  : launch_mx<__half>(h, P, format, s);
  return e != cudaSuccess || cudaGetLastError() != cudaSuccess ? A2AV_ERR_CUDA : A2AV_OK;
}
