// experts.cu -- one product per expert over the rows a dispatch delivered
// (a2av_expert_matmul) and its gradients; the interface is in
// include/a2av_moe.h.
#include "experts.cuh"

namespace {

// ------------------------------------------------- products by plain FMAs --
// For shapes and buffers that the tensor-core kernels' copies cannot take
// (rows that are not multiples of 16 bytes, or not aligned to them).  64 x 64
// tiles of the result, 16 of the contraction in shared memory at a time, 4 x 4
// results a thread.
constexpr int kTile = 64, kDepth = 16, kPlainThreads = 256;

// out rows x features: sum over c of x[row][c] * w(feature, c), where
// w(f, c) is at w[f * wf + c * wc] of the expert.  kGated: features f and
// f + N together.
template <typename T, bool kGated>
__global__ void __launch_bounds__(kPlainThreads)
    expert_plain_kernel(const __grid_constant__ ExpertParams P, long long C, long long F,
                        long long wf, long long wc) {
  chain();
  __shared__ GroupTable g;
  __shared__ GroupTiles tiles;
  __shared__ float xs[kDepth][kTile + 1], ws[kGated ? 2 : 1][kDepth][kTile + 1];
  const int nf = (int)((F + kTile - 1) / kTile);
  if (!build_groups(P.g, g, &tiles, kTile, nf)) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (long long tile = blockIdx.x; tile < tiles.first[g.entries]; tile += gridDim.x) {
    const GroupTile gt = find_tile(P.g, g, tiles, tile, kTile, nf);
    const long long f0 = gt.local % nf * kTile, m0 = gt.local / nf * kTile;
    const T* x = static_cast<const T*>(P.x[gt.p]) + (gt.first + m0) * C;
    const T* w = static_cast<const T*>(P.w[gt.p]) + (long long)gt.e * P.Z * P.D;
    const int rows = (int)min((long long)kTile, gt.rows - m0);
    float acc[kGated ? 2 : 1][4][4] = {};
    for (long long c0 = 0; c0 < C; c0 += kDepth) {
      for (int i = tid; i < kTile * kDepth; i += kPlainThreads) {
        const int c = i % kDepth, m = i / kDepth;
        xs[c][m] = m < rows && c0 + c < C ? to_float(x[(long long)m * C + c0 + c]) : 0.0f;
        const int fc = wc == 1 ? i % kDepth : i / kTile, f = wc == 1 ? i / kDepth : i % kTile;
        const bool in = f0 + f < F && c0 + fc < C;
        const long long at = (f0 + f) * wf + (c0 + fc) * wc;
        ws[0][fc][f] = in ? to_float(w[at]) : 0.0f;
        if (kGated) ws[kGated ? 1 : 0][fc][f] = in ? to_float(w[at + P.N * wf]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kDepth; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[0][i][j] += xs[c][ty + 16 * i] * ws[0][c][tx + 16 * j];
            if (kGated) acc[kGated ? 1 : 0][i][j] += xs[c][ty + 16 * i] * ws[kGated ? 1 : 0][c][tx + 16 * j];
          }
      __syncthreads();
    }
    const T* bias = P.bias[gt.p] != nullptr
                        ? static_cast<const T*>(P.bias[gt.p]) + gt.e * P.Z : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = ty + 16 * i;
      if (m >= rows) continue;
      const long long row = gt.first + m0 + m;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long f = f0 + tx + 16 * j;
        if (f >= F) continue;
        float z = acc[0][i][j] + (bias != nullptr ? to_float(bias[f]) : 0.0f);
        float y;
        if (P.pre[gt.p] != nullptr)
          static_cast<T*>(P.pre[gt.p])[row * P.Z + f] = from_float<T>(z);
        if (kGated) {
          const float u = acc[kGated ? 1 : 0][i][j] + (bias != nullptr ? to_float(bias[P.N + f]) : 0.0f);
          if (P.pre[gt.p] != nullptr)
            static_cast<T*>(P.pre[gt.p])[row * P.Z + P.N + f] = from_float<T>(u);
          y = act_fn(P.act, z) * u;
        } else {
          y = act_fn(P.act, z);
        }
        if (P.residual[gt.p] != nullptr)
          y += to_float(static_cast<const T*>(P.residual[gt.p])[row * F + f]);
        static_cast<T*>(P.out[gt.p])[row * F + f] = from_float<T>(y);
      }
    }
  }
}

// d_w[e][z][d] = sum over the expert's rows of dz[row][z] * x[row][d].
template <typename T>
__global__ void __launch_bounds__(kPlainThreads)
    expert_plain_wgrad_kernel(const __grid_constant__ ExpertParams P) {
  chain();
  __shared__ GroupTable g;
  __shared__ float zs[kDepth][kTile + 1], xs[kDepth][kTile + 1];
  if (!build_groups(P.g, g)) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int W = P.g.W, K = P.g.K;
  const long long nz = (P.Z + kTile - 1) / kTile, nd = (P.D + kTile - 1) / kTile;
  for (long long tile = blockIdx.x; tile < (long long)W * K * nz * nd; tile += gridDim.x) {
    const int pe = (int)(tile / (nz * nd)), p = pe / K, e = pe % K;
    const long long z0 = tile / nd % nz * kTile, d0 = tile % nd * kTile;
    const T* dz = static_cast<const T*>(P.dy[p]);
    const T* x = static_cast<const T*>(P.x[p]);
    float acc[4][4] = {};
    for (int r = 0; r < W; ++r) {
      int rows;
      const long long first = find_group(P.g, g, (p * W + r) * K + e, &rows);
      for (unsigned m0 = 0; m0 < (unsigned)rows; m0 += kDepth) {  // (up to 2^31 - 1 rows)
        for (int i = tid; i < kTile * kDepth; i += kPlainThreads) {
          const int c = i % kTile, m = i / kTile;
          const long long row = first + m0 + m;
          const bool in = m0 + m < (unsigned)rows;
          zs[m][c] = in && z0 + c < P.Z ? to_float(dz[row * P.Z + z0 + c]) : 0.0f;
          xs[m][c] = in && d0 + c < P.D ? to_float(x[row * P.D + d0 + c]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kDepth; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += zs[m][ty + 16 * i] * xs[m][tx + 16 * j];
        __syncthreads();
      }
    }
    T* out = static_cast<T*>(P.d_w[p]) + (long long)e * P.Z * P.D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long z = z0 + ty + 16 * i, d = d0 + tx + 16 * j;
        if (z < P.Z && d < P.D) out[z * P.D + d] = from_float<T>(acc[i][j]);
      }
  }
}

// ---------------------------------------------- activation's gradient --
// dz from dy and the saved pre-activations: a warp takes a row, or a part of one, a vector of N
// elements a lane at a time.  It is rounded to the operands' type, once, because
// the tensor cores take that: the gradients of rows and weights are then off by
// 0.0024 of their norm where 32 bits of dz leave 0.0017, their own rounding, and in
// f16 a dz above 65504 is infinite.  d_bias adds up the rounded values, so that it is
// the gradient of the same product.  Memory bound: with a gate 5 N elements of 2
// bytes are read and written a row (32,768 rows, N 2048, SiLU: 671 MB in 117 to 128
// us, 5.2 to 5.7 TB/s).
template <typename T, int N>
__global__ void __launch_bounds__(256)
    expert_dz_kernel(const __grid_constant__ ExpertParams P) {
  chain();
  __shared__ GroupTable g;
  if (!build_groups(P.g, g)) return;
  using Q = Piece<T, N>;
  using V = typename Q::Raw;
  const int nv = (int)(P.N / N), lane = threadIdx.x & 31;
  // (unsigned: up to 2^31 - 1 rows, and a stride past them)
  const unsigned warps = gridDim.x * (blockDim.x / 32), all = g.peer_base[P.g.W];
  const RowParts split(all, warps, nv);
  int p = 0;
  for (unsigned unit = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; unit < all * split.parts;
       unit += warps) {
    const int at = unit / split.parts;
    int from, to;
    split.run(unit - at * split.parts, nv, &from, &to);
    while (at >= g.peer_base[p + 1]) ++p;
    const long long row = at - g.peer_base[p];
    const V* dy = reinterpret_cast<const V*>(static_cast<const T*>(P.dy[p]) + row * P.N);
    const V* pre = reinterpret_cast<const V*>(static_cast<const T*>(P.pre_in[p]) + row * P.Z);
    V* dz = reinterpret_cast<V*>(static_cast<T*>(P.dz[p]) + row * P.Z);
#pragma unroll 2
    for (int v = from + lane; v < to; v += 32) {
      float d[N], z[N], u[N];
      Q::unpack(dy[v], d);
      Q::unpack(pre[v], z);
      if (P.gated) {
        Q::unpack(pre[nv + v], u);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          u[k] *= d[k] * act_slope(P.act, z[k]);
          d[k] *= act_fn(P.act, z[k]);
        }
        dz[v] = Q::pack(u);
        dz[nv + v] = Q::pack(d);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) d[k] *= act_slope(P.act, z[k]);
        dz[v] = Q::pack(d);
      }
    }
  }
}

// d_bias[e][z]: a block takes 16 vectors of N columns of an expert, each of its
// 32 half warps every 32nd row of a group; their sums are joined in shared
// memory in a fixed order.  It reads dz once, so the memory's rate is its floor
// (40 us for 32,768 rows of 4096 over 64 skewed experts); it takes 116, the
// dependent rounds of the expert with the most rows.  Eight or sixteen rows in
// flight a thread instead of four take 154 and 220: the registers cost blocks.
constexpr int kBiasThreads = 512, kBiasRows = kBiasThreads / 16;

template <typename T, int N>
__global__ void __launch_bounds__(kBiasThreads)
    expert_dbias_kernel(const __grid_constant__ ExpertParams P) {
  chain();
  __shared__ GroupTable g;
  __shared__ float part[kBiasRows][16 * N + 1];
  if (!build_groups(P.g, g)) return;
  using Q = Piece<T, N>;
  using V = typename Q::Raw;
  const int at = threadIdx.x % 16, team = threadIdx.x / 16;
  const int W = P.g.W, K = P.g.K;
  const long long nz = (P.Z + 16 * N - 1) / (16 * N);
  for (long long tile = blockIdx.x; tile < (long long)W * K * nz; tile += gridDim.x) {
    const int pe = (int)(tile / nz), p = pe / K, e = pe % K;
    const long long z = tile % nz * 16 * N + at * N;
    float sum[N] = {};
    for (int r = 0; r < W; ++r) {
      int rows;
      const long long first = find_group(P.g, g, (p * W + r) * K + e, &rows);
      if (z >= P.Z) continue;
      const T* from = static_cast<const T*>(P.dy[p]) + first * P.Z + z;
      constexpr int kAhead = 4;  // loads in flight
      for (unsigned m = team; m < (unsigned)rows; m += kAhead * kBiasRows) {  // (up to 2^31 - 1)
        V v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (m + u * kBiasRows < (unsigned)rows)
            v[u] = *reinterpret_cast<const V*>(from + (long long)(m + u * kBiasRows) * P.Z);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (m + u * kBiasRows < (unsigned)rows) {
            float f[N];
            Q::unpack(v[u], f);
#pragma unroll
            for (int k = 0; k < N; ++k) sum[k] += f[k];
          }
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) part[team][at * N + k] = sum[k];
    __syncthreads();
    for (int c = threadIdx.x; c < 16 * N; c += kBiasThreads) {
      const long long col = tile % nz * 16 * N + c;
      if (col < P.Z) {
        float all = 0.0f;
        for (int i = 0; i < kBiasRows; ++i) all += part[i][c];
        static_cast<T*>(P.d_bias[p])[e * P.Z + col] = from_float<T>(all);
      }
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------- host side --
int shape_ok(const a2av_expert_t* c, int W) {
  if (c == nullptr || c->experts_per_peer < 1 || c->in_features < 1 || c->out_features < 1 ||
      (c->dtype != A2AV_BF16 && c->dtype != A2AV_F16) || c->activation < A2AV_ACT_NONE ||
      c->activation > A2AV_ACT_SILU)
    return A2AV_ERR_INVALID_ARG;
  if ((long long)W * c->experts_per_peer > A2AV_MAX_DISPATCH_KEYS ||
      c->in_features > (1 << 24) || c->out_features > (c->gated ? 1 << 23 : 1 << 24))
    return A2AV_ERR_UNSUPPORTED;
  return A2AV_OK;
}

// Copies a list of W pointers (`need`: rows or experts of peer p want one).
bool take(const void** to, const void* const* from, int W, const int64_t* rows, int size) {
  for (int p = 0; p < W; ++p) {
    to[p] = from != nullptr && (rows == nullptr || rows[p] > 0) ? from[p] : nullptr;
    if (from != nullptr && (rows == nullptr || rows[p] > 0) && to[p] == nullptr) return false;
    if (!aligned_to(to[p], size)) return false;
  }
  return true;
}

bool take(void** to, void* const* from, int W, const int64_t* rows, int size) {
  return take(const_cast<const void**>(to), from, W, rows, size);
}

int expert_params(a2av_handle* h, const a2av_expert_t* c, const int64_t* rows_per_peer,
                  const int64_t* counts, ExpertParams* P) {
  if (h == nullptr || rows_per_peer == nullptr || counts == nullptr || !aligned_to(counts, 8))
    return A2AV_ERR_INVALID_ARG;
  const int rc = shape_ok(c, h->W);
  if (rc != A2AV_OK) return rc;
  std::memset(P, 0, sizeof(*P));
  int64_t all = 0;
  for (int p = 0; p < h->W; ++p) {
    if (rows_per_peer[p] < 0) return A2AV_ERR_INVALID_ARG;
    if (rows_per_peer[p] > kMaxCount - all) return A2AV_ERR_UNSUPPORTED;
    all += rows_per_peer[p];
    P->g.cap[p] = rows_per_peer[p];
  }
  P->g.counts = reinterpret_cast<const long long*>(counts);
  P->g.status = h->d_status;
  P->g.W = h->W;
  P->g.K = c->experts_per_peer;
  P->D = c->in_features;
  P->N = c->out_features;
  P->Z = c->gated ? 2 * c->out_features : c->out_features;
  P->act = c->activation;
  P->gated = c->gated != 0;
  return current_device(h);
}

template <typename T>
cudaError_t launch_forward(a2av_handle* h, const ExpertParams& P, int dtype, cudaStream_t s) {
  cudaError_t e;
  if (a2av_expert_mma(h, P, dtype, 0, s, &e)) return e;
  const dim3 grid(4 * h->sms);
  return P.gated ? launch_chained(expert_plain_kernel<T, true>, grid, kPlainThreads, 0, s, h->pdl,
                                  P, P.D, P.N, P.D, 1LL)
                 : launch_chained(expert_plain_kernel<T, false>, grid, kPlainThreads, 0, s, h->pdl,
                                  P, P.D, P.N, P.D, 1LL);
}

template <typename T>
cudaError_t launch_backward(a2av_handle* h, ExpertParams P, void* const* d_rows, bool dz_needed,
                            int dtype, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const dim3 grid(4 * h->sms);
  if (dz_needed) {
    bool vec = P.N % 8 == 0;
    for (int p = 0; p < h->W; ++p)
      vec = vec && aligned_to(P.dy[p], 16) && aligned_to(P.pre_in[p], 16) && aligned_to(P.dz[p], 16);
    e = launch_chained(vec ? expert_dz_kernel<T, 8> : expert_dz_kernel<T, 1>, grid, 256, 0, s,
                       h->pdl, P);
    if (e != cudaSuccess) return e;
    for (int p = 0; p < h->W; ++p) P.dy[p] = P.dz[p];
  }
  if (P.d_w[0] != nullptr && !a2av_expert_mma(h, P, dtype, 2, s, &e))
    e = launch_chained(expert_plain_wgrad_kernel<T>, grid, kPlainThreads, 0, s, h->pdl, P);
  if (e != cudaSuccess) return e;
  if (P.d_bias[0] != nullptr) {
    bool vec = P.Z % 8 == 0;
    for (int p = 0; p < h->W; ++p) vec = vec && aligned_to(P.dy[p], 16);
    e = launch_chained(vec ? expert_dbias_kernel<T, 8> : expert_dbias_kernel<T, 1>, grid,
                       kBiasThreads, 0, s, h->pdl, P);
    if (e != cudaSuccess) return e;
  }
  if (d_rows != nullptr) {
    for (int p = 0; p < h->W; ++p) {
      P.x[p] = P.dy[p];
      P.out[p] = P.g.cap[p] > 0 ? d_rows[p] : nullptr;
    }
    P.act = A2AV_ACT_NONE;
    if (!a2av_expert_mma(h, P, dtype, 1, s, &e))
      e = launch_chained(expert_plain_kernel<T, false>, grid, kPlainThreads, 0, s, h->pdl, P,
                         P.Z, P.D, 1LL, P.D);
  }
  return e;
}

}  // namespace

extern "C" int a2av_expert_matmul(a2av_handle* h, const a2av_expert_t* shape,
                                  const void* const* rows_ptrs, const int64_t* rows_per_peer,
                                  const int64_t* counts_dev, const void* const* weight_ptrs,
                                  const void* const* bias_ptrs, const void* const* residual_ptrs,
                                  void* const* out_ptrs, void* const* pre_ptrs, void* stream) {
  if (rows_ptrs == nullptr || weight_ptrs == nullptr || out_ptrs == nullptr)
    return A2AV_ERR_INVALID_ARG;
  ExpertParams P;
  const int rc = expert_params(h, shape, rows_per_peer, counts_dev, &P);
  if (rc != A2AV_OK) return rc;
  const int W = h->W, size = dtype_bytes(shape->dtype);
  if (!take(P.x, rows_ptrs, W, rows_per_peer, size) || !take(P.w, weight_ptrs, W, nullptr, size) ||
      !take(P.bias, bias_ptrs, W, nullptr, size) ||
      !take(P.residual, residual_ptrs, W, rows_per_peer, size) ||
      !take(P.out, out_ptrs, W, rows_per_peer, size) ||
      !take(P.pre, pre_ptrs, W, rows_per_peer, size))
    return A2AV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = shape->dtype == A2AV_BF16 ? launch_forward<__nv_bfloat16>(h, P, shape->dtype, s)
                                                  : launch_forward<__half>(h, P, shape->dtype, s);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return A2AV_ERR_CUDA;
  return A2AV_OK;
}

extern "C" int64_t a2av_expert_matmul_workspace_bytes(int world_size, const a2av_expert_t* shape,
                                                      int64_t total_rows) {
  if (world_size < 1 || world_size > kW || total_rows < 0 ||
      total_rows > kMaxCount || shape_ok(shape, world_size) != A2AV_OK)
    return -1;
  const int64_t Z = shape->gated ? 2 * shape->out_features : shape->out_features;
  const int64_t dz = shape->activation == A2AV_ACT_NONE && !shape->gated ? 0 : total_rows * Z;
  const int64_t tails = a2av_expert_tail_rows(world_size, shape->experts_per_peer, total_rows);
  const int64_t size = dtype_bytes(shape->dtype);
  return (dz * size + 255) / 256 * 256 + tails * (Z + shape->in_features) * size;
}

extern "C" int a2av_expert_matmul_backward(
    a2av_handle* h, const a2av_expert_t* shape, const void* const* rows_ptrs,
    const int64_t* rows_per_peer, const int64_t* counts_dev, const void* const* weight_ptrs,
    const void* const* pre_ptrs, const void* const* d_out_ptrs, void* const* d_rows_ptrs,
    void* const* d_weight_ptrs, void* const* d_bias_ptrs, void* workspace,
    int64_t workspace_bytes, void* stream) {
  if (rows_ptrs == nullptr || weight_ptrs == nullptr || d_out_ptrs == nullptr ||
      (d_rows_ptrs == nullptr && d_weight_ptrs == nullptr && d_bias_ptrs == nullptr))
    return A2AV_ERR_INVALID_ARG;
  ExpertParams P;
  const int rc = expert_params(h, shape, rows_per_peer, counts_dev, &P);
  if (rc != A2AV_OK) return rc;
  const int W = h->W, size = dtype_bytes(shape->dtype);
  const bool dz_needed = shape->activation != A2AV_ACT_NONE || shape->gated;
  if (dz_needed && pre_ptrs == nullptr) return A2AV_ERR_INVALID_ARG;
  if (!take(P.x, rows_ptrs, W, rows_per_peer, size) || !take(P.w, weight_ptrs, W, nullptr, size) ||
      !take(P.dy, d_out_ptrs, W, rows_per_peer, size) ||
      !take(P.pre_in, dz_needed ? pre_ptrs : nullptr, W, rows_per_peer, size) ||
      !take(P.out, d_rows_ptrs, W, rows_per_peer, size) ||
      !take(P.d_w, d_weight_ptrs, W, nullptr, size) ||
      !take(P.d_bias, d_bias_ptrs, W, nullptr, size))
    return A2AV_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int p = 0; p < W; ++p) total += rows_per_peer[p];
  const int64_t need = a2av_expert_matmul_workspace_bytes(W, shape, total);
  if (workspace_bytes < need || !aligned_to(workspace, 256) || (need > 0 && workspace == nullptr))
    return A2AV_ERR_INVALID_ARG;
  int64_t at = 0;
  for (int p = 0; p < W && dz_needed; ++p) {
    P.dz[p] = static_cast<unsigned char*>(workspace) + at * P.Z * size;
    at += rows_per_peer[p];
  }
  P.tails = static_cast<unsigned char*>(workspace) + (at * P.Z * size + 255) / 256 * 256;
  P.tail_rows = a2av_expert_tail_rows(W, P.g.K, total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      shape->dtype == A2AV_BF16
          ? launch_backward<__nv_bfloat16>(h, P, d_rows_ptrs, dz_needed, shape->dtype, s)
          : launch_backward<__half>(h, P, d_rows_ptrs, dz_needed, shape->dtype, s);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return A2AV_ERR_CUDA;
  return A2AV_OK;
}
