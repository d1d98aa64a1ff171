// weighted.cu -- the weighted return path of an MoE layer
// (a2av_combine_weighted) and its gradient; the interface is in
// include/a2av_moe.h.
//
// A block takes a token: its first k threads read the items' keys and
// positions and turn them into row addresses (the split matrix's prefix sums
// are in shared memory), then the block's threads walk the row, 16 bytes of it
// at a time, with all k rows' loads in flight together.
#include "moe_device.cuh"

namespace {

struct WeightedParams {
  const void* peer[kW];        // rows in the dispatch layout
  void* d_peer[kW];            // their gradients, in the same layout
  long long peer_rows[kW];     // rows that these buffers hold
  const int* key[kW];
  const long long* pos[kW];
  const float* weight[kW];     // NULL: 1
  const void* token_in[kW];    // forward: residual or NULL; backward: dy
  void* out[kW];
  float* d_weight[kW];
  long long token_first[kW + 1];
  const long long* splits;     // S [W][W]
  long long limit;             // largest valid split
  int* status;
  long long H;
  int W, K, k;
  int reads, writes;           // whether peer / d_peer are used
};

struct Offsets {
  long long in_off[kW][kW + 1];  // [r][p], rows of rank r before peer p; [r][W] all of them
  long long base[kW][kW];        // [r][p]: row in peer p = base + position
  int bad;
};

// The prefix sums of S, by the first warp; false (in every thread) and the
// status word set when S is not valid.
__device__ __forceinline__ bool build_offsets(const WeightedParams& P, Offsets& o) {
  const int W = P.W, tid = threadIdx.x;
  if (tid == 0) o.bad = 0;
  __syncthreads();
  for (int e = tid; e < W * W; e += blockDim.x) {
    const long long s = __ldcg(P.splits + e);
    if (s < 0 || s > P.limit) o.bad = 1;
    o.base[e / W][e % W] = s;  // S for now
  }
  __syncthreads();
  if (!o.bad) {
    if (tid < W) {
      long long row = 0;
      for (int p = 0; p < W; ++p) {
        o.in_off[tid][p] = row;
        row += o.base[tid][p];
      }
      o.in_off[tid][W] = row;
    }
    __syncthreads();
    if (tid < W) {
      long long col = 0;
      for (int r = 0; r < W; ++r) {
        const long long s = o.base[r][tid];
        o.base[r][tid] = col - o.in_off[r][tid];
        col += s;
      }
      if (col > P.peer_rows[tid]) o.bad = 1;
    }
    __syncthreads();
  }
  if (o.bad && blockIdx.x == 0 && tid == 0) note_error(P.status, A2AV_ERR_BAD_SPLITS);
  return !o.bad;
}

template <typename T>
__device__ __forceinline__ void find_items(const WeightedParams& P, const Offsets& o, int r,
                                           long long t, const T** row, T** d_row, float* w,
                                           int* bad) {
  const int j = threadIdx.x;
  if (j < P.k) {
    const long long i = t * P.k + j;
    const int key = P.key[r][i];
    const long long pos = P.pos[r][i];
    bool ok = key >= 0 && key < P.W * P.K;
    const int p = ok ? key / P.K : 0;
    ok = ok && pos >= o.in_off[r][p] && pos < o.in_off[r][p + 1];
    const long long at = ok ? (o.base[r][p] + pos) * P.H : 0;
    row[j] = static_cast<const T*>(P.peer[p]) + at;
    if (d_row != nullptr) d_row[j] = static_cast<T*>(P.d_peer[p]) + at;
    w[j] = P.weight[r] != nullptr ? P.weight[r][i] : 1.0f;
    if (!ok) *bad = 1;
  }
}

constexpr int kWeightedThreads = 256;

template <typename T, int N>
__global__ void __launch_bounds__(kWeightedThreads)
    combine_weighted_kernel(const __grid_constant__ WeightedParams P) {
  chain();
  __shared__ Offsets o;
  __shared__ const T* row[A2AV_MAX_TOPK];
  __shared__ float w[A2AV_MAX_TOPK];
  __shared__ int bad;
  if (!build_offsets(P, o)) return;
  using V = Vec<T, N>;
  const long long nv = P.H / N;
  for (long long g = blockIdx.x; g < P.token_first[P.W]; g += gridDim.x) {
    int r = 0;
    while (P.token_first[r + 1] <= g) ++r;
    const long long t = g - P.token_first[r];
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    find_items<T>(P, o, r, t, row, nullptr, w, &bad);
    __syncthreads();
    if (bad) {
      if (threadIdx.x == 0) note_error(P.status, A2AV_ERR_BAD_INDEX);
    } else {
      const T* res = P.token_in[r] != nullptr
                         ? static_cast<const T*>(P.token_in[r]) + t * P.H : nullptr;
      T* out = static_cast<T*>(P.out[r]) + t * P.H;
      for (long long v = threadIdx.x; v < nv; v += blockDim.x) {
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.0f;
        for (int j = 0; j < P.k; ++j) {
          const V x = reinterpret_cast<const V*>(row[j])[v];
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] += w[j] * to_float(x.v[i]);
        }
        if (res != nullptr) {
          const V x = reinterpret_cast<const V*>(res)[v];
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] += to_float(x.v[i]);
        }
        V y;
#pragma unroll
        for (int i = 0; i < N; ++i) y.v[i] = from_float<T>(acc[i]);
        reinterpret_cast<V*>(out)[v] = y;
      }
    }
    __syncthreads();
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(kWeightedThreads)
    combine_weighted_backward_kernel(const __grid_constant__ WeightedParams P) {
  chain();
  __shared__ Offsets o;
  __shared__ const T* row[A2AV_MAX_TOPK];
  __shared__ T* d_row[A2AV_MAX_TOPK];
  __shared__ float w[A2AV_MAX_TOPK];
  __shared__ float part[kWeightedThreads / 32];
  __shared__ int bad;
  if (!build_offsets(P, o)) return;
  using V = Vec<T, N>;
  const long long nv = P.H / N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long g = blockIdx.x; g < P.token_first[P.W]; g += gridDim.x) {
    int r = 0;
    while (P.token_first[r + 1] <= g) ++r;
    const long long t = g - P.token_first[r];
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    find_items<T>(P, o, r, t, row, d_row, w, &bad);
    __syncthreads();
    if (bad) {
      if (threadIdx.x == 0) note_error(P.status, A2AV_ERR_BAD_INDEX);
      __syncthreads();
      continue;
    }
    const T* dy = static_cast<const T*>(P.token_in[r]) + t * P.H;
    for (int j = 0; j < P.k; ++j) {
      float dot = 0.0f;
      for (long long v = threadIdx.x; v < nv; v += blockDim.x) {
        const V x = reinterpret_cast<const V*>(dy)[v];
        if (P.reads) {
          const V y = reinterpret_cast<const V*>(row[j])[v];
#pragma unroll
          for (int i = 0; i < N; ++i) dot += to_float(x.v[i]) * to_float(y.v[i]);
        }
        if (P.writes) {
          V d;
#pragma unroll
          for (int i = 0; i < N; ++i) d.v[i] = from_float<T>(w[j] * to_float(x.v[i]));
          reinterpret_cast<V*>(d_row[j])[v] = d;
        }
      }
      if (P.reads) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(kAll, dot, s);
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
          float sum = 0.0f;
          for (int i = 0; i < (int)blockDim.x / 32; ++i) sum += part[i];
          P.d_weight[r][t * P.k + j] = sum;
        }
        __syncthreads();
      }
    }
    __syncthreads();
  }
}

using WeightedKernel = void (*)(WeightedParams);

template <typename T>
WeightedKernel weighted_kernel_of(bool vec, bool backward) {
  constexpr int kV = 16 / sizeof(T);
  if (backward)
    return vec ? combine_weighted_backward_kernel<T, kV> : combine_weighted_backward_kernel<T, 1>;
  return vec ? combine_weighted_kernel<T, kV> : combine_weighted_kernel<T, 1>;
}

WeightedKernel weighted_kernel_of(int dtype, bool vec, bool backward) {
  if (dtype == A2AV_F32) return weighted_kernel_of<float>(vec, backward);
  if (dtype == A2AV_BF16) return weighted_kernel_of<__nv_bfloat16>(vec, backward);
  return weighted_kernel_of<__half>(vec, backward);
}

// Both directions: `peers` read, `d_peers` written (either may be NULL as the
// call allows), `token_in` residual or dy, `out` / `d_weight` written.
int weighted_call(a2av_handle* h, int K, int k, int64_t H, int dtype, const void* const* peers,
                  const int64_t* rows_per_peer, const int64_t* splits, const int32_t* const* keys, const int64_t* const* pos,
                  const float* const* weights, const int64_t* tokens,
                  const void* const* token_in, void* const* out, void* const* d_peers,
                  float* const* d_weights, bool backward, void* stream) {
  if (h == nullptr || rows_per_peer == nullptr || splits == nullptr || keys == nullptr || pos == nullptr || tokens == nullptr)
    return A2AV_ERR_INVALID_ARG;
  const int size = dtype_bytes(dtype);
  if (K < 1 || k < 1 || H < 1 || size == 0 || !aligned_to(splits, 8)) return A2AV_ERR_INVALID_ARG;
  const int W = h->W;
  if ((long long)W * K > A2AV_MAX_DISPATCH_KEYS || k > A2AV_MAX_TOPK || H > (1LL << 32))
    return A2AV_ERR_UNSUPPORTED;
  WeightedParams P;
  std::memset(&P, 0, sizeof(P));
  bool vec = H * size % 16 == 0;
  for (int r = 0; r < W; ++r) {
    const int64_t n = tokens[r];
    if (n < 0 || rows_per_peer[r] < 0) return A2AV_ERR_INVALID_ARG;
    P.peer_rows[r] = rows_per_peer[r];
    if (n > kMaxCount / k) return A2AV_ERR_UNSUPPORTED;
    P.token_first[r + 1] = P.token_first[r] + n;
    if (peers != nullptr) P.peer[r] = peers[r];
    if (d_peers != nullptr) P.d_peer[r] = d_peers[r];
    if (rows_per_peer[r] > 0 && ((peers != nullptr && P.peer[r] == nullptr) ||
                                 (d_peers != nullptr && P.d_peer[r] == nullptr)))
      return A2AV_ERR_INVALID_ARG;
    if (!aligned_to(P.peer[r], size) || !aligned_to(P.d_peer[r], size)) return A2AV_ERR_INVALID_ARG;
    vec = vec && aligned_to(P.peer[r], 16) && aligned_to(P.d_peer[r], 16);
    if (n == 0) continue;
    P.key[r] = keys[r];
    P.pos[r] = reinterpret_cast<const long long*>(pos[r]);
    P.weight[r] = weights != nullptr ? weights[r] : nullptr;
    P.token_in[r] = token_in != nullptr ? token_in[r] : nullptr;
    P.out[r] = out != nullptr ? out[r] : nullptr;
    P.d_weight[r] = d_weights != nullptr ? d_weights[r] : nullptr;
    if (P.key[r] == nullptr || P.pos[r] == nullptr || (weights != nullptr && !P.weight[r]) ||
        (token_in != nullptr && !P.token_in[r]) || (out != nullptr && !P.out[r]) ||
        (d_weights != nullptr && !P.d_weight[r]) || !aligned_to(P.key[r], 4) ||
        !aligned_to(P.pos[r], 8) || !aligned_to(P.weight[r], 4) ||
        !aligned_to(P.token_in[r], size) || !aligned_to(P.out[r], size) ||
        !aligned_to(P.d_weight[r], 4))
      return A2AV_ERR_INVALID_ARG;
    vec = vec && aligned_to(P.token_in[r], 16) && aligned_to(P.out[r], 16);
  }
  const int rc = current_device(h);
  if (rc != A2AV_OK) return rc;
  if (P.token_first[W] == 0) return A2AV_OK;
  P.splits = reinterpret_cast<const long long*>(splits);
  P.limit = (1LL << 62) / ((long long)W * H * size);
  P.status = h->d_status;
  P.H = H;
  P.W = W;
  P.K = K;
  P.k = k;
  P.reads = peers != nullptr;
  P.writes = d_peers != nullptr;
  const long long fit = 8LL * h->sms;
  const unsigned grid = (unsigned)(P.token_first[W] < fit ? P.token_first[W] : fit);
  const cudaError_t e =
      launch_chained(weighted_kernel_of(dtype, vec, backward), dim3(grid), kWeightedThreads, 0,
                     static_cast<cudaStream_t>(stream), h->pdl, P);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return A2AV_ERR_CUDA;
  return A2AV_OK;
}

}  // namespace

extern "C" int a2av_combine_weighted(a2av_handle* h, int keys_per_peer, int topk, int64_t hidden,
                                     int dtype, const void* const* peer_ptrs,
                                     const int64_t* rows_per_peer, const int64_t* in_splits_dev,
                                     const int32_t* const* key_ptrs,
                                     const int64_t* const* sorted_pos_ptrs,
                                     const float* const* weight_ptrs,
                                     const int64_t* tokens_per_rank,
                                     const void* const* residual_ptrs, void* const* out_ptrs,
                                     void* stream) {
  if (peer_ptrs == nullptr || out_ptrs == nullptr) return A2AV_ERR_INVALID_ARG;
  return weighted_call(h, keys_per_peer, topk, hidden, dtype, peer_ptrs, rows_per_peer, in_splits_dev, key_ptrs,
                       sorted_pos_ptrs, weight_ptrs, tokens_per_rank, residual_ptrs, out_ptrs,
                       nullptr, nullptr, false, stream);
}

extern "C" int a2av_combine_weighted_backward(
    a2av_handle* h, int keys_per_peer, int topk, int64_t hidden, int dtype,
    const void* const* peer_ptrs, const int64_t* rows_per_peer, const int64_t* in_splits_dev,
    const int32_t* const* key_ptrs, const int64_t* const* sorted_pos_ptrs, const float* const* weight_ptrs,
    const int64_t* tokens_per_rank, const void* const* d_out_ptrs, void* const* d_peer_ptrs,
    float* const* d_weight_ptrs, void* stream) {
  if (d_out_ptrs == nullptr || (d_peer_ptrs == nullptr && d_weight_ptrs == nullptr) ||
      (d_weight_ptrs != nullptr && peer_ptrs == nullptr))
    return A2AV_ERR_INVALID_ARG;
  return weighted_call(h, keys_per_peer, topk, hidden, dtype,
                       d_weight_ptrs != nullptr ? peer_ptrs : nullptr, rows_per_peer, in_splits_dev, key_ptrs,
                       sorted_pos_ptrs, weight_ptrs, tokens_per_rank, d_out_ptrs, nullptr,
                       d_peer_ptrs, d_weight_ptrs, true, stream);
}
