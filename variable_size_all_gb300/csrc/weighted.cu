// weighted.cu -- the weighted return path of an MoE layer
// (a2av_combine_weighted) and its gradient; the interface is in
// include/a2av_moe.h.
//
// Memory bound: each row is read once and each token written once.  A warp takes
// 2 KiB of a token's rows (the backward pass, which sums over the row, a token,
// 1 KiB of it at a time): its first k lanes read the items' keys, positions and weights and turn them into
// row addresses (the split matrix's prefix sums are in shared memory), those of
// its next piece being in flight meanwhile; then two rows at a time are read,
// with no barrier between an SM's warps.  Neighbouring warps are in the same
// rows, which memory likes better than one row a warp: 131,072 rows of 14 KiB
// summed by twos 444 to 449 us (0.93 of the copy rate) against 466 to 585, and the more
// warps an SM holds in other rows the slower (two blocks of eight: 466, four: 585).
// The backward pass of the same rows (dy and the rows read, their gradients
// written) takes 695 us, the copy rate.
// (Of few tokens a block takes one: a decoding step of 16 tokens on each of 8
// ranks, 5.6 us against 13.)
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

// One lane's item of a token.
struct Item {
  int r, key;
  long long t, pos;
  float w;
};

// Token g of all ranks' (rank-major); its item j to lane j < k.
__device__ __forceinline__ Item fetch_item(const WeightedParams& P, long long g, int lane) {
  Item x;
  x.r = 0;
  while (P.token_first[x.r + 1] <= g) ++x.r;
  x.t = g - P.token_first[x.r];
  x.key = 0;
  x.pos = 0;
  x.w = 1.0f;
  if (lane < P.k) {
    const long long i = x.t * P.k + lane;
    x.key = P.key[x.r][i];
    x.pos = P.pos[x.r][i];
    if (P.weight[x.r] != nullptr) x.w = P.weight[x.r][i];
  }
  return x;
}

// The item's peer and row (lanes below k); false, in every lane, when one of
// the token's items has none.
__device__ __forceinline__ bool find_row(const WeightedParams& P, const Offsets& o, const Item& x,
                                         int lane, int* peer, long long* row) {
  bool ok = x.key >= 0 && x.key < P.W * P.K;
  const int p = ok ? x.key / P.K : 0;
  ok = ok && x.pos >= o.in_off[x.r][p] && x.pos < o.in_off[x.r][p + 1];
  *peer = p;
  *row = o.base[x.r][p] + x.pos;
  const bool all = __all_sync(kAll, ok || lane >= P.k);
  if (!all && lane == 0) note_error(P.status, A2AV_ERR_BAD_INDEX);
  return all;
}

template <typename P>
__device__ __forceinline__ P* from_lane(P* p, int lane) {
  return reinterpret_cast<P*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(p), lane));
}

constexpr int kWeightedThreads = 256;

// U vectors of a row, 32 apart.
template <typename T, int N, int U>
__device__ __forceinline__ void load_slice(typename Piece<T, N>::Raw (&x)[U], const T* row,
                                           long long v0, long long nv) {
  using V = typename Piece<T, N>::Raw;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (v0 + 32 * u < nv) x[u] = reinterpret_cast<const V*>(row)[v0 + 32 * u];
}

template <typename T, int N>
__global__ void __launch_bounds__(kWeightedThreads, 2)
    combine_weighted_kernel(const __grid_constant__ WeightedParams P) {
  chain();
  __shared__ Offsets o;
  using Q = Piece<T, N>;
  using V = typename Q::Raw;
  constexpr int kVectors = N * sizeof(T) == 16 ? 4 : 8, kSlice = 32 * kVectors;
  const int lane = threadIdx.x & 31;
  const long long nv = P.H / N, slices = (nv + kSlice - 1) / kSlice;
  const long long warps = (long long)gridDim.x * (kWeightedThreads / 32);
  const long long first = (long long)blockIdx.x * (kWeightedThreads / 32) + threadIdx.x / 32;
  const long long tokens = P.token_first[P.W];
  // token and slice of this warp, and the way to its next
  long long g = first / slices, s = first - g * slices;
  const long long g_on = warps / slices, s_on = warps - g_on * slices;
  Item item;
  if (g < tokens) item = fetch_item(P, g, lane);
  if (!build_offsets(P, o)) return;
  while (g < tokens) {
    const Item it = item;
    const long long v0 = s * kSlice + lane;
    g += g_on;
    s += s_on;
    if (s >= slices) {
      s -= slices;
      ++g;
    }
    if (g < tokens) item = fetch_item(P, g, lane);
    int p;
    long long at;
    if (!find_row(P, o, it, lane, &p, &at)) continue;
    const T* row = static_cast<const T*>(P.peer[p]) + at * P.H;  // (lanes below k)
    const T* res = static_cast<const T*>(P.token_in[it.r]);
    if (res != nullptr) res += it.t * P.H;
    V* out = reinterpret_cast<V*>(static_cast<T*>(P.out[it.r]) + it.t * P.H);
    V z[kVectors];
    if (res != nullptr) load_slice<T, N, kVectors>(z, res, v0, nv);
    float acc[kVectors][N];
#pragma unroll
    for (int u = 0; u < kVectors; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[u][i] = 0.0f;
    for (int j = 0; j < P.k; j += 2) {
      V x[kVectors], y[kVectors];
      const bool two = j + 1 < P.k;
      load_slice<T, N, kVectors>(x, from_lane(row, j), v0, nv);
      const T* next = from_lane(row, two ? j + 1 : j);
      if (two) load_slice<T, N, kVectors>(y, next, v0, nv);
      const float wx = __shfl_sync(kAll, it.w, j), wy = __shfl_sync(kAll, it.w, two ? j + 1 : j);
#pragma unroll
      for (int u = 0; u < kVectors; ++u) {
        float f[N];
        Q::unpack(x[u], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[u][i] += wx * f[i];
        if (two) {
          Q::unpack(y[u], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[u][i] += wy * f[i];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kVectors; ++u)
      if (v0 + 32 * u < nv) {
        if (res != nullptr) {
          float f[N];
          Q::unpack(z[u], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[u][i] += f[i];
        }
        out[v0 + 32 * u] = Q::pack(acc[u]);
      }
  }
}

// kBlock: a block takes a token, its warps every eighth slice of the rows; else
// a warp does.
template <typename T, int N, bool kBlock>
__global__ void __launch_bounds__(kWeightedThreads)
    combine_weighted_backward_kernel(const __grid_constant__ WeightedParams P) {
  chain();
  constexpr int kWarps = kWeightedThreads / 32;
  __shared__ Offsets o;
  __shared__ float part[kBlock ? A2AV_MAX_TOPK : 1][kWarps];  // the warps' sums of an item
  using Q = Piece<T, N>;
  using V = typename Q::Raw;
  constexpr int kVectors = N == 1 ? 8 : 16 / N, kSlice = 32 * kVectors;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const long long nv = P.H / N, tokens = P.token_first[P.W];
  const long long by = kBlock ? gridDim.x : (long long)gridDim.x * kWarps;
  long long g = kBlock ? blockIdx.x : (long long)blockIdx.x * kWarps + warp;
  Item item;
  if (g < tokens) item = fetch_item(P, g, lane);
  if (!build_offsets(P, o)) return;
  while (g < tokens) {
    const Item it = item;
    g += by;
    if (g < tokens) item = fetch_item(P, g, lane);
    int p;
    long long at;
    if (!find_row(P, o, it, lane, &p, &at)) continue;
    const T* row = static_cast<const T*>(P.peer[p]) + at * P.H;
    T* d_row = static_cast<T*>(P.d_peer[p]) + at * P.H;
    const T* dy = static_cast<const T*>(P.token_in[it.r]) + it.t * P.H;
    for (int j = 0; j < P.k; j += 2) {
      const bool two = j + 1 < P.k;
      const int j1 = two ? j + 1 : j;
      const T *r0 = from_lane(row, j), *r1 = from_lane(row, j1);
      T *d0 = from_lane(d_row, j), *d1 = from_lane(d_row, j1);
      const float w0 = __shfl_sync(kAll, it.w, j), w1 = __shfl_sync(kAll, it.w, j1);
      float dot0 = 0.0f, dot1 = 0.0f;
      for (long long v0 = lane + (kBlock ? warp * kSlice : 0); v0 < nv;
           v0 += kBlock ? kWarps * kSlice : kSlice) {
        V d[kVectors], x[kVectors], y[kVectors];
        load_slice<T, N, kVectors>(d, dy, v0, nv);
        if (P.reads) {
          load_slice<T, N, kVectors>(x, r0, v0, nv);
          if (two) load_slice<T, N, kVectors>(y, r1, v0, nv);
        }
#pragma unroll
        for (int u = 0; u < kVectors; ++u) {
          const long long v = v0 + 32 * u;
          if (v >= nv) continue;
          float f[N], h[N];
          Q::unpack(d[u], f);
          if (P.reads) {
            Q::unpack(x[u], h);
#pragma unroll
            for (int i = 0; i < N; ++i) dot0 += f[i] * h[i];
            if (two) {
              Q::unpack(y[u], h);
#pragma unroll
              for (int i = 0; i < N; ++i) dot1 += f[i] * h[i];
            }
          }
          if (P.writes) {
#pragma unroll
            for (int i = 0; i < N; ++i) h[i] = w0 * f[i];
            reinterpret_cast<V*>(d0)[v] = Q::pack(h);
            if (two) {
#pragma unroll
              for (int i = 0; i < N; ++i) h[i] = w1 * f[i];
              reinterpret_cast<V*>(d1)[v] = Q::pack(h);
            }
          }
        }
      }
      if (P.reads) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
          dot0 += __shfl_xor_sync(kAll, dot0, s);
          dot1 += __shfl_xor_sync(kAll, dot1, s);
        }
        float* dw = kBlock ? &part[j][warp] : P.d_weight[it.r] + it.t * P.k + j;
        if (lane == 0) dw[0] = dot0;
        if (lane == 1 && two) dw[kBlock ? kWarps : 1] = dot1;
      }
    }
    if (kBlock && P.reads) {
      __syncthreads();
      if (threadIdx.x < P.k) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += part[threadIdx.x][i];
        P.d_weight[it.r][it.t * P.k + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
}

using WeightedKernel = void (*)(WeightedParams);

enum WeightedForm { kForward, kBackward, kBackwardBlock };

// `bytes`: of a vector, 16, 4 or one element, as every row and buffer allows.
template <typename T, int N>
WeightedKernel weighted_kernel_of(WeightedForm form) {
  if (form == kForward) return combine_weighted_kernel<T, N>;
  return form == kBackward ? combine_weighted_backward_kernel<T, N, false>
                           : combine_weighted_backward_kernel<T, N, true>;
}

template <typename T>
WeightedKernel weighted_kernel_of(int bytes, WeightedForm form) {
  if (bytes == 16) return weighted_kernel_of<T, 16 / sizeof(T)>(form);
  return bytes == 4 ? weighted_kernel_of<T, 4 / sizeof(T)>(form) : weighted_kernel_of<T, 1>(form);
}

WeightedKernel weighted_kernel_of(int dtype, int bytes, WeightedForm form) {
  if (dtype == A2AV_F32) return weighted_kernel_of<float>(bytes, form);
  if (dtype == A2AV_BF16) return weighted_kernel_of<__nv_bfloat16>(bytes, form);
  return weighted_kernel_of<__half>(bytes, form);
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
  uintptr_t low = (uintptr_t)(H * size);  // the bits below a common alignment
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
    low |= (uintptr_t)P.peer[r] | (uintptr_t)P.d_peer[r];
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
    low |= (uintptr_t)P.token_in[r] | (uintptr_t)P.out[r];
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
  const int bytes = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : size;
  // A block a token where that keeps more bytes in flight: rows of 8 KiB, a slice
  // for each of its warps, until the tokens' warps fill the GPU several times over
  // (14 KiB rows by twos, 128 tokens 13.0 -> 5.6 us, 4096: 64 -> 50; 8 KiB, 4096:
  // 39 -> 33, but 16,384: 109 -> 114), shorter ones only with few tokens (4 KiB,
  // 128: 6.4 -> 4.1; 4096: 16 -> 21).
  const long long kib = (H * size + 1023) / 1024;
  const bool by_block = backward && P.token_first[W] < h->sms * (kib >= 8 ? 64 : kib);
  const WeightedKernel kernel =
      weighted_kernel_of(dtype, bytes, !backward ? kForward : by_block ? kBackwardBlock : kBackward);
  int fit = 0;  // blocks an SM holds
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, kWeightedThreads, 0) != cudaSuccess)
    return A2AV_ERR_CUDA;
  const long long most = (long long)fit * h->sms, warps = kWeightedThreads / 32;
  const int slice = bytes == 16 ? 128 : 256;  // vectors of a forward warp's slice
  const long long slices = backward ? 1 : (H * size / bytes + slice - 1) / slice;
  const long long blocks =
      by_block ? P.token_first[W] : (P.token_first[W] * slices + warps - 1) / warps;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  const cudaError_t e = launch_chained(kernel, dim3(grid), kWeightedThreads, 0,
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
