// route.cu -- routing to experts (a2av_route) and its gradient
// (a2av_route_backward); the interface is in include/a2av_moe.h.
//
// A warp takes a token.  Lane l holds the experts [l NJ, (l + 1) NJ), NJ the
// power of two >= E / 32, so that among equal choices the lowest expert is the
// lowest lane's lowest: a round of the top-k is one redux.max over the lanes'
// best, one ballot for the first lane that has it, and a search of that lane's
// NJ values.  Choices are compared as unsigned integers in the order of the
// floats they stand for (0 = not an expert, or already taken).
#include "moe_device.cuh"

namespace {

constexpr int kRouteWarps = 8;

struct RouteParams {
  const void* logits[kW];
  int* key[kW];
  float* weight[kW];
  const float* d_weight[kW];
  void* d_logits[kW];
  int tokens[kW];
  const float* bias;
  unsigned long long* counts;
  int* status;
  int E, k, score, groups, top_groups, group_top, renormalise;
  int group_size;
  float scale;
  int add_counts;  // several blocks a rank: counts (cleared before) are added to
};

constexpr unsigned kNegInf = 0x007fffffu;  // order_of(-inf)

// Floats in their order as unsigned integers; NaN as -inf, -0 as 0.
__device__ __forceinline__ unsigned order_of(float c) {
  if (c != c) return kNegInf;
  const unsigned u = __float_as_uint(c + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float float_of(unsigned o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// The accurate exponential and an IEEE division: choices are decided by these
// scores, and equal logits must give equal ones on every path.
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// exp(x - m) where m is the largest of the x's it belongs to; 0 where all are -inf.
__device__ __forceinline__ float exp_below(float x, float m) {
  return m == -INFINITY ? 0.0f : expf(x - m);
}

// The lane's NJ logits (-inf past the last expert).
template <typename T, int NJ, bool kVec>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&x)[NJ]) {
  if (kVec) {  // rows and lanes are vectors of kV elements
    constexpr int kV = NJ * sizeof(T) <= 16 ? NJ : 16 / sizeof(T);
#pragma unroll
    for (int b = 0; b < NJ; b += kV) {
      const int e = lane * NJ + b;
      if (e < E) {
        const Vec<T, kV> v = *reinterpret_cast<const Vec<T, kV>*>(row + e);
#pragma unroll
        for (int j = 0; j < kV; ++j) x[b + j] = to_float(v.v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) x[b + j] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane * NJ + j;
      x[j] = e < E ? to_float(row[e]) : -INFINITY;
    }
  }
}

template <typename T, int NJ, bool kVec>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ RouteParams P) {
  chain();
  extern __shared__ int hist[];
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.E, k = P.k;
  if (P.counts != nullptr) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const bool by_logit = P.score == A2AV_SCORE_SOFTMAX && P.bias == nullptr && P.group_top == 1;
  const bool softmax = P.score == A2AV_SCORE_SOFTMAX;
  const bool need_sum = softmax && (!by_logit || !P.renormalise);
  const int n = P.tokens[r];
  for (int t = blockIdx.x * kRouteWarps + warp; t < n; t += gridDim.x * kRouteWarps) {
    float x[NJ];
    load_logits<T, NJ, kVec>(static_cast<const T*>(P.logits[r]) + (long long)t * E, E, lane, x);
    float m = 0.0f, total = 1.0f;
    if (need_sum) {
      m = x[0];
#pragma unroll
      for (int j = 1; j < NJ; ++j) m = fmaxf(m, x[j]);
      m = warp_max(m);
      total = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) total += exp_below(x[j], m);
      total = warp_sum(total);
    }
    unsigned c[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane * NJ + j;
      float v = x[j];
      if (!softmax)
        v = sigmoid(v);
      else if (!by_logit)
        v = m == -INFINITY ? 0.0f : expf(v - m) / total;
      if (P.bias != nullptr && e < E) v += P.bias[e];
      c[j] = e < E ? order_of(v) : 0u;
    }
    if (P.groups > 1) {
      // lane g gets group g's score: its best choice, or its two best, summed
      unsigned score = 0;
      for (int g = 0; g < P.groups; ++g) {
        unsigned a = 0, b = 0;  // this lane's two best in group g
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int e = lane * NJ + j;
          if (e >= g * P.group_size && e < (g + 1) * P.group_size) {
            if (c[j] > a) {
              b = a;
              a = c[j];
            } else if (c[j] > b) {
              b = c[j];
            }
          }
        }
        unsigned best = __reduce_max_sync(kAll, a);
        if (P.group_top == 2) {
          const int first = __ffs(__ballot_sync(kAll, a == best)) - 1;
          const unsigned second = __reduce_max_sync(kAll, lane == first ? b : a);
          best = order_of(float_of(best) + float_of(second));
        }
        if (lane == g) score = best;
      }
      unsigned keep = 0;
      for (int i = 0; i < P.top_groups; ++i) {
        const unsigned best = __reduce_max_sync(kAll, score);
        const int g = __ffs(__ballot_sync(kAll, score == best)) - 1;
        keep |= 1u << g;
        if (lane == g) score = 0;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = lane * NJ + j;
        if (e < E && !((keep >> (e / P.group_size)) & 1)) c[j] = kNegInf;
      }
    }
    // top k: lane i keeps the i-th choice and its logit
    int my_key = 0;
    float my_x = -INFINITY;
    unsigned mine = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) mine = max(mine, c[j]);
    for (int i = 0; i < k; ++i) {
      const unsigned best = __reduce_max_sync(kAll, mine);
      const int owner = __ffs(__ballot_sync(kAll, mine == best)) - 1;
      int at = 0;
      float xv = 0.0f;
      if (lane == owner) {
#pragma unroll
        for (int j = NJ - 1; j >= 0; --j)
          if (c[j] == best) {
            at = j;
            xv = x[j];
          }
        mine = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if (j == at) c[j] = 0;
          mine = max(mine, c[j]);
        }
        at += lane * NJ;
      }
      at = __shfl_sync(kAll, at, owner);
      xv = __shfl_sync(kAll, xv, owner);
      if (lane == i) {
        my_key = at;
        my_x = xv;
      }
    }
    // weights, from the chosen logits alone where they are renormalised
    float w;
    if (!softmax) {
      w = sigmoid(my_x);
    } else if (P.renormalise) {
      // NaN logits are chosen last; fmaxf passes them over and the sum does not
      w = exp_below(my_x, warp_max(lane < k ? my_x : -INFINITY));
    } else {
      w = m == -INFINITY ? 0.0f : expf(my_x - m) / total;
    }
    if (P.renormalise) {
      const float sum = warp_sum(lane < k ? w : 0.0f);
      w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (lane < k) {
      const long long i = (long long)t * k + lane;
      P.key[r][i] = my_key;
      P.weight[r][i] = w * P.scale;
      if (P.counts != nullptr) atomicAdd(&hist[my_key], 1);
    }
  }
  if (P.counts == nullptr) return;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    unsigned long long* to = P.counts + (long long)r * E + e;
    if (!P.add_counts)
      *to = (unsigned long long)hist[e];
    else if (hist[e] != 0)
      atomicAdd(to, (unsigned long long)hist[e]);
  }
}

template <typename T, int NJ, bool kVec>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_kernel(const __grid_constant__ RouteParams P) {
  chain();
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.E, k = P.k;
  const bool softmax = P.score == A2AV_SCORE_SOFTMAX;
  const bool dense = softmax && !P.renormalise;
  const int n = P.tokens[r];
  for (int t = blockIdx.x * kRouteWarps + warp; t < n; t += gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(P.logits[r]) + (long long)t * E;
    const long long i0 = (long long)t * k;
    int key = 0;
    float g = 0.0f, xs = -INFINITY;
    if (lane < k) {
      key = P.key[r][i0 + lane];
      g = P.d_weight[r][i0 + lane] * P.scale;
    }
    const bool bad = __any_sync(kAll, key < 0 || key >= E);
    if (bad && lane == 0) note_error(P.status, A2AV_ERR_BAD_INDEX);
    if (lane < k && !bad) xs = to_float(row[key]);
    float d[NJ];  // the row's gradient
#pragma unroll
    for (int j = 0; j < NJ; ++j) d[j] = 0.0f;
    float onto = 0.0f;  // what the lane's choice gets
    if (!bad) {
      if (dense) {
        float x[NJ];
        load_logits<T, NJ, kVec>(row, E, lane, x);
        float m = x[0];
#pragma unroll
        for (int j = 1; j < NJ; ++j) m = fmaxf(m, x[j]);
        m = warp_max(m);
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          x[j] = exp_below(x[j], m);
          total += x[j];
        }
        total = warp_sum(total);
        const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
        const float p = lane < k ? exp_below(xs, m) * inv : 0.0f;
        const float dot = warp_sum(lane < k ? g * p : 0.0f);
#pragma unroll
        for (int j = 0; j < NJ; ++j) d[j] = -(x[j] * inv) * dot;
        onto = p * g;  // added to -p * dot of the same expert
      } else if (softmax) {
        const float m = warp_max(xs);  // (xs is -inf in the lanes past k)
        const float e = lane < k ? exp_below(xs, m) : 0.0f;
        const float sum = warp_sum(e);
        const float q = sum == 0.0f ? 0.0f : e / sum;
        const float dot = warp_sum(lane < k ? g * q : 0.0f);
        onto = q * (g - dot);
      } else {
        const float s = lane < k ? sigmoid(xs) : 0.0f;
        float ds = g;
        if (P.renormalise) {
          const float sum = warp_sum(s);
          const float dot = warp_sum(lane < k ? g * s : 0.0f);
          ds = sum == 0.0f ? 0.0f : (g - dot / sum) / sum;
        }
        onto = ds * s * (1.0f - s);
      }
      for (int i = 0; i < k; ++i) {
        const int e = __shfl_sync(kAll, key, i);
        const float v = __shfl_sync(kAll, onto, i);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (e == lane * NJ + j) d[j] += v;
      }
    }
    T* out = static_cast<T*>(P.d_logits[r]) + (long long)t * E;
    if (kVec) {
      constexpr int kV = NJ * sizeof(T) <= 16 ? NJ : 16 / sizeof(T);
#pragma unroll
      for (int b = 0; b < NJ; b += kV) {
        const int e = lane * NJ + b;
        if (e < E) {
          Vec<T, kV> v;
#pragma unroll
          for (int j = 0; j < kV; ++j) v.v[j] = from_float<T>(d[b + j]);
          *reinterpret_cast<Vec<T, kV>*>(out + e) = v;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = lane * NJ + j;
        if (e < E) out[e] = from_float<T>(d[j]);
      }
    }
  }
}

using RouteKernel = void (*)(RouteParams);

template <typename T, bool kVec>
RouteKernel route_kernel_of(int nj, bool backward) {
  switch (nj) {
    case 1: return backward ? route_backward_kernel<T, 1, kVec> : route_kernel<T, 1, kVec>;
    case 2: return backward ? route_backward_kernel<T, 2, kVec> : route_kernel<T, 2, kVec>;
    case 4: return backward ? route_backward_kernel<T, 4, kVec> : route_kernel<T, 4, kVec>;
    case 8: return backward ? route_backward_kernel<T, 8, kVec> : route_kernel<T, 8, kVec>;
    case 16: return backward ? route_backward_kernel<T, 16, kVec> : route_kernel<T, 16, kVec>;
    default: return backward ? route_backward_kernel<T, 32, kVec> : route_kernel<T, 32, kVec>;
  }
}

RouteKernel route_kernel_of(int dtype, int nj, bool vec, bool backward) {
  if (dtype == A2AV_F32)
    return vec ? route_kernel_of<float, true>(nj, backward)
               : route_kernel_of<float, false>(nj, backward);
  if (dtype == A2AV_BF16)
    return vec ? route_kernel_of<__nv_bfloat16, true>(nj, backward)
               : route_kernel_of<__nv_bfloat16, false>(nj, backward);
  return vec ? route_kernel_of<__half, true>(nj, backward)
             : route_kernel_of<__half, false>(nj, backward);
}

// The checks both calls share; fills what both need.
int route_params(a2av_handle* h, const a2av_route_t* c, const void* const* logits,
                 const int64_t* tokens, const int32_t* const* keys, const float* const* weights,
                 void* const* d_logits, RouteParams* P, int* nj, bool* vec, int* most) {
  if (h == nullptr || c == nullptr || logits == nullptr || tokens == nullptr || keys == nullptr ||
      weights == nullptr)
    return A2AV_ERR_INVALID_ARG;
  const int size = dtype_bytes(c->dtype);
  if (c->experts < 1 || c->topk < 1 || size == 0 || c->groups < 1 || c->top_groups < 1 ||
      (c->score != A2AV_SCORE_SOFTMAX && c->score != A2AV_SCORE_SIGMOID) ||
      (c->group_top != 1 && c->group_top != 2))
    return A2AV_ERR_INVALID_ARG;
  if (c->experts > A2AV_MAX_DISPATCH_KEYS || c->topk > A2AV_MAX_TOPK ||
      c->groups > A2AV_MAX_ROUTE_GROUPS)
    return A2AV_ERR_UNSUPPORTED;
  if (c->experts % c->groups != 0 || c->top_groups > c->groups) return A2AV_ERR_INVALID_ARG;
  const int group_size = c->experts / c->groups;
  if (c->topk > c->top_groups * group_size || c->group_top > group_size)
    return A2AV_ERR_INVALID_ARG;
  std::memset(P, 0, sizeof(*P));
  *nj = 1;
  while (*nj * 32 < c->experts) *nj *= 2;
  // Vectors when every lane's run of NJ logits is whole and aligned: the row
  // is a multiple of a lane's vector and every buffer is aligned to it.
  const int lane_bytes = *nj * size < 16 ? *nj * size : 16;
  *vec = (long long)c->experts * size % lane_bytes == 0;
  *most = 0;
  for (int r = 0; r < h->W; ++r) {
    const int64_t n = tokens[r];
    if (n < 0) return A2AV_ERR_INVALID_ARG;
    if (n > kMaxCount / c->topk) return A2AV_ERR_UNSUPPORTED;
    P->tokens[r] = (int)n;
    if (n == 0) continue;
    const void* d = d_logits != nullptr ? d_logits[r] : logits[r];
    if (logits[r] == nullptr || keys[r] == nullptr || weights[r] == nullptr || d == nullptr ||
        !aligned_to(logits[r], size) || !aligned_to(d, size) || !aligned_to(keys[r], 4) ||
        !aligned_to(weights[r], 4))
      return A2AV_ERR_INVALID_ARG;
    *vec = *vec && aligned_to(logits[r], lane_bytes) && aligned_to(d, lane_bytes);
    P->logits[r] = logits[r];
    P->key[r] = const_cast<int*>(keys[r]);
    if (n > *most) *most = (int)n;
  }
  P->E = c->experts;
  P->k = c->topk;
  P->score = c->score;
  P->groups = c->groups;
  P->top_groups = c->top_groups;
  P->group_top = c->group_top;
  P->group_size = group_size;
  P->renormalise = c->renormalise != 0;
  P->scale = c->scale;
  P->status = h->d_status;
  return current_device(h);
}

// Blocks a rank: enough for every token to have its warp, up to eight blocks an SM.
int route_blocks(const a2av_handle* h, int most) {
  const int all = (most + kRouteWarps - 1) / kRouteWarps;
  const int fit = (8 * h->sms + h->W - 1) / h->W;
  return all < 1 ? 1 : all < fit ? all : fit;
}

}  // namespace

extern "C" int a2av_route(a2av_handle* h, const a2av_route_t* route,
                          const void* const* logits_ptrs, const int64_t* tokens_per_rank,
                          const float* bias_dev, int32_t* const* key_ptrs,
                          float* const* weight_ptrs, int64_t* counts_dev, void* stream) {
  RouteParams P;
  int nj = 0, most = 0;
  bool vec = false;
  const int rc = route_params(h, route, logits_ptrs, tokens_per_rank, key_ptrs, weight_ptrs,
                              nullptr, &P, &nj, &vec, &most);
  if (rc != A2AV_OK) return rc;
  if (!aligned_to(bias_dev, 4) || !aligned_to(counts_dev, 8)) return A2AV_ERR_INVALID_ARG;
  for (int r = 0; r < h->W; ++r) P.weight[r] = P.tokens[r] > 0 ? weight_ptrs[r] : nullptr;
  P.bias = bias_dev;
  P.counts = reinterpret_cast<unsigned long long*>(counts_dev);
  if (most == 0 && counts_dev == nullptr) return A2AV_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int blocks = route_blocks(h, most);
  if (P.counts != nullptr && blocks > 1) {
    P.add_counts = 1;
    if (cudaMemsetAsync(counts_dev, 0, sizeof(int64_t) * h->W * P.E, s) != cudaSuccess)
      return A2AV_ERR_CUDA;
  }
  const cudaError_t e =
      launch_chained(route_kernel_of(route->dtype, nj, vec, false), dim3(blocks, h->W),
                     32 * kRouteWarps, sizeof(int) * P.E, s, h->pdl, P);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return A2AV_ERR_CUDA;
  return A2AV_OK;
}

extern "C" int a2av_route_backward(a2av_handle* h, const a2av_route_t* route,
                                   const void* const* logits_ptrs, const int64_t* tokens_per_rank,
                                   const int32_t* const* key_ptrs,
                                   const float* const* d_weight_ptrs, void* const* d_logits_ptrs,
                                   void* stream) {
  if (d_logits_ptrs == nullptr) return A2AV_ERR_INVALID_ARG;
  RouteParams P;
  int nj = 0, most = 0;
  bool vec = false;
  const int rc = route_params(h, route, logits_ptrs, tokens_per_rank, key_ptrs, d_weight_ptrs,
                              d_logits_ptrs, &P, &nj, &vec, &most);
  if (rc != A2AV_OK) return rc;
  for (int r = 0; r < h->W; ++r) {
    P.d_weight[r] = P.tokens[r] > 0 ? d_weight_ptrs[r] : nullptr;
    P.d_logits[r] = P.tokens[r] > 0 ? d_logits_ptrs[r] : nullptr;
  }
  if (most == 0) return A2AV_OK;
  const cudaError_t e = launch_chained(route_kernel_of(route->dtype, nj, vec, true),
                                       dim3(route_blocks(h, most), h->W), 32 * kRouteWarps, 0,
                                       static_cast<cudaStream_t>(stream), h->pdl, P);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return A2AV_ERR_CUDA;
  return A2AV_OK;
}
