// route.cu -- routing to experts (a2av_route) and its gradient
// (a2av_route_backward); the interface is in include/a2av_moe.h.
//
// L lanes of a warp take a token, the warp 32 / L tokens.  Lane l of them holds
// the experts [l NJ, (l + 1) NJ), so that the order of (lane, place) is that of
// the experts, which decides ties.  With few tokens L is 32, for the shortest
// way through one; with many, NJ is 16 and L as many as the experts need:
// what is done once a token, whatever its experts (prefix sums, rounds,
// ranking, the weights), is then shared by the tokens of the warp.
//
// The top k without k rounds over all the experts: the k-th largest of the
// maxima of eight is at most the k-th largest of all, so only choices that
// reach it are candidates, a little over k of them.  They are written side by
// side, and each one's place is the number of candidates that come before it.
// A round over the maxima is a few instructions; one that also removes a choice
// and finds the next costs some for every expert.  (Many equal choices can make
// more candidates than there is room for; then those rounds are run.)
//
// Bound by steps that wait for one another: 65,536 tokens of 256 experts (f32,
// sigmoid, 4 of 8 groups, top 8) take 52 us against 10.5 for the memory.  A token
// takes 597 of a warp's instructions, which fill 65 % of the issue slots at 44 %
// of the warps an SM holds; between two of them a warp waits 2.8 cycles for
// shuffles and shared memory, 2.3 for the arithmetic before, 1.3 for loads.  (The
// exact exponential and division of every score, which decide ties, are a tenth of
// the instructions; without them it took as long.)  65,536 tokens of 64 experts
// (bf16, top 2) take 10.7 us with the clearing of the counts, of a warp's waits
// 3.6 for shuffles and shared memory, 2.2 and 1.9 for the others; 4 tokens on each
// of 8 ranks 3.5, one small launch.
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
  int group_lanes;  // lanes of a group, where that is a power of two of whole lanes; else 0
  float scale;
  int add_counts;  // several blocks a rank: counts (cleared by a kernel before) are added to
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

// Over the L lanes of a token.
template <int L = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// exp(x - m) where m is the largest of the x's it belongs to; 0 where all are -inf.
__device__ __forceinline__ float exp_below(float x, float m) {
  return m == -INFINITY ? 0.0f : expf(x - m);
}

// The sum of exp(x - m) over a token's experts, NJ a lane: the binary tree of
// neighbours over their numbers, which is the same however many lanes and experts
// a lane share it out (what is past the last expert adds 0).  So a token gets the
// same scores in a batch of any size.  lane_sum: of the lane's, depth first (an
// array of them, summed level by level, cost a call that has no use for the sum
// 2 % by its registers); experts_sum: of the lanes'.
template <int kFrom, int kOf, int NJ>
__device__ __forceinline__ float lane_sum(const float (&x)[NJ], float m) {
  if constexpr (kOf == 1) {
    return exp_below(x[kFrom], m);
  } else {
    const float first = lane_sum<kFrom, kOf / 2>(x, m);
    return __fadd_rn(first, lane_sum<kFrom + kOf / 2, kOf / 2>(x, m));
  }
}

template <int L>
__device__ __forceinline__ float experts_sum(float sum) {
#pragma unroll
  for (int o = 1; o < L; o *= 2) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, o));
  return sum;
}

// The same for k of 32 choices, choice lane + L s in v[s]: the tree that joins those
// 16 apart first, then 8, ... (levels that would add nothing but 0 are left out).
template <int L, int N>
__device__ __forceinline__ float choices_sum(float (&v)[N], int k) {
  static_assert(L * N == 32, "32 choices");
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2)
    if (k > L * n) {
#pragma unroll
      for (int s = 0; s < n; ++s) v[s] = __fadd_rn(v[s], v[s + n]);
    }
  float sum = v[0];
#pragma unroll
  for (int o = L / 2; o > 0; o /= 2) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, o));
  return sum;
}

template <int L = 32>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

template <int L>
__device__ __forceinline__ unsigned lanes_max(unsigned v) {
  if constexpr (L == 32) {
    v = __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  }
  return v;
}

// The accurate exponential and an IEEE division: choices are decided by these
// scores, and equal logits must give equal ones on every path.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

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

// Whether the lane's group is one of the top_groups, when every lane's experts
// are of one group and a group has a power of two of lanes (`width`).
template <int L, int NJ>
__device__ __forceinline__ bool keep_by_lanes(const RouteParams& P, const float (&c)[NJ], int width,
                                              int sl) {
  float a = -INFINITY, b = -INFINITY;  // the group's two best
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    b = fmaxf(b, fminf(a, c[j]));
    a = fmaxf(a, c[j]);
  }
  for (int o = 1; o < width; o <<= 1) {
    const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
    b = fmaxf(fmaxf(b, b2), fminf(a, a2));
    a = fmaxf(a, a2);
  }
  const unsigned score = order_of(P.group_top == 2 ? a + b : a);
  const int mine = sl / width;
  int before = 0;  // groups chosen before this one
  for (int g = 0; g < P.groups; ++g) {
    const unsigned s = __shfl_sync(kAll, score, g * width, L);
    before += s > score || (s == score && g < mine);
  }
  return before < P.top_groups;
}

// The same for groups of any size (L = 32): a bit for each group that stays.
template <int NJ>
__device__ __forceinline__ unsigned keep_groups(const RouteParams& P, const float (&c)[NJ], int lane) {
  unsigned score = 0;  // lane g: of group g
  for (int g = 0; g < P.groups; ++g) {
    unsigned a = 0, b = 0;  // this lane's two best in group g
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane * NJ + j;
      if (e >= g * P.group_size && e < (g + 1) * P.group_size) {
        const unsigned o = order_of(c[j]);
        b = max(b, min(a, o));
        a = max(a, o);
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
  return keep;
}

constexpr int kListed = 32;  // candidates a token has room for
struct Candidate {
  float c;
  int e;
};

// The top k by k rounds, to `chosen`.
template <int L, int NJ>
__device__ __forceinline__ void choose_by_rounds(const float (&c)[NJ], int k, int sl, int* chosen) {
  unsigned o[NJ], mine = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    o[j] = c[j] == c[j] ? order_of(c[j]) : 0u;
    mine = max(mine, o[j]);
  }
  for (int i = 0; i < k; ++i) {
    const unsigned best = lanes_max<L>(mine);
    // the first lane that has it, and its first expert
    int at = 32 * NJ;
#pragma unroll
    for (int j = NJ - 1; j >= 0; --j)
      if (o[j] == best) at = sl * NJ + j;
#pragma unroll
    for (int s = L / 2; s > 0; s >>= 1) at = min(at, __shfl_xor_sync(kAll, at, s));
    mine = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (sl * NJ + j == at) o[j] = 0;
      mine = max(mine, o[j]);
    }
    if (sl == 0) chosen[i] = at;
  }
}

template <typename T, int L, int NJ, bool kVec>
__global__ void __launch_bounds__(32 * kRouteWarps, L < 32 ? 4 : 1) route_kernel(const __grid_constant__ RouteParams P) {
  chain();
  constexpr int kTokens = 32 / L;  // of a warp
  extern __shared__ int hist[];
  constexpr int kEight = NJ < 8 ? NJ : 8, kMaxima = NJ / kEight;
  __shared__ __align__(16) float choices[kRouteWarps * kTokens][L * NJ];
  __shared__ __align__(16) float biases[L * NJ];
  __shared__ Candidate lists[kRouteWarps * kTokens][kListed];
  __shared__ int picks[kRouteWarps * kTokens][A2AV_MAX_TOPK];
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / L, sl = lane % L;
  const int E = P.E, k = P.k;
  if (P.counts != nullptr)
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  if (P.bias != nullptr)
    for (int e = threadIdx.x; e < L * NJ; e += blockDim.x) biases[e] = e < E ? P.bias[e] : 0.0f;
  __syncthreads();
  const bool by_logit = P.score == A2AV_SCORE_SOFTMAX && P.bias == nullptr && P.group_top == 1;
  const bool softmax = P.score == A2AV_SCORE_SOFTMAX;
  const bool need_sum = softmax && (!by_logit || !P.renormalise);
  // (unsigned: a stride past 2^31 - 1 tokens fits)
  const unsigned n = P.tokens[r];
  // the experts of this lane (the first `present` of its NJ; -inf where a group
  // that is dropped has one, NaN where there is none)
  const int present = E - sl * NJ;
  const bool whole = E == L * NJ;
  Candidate* list = lists[warp * kTokens + sub];
  float* row_c = choices[warp * kTokens + sub];
  int* chosen = picks[warp * kTokens + sub];
  for (unsigned t0 = (blockIdx.x * kRouteWarps + warp) * kTokens; t0 < n;
       t0 += gridDim.x * kRouteWarps * kTokens) {
    const bool live = t0 + sub < n;
    const unsigned t = live ? t0 + sub : n - 1;  // (lanes without a token repeat the last one)
    const T* row = static_cast<const T*>(P.logits[r]) + (long long)t * E;
    float c[NJ];  // the logits, then the choices
    load_logits<T, NJ, kVec>(row, E, sl, c);
    float m = 0.0f, total = 1.0f;
    if (need_sum) {
      m = c[0];
#pragma unroll
      for (int j = 1; j < NJ; ++j) m = fmaxf(m, c[j]);
      m = lanes_max<L>(m);
      total = experts_sum<L>(lane_sum<0, NJ>(c, m));
    }
    if (!softmax || !by_logit) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        c[j] = !softmax         ? sigmoid(c[j])
               : m == -INFINITY ? 0.0f
                                : expf(c[j] - m) / total;
    }
    if (P.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) c[j] += biases[sl * NJ + j];
    }
    // a choice that is NaN counts as -inf; from here on NaN is no expert at all
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      c[j] = fmaxf(c[j], -INFINITY);
      if (!whole && j >= present) c[j] = NAN;
    }
    if (P.groups > 1) {
      if (L < 32 || P.group_lanes > 0) {
        const bool keep = keep_by_lanes<L>(P, c, P.group_lanes, sl);
        const float gone = present > 0 ? -INFINITY : NAN;  // (lanes are whole here)
#pragma unroll
        for (int j = 0; j < NJ; ++j) c[j] = keep ? c[j] : gone;
      } else {
        const unsigned keep = keep_groups(P, c, lane);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (c[j] == c[j] && !((keep >> ((lane * NJ + j) / P.group_size)) & 1)) c[j] = -INFINITY;
      }
    }
    // the k-th largest of the maxima of eight
    unsigned most[kMaxima], best = 0;
#pragma unroll
    for (int q = 0; q < kMaxima; ++q) {
      float v = c[q * kEight];
#pragma unroll
      for (int j = 1; j < kEight; ++j) v = fmaxf(v, c[q * kEight + j]);
      most[q] = v == v ? order_of(v) : 0u;
    }
    for (int i = 0; i < k; ++i) {
      unsigned v = most[0];
#pragma unroll
      for (int q = 1; q < kMaxima; ++q) v = max(v, most[q]);
      best = lanes_max<L>(v);
#pragma unroll
      for (int q = 0; q < kMaxima; ++q)
        if (most[q] == best) most[q] = 0;
    }
    const float least = best != 0 ? float_of(best) : -INFINITY;
    unsigned marks = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) marks |= (c[j] >= least ? 1u : 0u) << j;
    const int own = __popc(marks);
    int upto = own;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      const int v = __shfl_up_sync(kAll, upto, o, L);
      if (sl >= o) upto += v;
    }
    const int count = __shfl_sync(kAll, upto, L - 1, L);
    if (!__any_sync(kAll, count > kListed)) {
      // (a lane has one or two: taken by their numbers from its choices in memory)
      float* to_c = row_c + sl * NJ;
#pragma unroll
      for (int j = 0; j < NJ; ++j) to_c[j] = c[j];
      Candidate* to = list + (upto - own);
      for (; marks != 0; marks &= marks - 1) {
        const int j = __ffs(marks) - 1;
        *to++ = Candidate{to_c[j], sl * NJ + j};
      }
      __syncwarp();
      for (int i = sl; i < count; i += L) {
        const Candidate x = list[i];
        int place = 0;
        for (int q = 0; q < count; ++q) {
          const float other = list[q].c;
          place += other > x.c || (other == x.c && q < i);
        }
        if (place < k) chosen[place] = x.e;
      }
    } else {
      choose_by_rounds<L, NJ>(c, k, sl, chosen);
    }
    __syncwarp();
    // weights, from the chosen logits alone where they are renormalised
    float w[kTokens], part[kTokens];
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int s = 0; s < kTokens; ++s) {
      const int i = sl + L * s;
      w[s] = i < k ? to_float(row[chosen[i]]) : -INFINITY;
      top = fmaxf(top, w[s]);  // (passes NaN over; the sum does not)
    }
    if (softmax && P.renormalise) top = lanes_max<L>(top);
#pragma unroll
    for (int s = 0; s < kTokens; ++s) {
      part[s] = 0.0f;
      if (sl + L * s < k) {
        w[s] = !softmax             ? sigmoid(w[s])
               : P.renormalise      ? exp_below(w[s], top)
               : m == -INFINITY     ? 0.0f
                                    : expf(w[s] - m) / total;
        part[s] = w[s];
      }
    }
    if (P.renormalise) sum = choices_sum<L>(part, k);
#pragma unroll
    for (int s = 0; s < kTokens; ++s) {
      const int i = sl + L * s;
      if (i < k && live) {
        if (P.renormalise) w[s] = sum == 0.0f ? 0.0f : w[s] / sum;
        const int e = chosen[i];
        P.key[r][(long long)t * k + i] = e;
        P.weight[r][(long long)t * k + i] = w[s] * P.scale;
        if (P.counts != nullptr) atomicAdd(&hist[e], 1);
      }
    }
    __syncwarp();
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

// A warp takes a token, a lane NJ experts: consecutive ones as vectors, or, where
// rows are not aligned for those, every 32nd.  Memory bound: the logits are read
// (softmax over all the experts) and their gradients written once, 65,536 tokens
// of 256 experts, f32: 139 MB in 27 us, 0.75 of the copy rate.
template <typename T, int NJ, bool kVec>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_kernel(const __grid_constant__ RouteParams P) {
  chain();
  // what the chosen experts get, at their places in the row: zeros between tokens
  __shared__ __align__(16) float scatter[kRouteWarps][32 * NJ];
  for (int i = threadIdx.x; i < kRouteWarps * 32 * NJ; i += blockDim.x) (&scatter[0][0])[i] = 0.0f;
  __syncthreads();
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.E, k = P.k;
  const bool softmax = P.score == A2AV_SCORE_SOFTMAX;
  const bool dense = softmax && !P.renormalise;
  const unsigned n = P.tokens[r];  // (unsigned: as in the router)
  for (unsigned t = blockIdx.x * kRouteWarps + warp; t < n; t += gridDim.x * kRouteWarps) {
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
    if (!bad) {
      const float* own = scatter[warp] + (kVec ? lane * NJ : lane);
      constexpr int kStep = kVec ? 1 : 32;
      if (dense) {
        float x[NJ];
        if (kVec) {
          load_logits<T, NJ, true>(row, E, lane, x);
        } else {
#pragma unroll
          for (int j = 0; j < NJ; ++j) x[j] = lane + 32 * j < E ? to_float(row[lane + 32 * j]) : -INFINITY;
        }
        float m = x[0];
#pragma unroll
        for (int j = 1; j < NJ; ++j) m = fmaxf(m, x[j]);
        m = lanes_max<32>(m);
        float total = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          x[j] = exp_below(x[j], m);
          total += x[j];
        }
        total = lanes_sum<32>(total);
        const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
        const float p = lane < k ? exp_below(xs, m) * inv : 0.0f;
        const float dot = lanes_sum<32>(lane < k ? g * p : 0.0f);
        if (lane < k) scatter[warp][key] = g;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NJ; ++j) d[j] = x[j] * inv * (own[j * kStep] - dot);
      } else {
        float onto;  // what the lane's choice gets
        if (softmax) {
          const float m = lanes_max<32>(xs);  // (xs is -inf in the lanes past k)
          const float e = lane < k ? exp_below(xs, m) : 0.0f;
          const float sum = lanes_sum<32>(e);
          const float q = sum == 0.0f ? 0.0f : e / sum;
          onto = q * (g - lanes_sum<32>(lane < k ? g * q : 0.0f));
        } else {
          const float s = lane < k ? sigmoid(xs) : 0.0f;
          float ds = g;
          if (P.renormalise) {
            const float sum = lanes_sum<32>(s);
            const float dot = lanes_sum<32>(lane < k ? g * s : 0.0f);
            ds = sum == 0.0f ? 0.0f : (g - dot / sum) / sum;
          }
          // (1 - s as sigmoid(-x): of a score near 1 a difference would leave nothing)
          onto = lane < k ? ds * s * sigmoid(-xs) : 0.0f;
        }
        if (lane < k) scatter[warp][key] = onto;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NJ; ++j) d[j] = own[j * kStep];
      }
      __syncwarp();
      if (lane < k) scatter[warp][key] = 0.0f;
      __syncwarp();
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
        const int e = lane + 32 * j;
        if (e < E) out[e] = from_float<T>(d[j]);
      }
    }
  }
}

// (A kernel, which the router's chains to, and no memset, which it would have to
// wait out: 65,536 tokens of 64 experts take 10.7 us against 14.3, 256 tokens on
// each of 8 ranks 5.0 against 8.2.  A cluster for the blocks of a rank, which
// read each other's counts, took 4.1 against 5.0 for 64 cheap tokens a rank, one
// launch instead of two, and 6.4 against 5.2 for dear ones; not kept.)
__global__ void clear_counts_kernel(unsigned long long* counts, int n) {
  chain();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) counts[i] = 0;
}

using RouteKernel = void (*)(RouteParams);

// Lanes and experts a lane for a call: few tokens, or many.  (Measured at 65,536
// tokens over 256 experts in 8 groups: 16 lanes x 16 experts with four blocks an
// SM 65 us, 8 x 32 with two or three 84, 32 x 8 73.)
constexpr int kManyNj = 16;
struct RouteShape {
  int lanes, nj;
};

template <typename T, bool kVec>
RouteKernel route_kernel_of(RouteShape f) {
  if (f.lanes == 4) return route_kernel<T, 4, kManyNj, kVec>;  // (many tokens)
  if (f.lanes == 8) return route_kernel<T, 8, kManyNj, kVec>;
  if (f.lanes == 16) return route_kernel<T, 16, kManyNj, kVec>;
  switch (f.nj) {
    case 1: return route_kernel<T, 32, 1, kVec>;
    case 2: return route_kernel<T, 32, 2, kVec>;
    case 4: return route_kernel<T, 32, 4, kVec>;
    case 8: return route_kernel<T, 32, 8, kVec>;
    case 16: return route_kernel<T, 32, 16, kVec>;
    default: return route_kernel<T, 32, 32, kVec>;
  }
}

template <typename T, bool kVec>
RouteKernel backward_kernel_of(int nj) {
  switch (nj) {
    case 1: return route_backward_kernel<T, 1, kVec>;
    case 2: return route_backward_kernel<T, 2, kVec>;
    case 4: return route_backward_kernel<T, 4, kVec>;
    case 8: return route_backward_kernel<T, 8, kVec>;
    case 16: return route_backward_kernel<T, 16, kVec>;
    default: return route_backward_kernel<T, 32, kVec>;
  }
}

template <typename T>
RouteKernel route_kernel_of(RouteShape f, bool vec, bool backward) {
  if (backward) return vec ? backward_kernel_of<T, true>(f.nj) : backward_kernel_of<T, false>(f.nj);
  return vec ? route_kernel_of<T, true>(f) : route_kernel_of<T, false>(f);
}

RouteKernel route_kernel_of(int dtype, RouteShape f, bool vec, bool backward) {
  if (dtype == A2AV_F32) return route_kernel_of<float>(f, vec, backward);
  if (dtype == A2AV_BF16) return route_kernel_of<__nv_bfloat16>(f, vec, backward);
  return route_kernel_of<__half>(f, vec, backward);
}

// Tokens from which on several share a warp (also where rows take no vectors:
// 65,536 tokens of 61 experts, bf16, 11.3 us against 25).
constexpr long long kManyTokens = 2048;

// The checks both calls share; fills what both need.
int route_params(a2av_handle* h, const a2av_route_t* c, const void* const* logits,
                 const int64_t* tokens, const int32_t* const* keys, const float* const* weights,
                 void* const* d_logits, RouteParams* P, RouteShape* shape, bool* vec, int* most) {
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
  bool aligned = true;
  long long all = 0;
  *most = 0;
  for (int r = 0; r < h->W; ++r) {
    const int64_t n = tokens[r];
    if (n < 0) return A2AV_ERR_INVALID_ARG;
    if (n > kMaxCount / c->topk) return A2AV_ERR_UNSUPPORTED;
    P->tokens[r] = (int)n;
    if (n == 0) continue;
    const void* d = d_logits != nullptr ? d_logits[r] : logits[r];
    all += n;
    if (logits[r] == nullptr || keys[r] == nullptr || weights[r] == nullptr || d == nullptr ||
        !aligned_to(logits[r], size) || !aligned_to(d, size) || !aligned_to(keys[r], 4) ||
        !aligned_to(weights[r], 4))
      return A2AV_ERR_INVALID_ARG;
    aligned = aligned && aligned_to(logits[r], 16) && aligned_to(d, 16);
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
  // A group's lanes, where they are a power of two of whole lanes.
  const auto group_lanes = [&](int nj) {
    const int lanes = group_size / nj;
    return group_size % nj == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  };
  shape->lanes = 32;
  shape->nj = 1;
  while (shape->nj * 32 < c->experts) shape->nj *= 2;
  if (d_logits == nullptr && all >= kManyTokens && c->experts <= 16 * kManyNj) {
    RouteShape many = {4, kManyNj};
    while (many.lanes * many.nj < c->experts) many.lanes *= 2;
    if (c->groups == 1 || group_lanes(many.nj) > 0) *shape = many;
  }
  P->group_lanes = group_lanes(shape->nj);
  // Vectors when every lane's run of NJ logits is whole and aligned: the row
  // is a multiple of a lane's vector, and the buffers are aligned.
  const int lane_bytes = shape->nj * size < 16 ? shape->nj * size : 16;
  *vec = aligned && (long long)c->experts * size % lane_bytes == 0;
  P->renormalise = c->renormalise != 0;
  P->scale = c->scale;
  P->status = h->d_status;
  return current_device(h);
}

// Blocks a rank: enough for every token to have its lanes, up to eight blocks an
// SM, or the four that the kernels of several tokens a warp have room for (53
// against 55 us at 65,536 tokens over 256 experts).
int route_blocks(const a2av_handle* h, int most, int lanes) {
  const int tokens = kRouteWarps * 32 / lanes;
  const int all = (most - 1) / tokens + 1;  // (a rank without tokens: 1)
  const int fit = ((lanes < 32 ? 4 : 8) * h->sms + h->W - 1) / h->W;
  return all < 1 ? 1 : all < fit ? all : fit;
}

}  // namespace

extern "C" int a2av_route(a2av_handle* h, const a2av_route_t* route,
                          const void* const* logits_ptrs, const int64_t* tokens_per_rank,
                          const float* bias_dev, int32_t* const* key_ptrs,
                          float* const* weight_ptrs, int64_t* counts_dev, void* stream) {
  RouteParams P;
  RouteShape shape;
  int most = 0;
  bool vec = false;
  const int rc = route_params(h, route, logits_ptrs, tokens_per_rank, key_ptrs, weight_ptrs,
                              nullptr, &P, &shape, &vec, &most);
  if (rc != A2AV_OK) return rc;
  if (!aligned_to(bias_dev, 4) || !aligned_to(counts_dev, 8)) return A2AV_ERR_INVALID_ARG;
  for (int r = 0; r < h->W; ++r) P.weight[r] = P.tokens[r] > 0 ? weight_ptrs[r] : nullptr;
  P.bias = bias_dev;
  P.counts = reinterpret_cast<unsigned long long*>(counts_dev);
  if (most == 0 && counts_dev == nullptr) return A2AV_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = route_blocks(h, most, shape.lanes);
  if (P.counts != nullptr && blocks > 1) {
    P.add_counts = 1;
    const int n = h->W * P.E, clear = (n + 255) / 256;
    if (launch_chained(clear_counts_kernel, dim3(clear < h->sms ? clear : h->sms), 256, 0, s, h->pdl,
                       P.counts, n) != cudaSuccess)
      return A2AV_ERR_CUDA;
  }
  const cudaError_t e =
      launch_chained(route_kernel_of(route->dtype, shape, vec, false), dim3(blocks, h->W),
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
  RouteShape shape;
  int most = 0;
  bool vec = false;
  const int rc = route_params(h, route, logits_ptrs, tokens_per_rank, key_ptrs, d_weight_ptrs,
                              d_logits_ptrs, &P, &shape, &vec, &most);
  if (rc != A2AV_OK) return rc;
  for (int r = 0; r < h->W; ++r) {
    P.d_weight[r] = P.tokens[r] > 0 ? d_weight_ptrs[r] : nullptr;
    P.d_logits[r] = P.tokens[r] > 0 ? d_logits_ptrs[r] : nullptr;
  }
  if (most == 0) return A2AV_OK;
  const cudaError_t e = launch_chained(route_kernel_of(route->dtype, shape, vec, true),
                                       dim3(route_blocks(h, most, 32), h->W), 32 * kRouteWarps, 0,
                                       static_cast<cudaStream_t>(stream), h->pdl, P);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return A2AV_ERR_CUDA;
  return A2AV_OK;
}
