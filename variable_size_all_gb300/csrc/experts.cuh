// experts.cuh -- the groups of rows that the experts' products work on: where
// each begins, and which tile of work belongs to which (device side), and the
// epilogue's activations.
#pragma once

#include "moe_device.cuh"

// Groups are numbered in the order of their rows: peer p, source rank r, local
// expert e -> (p * W + r) * K + e, its count at counts[r][p * K + e].
struct A2avGroups {
  const long long* counts;  // [W][W * K]
  long long cap[A2AV_MAX_RANKS];        // rows the peer's buffers hold
  int* status;
  int W, K;
};

// One call of the experts' products.
struct A2avExperts {
  A2avGroups g;
  const void* x[A2AV_MAX_RANKS];         // rows that are multiplied (forward: x; d_rows: dz)
  const void* w[A2AV_MAX_RANKS];         // [K][Z][D]
  const void* bias[A2AV_MAX_RANKS];
  const void* residual[A2AV_MAX_RANKS];
  void* out[A2AV_MAX_RANKS];
  void* pre[A2AV_MAX_RANKS];
  const void* dy[A2AV_MAX_RANKS];        // backward
  const void* pre_in[A2AV_MAX_RANKS];
  void* dz[A2AV_MAX_RANKS];
  void* d_w[A2AV_MAX_RANKS];
  void* d_bias[A2AV_MAX_RANKS];
  void* tails;               // workspace of the weights' gradient
  long long tail_rows;
  long long D, N, Z;
  int act, gated;
};

namespace {

using GroupParams = A2avGroups;
using ExpertParams = A2avExperts;

// The prefix sums over the groups' rows and tiles, kept in shared memory for
// every 2^shift-th group; the groups between two entries are walked.
constexpr int kEntries = 512;
struct GroupTable {
  int rows[kEntries + 1];
  int peer_base[kW + 1];  // rows before peer p
  long long warp_rows[32], warp_tiles[32];
  int shift, entries, bad;
};

// The tiles before every 2^shift-th group, for kernels whose tiles are cut
// from single groups.
struct GroupTiles {
  long long first[kEntries + 1];
};

// How a row's vectors are shared out: one warp takes them all, or, where there
// are fewer rows than warps, several take a run of them each (of 64 at least).
struct RowParts {
  int parts;
  __device__ __forceinline__ RowParts(int rows, int warps, int vectors)
      : parts(max(1, min(warps / max(rows, 1), (vectors + 63) / 64))) {}
  // the run of `vectors` that part i has
  __device__ __forceinline__ void run(int i, int vectors, int* from, int* to) const {
    const int len = (vectors + 32 * parts - 1) / (32 * parts) * 32;
    *from = min(i * len, vectors);
    *to = min(*from + len, vectors);
  }
};

struct GroupTile {
  int p, e;          // peer, local expert
  int rows;          // rows of the group
  long long first;   // its first row in the peer's buffers
  long long local;   // the tile's number within the group
};

__device__ __forceinline__ long long group_count(const GroupParams& G, int s) {
  const int E = G.W * G.K;
  const int p = s / E, in = s - p * E;
  const int r = in / G.K, e = in - r * G.K;
  return __ldcg(G.counts + (long long)r * E + p * G.K + e);
}

// Tiles of a group of n rows: `features` for each `tile_rows` of them.
__device__ __forceinline__ long long group_tiles(long long n, int tile_rows, int features) {
  return (n + tile_rows - 1) / tile_rows * features;
}

// By the whole block.  False (in every thread) when a count is negative or a
// peer's rows do not fit its buffers; block 0 then records A2AV_ERR_BAD_SPLITS.
__device__ bool build_groups(const GroupParams& G, GroupTable& g, GroupTiles* gt = nullptr,
                             int tile_rows = 1, int features = 1) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int E = G.W * G.K, n = G.W * E;
  if (tid == 0) {
    g.bad = 0;
    int shift = 0;
    while ((n + (1 << shift) - 1) >> shift > kEntries) ++shift;
    g.shift = shift;
    g.entries = (n + (1 << shift) - 1) >> shift;
  }
  __syncthreads();
  const int shift = g.shift, entries = g.entries;
  const int per = (entries + nt - 1) / nt;
  const int e0 = min(tid * per, entries), e1 = min(e0 + per, entries);
  const int s0 = min(e0 << shift, n), s1 = min(e1 << shift, n);
  long long rows = 0, tiles = 0, held[4];  // (the first four counts, for the second pass)
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) held[i] = s0 + i < s1 ? group_count(G, s0 + i) : 0;
  const auto count_of = [&](int s) {
    const int i = s - s0;
    return i == 0 ? held[0] : i == 1 ? held[1] : i == 2 ? held[2] : i == 3 ? held[3] : group_count(G, s);
  };
  for (int s = s0; s < s1; ++s) {
    const long long c = count_of(s);
    if (c < 0 || c > kMaxCount) {
      bad = true;
    } else {
      rows += c;
      tiles += group_tiles(c, tile_rows, features);
    }
  }
  if (bad) g.bad = 1;
  long long ir = rows, it = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(kAll, ir, o), b = __shfl_up_sync(kAll, it, o);
    if (lane >= o) {
      ir += a;
      it += b;
    }
  }
  if (lane == 31) {
    g.warp_rows[warp] = ir;
    g.warp_tiles[warp] = it;
  }
  __syncthreads();
  long long r0 = ir - rows, t0 = it - tiles;
  for (int w = 0; w < warp; ++w) {
    r0 += g.warp_rows[w];
    t0 += g.warp_tiles[w];
  }
  for (int s = s0; s < s1; ++s) {
    if ((s & ((1 << shift) - 1)) == 0) {
      g.rows[s >> shift] = (int)r0;
      if (gt != nullptr) gt->first[s >> shift] = t0;
    }
    if (r0 > kMaxCount) {  // more than all the buffers hold together
      g.bad = 1;
      break;
    }
    if (s % E == 0) g.peer_base[s / E] = (int)r0;
    const long long c = count_of(s);
    if (c < 0 || c > kMaxCount) break;
    r0 += c;
    t0 += group_tiles(c, tile_rows, features);
    if (s == n - 1) {
      if (r0 > kMaxCount) g.bad = 1;
      g.rows[entries] = (int)r0;
      if (gt != nullptr) gt->first[entries] = t0;
      g.peer_base[G.W] = (int)r0;
    }
  }
  __syncthreads();
  if (!g.bad && tid < G.W && g.peer_base[tid + 1] - g.peer_base[tid] > G.cap[tid]) g.bad = 1;
  __syncthreads();
  if (g.bad && blockIdx.x == 0 && tid == 0) note_error(G.status, A2AV_ERR_BAD_SPLITS);
  return !g.bad;
}

// The group that tile t (below the table's last entry) belongs to.
__device__ __forceinline__ GroupTile find_tile(const GroupParams& G, const GroupTable& g,
                                               const GroupTiles& gt, long long t, int tile_rows,
                                               int features) {
  int lo = 0, hi = g.entries;  // first[lo] <= t < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (gt.first[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  int s = lo << g.shift;
  long long first = g.rows[lo], at = gt.first[lo];
  long long c = g.shift == 0 ? g.rows[lo + 1] - first : group_count(G, s);
  while (true) {
    const long long more = group_tiles(c, tile_rows, features);
    if (t < at + more) break;
    at += more;
    first += c;
    c = group_count(G, ++s);
  }
  GroupTile x;
  const int E = G.W * G.K;
  x.p = s / E;
  x.e = s % G.K;
  x.rows = (int)c;
  x.first = first - g.peer_base[x.p];
  x.local = t - at;
  return x;
}

// First row (in its peer's buffers) and rows of group s.
__device__ __forceinline__ long long find_group(const GroupParams& G, const GroupTable& g, int s,
                                                int* rows) {
  long long first = g.rows[s >> g.shift];
  if (g.shift == 0) {
    *rows = (int)(g.rows[s + 1] - first);
    return first - g.peer_base[s / (G.W * G.K)];
  }
  for (int i = s >> g.shift << g.shift; i < s; ++i) first += group_count(G, i);
  *rows = (int)group_count(G, s);
  return first - g.peer_base[s / (G.W * G.K)];
}

// --------------------------------------------------------- activations --
// In 32 bits, with the hardware's approximate exponential and reciprocal (2^-22
// of their results, and what the rounding of a large argument makes of them: with
// SiLU and GELU up to 2^-17): a value is rounded to 8 or 11 bits right after.  Instructions
// count here: a warp of the epilogue has 128 values of a tile for each lane.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504f;

// Where exp(-z^2 / 2) and exp(-|z|) are 0 in 32 bits: beyond, a product with them
// takes this in place of |z|, or it would be infinity times 0 where |z| is infinite
// (a pre-activation out of 16 bits' range is saved as an infinity).  min and max
// drop a NaN, so each result has a factor in which z has not been through them.
constexpr float kFar = 16.0f, kFarExp = 128.0f;

// The normal distribution's upper tail at |z|, with *density = exp(-z^2 / 2); x is
// min(|z|, kFar): density * t P(t), t = 1 / (1 + 0.362 x).  The six powers and the
// 0.362 are a fit of erfc(x / sqrt 2) exp(x^2 / 2) / 2 over 0 <= x <= 13.5 with
// the least largest relative error, 7.4e-7 (1.03e-6 as evaluated in 32 bits): what
// 16 bits keep of z Phi(z) is right down to the smallest results, where the
// exponential's argument adds z^2 2^-24.  Kept as a tail, it costs no cancellation
// for negative z.  (The library's error function made the epilogue of a short
// contraction take longer than its products: 4864 rows, 2048 -> 7168, 100 us,
// 86 with SiLU.)
__device__ __forceinline__ float normal_tail(float z, float x, float* density) {
  const float t = reciprocal_fast(fmaf(0.362f, x, 1.0f));
  *density = exp2_fast(z * z * (-0.5f * kLog2e));
  float p = fmaf(t, 0.0480388328f, -0.180348456f);
  p = fmaf(t, p, 0.177071229f);
  p = fmaf(t, p, 0.0285236593f);
  p = fmaf(t, p, 0.139540434f);
  p = fmaf(t, p, 0.14266938f);
  p = fmaf(t, p, 0.144505292f);
  return t * p * *density;
}

__device__ __forceinline__ float act_fn(int a, float z) {
  switch (a) {
    case A2AV_ACT_RELU: return z < 0.0f ? 0.0f : z;  // (a NaN stays)
    case A2AV_ACT_GELU: {
      float density;
      const float x = fminf(fabsf(z), kFar);
      return fmaf(-x, normal_tail(z, x, &density), fmaxf(z, 0.0f));
    }
    case A2AV_ACT_SILU:
      return fmaxf(z, -kFarExp) * reciprocal_fast(1.0f + exp2_fast(z * -kLog2e));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(int a, float z) {
  switch (a) {
    case A2AV_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case A2AV_ACT_GELU: {
      float density;
      const float x = fminf(fabsf(z), kFar);
      const float q = normal_tail(z, x, &density);  // the slope at -|z|:
      const float low = fmaf(x * -0.39894228f, density, q);
      return z < 0.0f ? low : 1.0f - low;
    }
    case A2AV_ACT_SILU: {
      const float s = reciprocal_fast(1.0f + exp2_fast(z * -kLog2e));
      return s * fmaf(fminf(fmaxf(z, -kFarExp), kFarExp), 1.0f - s, 1.0f);
    }
    default: return 1.0f;
  }
}

// ----------------------------------------------------------- host side --
// Copies a list of W pointers (`need`: rows or experts of peer p want one).
inline bool take(const void** to, const void* const* from, int W, const int64_t* rows, int size) {
  for (int p = 0; p < W; ++p) {
    to[p] = from != nullptr && (rows == nullptr || rows[p] > 0) ? from[p] : nullptr;
    if (from != nullptr && (rows == nullptr || rows[p] > 0) && to[p] == nullptr) return false;
    if (!aligned_to(to[p], size)) return false;
  }
  return true;
}

inline bool take(void** to, void* const* from, int W, const int64_t* rows, int size) {
  return take(const_cast<const void**>(to), from, W, rows, size);
}

}  // namespace

// experts_mma.cu: the same products on the tensor cores.  `direction` 0: out =
// epilogue(x w^T); 1: out = x w, x being dz; 2: d_w = dy^T x.  False when the
// shape or a buffer is not one their copies can take (then nothing is
// launched); *error gets the launch's error.
__attribute__((visibility("hidden"))) bool a2av_expert_mma(a2av_handle* h, const A2avExperts& P,
                                                           int dtype, int direction,
                                                           cudaStream_t s, cudaError_t* error);

// Rows of the weights' gradient's packed remainders (see experts_mma.cu), at
// most; and their place: Z elements each for dz, then D each for x.
__attribute__((visibility("hidden"))) int64_t a2av_expert_tail_rows(int W, int K, int64_t rows);

// experts.cu: a call's groups and shape, checked; the buffers are still to be taken.
__attribute__((visibility("hidden"))) int a2av_expert_params(a2av_handle* h, const a2av_expert_t* c,
                                                             const int64_t* rows_per_peer,
                                                             const int64_t* counts, A2avExperts* P);
