// norm.cu -- the root-mean-square norm with the residual's addition (a2av_norm),
// its gradients, and packed rows (a2av_quantise, a2av_dequantise); the interface is
// in include/a2av_mx.h.
//
// All are bound by memory: what a row has is read once and written once.  Of 65,536
// rows of 7168 in bf16, at a copy rate of 6.68 TB/s: the norm with a residual, 8-bit results
// 529 to 543 us (91 to 93 %); its gradients, 618 to 640 us (88 to 91 %); rows to 8 bits 214 us (99 %), 131,072
// of them back 467 us (91 %); 458,752 rows of 2048 to 4 bits and back 785 us (91 %).
//
// The norm: a block (a warp, for short rows) takes a row, holds it in registers
// between its sums and its results, and goes on.  What decides is how much is in flight
// meanwhile: bulk copies bring the block's next two rows to shared memory (rows read when
// they are needed took 627 and 1441 us instead, cp.async by each thread 523 and 841, with two
// registers of addresses for each array in every thread), and the weight is read from L1
// for each row, because 32 registers less are a block more on an SM.  (A spill costs far more
// than a block: its loads miss the little L1 that the rows leave, 1730 us.  The gradients of
// rows above 8192 features spill all the same where a block needs 1024 threads, which leaves each
// 64 registers: f32, and rows that take no vectors.  8192 rows of 16,384 in f32 547 us, of
// 16,383 708, of 16,383 in bf16 517; floors 321, 321 and 161.)
//
// Instructions count as well: values are multiplied in pairs, magnitudes of 16-bit rows
// compared in pairs, ranks and slices followed without divisions.
#include "mma.cuh"
#include "mx_device.cuh"

#include <algorithm>
#include <cfloat>

namespace {

struct NormParams {
  const void* x[kW];         // backward: s
  const void* residual[kW];  // or NULL; backward: d_sums
  void* sums[kW];            // or NULL
  void* out[kW];             // y; backward: d_x
  void* plain[kW];           // y in the rows' type as well, or NULL
  const void* d_out[kW];     // backward: dy
  long long first[kW + 1];   // tokens before each rank's
  const float* weight;
  float* part;               // backward: [blocks][H], or NULL
  MxRow row;                 // of packed results
  int* status;
  int W, H;
  float eps, per_feature, per_feature_low;  // 1 / H, and what its rounding left
  int weight_aligned;        // to 16 bytes
};

// Token t of all ranks' (rank-major), in rank r or a later one.
__device__ __forceinline__ void find_rank(const long long* first, long long t, int* r) {
  while (first[*r + 1] <= t) ++*r;
}

// Sums of kSums values over a warp, or over the block: `shared` is not that of the
// row before, whose sums others may still be reading.
template <bool kWarp, int kSums>
__device__ __forceinline__ void row_sum(float (&x)[kSums], float (*shared)[kSums]) {
#pragma unroll
  for (int i = 0; i < kSums; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x[i] += __shfl_xor_sync(kAll, x[i], o);
  if constexpr (!kWarp) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < kSums; ++i) shared[warp][i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      x[i] = lane < warps ? shared[lane][i] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x[i] += __shfl_xor_sync(kAll, x[i], o);
    }
  }
}

// How a row lies on its threads: in vectors of 16 bytes, thread i having the vectors
// i, i + threads, ..., of these many values in all.  The backward pass keeps the weight's
// gradient of its values as well; rows that take no vectors are not fetched ahead, and want
// more threads instead (16,384 rows of 7161, bf16: the norm 226 us with 16 values a thread,
// 270 with 32; the gradients of 32,768 rows of 1001 80 us with 8, 92 with 16).
template <bool kAligned>
constexpr int kHeld = kAligned ? 32 : 16;
__host__ __device__ constexpr int held_backward(bool aligned, int size, int64_t H) {
  return aligned ? (size == 2 ? 32 : 16) : H <= 8192 ? 8 : 16;  // (1024 threads have 8192 or 16,384)
}

// Rows on their way to shared memory, by bulk copies, while others are worked on: two
// rows of `arrays` arrays of `bytes` each, for the block or for each of its warps.
struct Ahead {
  uint32_t place, bar;  // of the stage that is read next
  uint32_t step;        // bytes of a stage
  int turn, parity;
  bool lost;            // a copy has not come

  __device__ __forceinline__ uint32_t at(int stage) const { return place + (stage ? step : 0); }
  // By the thread that copies; a list of `count` arrays.
  __device__ __forceinline__ void expect(int stage, unsigned total) const {
    bar_arrive_tx(bar + 8 * stage, total);
  }
  __device__ __forceinline__ void fetch(int stage, int array, const void* from, unsigned bytes) const {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            at(stage) + array * bytes),
        "l"(from), "r"(bytes), "r"(bar + 8 * stage)
        : "memory");
  }
  __device__ __forceinline__ void wait() {
    if (!lost) lost = !bar_wait(bar + 8 * turn, parity);
  }
  __device__ __forceinline__ void next() {
    parity ^= turn;
    turn ^= 1;
  }
};

// A copy has not come: this is recorded, and what is in flight waited for, with a limit,
// before the block may leave.
__device__ __noinline__ void give_up(const Ahead& ahead, int* status) {
  note_error(status, A2AV_ERR_TIMEOUT);
  bar_wait(ahead.bar + 8 * ahead.turn, ahead.parity);
  bar_wait(ahead.bar + 8 * (ahead.turn ^ 1), ahead.parity ^ ahead.turn);
}

// A thread's U vectors of a row: from shared memory, where it has been fetched to `here`,
// from memory, or (kAligned false) the elements that it has instead.
template <typename T, bool kAhead, bool kAligned, int U, typename V>
__device__ __forceinline__ void take_row(V (&to)[U], uint32_t here, const T* row, int i0, int threads, int H) {
  if constexpr (!kAligned) {
    Loose<T>::load(to, row, i0 - threadIdx.x % 32, threads, H);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = i0 + u * threads;
      if (v * Pairs<T>::N >= H) continue;
      if constexpr (kAhead)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(to[u].w[0]), "=r"(to[u].w[1]), "=r"(to[u].w[2]), "=r"(to[u].w[3])
                     : "r"(here + 16 * v)
                     : "memory");
      else
        to[u] = reinterpret_cast<const V*>(row)[v];
    }
  }
}

// And back to memory.
template <typename T, bool kAligned, int U, typename V>
__device__ __forceinline__ void give_row(T* row, const V (&from)[U], int i0, int threads, int H) {
  if constexpr (!kAligned) {
    Loose<T>::store(row, from, i0 - threadIdx.x % 32, threads, H);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = i0 + u * threads;
      if (v * Pairs<T>::N < H) reinterpret_cast<V*>(row)[v] = from[u];
    }
  }
}

// Whether a thread has anything of a row in vector v, and the column of its value i there.
template <typename T, bool kVectors>
__device__ __forceinline__ bool has_part(int v, int H) {
  return (kVectors ? v : v - (int)(threadIdx.x % 32)) * Pairs<T>::N < H;
}
template <typename T, bool kVectors>
__device__ __forceinline__ int column_of(int v, int i) {
  return kVectors ? v * Pairs<T>::N + i : Loose<T>::element(v - threadIdx.x % 32, i);
}

// A token's place: its rank and its first element in the rank's buffers.
struct Token {
  int r;
  long long at;
};
template <typename T>
__device__ __forceinline__ const T* row_of(const void* const* list, const Token& t) {
  return static_cast<const T*>(list[t.r]) + t.at;
}
template <typename T>
__device__ __forceinline__ T* row_of(void* const* list, const Token& t) {
  return static_cast<T*>(list[t.r]) + t.at;
}
// Token g of all ranks', g being no smaller than the last one.
__device__ __forceinline__ void find_token(const NormParams& P, long long g, Token* t) {
  find_rank(P.first, g, &t->r);
  t->at = (g - P.first[t->r]) * P.H;
}

// The weight's values of vector v, zeros past the row.  They are read again for every
// row, from L1: in registers they would cost the block that an SM has beside this one.
template <typename T, bool kAligned, bool kVectors>
__device__ __forceinline__ void take_weight(float2 (&w)[Pairs<T>::N / 2], const NormParams& P, int v) {
  constexpr int N = Pairs<T>::N;
  const float* from = P.weight + v * N;
  if (kAligned || (kVectors && P.weight_aligned && v * N + N <= P.H)) {
#pragma unroll
    for (int i = 0; i < N / 2; i += 2)
      asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(w[i].x), "=f"(w[i].y), "=f"(w[i + 1].x), "=f"(w[i + 1].y)
                   : "l"(from + 2 * i));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const int a = column_of<T, kVectors>(v, 2 * i), b = column_of<T, kVectors>(v, 2 * i + 1);
      w[i].x = a < P.H ? P.weight[a] : 0.0f;
      w[i].y = b < P.H ? P.weight[b] : 0.0f;
    }
  }
}

// A value as a sum of two floats.  (The norm's codes, and their blocks' scales, go by
// which side of a border a value is on.  With what the last sums, the mean, the root and
// the two products after it round off kept, a result is mostly the exact one's rounding to
// 32 bits.  Of 7.05e9 values, 15 draws, 608 codes and 3 scales are not those of that
// rounding, against 1698 and 12 with 32 bits alone, for 8 of 543 us.  Codes rounded from
// 64 bits at once differ in 3371 against 3427: there the rounding to 32 bits decides.)
struct Two {
  float high, low;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two add_two(Two a, Two b) {
  const Two s = two_sum(a.high, b.high);
  const float low = s.low + (a.low + b.low), high = s.high + low;
  return isfinite(s.high) ? Two{high, low - (high - s.high)} : Two{s.high, 0.0f};
}
__device__ __forceinline__ Two lanes_sum(Two x, const int from) {
#pragma unroll
  for (int o = from; o > 0; o >>= 1)
    x = add_two(x, {__shfl_xor_sync(kAll, x.high, o), __shfl_xor_sync(kAll, x.low, o)});
  return x;
}

// The weight that what a value's rounding left is multiplied by: an infinite one's largest
// finite neighbour, so that the value's own product decides.
__device__ __forceinline__ float2 finite(float2 w) {
  float2 r;
  asm("min.xorsign.abs.f32 %0, %1, 0f7F7FFFFF;" : "=f"(r.x) : "f"(w.x));
  asm("min.xorsign.abs.f32 %0, %1, 0f7F7FFFFF;" : "=f"(r.y) : "f"(w.y));
  return r;
}

// The sum of x over a warp, or over the block (`shared` as in row_sum).  A block's first
// steps are between so many partial sums that their roundings average out.
template <bool kWarp, int kThreads>
__device__ __forceinline__ Two precise_sum(float2 x, Two* shared) {
  if constexpr (kWarp) return lanes_sum(add_two({x.x, 0.0f}, {x.y, 0.0f}), 16);
  float s = x.x + x.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  // (every lane ends up with the sum: they take the warps' in turn, several times over)
  constexpr int kMost = kThreads / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  if (lane == 0) shared[warp] = {s, 0.0f};
  __syncthreads();
  return lanes_sum(lane % kMost < warps ? shared[lane % kMost] : Two{0.0f, 0.0f}, kMost / 2);
}

// 1 / sqrt(mean + eps): what the first float is off, from its square.
__device__ __forceinline__ Two inverse_root(const NormParams& P, Two sum) {
  const float p = sum.high * P.per_feature;
  const float rest = fmaf(sum.high, P.per_feature, -p) + (sum.low * P.per_feature + sum.high * P.per_feature_low);
  const Two x = two_sum(p, P.eps);
  const float r = rsqrtf(x.high), t = x.high * r;
  const float off = fmaf(-t, r, 1.0f) - fmaf(x.high, r, -t) * r - (x.low + rest) * r * r;
  const float low = 0.5f * r * off;
  return {r, isfinite(low) ? low : 0.0f};  // (a mean of 0 or infinity)
}

template <typename T, bool kAligned, int kFormat, bool kWarp, int kThreads, bool kAhead>
__global__ void __maxnreg__(kThreads > 512 ? 64 : !kAligned ? 72 : sizeof(T) == 4 ? 128 : kAhead && !kWarp ? 80 : 96)
    norm_kernel(const __grid_constant__ NormParams P) {
  chain();
  using Q = Pairs<T>;
  using V = typename Q::Raw;
  using F = float2;
  constexpr int N = Q::N, U = kHeld<kAligned> / N, M = N / 2;
  extern __shared__ uint4 room[];
  __shared__ Two sums[2][kThreads / 32];
  __shared__ unsigned long long bars[kWarp ? 2 * kThreads / 32 : 2];
  // (rows that take no vectors have them for codes alone)
  constexpr bool kVectors = kAligned || kFormat != A2AV_PLAIN, kSpread = kVectors && !kAligned;
  __shared__ uint4 places[kSpread ? kThreads / 32 : 1][kSpread ? U : 1][32];
  uint4(*place)[32] = places[kSpread ? threadIdx.x / 32 : 0];
  const int threads = kWarp ? 32 : blockDim.x, i0 = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int nv = (P.H + N - 1) / N;
  // vectors of a packed row, zeros behind the row's own
  const int np = kFormat == A2AV_PLAIN ? nv : P.row.scales * (kMxBlock / N);
  const int per = kWarp ? blockDim.x / 32 : 1;
  const long long rows = P.first[P.W], by = (long long)gridDim.x * per;
  long long g = (long long)blockIdx.x * per + (kWarp ? threadIdx.x / 32 : 0);
  Ahead ahead;
  // (the thread that copies: the block's or the warp's first)
  const unsigned bytes = (unsigned)P.H * sizeof(T);
  const auto fetch = [&](int stage, const Token& t) {
    const bool more = P.residual[t.r] != nullptr;
    ahead.expect(stage, (more ? 2 : 1) * bytes);
    ahead.fetch(stage, 0, row_of<T>(P.x, t), bytes);
    if (more) ahead.fetch(stage, 1, row_of<T>(P.residual, t), bytes);
  };
  Token coming = {0, 0};
  if constexpr (kAhead) {
    const int own = kWarp ? threadIdx.x / 32 : 0;
    ahead.step = 2 * bytes;
    ahead.place = smem_addr(room) + own * 2 * ahead.step;
    ahead.bar = smem_addr(&bars[2 * own]);
    ahead.turn = ahead.parity = 0;
    ahead.lost = false;
    if (i0 == 0) {
      bar_init(ahead.bar, 1);
      bar_init(ahead.bar + 8, 1);
      bar_init_done();
      for (int i = 0; i < 2 && g + i * by < rows; ++i) {
        find_token(P, g + i * by, &coming);
        fetch(i, coming);
      }
    }
    __syncthreads();
  }
  Token t = {0, 0};
  for (int parity = 0; g < rows; g += by, parity ^= 1) {
    find_token(P, g, &t);
    T* kept = row_of<T>(P.sums, t);
    const bool add = P.residual[t.r] != nullptr, keep = P.sums[t.r] != nullptr;
    uint32_t here = 0;
    if constexpr (kAhead) {
      ahead.wait();
      here = ahead.at(ahead.turn);
    }
    V s[U], a[U];
    take_row<T, kAhead, kAligned>(s, here, row_of<T>(P.x, t), i0, threads, P.H);
    if (add) take_row<T, kAhead, kAligned>(a, here + bytes, row_of<T>(P.residual, t), i0, threads, P.H);
    F total2 = both(0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (has_part<T, kAligned>(i0 + u * threads, P.H)) {
        F f[M];
        Q::unpack(s[u], f);
        if (add) {
          F b[M];
          Q::unpack(a[u], b);
#pragma unroll
          for (int i = 0; i < M; ++i) f[i] = add2(f[i], b[i]);
          s[u] = Q::pack(f);
          Q::unpack(s[u], f);
        }
        F squares = mul2(f[0], f[0]);
#pragma unroll
        for (int i = 1; i < M; ++i) squares = fma2(f[i], f[i], squares);
        total2 = add2(total2, squares);
      }
    }
    if (keep) give_row<T, kAligned>(kept, s, i0, threads, P.H);
    if constexpr (kSpread) Loose<T>::spread(s, place);
    const Two total = precise_sum<kWarp, kThreads>(total2, sums[parity]);
    // (all threads have taken their part of the row: its place is free)
    if constexpr (kAhead) {
      if (kWarp) __syncwarp();
      if (i0 == 0 && g + 2 * by < rows && !ahead.lost) {
        find_token(P, g + 2 * by, &coming);
        fetch(ahead.turn, coming);
      }
      ahead.next();
    }
    const Two root = inverse_root(P, total);
    const F high = both(root.high), low = both(root.low);
    unsigned char* packed = nullptr;
    T* out = row_of<T>(kFormat == A2AV_PLAIN ? P.out : P.plain, t);
    const bool plain = kFormat == A2AV_PLAIN || P.plain[t.r] != nullptr;
    if constexpr (kFormat != A2AV_PLAIN)
      packed = static_cast<unsigned char*>(P.out[t.r]) + (g - P.first[t.r]) * P.row.bytes;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = i0 + u * threads;
      F f[M];
#pragma unroll
      for (int i = 0; i < M; ++i) f[i] = both(0.0f);
      if (has_part<T, kVectors>(v, P.H)) {
        F w[M];
        take_weight<T, kAligned, kVectors>(w, P, v);
        Q::unpack(s[u], f);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const F a = mul2(f[i], high), rest = fma2(f[i], low, fma2(f[i], high, minus(a)));
          f[i] = fma2(a, w[i], mul2(rest, kFormat == A2AV_PLAIN ? finite(w[i]) : w[i]));
        }
      }
      const float top = kFormat == A2AV_PLAIN ? 0.0f : largest(f);
      if (plain) {
        // (of a packed row's block nothing is left where a weight is infinite, so that the plain
        // row alone is put right: finite() for every value cost 5 us of 533)
        if (kFormat != A2AV_PLAIN && isnan(top)) {
          F w[M], x[M];
          take_weight<T, kAligned, kVectors>(w, P, v);
          Q::unpack(s[u], x);
#pragma unroll
          for (int i = 0; i < M; ++i) {
            const F y = mul2(mul2(x[i], high), w[i]);
            if (isinf(y.x)) f[i].x = y.x;
            if (isinf(y.y)) f[i].y = y.y;
          }
        }
        V y[1] = {Q::pack(f)};
        if constexpr (kSpread) Loose<T>::gather(y, place);
        give_row<T, kAligned>(out, y, v, 0, P.H);
      }
      if constexpr (kFormat != A2AV_PLAIN) {
        // whether one of the values of these bits is larger than them, rounded down
        const auto above = [&](unsigned bits) {
          bool any = false;
          if (has_part<T, kVectors>(v, P.H)) {
            F w[M], x[M];
            take_weight<T, kAligned, kVectors>(w, P, v);
            Q::unpack(s[u], x);
#pragma unroll
            for (int i = 0; i < M; ++i) {
              const F a = mul2(x[i], high), rest = fma2(x[i], low, fma2(x[i], high, minus(a)));
              const F c = mul2(rest, w[i]), y = fma2(a, w[i], c), off = add2(fma2(a, w[i], minus(y)), c);
              any = any || (__float_as_uint(fabsf(y.x)) == bits && (y.x > 0.0f ? off.x : -off.x) > 0.0f) ||
                    (__float_as_uint(fabsf(y.y)) == bits && (y.y > 0.0f ? off.y : -off.y) > 0.0f);
            }
          }
          return any;
        };
        if (u * threads < np)
          mx_store<kFormat, N>(packed, P.row.values, v, f, __float_as_uint(top), v < np, above);
      }
    }
    if constexpr (kFormat != A2AV_PLAIN) {
      const int used = P.row.values + P.row.scales;
      if (used + i0 < P.row.bytes) packed[used + i0] = 0;  // (31 at most)
    }
  }
  if constexpr (kAhead)
    if (ahead.lost) give_up(ahead, P.status);
}

// d_x, and a block's part of the weight's gradient, kept in registers over its
// rows.
template <typename T, bool kAligned, int kValues, bool kWarp, int kThreads, bool kAhead>
__global__ void __maxnreg__(kThreads > 512 ? 64 : 128)
    norm_backward_kernel(const __grid_constant__ NormParams P) {
  chain();
  using Q = Pairs<T>;
  using V = typename Q::Raw;
  using F = float2;
  constexpr int N = Q::N, U = kValues / N, M = N / 2;
  extern __shared__ uint4 room[];
  __shared__ float sums[2][kThreads / 32][2];
  __shared__ unsigned long long bars[kWarp ? 2 * kThreads / 32 : 2];
  const int threads = kWarp ? 32 : blockDim.x, i0 = kWarp ? threadIdx.x % 32 : threadIdx.x;
  const int per = kWarp ? blockDim.x / 32 : 1;
  const long long rows = P.first[P.W], by = (long long)gridDim.x * per;
  long long g = (long long)blockIdx.x * per + (kWarp ? threadIdx.x / 32 : 0);
  Ahead ahead;
  // (the thread that copies: the block's or the warp's first)
  const unsigned bytes = (unsigned)P.H * sizeof(T);
  const auto fetch = [&](int stage, const Token& t) {
    const bool more = P.residual[t.r] != nullptr;
    ahead.expect(stage, (more ? 3 : 2) * bytes);
    ahead.fetch(stage, 0, row_of<T>(P.x, t), bytes);
    ahead.fetch(stage, 1, row_of<T>(P.d_out, t), bytes);
    if (more) ahead.fetch(stage, 2, row_of<T>(P.residual, t), bytes);
  };
  Token coming = {0, 0};
  if constexpr (kAhead) {
    const int own = kWarp ? threadIdx.x / 32 : 0;
    ahead.step = 3 * bytes;
    ahead.place = smem_addr(room) + own * 2 * ahead.step;
    ahead.bar = smem_addr(&bars[2 * own]);
    ahead.turn = ahead.parity = 0;
    ahead.lost = false;
    if (i0 == 0) {
      bar_init(ahead.bar, 1);
      bar_init(ahead.bar + 8, 1);
      bar_init_done();
      for (int i = 0; i < 2 && g + i * by < rows; ++i) {
        find_token(P, g + i * by, &coming);
        fetch(i, coming);
      }
    }
    __syncthreads();
  }
  Token t = {0, 0};
  F dw[U][M];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < M; ++i) dw[u][i] = both(0.0f);
  for (int parity = 0; g < rows; g += by, parity ^= 1) {
    find_token(P, g, &t);
    T* out = row_of<T>(P.out, t);
    const bool add = P.residual[t.r] != nullptr;
    uint32_t here = 0;
    if constexpr (kAhead) {
      ahead.wait();
      here = ahead.at(ahead.turn);
    }
    V s[U], d[U], a[U];
    take_row<T, kAhead, kAligned>(s, here, row_of<T>(P.x, t), i0, threads, P.H);
    take_row<T, kAhead, kAligned>(d, here + bytes, row_of<T>(P.d_out, t), i0, threads, P.H);
    if (add) take_row<T, kAhead, kAligned>(a, here + 2 * bytes, row_of<T>(P.residual, t), i0, threads, P.H);
    F squares = both(0.0f), products = both(0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (has_part<T, kAligned>(i0 + u * threads, P.H)) {
        F f[M], e[M], w[M];
        take_weight<T, kAligned, kAligned>(w, P, i0 + u * threads);
        Q::unpack(s[u], f);
        Q::unpack(d[u], e);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          squares = fma2(f[i], f[i], squares);
          products = fma2(f[i], mul2(e[i], w[i]), products);
        }
      }
    float total[2] = {squares.x + squares.y, products.x + products.y};
    row_sum<kWarp, 2>(total, sums[parity]);
    // (all threads have taken their part of the row: its place is free)
    if constexpr (kAhead) {
      if (kWarp) __syncwarp();
      if (i0 == 0 && g + 2 * by < rows && !ahead.lost) {
        find_token(P, g + 2 * by, &coming);
        fetch(ahead.turn, coming);
      }
      ahead.next();
    }
    const float one = rsqrtf(fmaf(total[0], P.per_feature, P.eps));
    // (1 / length^2 may not fit where the product does; of an infinite length nothing is left)
    const F scale = both(one), along = both(one == 0.0f ? 0.0f : -one * (one * (total[1] * P.per_feature)));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = i0 + u * threads;
      F f[M], e[M], y[M], w[M];
      if (has_part<T, kAligned>(v, P.H)) {
        take_weight<T, kAligned, kAligned>(w, P, v);
        Q::unpack(s[u], f);
        Q::unpack(d[u], e);
        if (add) Q::unpack(a[u], y);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          dw[u][i] = fma2(e[i], mul2(f[i], scale), dw[u][i]);
          const F z = fma2(f[i], along, mul2(e[i], w[i]));
          y[i] = add ? fma2(z, scale, y[i]) : mul2(z, scale);
        }
      }
      a[u] = Q::pack(y);
    }
    give_row<T, kAligned>(out, a, i0, threads, P.H);
  }
  if constexpr (kAhead)
    if (ahead.lost) give_up(ahead, P.status);
  if (P.part == nullptr) return;
  float* part = P.part + (long long)blockIdx.x * P.H;
  if constexpr (kWarp) {  // the block's warps one after the other
    __shared__ float all[32 * U * N];
    for (int k = 0; k < per; ++k) {
      if (threadIdx.x / 32 == k)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float* at = all + column_of<T, kAligned>(i0 + u * 32, i);
            const float x = value_of(dw[u], i);
            *at = k == 0 ? x : *at + x;
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < P.H; c += blockDim.x) part[c] = all[c];
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = column_of<T, kAligned>(i0 + u * threads, i);
        if (c < P.H) part[c] = value_of(dw[u], i);
      }
  }
}

// The blocks' parts of 32 columns, summed by 32 warps and joined (304 parts of 7168: 7 us
// of the 620).  The order is that of the blocks, which go by the sizes alone.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* part, int blocks, int H,
                                                           float* d_weight) {
  chain();
  __shared__ float sums[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (c < H)
#pragma unroll 4
    for (int b = warp; b < blocks; b += 32) sum += part[(long long)b * H + c];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < H) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sums[i][lane];
    d_weight[c] = sum;
  }
}

// ---------------------------------------------------------- packed rows --
struct PackParams {
  const void* from[kW];
  void* to[kW];
  long long first[kW + 1];  // rows before each rank's, as many as the buffers hold
  const long long* splits;  // S [W][W]: the rows that are there; or NULL, all of them
  int* status;
  MxRow row;
  int D, W;
};

// Rows before each rank's that are worked on, by the whole block; false (in every
// thread) and the status word set where S is not valid.
__device__ __forceinline__ bool count_received(const PackParams& P, long long (&first)[kW + 1]) {
  __shared__ int bad;
  const int tid = threadIdx.x, W = P.W;
  __shared__ long long rows[kW];
  if (tid == 0) bad = 0;
  __syncthreads();
  if (tid < W) {
    long long n = 0;
    const long long most = P.first[tid + 1] - P.first[tid];
    for (int r = 0; r < W; ++r) {
      const long long s = __ldcg(P.splits + r * W + tid);
      if (s < 0 || s > most - n) bad = 1;
      n = s < 0 || s > most - n ? n : n + s;
    }
    rows[tid] = n;
  }
  __syncthreads();
  if (tid <= W) {
    long long at = 0;
    for (int p = 0; p < tid; ++p) at += rows[p];
    first[tid] = at;
  }
  __syncthreads();
  if (bad && blockIdx.x == 0 && tid == 0) note_error(P.status, A2AV_ERR_BAD_SPLITS);
  return !bad;
}

constexpr int kPackThreads = 256;

// The rows' slices, shared out among all warps; a warp's next is found without a
// division.
struct Slice {
  long long t;  // row
  int slice;
};
struct Slices {
  long long rows, t_on;
  int slices, slice_on;
  __device__ __forceinline__ Slices(long long rows, int slices) : rows(rows), slices(slices) {
    const long long warps = (long long)gridDim.x * (kPackThreads / 32);
    t_on = warps / slices;
    slice_on = (int)(warps - t_on * slices);
  }
  __device__ __forceinline__ Slice first() const {
    const long long g = (long long)blockIdx.x * (kPackThreads / 32) + threadIdx.x / 32;
    return {g / slices, (int)(g % slices)};
  }
  __device__ __forceinline__ void next(Slice* at) const {
    at->t += t_on;
    at->slice += slice_on;
    if (at->slice >= slices) {
      at->slice -= slices;
      ++at->t;
    }
  }
};

// The bits, in 32, of the largest magnitude of a vector: of pairs of 16 bits by
// one instruction each.
template <typename T>
__device__ __forceinline__ unsigned top_bits(const typename Pairs<T>::Raw& r, const float2 (&f)[Pairs<T>::N / 2]) {
  if constexpr (sizeof(T) == 2) {
    using T2 = std::conditional_t<__is_same(T, __half), __half2, __nv_bfloat162>;
    T2 m = __habs2(reinterpret_cast<const T2&>(r.w[0]));
#pragma unroll
    for (int i = 1; i < Pairs<T>::N / 2; ++i) m = __hmax2_nan(m, __habs2(reinterpret_cast<const T2&>(r.w[i])));
    return __float_as_uint(to_float(__hmax_nan(m.x, m.y))) & 0x7fffffffu;
  } else {
    return __float_as_uint(largest(f));
  }
}

// (either stays in its own kind of memory)
template <bool kReceived>
__device__ __forceinline__ const auto& firsts(const PackParams& P, const long long (&received)[kReceived ? kW + 1 : 1]) {
  if constexpr (kReceived)
    return received;
  else
    return P.first;
}

constexpr int kPackVectors = 4;  // of a lane at a time

// A warp takes 32 x kPackVectors neighbouring vectors of a row.
template <typename T, bool kAligned, int kFormat, bool kReceived>
__global__ void __launch_bounds__(kPackThreads) quantise_kernel(const __grid_constant__ PackParams P) {
  chain();
  using Q = Pairs<T>;
  constexpr int N = Q::N, U = kPackVectors;
  __shared__ uint4 places[kAligned ? 1 : kPackThreads / 32][kAligned ? 1 : U][32];
  const int lane = threadIdx.x % 32;
  const int nv = (P.D + N - 1) / N, np = P.row.scales * (kMxBlock / N);
  __shared__ long long received[kReceived ? kW + 1 : 1];
  if constexpr (kReceived)
    if (!count_received(P, received)) return;
  const auto& first = firsts<kReceived>(P, received);
  const Slices cut(first[P.W], (np + 32 * U - 1) / (32 * U));
  int r = 0;
  for (Slice at = cut.first(); at.t < cut.rows; cut.next(&at)) {
    find_rank(first, at.t, &r);
    const long long t = at.t - first[r];
    const int v0 = at.slice * (32 * U) + lane;
    const T* x = static_cast<const T*>(P.from[r]) + t * P.D;
    unsigned char* to = static_cast<unsigned char*>(P.to[r]) + t * P.row.bytes;
    typename Q::Raw s[U];
    if constexpr (kAligned) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + 32 * u < nv) s[u] = reinterpret_cast<const typename Q::Raw*>(x)[v0 + 32 * u];
    } else {
      Loose<T>::load(s, x, v0 - lane, 32, P.D);
      Loose<T>::spread(s, places[threadIdx.x / 32]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 32 * u;
      float2 f[N / 2];
      unsigned top = 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) f[i] = both(0.0f);
      if (v < nv) {
        Q::unpack(s[u], f);
        top = top_bits<T>(s[u], f);
      }
      if (v - lane < np) mx_store<kFormat, N>(to, P.row.values, v, f, top, v < np, Exact());
    }
    const int used = P.row.values + P.row.scales;
    if (at.slice == cut.slices - 1 && used + lane < P.row.bytes) to[used + lane] = 0;
  }
}

template <typename T, bool kAligned, int kFormat, bool kReceived>
__global__ void __launch_bounds__(kPackThreads) dequantise_kernel(const __grid_constant__ PackParams P) {
  chain();
  using Q = Pairs<T>;
  constexpr int N = Q::N, U = kPackVectors, kBits = kFormat == A2AV_MXFP8 ? 8 : 4;
  __shared__ uint4 places[kAligned ? 1 : kPackThreads / 32][kAligned ? 1 : U][32];
  const int lane = threadIdx.x % 32;
  const int nv = (P.D + N - 1) / N;
  __shared__ long long received[kReceived ? kW + 1 : 1];
  if constexpr (kReceived)
    if (!count_received(P, received)) return;
  const auto& first = firsts<kReceived>(P, received);
  const Slices cut(first[P.W], (nv + 32 * U - 1) / (32 * U));
  int r = 0;
  for (Slice at = cut.first(); at.t < cut.rows; cut.next(&at)) {
    find_rank(first, at.t, &r);
    const long long t = at.t - first[r];
    const int v0 = at.slice * (32 * U) + lane;
    const unsigned char* from = static_cast<const unsigned char*>(P.from[r]) + t * P.row.bytes;
    T* out = static_cast<T*>(P.to[r]) + t * P.D;
    unsigned w[U][N * kBits >= 32 ? N * kBits / 32 : 1], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 32 * u;
      s[u] = 0;
#pragma unroll
      for (unsigned& x : w[u]) x = 0;
      if (v < nv) {
        s[u] = from[P.row.values + v / (kMxBlock / N)];
        if constexpr (N * kBits == 64) {
          const uint2 c = reinterpret_cast<const uint2*>(from)[v];
          w[u][0] = c.x;
          w[u][1] = c.y;
        } else if constexpr (N * kBits == 32) {
          w[u][0] = reinterpret_cast<const unsigned*>(from)[v];
        } else {
          w[u][0] = reinterpret_cast<const unsigned short*>(from)[v];
        }
      }
    }
    typename Q::Raw values[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float2 by = both(mx_scale_value(s[u]));
      float2 f[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const unsigned c = w[u][2 * i * kBits / 32] >> (2 * i * kBits % 32);
        f[i] = mul2(kBits == 8 ? e4m3_values(c) : e2m1_values(c), by);
      }
      values[u] = Q::pack(f);
    }
    if constexpr (!kAligned) Loose<T>::gather(values, places[threadIdx.x / 32]);
    give_row<T, kAligned>(out, values, v0, 32, P.D);
  }
}

// ------------------------------------------------------------ host side --
// Copies a list of W pointers of ranks that have rows; the bits below their common
// alignment go to *low.
bool take_rows(const void** to, const void* const* from, int W, const int64_t* rows, int size,
               uintptr_t* low) {
  for (int r = 0; r < W; ++r) {
    to[r] = rows[r] > 0 ? from[r] : nullptr;
    if ((rows[r] > 0 && to[r] == nullptr) || !aligned_to(to[r], size)) return false;
    *low |= (uintptr_t)to[r];
  }
  return true;
}

bool take_rows(void** to, void* const* from, int W, const int64_t* rows, int size, uintptr_t* low) {
  return take_rows(const_cast<const void**>(to), from, W, rows, size, low);
}

// Rows before each rank's.
int count_rows(const a2av_handle* h, const int64_t* rows, long long* first) {
  for (int r = 0; r < h->W; ++r) {
    if (rows[r] < 0) return A2AV_ERR_INVALID_ARG;
    if (rows[r] > kMaxCount - first[r]) return A2AV_ERR_UNSUPPORTED;
    first[r + 1] = first[r] + rows[r];
  }
  return A2AV_OK;
}

bool is_packed(int format) { return format == A2AV_MXFP8 || format == A2AV_MXFP4; }

constexpr int kNormParts = 1024;  // most blocks that keep a part of the weight's gradient

using NormKernel = void (*)(NormParams);

// How a norm's rows are shared out: a warp a row where it can
// hold one, else a block of up to 256, 512 or 1024 threads.
struct NormForm {
  bool aligned, warp, ahead;
  int threads, most;  // of a block, and what its kernel is made for
  int held;           // values a thread has room for
};

NormForm norm_form(int64_t H, int size, uintptr_t low, long long rows, int sms, bool backward) {
  NormForm f;
  f.aligned = low % 16 == 0 && H * size % 16 == 0;
  f.ahead = false;
  const int n = 16 / size, nv = ((int)H + n - 1) / n;
  int held = backward ? held_backward(f.aligned, size, H) : f.aligned ? kHeld<true> : kHeld<false>;
  f.held = held;
  held /= n;
  f.warp = nv <= 32 * held;
  f.threads = 256;
  if (!f.warp) {
    // few rows: more threads a row, with less to do each
    while (rows < 2 * sms && held > 1 && (nv + held / 2 - 1) / (held / 2) <= 512) held /= 2;
    f.threads = ((nv + held - 1) / held + 31) / 32 * 32;
  }
  f.most = f.threads <= 256 ? 256 : f.threads <= 512 ? 512 : 1024;
  return f;
}

template <typename T, int kFormat>
NormKernel norm_kernel_of(const NormForm& f) {
  if (f.ahead) {
    if (f.warp) return norm_kernel<T, true, kFormat, true, 256, true>;
    return f.most == 256 ? norm_kernel<T, true, kFormat, false, 256, true>
                         : norm_kernel<T, true, kFormat, false, 512, true>;
  }
  if (f.aligned)
    return f.warp ? norm_kernel<T, true, kFormat, true, 256, false> : norm_kernel<T, true, kFormat, false, 512, false>;
  if (f.most > 512) return norm_kernel<T, false, kFormat, false, 1024, false>;
  return f.warp ? norm_kernel<T, false, kFormat, true, 256, false> : norm_kernel<T, false, kFormat, false, 512, false>;
}

template <typename T>
NormKernel norm_kernel_of(int format, const NormForm& f) {
  if (format == A2AV_MXFP8) return norm_kernel_of<T, A2AV_MXFP8>(f);
  return format == A2AV_MXFP4 ? norm_kernel_of<T, A2AV_MXFP4>(f) : norm_kernel_of<T, A2AV_PLAIN>(f);
}

template <typename T>
NormKernel norm_backward_kernel_of(const NormForm& f) {
  constexpr int kOwn = held_backward(true, sizeof(T), 0);
  if (f.ahead) {
    if (f.warp) return norm_backward_kernel<T, true, kOwn, true, 256, true>;
    return f.most == 256 ? norm_backward_kernel<T, true, kOwn, false, 256, true>
                         : norm_backward_kernel<T, true, kOwn, false, 512, true>;
  }
  if (f.aligned) {
    if constexpr (sizeof(T) == 4)  // (of 16 bits 512 threads hold any row)
      if (f.most > 512) return norm_backward_kernel<T, true, kOwn, false, 1024, false>;
    return f.warp ? norm_backward_kernel<T, true, kOwn, true, 256, false>
                  : norm_backward_kernel<T, true, kOwn, false, 512, false>;
  }
  if (f.held == 16) return norm_backward_kernel<T, false, 16, false, 1024, false>;
  if (f.most > 512) return norm_backward_kernel<T, false, 8, false, 1024, false>;
  return f.warp ? norm_backward_kernel<T, false, 8, true, 256, false>
                : norm_backward_kernel<T, false, 8, false, 512, false>;
}

NormKernel norm_kernel_of(int dtype, int format, const NormForm& f) {
  if (dtype == A2AV_F32) return norm_kernel_of<float>(format, f);
  return dtype == A2AV_BF16 ? norm_kernel_of<__nv_bfloat16>(format, f) : norm_kernel_of<__half>(format, f);
}

NormKernel norm_backward_kernel_of(int dtype, const NormForm& f) {
  if (dtype == A2AV_F32) return norm_backward_kernel_of<float>(f);
  return dtype == A2AV_BF16 ? norm_backward_kernel_of<__nv_bfloat16>(f) : norm_backward_kernel_of<__half>(f);
}

constexpr size_t kMostRoom = 200 << 10;  // shared memory that a block fetches rows to

// Launches the kernel that kernel_of(form) is, whose rows take `row_bytes` of all arrays
// together.  The blocks are as many as the GPU holds, and not more than the rows need
// or `limit`; where they take several rows each, they fetch them ahead.
template <typename K>
cudaError_t launch_norm(const a2av_handle* h, K kernel_of, NormForm f, int row_bytes, long long rows,
                        long long limit, const NormParams& P, cudaStream_t s, unsigned* blocks) {
  const long long per = f.warp ? f.threads / 32 : 1, want = (rows + per - 1) / per;
  NormKernel kernel = kernel_of(f);
  int fit = 0;
  size_t room = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, f.threads, 0);
  if (e != cudaSuccess) return e;
  const size_t two_rows = (size_t)2 * per * row_bytes;
  if (f.aligned && f.most <= 512 && want > (long long)fit * h->sms && two_rows <= kMostRoom) {
    f.ahead = true;
    kernel = kernel_of(f);
    room = two_rows;
    // (the most that any call asks for, and never less: the limit is the kernel's, which
    // another thread may be about to launch with wider rows)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostRoom);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, f.threads, room);
    if (e != cudaSuccess) return e;
  }
  long long most = (long long)fit * h->sms;
  if (most > limit) most = limit;
  *blocks = (unsigned)(want < most ? want : most);
  return launch_chained(kernel, dim3(*blocks), f.threads, room, s, h->pdl, P);
}

int norm_ok(const a2av_handle* h, int64_t features, int dtype, float eps, const void* x,
            const int64_t* tokens, const float* weight, const void* out) {
  if (h == nullptr || x == nullptr || tokens == nullptr || weight == nullptr || out == nullptr ||
      features < 1 || dtype_bytes(dtype) == 0 || !(eps >= 0.0f) || eps > FLT_MAX || !aligned_to(weight, 4))
    return A2AV_ERR_INVALID_ARG;
  return features > A2AV_MAX_NORM_FEATURES ? A2AV_ERR_UNSUPPORTED : A2AV_OK;
}

using PackKernel = void (*)(PackParams);

struct PackForm {
  bool aligned, back, received;
};

template <typename T, int kFormat, bool kReceived>
PackKernel pack_kernel_of(const PackForm& f) {
  if (f.back)
    return f.aligned ? dequantise_kernel<T, true, kFormat, kReceived> : dequantise_kernel<T, false, kFormat, kReceived>;
  return f.aligned ? quantise_kernel<T, true, kFormat, kReceived> : quantise_kernel<T, false, kFormat, kReceived>;
}

template <typename T>
PackKernel pack_kernel_of(int format, const PackForm& f) {
  if (format == A2AV_MXFP8)
    return f.received ? pack_kernel_of<T, A2AV_MXFP8, true>(f) : pack_kernel_of<T, A2AV_MXFP8, false>(f);
  return f.received ? pack_kernel_of<T, A2AV_MXFP4, true>(f) : pack_kernel_of<T, A2AV_MXFP4, false>(f);
}

// Both directions; `plain` and `packed` are the buffers' lists.
int pack_call(a2av_handle* h, int64_t features, int dtype, int format, const void* const* plain,
              const int64_t* rows, const int64_t* splits, const void* const* packed, bool back, void* stream) {
  const int size = dtype_bytes(dtype);
  if (h == nullptr || plain == nullptr || rows == nullptr || packed == nullptr || features < 1 ||
      size == 0 || !is_packed(format) || !aligned_to(splits, 8))
    return A2AV_ERR_INVALID_ARG;
  if (features > A2AV_MAX_MX_FEATURES) return A2AV_ERR_UNSUPPORTED;
  PackParams P;
  std::memset(&P, 0, sizeof(P));
  int rc = count_rows(h, rows, P.first);
  if (rc != A2AV_OK) return rc;
  uintptr_t low = (uintptr_t)(features * size), other = 0;
  const void** from = P.from;
  const void** to = const_cast<const void**>(P.to);
  if (!take_rows(back ? to : from, plain, h->W, rows, size, &low) ||
      !take_rows(back ? from : to, packed, h->W, rows, 16, &other))
    return A2AV_ERR_INVALID_ARG;
  rc = current_device(h);
  if (rc != A2AV_OK) return rc;
  if (P.first[h->W] == 0 && splits == nullptr) return A2AV_OK;  // (splits are checked all the same)
  P.W = h->W;
  P.D = (int)features;
  P.splits = reinterpret_cast<const long long*>(splits);
  P.status = h->d_status;
  P.row = mx_row(features, format);
  const PackForm form = {low % 16 == 0, back, splits != nullptr};
  const PackKernel kernel = dtype == A2AV_F32    ? pack_kernel_of<float>(format, form)
                            : dtype == A2AV_BF16 ? pack_kernel_of<__nv_bfloat16>(format, form)
                                                 : pack_kernel_of<__half>(format, form);
  int fit = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, kPackThreads, 0) != cudaSuccess)
    return A2AV_ERR_CUDA;
  const long long vectors = (features * size + 15) / 16, warps = kPackThreads / 32;
  const long long slice = 32 * kPackVectors;
  const long long slices = (vectors + slice - 1) / slice;
  const long long want = std::max(1LL, (P.first[h->W] * slices + warps - 1) / warps), most = (long long)fit * h->sms;
  const cudaError_t e = launch_chained(kernel, dim3((unsigned)(want < most ? want : most)), kPackThreads, 0,
                                       static_cast<cudaStream_t>(stream), h->pdl, P);
  return e != cudaSuccess || cudaGetLastError() != cudaSuccess ? A2AV_ERR_CUDA : A2AV_OK;
}

}  // namespace

extern "C" int64_t a2av_mx_row_bytes(int64_t features, int format) {
  if (features < 1 || features > A2AV_MAX_MX_FEATURES || !is_packed(format)) return -1;
  return mx_row(features, format).bytes;
}

extern "C" int a2av_norm(a2av_handle* h, int64_t features, int dtype, int format, float eps,
                         const void* const* x_ptrs, const int64_t* tokens_per_rank,
                         const float* weight_dev, const void* const* residual_ptrs,
                         void* const* sum_ptrs, void* const* out_ptrs, void* const* plain_ptrs,
                         void* stream) {
  int rc = norm_ok(h, features, dtype, eps, x_ptrs, tokens_per_rank, weight_dev, out_ptrs);
  if (rc != A2AV_OK) return rc;
  if ((format != A2AV_PLAIN && !is_packed(format)) || (format == A2AV_PLAIN && plain_ptrs != nullptr))
    return A2AV_ERR_INVALID_ARG;
  NormParams P;
  std::memset(&P, 0, sizeof(P));
  rc = count_rows(h, tokens_per_rank, P.first);
  if (rc != A2AV_OK) return rc;
  const int W = h->W, size = dtype_bytes(dtype);
  uintptr_t low = (uintptr_t)weight_dev, other = 0;
  if (!take_rows(P.x, x_ptrs, W, tokens_per_rank, size, &low) ||
      (residual_ptrs != nullptr && !take_rows(P.residual, residual_ptrs, W, tokens_per_rank, size, &low)) ||
      (sum_ptrs != nullptr && !take_rows(P.sums, sum_ptrs, W, tokens_per_rank, size, &low)) ||
      !take_rows(P.out, out_ptrs, W, tokens_per_rank, format == A2AV_PLAIN ? size : 16,
                 format == A2AV_PLAIN ? &low : &other) ||
      (plain_ptrs != nullptr && !take_rows(P.plain, plain_ptrs, W, tokens_per_rank, size, &low)))
    return A2AV_ERR_INVALID_ARG;
  rc = current_device(h);
  if (rc != A2AV_OK) return rc;
  const long long rows = P.first[W];
  if (rows == 0) return A2AV_OK;
  P.weight = weight_dev;
  P.weight_aligned = aligned_to(weight_dev, 16);
  if (format != A2AV_PLAIN) P.row = mx_row(features, format);
  P.W = W;
  P.H = (int)features;
  P.eps = eps;
  P.status = h->d_status;
  P.per_feature = (float)(1.0 / (double)features);
  P.per_feature_low = (float)(1.0 / (double)features - (double)P.per_feature);
  const NormForm f = norm_form(features, size, low, rows, h->sms, false);
  unsigned blocks;
  const cudaError_t e = launch_norm(h, [&](const NormForm& g) { return norm_kernel_of(dtype, format, g); }, f,
                                    2 * (int)features * size, rows, rows, P,
                                    static_cast<cudaStream_t>(stream), &blocks);
  return e != cudaSuccess || cudaGetLastError() != cudaSuccess ? A2AV_ERR_CUDA : A2AV_OK;
}

extern "C" int64_t a2av_norm_workspace_bytes(int64_t features, int64_t total_rows) {
  if (features < 1 || features > A2AV_MAX_NORM_FEATURES || total_rows < 0 || total_rows > kMaxCount)
    return -1;
  return (total_rows < kNormParts ? total_rows : kNormParts) * features * 4;
}

extern "C" int a2av_norm_backward(a2av_handle* h, int64_t features, int dtype, float eps,
                                  const void* const* sum_ptrs, const int64_t* tokens_per_rank,
                                  const float* weight_dev, const void* const* d_out_ptrs,
                                  const void* const* d_sum_ptrs, void* const* d_x_ptrs,
                                  float* d_weight_dev, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
  int rc = norm_ok(h, features, dtype, eps, sum_ptrs, tokens_per_rank, weight_dev, d_x_ptrs);
  if (rc != A2AV_OK) return rc;
  if (d_out_ptrs == nullptr || !aligned_to(d_weight_dev, 4)) return A2AV_ERR_INVALID_ARG;
  NormParams P;
  std::memset(&P, 0, sizeof(P));
  rc = count_rows(h, tokens_per_rank, P.first);
  if (rc != A2AV_OK) return rc;
  const int W = h->W, size = dtype_bytes(dtype);
  uintptr_t low = (uintptr_t)weight_dev;
  if (!take_rows(P.x, sum_ptrs, W, tokens_per_rank, size, &low) ||
      !take_rows(P.d_out, d_out_ptrs, W, tokens_per_rank, size, &low) ||
      (d_sum_ptrs != nullptr && !take_rows(P.residual, d_sum_ptrs, W, tokens_per_rank, size, &low)) ||
      !take_rows(P.out, d_x_ptrs, W, tokens_per_rank, size, &low))
    return A2AV_ERR_INVALID_ARG;
  const long long rows = P.first[W];
  if (d_weight_dev != nullptr) {
    const int64_t need = a2av_norm_workspace_bytes(features, rows);
    if (workspace_bytes < need || !aligned_to(workspace, 256) || (need > 0 && workspace == nullptr))
      return A2AV_ERR_INVALID_ARG;
    P.part = static_cast<float*>(workspace);
  }
  rc = current_device(h);
  if (rc != A2AV_OK) return rc;
  P.weight = weight_dev;
  P.weight_aligned = aligned_to(weight_dev, 16);
  P.W = W;
  P.H = (int)features;
  P.eps = eps;
  P.status = h->d_status;
  P.per_feature = (float)(1.0 / (double)features);
  P.per_feature_low = (float)(1.0 / (double)features - (double)P.per_feature);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  unsigned blocks = 0;
  if (rows > 0) {
    const NormForm f = norm_form(features, size, low, rows, h->sms, true);
    e = launch_norm(h, [&](const NormForm& g) { return norm_backward_kernel_of(dtype, g); }, f,
                    3 * (int)features * size, rows, kNormParts, P, s, &blocks);
  }
  if (e == cudaSuccess && d_weight_dev != nullptr)
    e = launch_chained(norm_weight_kernel, dim3((unsigned)((features + 31) / 32)), 1024, 0, s, h->pdl,
                       (const float*)P.part, (int)blocks, (int)features, d_weight_dev);
  return e != cudaSuccess || cudaGetLastError() != cudaSuccess ? A2AV_ERR_CUDA : A2AV_OK;
}

extern "C" int a2av_quantise(a2av_handle* h, int64_t features, int dtype, int format,
                             const void* const* x_ptrs, const int64_t* rows_per_rank,
                             const int64_t* in_splits_dev, void* const* packed_ptrs, void* stream) {
  return pack_call(h, features, dtype, format, x_ptrs, rows_per_rank, in_splits_dev, packed_ptrs, false, stream);
}

extern "C" int a2av_dequantise(a2av_handle* h, int64_t features, int dtype, int format,
                               const void* const* packed_ptrs, const int64_t* rows_per_rank,
                               const int64_t* in_splits_dev, void* const* out_ptrs, void* stream) {
  return pack_call(h, features, dtype, format, out_ptrs, rows_per_rank, in_splits_dev, packed_ptrs, true, stream);
}
