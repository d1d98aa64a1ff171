// experts_mma.cu -- the experts' products on the tensor cores: the forward
// product and the rows' gradient (expert_mma_kernel), the weights' gradient
// (expert_wgrad_kernel).
//
// Both are persistent kernels of CTA pairs.  In each CTA warp 0 copies operand
// tiles into a ring of shared-memory stages (TMA, 128-byte swizzle), warp 1 of
// the pair's first CTA issues the products, and warps 4..7 take the sums of the
// tile before from TMEM, where two tiles' sums have room, while the next tile's
// products run.
//
// Experts' weights are the M = 256 side of a tile and rows (tokens) the N side:
// N can be any multiple of 32 up to 256, so that a ragged group's last tile
// costs what its rows cost, and a group of a few rows reads its weights with
// little else.  The rows' own multiple of 128 would be wasted on small groups.
#include "experts.cuh"
#include "mma.cuh"

namespace {

constexpr int kM = 256;               // of a pair
constexpr int kN = 256;               // most columns of a tile
constexpr int kK = 64;                // contraction per stage: 128 bytes of a row
constexpr int kSideBytes = 128 * 128; // one operand's part of a stage in one CTA
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kStages = 6;
constexpr int kRowBox = 32;           // rows of one copy of the N side
constexpr int kMmaThreads = 256;
constexpr unsigned kTmemColumns = 512;
constexpr int kPitch = 80;            // bytes between staged rows: 8 of them hit all banks once
constexpr int kStaging = 32 * kPitch; // per epilogue warp
constexpr size_t kMmaSmem = 1024 + (size_t)kStages * kStageBytes + 4 * kStaging;

struct MmaParams {
  CUtensorMap rows[kW];     // N side: [rows][C], or x of the weights' gradient
  CUtensorMap weights[kW];  // M side: [K][..][..], or dz
  GroupParams g;
  const void* bias[kW];
  const void* residual[kW];
  void* out[kW];
  void* pre[kW];
  int C, F, Z;  // contraction, features of the result, rows of an expert's weights
  int D;        // weights' gradient: its row length
  int act;
};

struct Bars {
  unsigned long long full[kStages];   // of the first CTA: both CTAs' copies have arrived
  unsigned long long empty[kStages];  // the products that read the stage are done
  unsigned long long tail[kStages];   // weights' gradient: this CTA's copies, before zeroing
  unsigned long long acc_full[2];     // a tile's sums are complete
  unsigned long long acc_empty[2];    // of the first CTA: both CTAs have taken them
  unsigned tmem;
};

// What the two kernels share before and after their roles.
__device__ __forceinline__ void pair_begin(Bars& b, int warp) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(smem_addr(&b.full[s]), 2);
      bar_init(smem_addr(&b.empty[s]), 1);
      bar_init(smem_addr(&b.tail[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&b.acc_full[i]), 1);
      bar_init(smem_addr(&b.acc_empty[i]), 8);
    }
    bar_init_done();
  }
  if (warp == 2) tmem_alloc(smem_addr(&b.tmem), kTmemColumns);
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
}

__device__ __forceinline__ void pair_end(Bars& b, int warp) {
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 2) tmem_free(b.tmem, kTmemColumns);
}

// A bounded wait has run out: the copies still in flight (counted on the first
// CTA's barriers) are waited for, with a limit, before the block may leave.
__device__ __noinline__ void drain(const Bars& b, uint32_t rank, unsigned issued) {
  if (rank != 0) return;
  for (unsigned i = 0; i < kStages && i < issued; ++i) {
    const unsigned at = issued - 1 - i;
    bar_wait(smem_addr(&b.full[at % kStages]), (at / kStages) & 1);
  }
}

// All copies are in: before the block leaves, the arrivals that the products
// still owe to this CTA's stages have to be there.
__device__ __forceinline__ bool settle(const Bars& b, unsigned issued) {
  bool ok = true;
  for (unsigned i = 0; i < kStages && i < issued && ok; ++i) {
    const unsigned at = issued - 1 - i;
    ok = bar_wait(smem_addr(&b.empty[at % kStages]), (at / kStages) & 1);
  }
  return ok;
}

__device__ __forceinline__ uint32_t columns_of(long long n) {
  return n >= kN ? kN : (uint32_t)((n + 31) / 32 * 32);
}

// The warp's 32 staged rows of kPieces x 16 bytes to rows `ld` apart; pieces
// past the first kSplit go `jump` elements further.
template <typename T, int kPieces, int kSplit>
__device__ __forceinline__ void write_rows(uint32_t stage, T* to, long long ld, int rows, int f,
                                           int F, long long jump, int lane) {
  constexpr int kPer = 32 / kPieces;
  const int piece = lane % kPieces, within = piece % kSplit;
  if (f + 8 * within >= F) return;
  T* at = to + f + 8 * within + (piece >= kSplit ? jump : 0);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = lane / kPieces + kPer * i;
    if (row < rows) {
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(stage + row * kPitch + piece * 16));
      *reinterpret_cast<uint4*>(at + row * ld) = v;
    }
  }
}

// The other way: rows into the warp's staging.
template <typename T, int kPieces>
__device__ __forceinline__ void read_rows(uint32_t stage, const T* from, long long ld, int rows,
                                          int f, int F, int lane) {
  constexpr int kPer = 32 / kPieces;
  const int piece = lane % kPieces;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = lane / kPieces + kPer * i;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows && f + 8 * piece < F)
      v = *reinterpret_cast<const uint4*>(from + row * ld + f + 8 * piece);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + row * kPitch + piece * 16),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
  }
}

// Sums of 16 features (lanes) x 32 rows (columns) to the staged rows' bytes
// [at, at + 32): two 8 x 8 blocks of features for each eight rows, transposed.
template <typename T>
__device__ __forceinline__ void stage_block(uint32_t stage, int at, const float (&v)[16], int lane) {
  const uint32_t a = stage + ((lane >> 4) * 8 + (lane & 7)) * kPitch + at + ((lane >> 3) & 1) * 16;
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    put4_t(a + i * 8 * kPitch, pack2(v[4 * i], v[4 * i + 1], T()), pack2(v[4 * i + 2], v[4 * i + 3], T()),
           pack2(v[4 * i + 4], v[4 * i + 5], T()), pack2(v[4 * i + 6], v[4 * i + 7], T()));
}

template <typename T>
__device__ __forceinline__ void add_block(uint32_t stage, int at, float (&v)[16], int lane) {
  const uint32_t a = stage + ((lane >> 4) * 8 + (lane & 7)) * kPitch + at + ((lane >> 3) & 1) * 16;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    uint32_t r[4];
    get4_t(a + i * 8 * kPitch, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = unpack2(r[j], T());
      v[4 * i + 2 * j] += x.x;
      v[4 * i + 2 * j + 1] += x.y;
    }
  }
}

template <int kAct>
__device__ __forceinline__ void apply_act(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = act_fn(kAct, v[i]);
}

__device__ __forceinline__ void apply_act(int act, float (&v)[16]) {
  if (act == A2AV_ACT_SILU)
    apply_act<A2AV_ACT_SILU>(v);
  else if (act == A2AV_ACT_GELU)
    apply_act<A2AV_ACT_GELU>(v);
  else if (act == A2AV_ACT_RELU)
    apply_act<A2AV_ACT_RELU>(v);
}

// ------------------------------------------------- rows times weights --
// kMn: the weights' contraction runs over their rows (the rows' gradient), so
// that they are the MN-major operand.  kGated: the tile's 256 weight rows are
// 128 of the first half and their partners of the second, 16 and 16 in turn:
// a thread of the epilogue finds both in its registers.
template <typename T, bool kMn, bool kGated>
__global__ void __launch_bounds__(kMmaThreads, 1) __cluster_dims__(2, 1, 1)
    expert_mma_kernel(const __grid_constant__ MmaParams P) {
  extern __shared__ unsigned char dynamic[];
  __shared__ GroupTable g;
  __shared__ Bars b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t base = (smem_addr(dynamic) + 1023) & ~1023u;
  constexpr int kTileF = kGated ? 128 : 256;   // features of the result per pair
  constexpr int kMyF = kTileF / 2;             // and per CTA
  chain();
  const int nf = (P.F + kTileF - 1) / kTileF;
  const bool good = build_groups(P.g, g, kN, nf);
  pair_begin(b, warp);
  const long long tiles = good ? g.tiles[g.entries] : 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int blocks = (P.C + kK - 1) / kK;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------ copies --
    const uint32_t full0 = map_to(smem_addr(&b.full[0]), 0);
    unsigned it = 0;
    for (long long t = pair; t < tiles && ok; t += pairs) {
      const GroupTile gt = find_tile(P.g, g, t, kN, nf);
      const int f0 = (int)(gt.local % nf) * kTileF + kMyF * rank;
      const long long m0 = gt.local / nf * kN;
      const uint32_t half = columns_of(gt.rows - m0) / 2;
      const int copies = (half + kRowBox - 1) / kRowBox;
      const int row = (int)(gt.first + m0 + half * rank);
      const CUtensorMap* wm = &P.weights[gt.p];
      const CUtensorMap* xm = &P.rows[gt.p];
      const unsigned bytes = kSideBytes + copies * kRowBox * 128;
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kStages;
        if (!bar_wait(smem_addr(&b.empty[s]), ((it / kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t full = full0 + s * 8;
        const uint32_t at = base + s * kStageBytes;
        bar_arrive_tx(full, bytes);
        const int c = kb * kK;
        if (kMn) {
          tma_load(at, wm, f0, c, gt.e, full);
          tma_load(at + kSideBytes / 2, wm, f0 + 64, c, gt.e, full);
        } else if (kGated) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tma_load(at + i * 4096, wm, c, f0 + 16 * i, gt.e, full);
            tma_load(at + i * 4096 + 2048, wm, c, P.F + f0 + 16 * i, gt.e, full);
          }
        } else {
          tma_load(at, wm, c, f0, gt.e, full);
        }
        for (int i = 0; i < copies; ++i)
          tma_load(at + kSideBytes + i * kRowBox * 128, xm, c, row + i * kRowBox, 0, full);
      }
    }
    if (!ok || !settle(b, it)) {
      note_error(P.g.status, A2AV_ERR_TIMEOUT);
      drain(b, rank, it);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---------------------------------------------------- products --
    constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
    unsigned it = 0, n_tile = 0;
    for (long long t = pair; t < tiles && ok; t += pairs, ++n_tile) {
      const GroupTile gt = find_tile(P.g, g, t, kN, nf);
      const uint32_t n = columns_of(gt.rows - gt.local / nf * kN);
      const uint32_t idesc = product(kBf16, kMn, false, kM, n);
      const unsigned buf = n_tile & 1;
      const uint32_t d = b.tmem + buf * kN;
      if (!bar_wait(smem_addr(&b.acc_empty[buf]), ((n_tile >> 1) & 1) ^ 1)) {
        ok = false;
        break;
      }
      fence_after_sync();
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kStages;
        if (!bar_wait(smem_addr(&b.full[s]), (it / kStages) & 1)) {
          ok = false;
          break;
        }
        fence_after_sync();
        const uint32_t at = base + s * kStageBytes;
        const uint64_t wd = operand(at, kMn ? kSideBytes / 2 : 16);
        const uint64_t xd = operand(at + kSideBytes, 16);
        // (the contraction's last block may have fewer steps of 16)
        const int left = P.C - kb * kK, steps = left >= kK ? 4 : (left + 15) / 16;
        for (int k = 0; k < steps; ++k)
          mma(d, wd + (kMn ? k * (2048 >> 4) : k * (32 >> 4)), xd + k * (32 >> 4), idesc,
              kb > 0 || k > 0);
        mma_commit(smem_addr(&b.empty[s]));
      }
      if (ok) mma_commit(smem_addr(&b.acc_full[buf]));
    }
    if (!ok) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp >= 4) {
    // ---------------------------------------------------- epilogue --
    const int q = warp - 4;
    const uint32_t stage = base + kStages * kStageBytes + q * kStaging;
    const uint32_t empty0 = map_to(smem_addr(&b.acc_empty[0]), 0);
    unsigned n_tile = 0;
    for (long long t = pair; t < tiles && ok; t += pairs, ++n_tile) {
      const GroupTile gt = find_tile(P.g, g, t, kN, nf);
      const long long m0 = gt.local / nf * kN;
      const int rows = (int)min((long long)kN, gt.rows - m0);
      // the warp's features: 32 of the result, or 16 and their partners
      const int f = (int)(gt.local % nf) * kTileF + kMyF * rank + (kGated ? 16 : 32) * q;
      const unsigned buf = n_tile & 1;
      const T* bias = P.bias[gt.p] != nullptr
                          ? static_cast<const T*>(P.bias[gt.p]) + (long long)gt.e * P.Z : nullptr;
      float ba[2] = {0.0f, 0.0f}, bb[2] = {0.0f, 0.0f};
      if (bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int fa = f + (lane >> 2) + 8 * i, fb = kGated ? fa : fa + 16;
          if (fa < P.F) ba[i] = to_float(bias[fa]);
          if (fb < P.F) bb[i] = to_float(bias[kGated ? P.F + fb : fb]);
        }
      }
      const long long row0 = gt.first + m0;
      T* out = static_cast<T*>(P.out[gt.p]) + row0 * P.F;
      T* pre = P.pre[gt.p] != nullptr ? static_cast<T*>(P.pre[gt.p]) + row0 * P.Z : nullptr;
      const T* res = P.residual[gt.p] != nullptr
                         ? static_cast<const T*>(P.residual[gt.p]) + row0 * P.F : nullptr;
      ok = __all_sync(kAll, bar_wait(smem_addr(&b.acc_full[buf]), (n_tile >> 1) & 1));
      if (!ok) break;
      fence_after_sync();
      for (int c = 0; c < rows; c += 32) {
        const int n = min(32, rows - c);
        const uint32_t at = b.tmem + buf * kN + c + ((uint32_t)(32 * q) << 16);
        float va[16], vb[16];
        tmem_load(at, va);
        tmem_load(at + (16u << 16), vb);
        tmem_load_wait();
        if (c + 32 >= rows) {  // the last of the tile's sums: the buffer is free
          fence_before_sync();
          __syncwarp();
          if (lane == 0) bar_arrive(empty0 + buf * 8);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          va[i] += ba[(i >> 1) & 1];
          vb[i] += bb[(i >> 1) & 1];
        }
        if (pre != nullptr) {
          stage_block<T>(stage, 0, va, lane);
          stage_block<T>(stage, 32, vb, lane);
          __syncwarp();
          if (kGated)
            write_rows<T, 4, 2>(stage, pre + (long long)c * P.Z, P.Z, n, f, P.F, P.F, lane);
          else
            write_rows<T, 4, 4>(stage, pre + (long long)c * P.Z, P.Z, n, f, P.F, 0, lane);
          __syncwarp();
        }
        apply_act(P.act, va);
        if (kGated) {
#pragma unroll
          for (int i = 0; i < 16; ++i) va[i] *= vb[i];
        } else {
          apply_act(P.act, vb);
        }
        if (res != nullptr) {
          read_rows<T, kGated ? 2 : 4>(stage, res + (long long)c * P.F, P.F, n, f, P.F, lane);
          __syncwarp();
          add_block<T>(stage, 0, va, lane);
          if (!kGated) add_block<T>(stage, 32, vb, lane);
          __syncwarp();
        }
        stage_block<T>(stage, 0, va, lane);
        if (!kGated) stage_block<T>(stage, 32, vb, lane);
        __syncwarp();
        constexpr int kPieces = kGated ? 2 : 4;
        write_rows<T, kPieces, kPieces>(stage, out + (long long)c * P.F, P.F, n, f, P.F, 0, lane);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  }
  __syncwarp();
  pair_end(b, warp);
}

// --------------------------------------------------- weights' gradient --
// d_w[e] = dz_e^T x_e: both operands are MN-major, the contraction is over the
// expert's rows, group after group.  The rows of a block past its group's end
// are the next group's; where they share a step of 16 with the group's own,
// warp 3 zeroes them in both operands (a zero in one would not stop a NaN in
// the other) between their arrival and the products.
template <typename T>
__global__ void __launch_bounds__(kMmaThreads, 1) __cluster_dims__(2, 1, 1)
    expert_wgrad_kernel(const __grid_constant__ MmaParams P) {
  extern __shared__ unsigned char dynamic[];
  __shared__ GroupTable g;
  __shared__ Bars b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t base = (smem_addr(dynamic) + 1023) & ~1023u;
  chain();
  const bool good = build_groups(P.g, g, kN, 1);
  pair_begin(b, warp);
  const int W = P.g.W, K = P.g.K;
  const int nz = (P.Z + kM - 1) / kM, nd = (P.D + kN - 1) / kN;
  const long long tiles = good ? (long long)W * K * nz * nd : 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  bool ok = true;
  unsigned it = 0;

  if (warp == 0 && lane == 0) {
    const uint32_t full0 = map_to(smem_addr(&b.full[0]), 0);
    for (long long t = pair; t < tiles && ok; t += pairs) {
      const int pe = (int)(t / ((long long)nz * nd)), p = pe / K, e = pe % K;
      const int z0 = (int)(t / nd % nz) * kM + 128 * rank, d0 = (int)(t % nd) * kN;
      const uint32_t half = columns_of(P.D - d0) / 2;
      const int copies = (half + 63) / 64;
      const unsigned bytes = kSideBytes + copies * 8192;
      for (int r = 0; r < W && ok; ++r) {
        int rows;
        const long long first = find_group(P.g, g, (p * W + r) * K + e, &rows);
        for (int m = 0; m < rows; m += kK, ++it) {
          const unsigned s = it % kStages;
          if (!bar_wait(smem_addr(&b.empty[s]), ((it / kStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          const bool ragged = rows - m < kK && (rows - m) % 16 != 0;
          const uint32_t bar = ragged ? smem_addr(&b.tail[s]) : full0 + s * 8;
          const uint32_t at = base + s * kStageBytes;
          const int row = (int)(first + m);
          bar_arrive_tx(ragged ? map_to(bar, rank) : bar, bytes);
          tma_load(at, &P.weights[p], z0, row, 0, bar);
          tma_load(at + 8192, &P.weights[p], z0 + 64, row, 0, bar);
          for (int i = 0; i < copies; ++i)
            tma_load(at + kSideBytes + i * 8192, &P.rows[p], d0 + half * rank + 64 * i, row, 0, bar);
        }
      }
    }
    if (!ok || !settle(b, it)) {
      note_error(P.g.status, A2AV_ERR_TIMEOUT);
      drain(b, rank, it);
    }
  } else if (warp == 3) {
    const uint32_t full0 = map_to(smem_addr(&b.full[0]), 0);
    unsigned parity = 0;  // a bit a stage
    for (long long t = pair; t < tiles && ok; t += pairs) {
      const int pe = (int)(t / ((long long)nz * nd)), p = pe / K, e = pe % K;
      const int d0 = (int)(t % nd) * kN;
      const uint32_t half = columns_of(P.D - d0) / 2;
      const int boxes = 2 + (half + 63) / 64;
      for (int r = 0; r < W && ok; ++r) {
        int rows;
        find_group(P.g, g, (p * W + r) * K + e, &rows);
        const unsigned n = (rows + kK - 1) / kK;
        const int left = rows % kK;
        it += n;
        if (left % 16 == 0) continue;
        const unsigned s = (it - 1) % kStages;
        ok = __all_sync(kAll, bar_wait(smem_addr(&b.tail[s]), (parity >> s) & 1));
        if (!ok) break;
        parity ^= 1u << s;
        const int lines = 16 - left % 16;
        const uint32_t at = base + s * kStageBytes + left * 128;
        for (int i = lane; i < boxes * lines * 8; i += 32) {
          const int box = i / (lines * 8), in = i % (lines * 8);
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + box * 8192 + in * 16),
                       "r"(0)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(full0 + s * 8);
      }
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr bool kBf16 = !__is_same(T, __half);
    unsigned n_tile = 0;
    for (long long t = pair; t < tiles && ok; t += pairs) {
      const int pe = (int)(t / ((long long)nz * nd)), p = pe / K, e = pe % K;
      const uint32_t idesc = product(kBf16, true, true, kM, columns_of(P.D - t % nd * kN));
      const unsigned buf = n_tile & 1;
      const uint32_t d = b.tmem + buf * kN;
      bool any = false;
      for (int r = 0; r < W && ok; ++r) {
        int rows;
        find_group(P.g, g, (p * W + r) * K + e, &rows);
        for (int m = 0; m < rows; m += kK, ++it) {
          if (!any && !bar_wait(smem_addr(&b.acc_empty[buf]), ((n_tile >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          const unsigned s = it % kStages;
          if (!bar_wait(smem_addr(&b.full[s]), (it / kStages) & 1)) {
            ok = false;
            break;
          }
          fence_after_sync();
          const uint32_t at = base + s * kStageBytes;
          const uint64_t zd = operand(at, 8192), xd = operand(at + kSideBytes, 8192);
          const int left = rows - m, steps = left >= kK ? 4 : (left + 15) / 16;
          for (int k = 0; k < steps; ++k) {
            mma(d, zd + k * (2048 >> 4), xd + k * (2048 >> 4), idesc, any);
            any = true;
          }
          mma_commit(smem_addr(&b.empty[s]));
        }
      }
      if (any && ok) {
        mma_commit(smem_addr(&b.acc_full[buf]));
        ++n_tile;
      }
    }
    if (!ok) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp >= 4) {
    const int q = warp - 4;
    const uint32_t stage = base + kStages * kStageBytes + q * kStaging;
    const uint32_t empty0 = map_to(smem_addr(&b.acc_empty[0]), 0);
    // the address a lane gives for its row of the 8 x 8 blocks (below)
    const uint32_t put = stage + (((lane >> 3) & 1) * 8 + (lane & 7)) * kPitch + (lane >> 4) * 16;
    unsigned n_tile = 0;
    for (long long t = pair; t < tiles && ok; t += pairs) {
      const int pe = (int)(t / ((long long)nz * nd)), p = pe / K, e = pe % K;
      const int z0 = (int)(t / nd % nz) * kM + 128 * rank + 32 * q, d0 = (int)(t % nd) * kN;
      long long all = 0;
      for (int r = 0; r < W; ++r) {
        int rows;
        find_group(P.g, g, (p * W + r) * K + e, &rows);
        all += rows;
      }
      const unsigned buf = n_tile & 1;
      if (all > 0) {
        ok = __all_sync(kAll, bar_wait(smem_addr(&b.acc_full[buf]), (n_tile >> 1) & 1));
        if (!ok) break;
        fence_after_sync();
        ++n_tile;
      }
      const int columns = min(kN, P.D - d0);
      T* out = static_cast<T*>(P.out[p]) + ((long long)e * P.Z + z0) * P.D;
      for (int c = 0; c < columns; c += 32) {
        float va[16] = {}, vb[16] = {};
        if (all > 0) {
          const uint32_t at = b.tmem + buf * kN + c + ((uint32_t)(32 * q) << 16);
          tmem_load(at, va);
          tmem_load(at + (16u << 16), vb);
          tmem_load_wait();
          if (c + 32 >= columns) {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(empty0 + buf * 8);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          put4(put + i * 16, pack2(va[4 * i], va[4 * i + 1], T()), pack2(va[4 * i + 2], va[4 * i + 3], T()),
               pack2(va[4 * i + 4], va[4 * i + 5], T()), pack2(va[4 * i + 6], va[4 * i + 7], T()));
          put4(put + i * 16 + 16 * kPitch, pack2(vb[4 * i], vb[4 * i + 1], T()),
               pack2(vb[4 * i + 2], vb[4 * i + 3], T()), pack2(vb[4 * i + 4], vb[4 * i + 5], T()),
               pack2(vb[4 * i + 6], vb[4 * i + 7], T()));
        }
        __syncwarp();
        write_rows<T, 4, 4>(stage, out, P.D, min(32, P.Z - z0), d0 + c, P.D, 0, lane);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  }
  __syncwarp();
  pair_end(b, warp);
}

// ----------------------------------------------------------- host side --
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

// A [depth][rows][inner] tensor of 16-bit elements in boxes of 64 x box_rows.
bool encode(CUtensorMap* m, const void* p, int dtype, long long inner, long long rows,
            long long depth, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)inner * rows * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, steps[3] = {1, 1, 1};
  return encoder()(m, dtype == A2AV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   3, const_cast<void*>(p), dims, strides, box, steps,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using MmaKernel = void (*)(MmaParams);

template <typename T>
MmaKernel mma_kernel_of(int direction, bool gated) {
  if (direction == 2) return expert_wgrad_kernel<T>;
  if (direction == 1) return expert_mma_kernel<T, true, false>;
  return gated ? expert_mma_kernel<T, false, true> : expert_mma_kernel<T, false, false>;
}

}  // namespace

bool a2av_expert_mma(a2av_handle* h, const A2avExperts& P, int dtype, int direction,
                     cudaStream_t s, cudaError_t* error) {
  *error = cudaSuccess;
  // TMA: rows of 16 bytes' multiples, buffers on 16 bytes; the strides of a
  // tensor map stay below 2^40
  if (P.D % 8 != 0 || P.N % 8 != 0 || encoder() == nullptr || P.Z * P.D >= (1LL << 38)) return false;
  static_assert(sizeof(MmaParams) <= 32764, "a kernel's parameters");
  MmaParams M;
  std::memset(&M, 0, sizeof(M));
  M.g = P.g;
  const bool gated = direction == 0 && P.gated;
  M.C = (int)(direction == 0 ? P.D : P.Z);
  M.F = (int)(direction == 0 ? P.N : P.D);
  M.Z = (int)P.Z;
  M.D = (int)P.D;
  M.act = direction == 0 ? P.act : A2AV_ACT_NONE;
  const long long C = M.C;
  for (int p = 0; p < h->W; ++p) {
    const long long rows = P.g.cap[p];
    const void* n_side = P.x[p];
    const void* m_side = direction == 2 ? P.dy[p] : P.w[p];
    void* out = direction == 2 ? P.d_w[p] : P.out[p];
    if (!aligned_to(n_side, 16) || !aligned_to(m_side, 16) || !aligned_to(out, 16) ||
        !aligned_to(P.pre[p], 16) || !aligned_to(P.residual[p], 16))
      return false;
    bool made = true;
    if (direction == 2) {
      if (rows > 0)
        made = encode(&M.rows[p], n_side, dtype, P.D, rows, 1, kK) &&
               encode(&M.weights[p], m_side, dtype, P.Z, rows, 1, kK);
    } else {
      if (rows > 0) made = encode(&M.rows[p], n_side, dtype, C, rows, 1, kRowBox);
      made = made && encode(&M.weights[p], m_side, dtype, P.D, P.Z, P.g.K,
                            direction == 1 ? kK : gated ? 16 : 128);
    }
    if (!made) return false;
    M.out[p] = out;
    if (direction == 0) {
      M.bias[p] = P.bias[p];
      M.residual[p] = P.residual[p];
      M.pre[p] = P.pre[p];
    }
  }
  const MmaKernel kernel = dtype == A2AV_BF16 ? mma_kernel_of<__nv_bfloat16>(direction, gated)
                                              : mma_kernel_of<__half>(direction, gated);
  *error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMmaSmem);
  if (*error != cudaSuccess) return true;
  *error = launch_chained(kernel, dim3(h->sms / 2 * 2), kMmaThreads, kMmaSmem, s, h->pdl, M);
  return true;
}
