// experts_mma.cu -- the experts' products on the tensor cores: the forward
// product and the rows' gradient (expert_mma_kernel), the weights' gradient
// (expert_wgrad_kernel).
//
// Both are persistent kernels of CTA pairs.  In each CTA warp 3 describes the
// tiles ahead of the others, warp 0 copies operand tiles into a ring of six
// 32 KB shared-memory stages (TMA, 128-byte swizzle; in the first kernel warp 2
// shares the copies), warp 1 of the pair's first CTA issues the products, and
// warps 4..11 take the sums of the tile before from TMEM, where two tiles' sums
// have room, while the next tile's products run.
//
// Experts' weights are the M = 256 side of a tile and rows (tokens) the N side.
// An expert's rows lie in W groups, one from each source rank; its tiles are
// runs of up to 32 granules, eight rows of one group each (a group's last may
// have fewer), whatever groups they are from.  So the products cost what the
// rows cost (to 8 a group, and 16 a tile), the weights of an expert with a few
// rows from every rank are read once, and a granule is what the 128-byte
// swizzle and a TMA copy can place by itself.
//
// What bounds them: with many rows an expert the tensor cores (a dense product,
// 8192 rows, 8192 -> 8192: 570 to 584 us, 1.88 to 1.93 PFLOP/s; its rows'
// gradient 1.75, its weights' gradient 1.68), with a few the memory (one or two
// rows for each of 64 gated experts, 7168 -> 2048: 3.7 GB of weights in 552 us,
// 6.7 TB/s).  In between, 16 experts with some 1024 rows each from 8 ranks, 4096
// -> 2 x 2048 gated: the tensor pipe is busy 80 % of the forward product, 83 % of
// the weights' gradient.
#include "experts_tile.cuh"

namespace {

constexpr int kN = 256;               // most columns of a tile
constexpr int kK = 64;                // contraction per stage: 128 bytes of a row
constexpr int kStages = 6;
constexpr int kMmaThreads = 128 + 32 * kEpilogueWarps;
constexpr size_t kMmaSmem = 1024 + (size_t)kStages * kStageBytes + kEpilogueWarps * kStaging;

struct MmaParams {
  CUtensorMap rows[kBoxes][kW];  // N side: [rows][C] in boxes of 1, 2 .. 16 granules
                                 // (weights' gradient: x, in [0])
  CUtensorMap tail_dz, tail_x;   // weights' gradient: the packed remainders
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

__device__ __forceinline__ uint32_t columns_of(long long n) {
  return n >= kN ? kN : (uint32_t)((n + 31) / 32 * 32);
}

// ------------------------------------------------- rows times weights --
// kMn: the weights' contraction runs over their rows (the rows' gradient), so
// that they are the MN-major operand.  kGated: the tile's 256 weight rows are
// 128 of the first half and their partners of the second, eight and eight in
// turn (one copy of a five-dimensional view of the weights puts them so): a
// thread of the epilogue finds both in its registers.
// (Zipf-skewed rows over 64 experts: 16,384 rows, 2048 -> 7168, 475 to 490 us,
// with the tensor pipe 56 % busy and the memory at 67 % of its nominal rate: tiles
// bound by one and by the other share the time, and neither is saturated; 131,072
// rows, 7168 -> 2 x 2048 gated, 4.96 to 5.15 ms, 1.5 PFLOP/s under the power cap, 3 %
// more where z is saved.  5001 rows of one, f16, 2048 -> 7168: 105 us, 560 tiles
// being 7.4 rounds of 76 pairs that take 8 (98 for 4864 rows, 7 rounds); bias adds
// nothing, SiLU 2 us, GELU 9, the residual 10, 123 with all of them: the 32 blocks
// of products of a tile are too few to hide its epilogue.)
template <typename T, bool kMn, bool kGated>
__global__ void __launch_bounds__(kMmaThreads, 1) __cluster_dims__(2, 1, 1)
    expert_mma_kernel(const __grid_constant__ MmaParams P) {
  extern __shared__ unsigned char dynamic[];
  __shared__ GroupTable g;
  __shared__ TileTable tt;
  __shared__ Slot slots[kSlots];
  __shared__ Bars<kStages> b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t base = (smem_addr(dynamic) + 1023) & ~1023u;
  const uint32_t ring = smem_addr(&b.empty[0]);
  constexpr int kTileF = kGated ? 128 : 256;  // features of the result per pair
  constexpr int kMyF = kTileF / 2;            // and per CTA
  pair_begin(b, warp, 2, kEpilogueWarps + 2 + (rank == 0 ? 1 : 0));
  chain();
  const int nf = (P.F + kTileF - 1) / kTileF;
  const bool good = build_groups(P.g, g);
  if (good) build_tiles<kTileGranules>(P.g, g, tt, nf);
  const long long tiles = good ? tt.first[P.g.W * P.g.K] + (long long)tt.singles * nf : 0;
  const unsigned pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int blocks = (P.C + kK - 1) / kK;
  bool ok = true;
  unsigned i = 0;  // tiles so far

  if (warp == 3) {
    // --------------------------------------------------- scheduler --
    for (long long t; (t = tile_of(i, pair, pairs)) < tiles; ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_empty[sl]), ((i / kSlots) & 1) ^ 1, ring));
      if (!ok) break;
      describe_tile<kTileGranules>(P.g, g, tt, t, tiles, nf, kTileF, slots[sl], lane);
      __syncwarp();
      if (lane == 0) plan_copies(slots[sl], rank);
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_full[sl]));
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp == 0 || warp == 2) {
    // ------------------------------------------------------ copies --
    // warp 0 announces a stage's bytes and copies the weights and the first half
    // of the rows' runs, warp 2 the others
    const uint32_t full0 = map_to(smem_addr(&b.full[0]), 0);
    unsigned it = 0;
    for (; ok && tile_of(i, pair, pairs) < tiles; ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring));
      if (!ok) break;
      const Slot& slot = slots[sl];
      const Copies& copies = slot.copies;
      const int p = slot.p, e = slot.e, f0 = slot.f + kMyF * rank;
      const int from = warp == 0 ? 0 : copies.count / 2, to = warp == 0 ? copies.count / 2 : copies.count;
      const unsigned bytes = kSideBytes + copies.bytes;
      const CUtensorMap* wm = &P.weights[p];
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kStages;
        ok = __all_sync(kAll, bar_wait(smem_addr(&b.empty[s]), ((it / kStages) & 1) ^ 1));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t full = full0 + s * 8;
          const uint32_t at = base + s * kStageBytes;
          const int c = kb * kK;
          if (warp == 0) {
            bar_arrive_tx(full, bytes);
            if (kMn) {
              tma_load(at, wm, f0, c, e, full);
              tma_load(at + kSideBytes / 2, wm, f0 + 64, c, e, full);
            } else if (kGated) {
              tma_load5(at, wm, c, 0, 0, f0 / 8, e, full);
            } else {
              tma_load(at, wm, c, f0, e, full);
            }
          }
          for (int n = from; n < to; ++n)
            tma_load(at + kSideBytes + copies.at[n] * 1024, &P.rows[copies.box[n]][p], c,
                     copies.row[n], 0, full);
        }
        __syncwarp();
      }
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
    }
    // (warp 2 may leave: what it copied is counted on the same stages)
    if (warp == 2 && lane == 0 && !ok) note_error(P.g.status, A2AV_ERR_TIMEOUT);
    if (warp == 0 && lane == 0 && (!ok || !settle(b, it))) {
      note_error(P.g.status, A2AV_ERR_TIMEOUT);
      drain(b, rank, it);
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------- products --
    // (the whole warp goes through the loop, and a predicate has one lane issue:
    // under a branch of its own an instruction of the warp, as these are, takes
    // up to a hundred cycles)
    constexpr bool kBf16 = !__is_same(T, __half);
    const bool issuer = elect_one();
    const uint32_t tmem = __shfl_sync(kAll, b.tmem, 0);
    unsigned it = 0;
    for (; ok && tile_of(i, pair, pairs) < tiles; ++i) {
      const unsigned sl = i % kSlots, buf = i & 1;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring) &&
                                bar_wait_tile(smem_addr(&b.acc_empty[buf]), ((i >> 1) & 1) ^ 1, ring));
      if (!ok) break;
      const uint32_t idesc = product(kBf16, kMn, false, kM, (slots[sl].granules + 1) / 2 * 2 * kGranule);
      __syncwarp();
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
      const uint32_t d = tmem + buf * kN;
      fence_after_sync();
      bool ready = false;
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kStages;
        if (!__all_sync(kAll, ready)) {
          ok = __all_sync(kAll, bar_wait(smem_addr(&b.full[s]), (it / kStages) & 1));
          if (!ok) break;
        }
        fence_after_sync();
        // (the next stage is looked at while this one's products are issued)
        const unsigned next = (it + 1) % kStages;
        ready = bar_test(smem_addr(&b.full[next]), ((it + 1) / kStages) & 1);
        const uint32_t at = base + s * kStageBytes;
        const uint64_t wd = operand(at, kMn ? kSideBytes / 2 : 16);
        const uint64_t xd = operand(at + kSideBytes, 16);
        // (the contraction's last block may have fewer steps of 16)
        const int left = P.C - kb * kK, steps = left >= kK ? 4 : (left + 15) / 16;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps)
            mma(d, wd + (kMn ? k * (2048 >> 4) : k * (32 >> 4)), xd + k * (32 >> 4), idesc,
                kb > 0 || k > 0, issuer);
        mma_commit(smem_addr(&b.empty[s]), issuer);
      }
      if (ok) mma_commit(smem_addr(&b.acc_full[buf]), issuer);
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp >= 4) {
    // ---------------------------------------------------- epilogue --
    // two warps share a quarter of the lanes, with every other 32 columns each
    const int q = warp % 4, c0 = warp >= 8 ? 32 : 0;
    const uint32_t stage = base + kStages * kStageBytes + (warp - 4) * kStaging;
    const uint32_t empty0 = map_to(smem_addr(&b.acc_empty[0]), 0);
    constexpr int kPieces = kGated ? 2 : 4;
    for (; ok && tile_of(i, pair, pairs) < tiles; ++i) {
      const unsigned sl = i % kSlots, buf = i & 1;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring));
      if (!ok) break;
      const Slot& slot = slots[sl];
      const int p = slot.p, columns = slot.granules * kGranule;
      // the warp's features: 32 of the result, or 16 and their partners
      const int f = slot.f + kMyF * rank + (kGated ? 16 : 32) * q;
      const T* bias = P.bias[p] != nullptr
                          ? static_cast<const T*>(P.bias[p]) + (long long)slot.e * P.Z : nullptr;
      float ba[2] = {0.0f, 0.0f}, bb[2] = {0.0f, 0.0f};
      if (bias != nullptr) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int fa = f + (lane >> 2) + 8 * h, fb = kGated ? fa : fa + 16;
          if (fa < P.F) ba[h] = to_float(bias[fa]);
          if (fb < P.F) bb[h] = to_float(bias[kGated ? P.F + fb : fb]);
        }
      }
      T* out = static_cast<T*>(P.out[p]);
      T* pre = static_cast<T*>(P.pre[p]);
      const T* res = static_cast<const T*>(P.residual[p]);
      uint4 held[kPieces];  // of the residual
      if (res != nullptr) load_rows<T, kPieces>(held, res, P.F, slot, c0 / kGranule, f, P.F, lane);
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.acc_full[buf]), (i >> 1) & 1, ring));
      if (!ok) break;
      fence_after_sync();
      if (c0 >= columns && lane == 0) bar_arrive_relaxed(empty0 + buf * 8);  // nothing to take
      for (int c = c0; c < columns; c += 64) {
        const int j = c / kGranule;
        const uint32_t at = b.tmem + buf * kN + c + ((uint32_t)(32 * q) << 16);
        float va[16], vb[16];
        tmem_load(at, va);
        tmem_load(at + (16u << 16), vb);
        tmem_load_wait();
        if (c + 64 >= columns) {  // the warp's last of the tile's sums: its share of the buffer is free
          fence_before_sync();
          __syncwarp();
          if (lane == 0) bar_arrive_relaxed(empty0 + buf * 8);
        }
        if (kGated) {  // lanes 0..7 and 8..15 of each are partners: va the first halves, vb the second
#pragma unroll
          for (int n = 0; n < 16; n += 4)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float second = va[n + 2 + x];
              va[n + 2 + x] = vb[n + x];
              vb[n + x] = second;
            }
        }
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          va[n] += ba[(n >> 1) & 1];
          vb[n] += bb[(n >> 1) & 1];
        }
        if (pre != nullptr) {
          stage_block<T>(stage, 0, va, lane);
          stage_block<T>(stage, 32, vb, lane);
          __syncwarp();
          write_rows<T, 4, kGated ? 2 : 4>(stage, pre, P.Z, slot, j, f, P.F, P.F, lane);
          __syncwarp();
        }
        apply_act(P.act, va);
        if (kGated) {
#pragma unroll
          for (int n = 0; n < 16; ++n) va[n] *= vb[n];
        } else {
          apply_act(P.act, vb);
        }
        if (res != nullptr) {
          keep_rows<kPieces>(stage, held, lane);
          load_rows<T, kPieces>(held, res, P.F, slot, j + 8, f, P.F, lane);
          __syncwarp();
          add_block<T>(stage, 0, va, lane);
          if (!kGated) add_block<T>(stage, 32, vb, lane);
          __syncwarp();
        }
        stage_block<T>(stage, 0, va, lane);
        if (!kGated) stage_block<T>(stage, 32, vb, lane);
        __syncwarp();
        write_rows<T, kPieces, kPieces>(stage, out, P.F, slot, j, f, P.F, 0, lane);
        __syncwarp();
      }
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  }
  __syncwarp();
  pair_end(b, warp);
}

// --------------------------------------------------- weights' gradient --
// d_w[e] = dz_e^T x_e: both operands are MN-major and the contraction is over
// the expert's rows, in blocks of 64.  A block has rows of one expert only (a
// foreign row's NaN would not be stopped by a zero in the other operand), so
// what each group has over a multiple of 64 is copied together first
// (expert_tails_kernel): the remainders of an expert's W groups one after the
// other, zeros up to the next multiple of 64.  The products then run over the
// groups' whole blocks where they lie and over the packed ones.  (The tiles go
// expert by expert: dealing large and small experts out evenly, as the forward
// product does, took 5 to 9 % longer here.)  32,768 skewed rows over 64 experts,
// 7168 x 4096 gradients: 1.44 to 1.54 ms and 116 us for the packing, bound by
// the products of large experts and by writing the gradients of small ones.
// Packing what is over 32, 16 or 8 rows instead takes 60, 43 or 33 us, and the
// products, of more and smaller copies, as much longer or more (1.70 ms at 16,
// 1.88 at 8).
struct TailTable {
  int first[A2AV_MAX_DISPATCH_KEYS + 1];  // packed row of each expert, multiples of 64
};

// Rows and remainders of an expert (by one thread): whole blocks, packed rows.
__device__ __forceinline__ void expert_blocks(const GroupParams& G, const GroupTable& g, int x,
                                              int* whole, int* tail) {
  const int p = x / G.K, e = x - p * G.K;
  *whole = *tail = 0;
  for (int r = 0; r < G.W; ++r) {
    int rows;
    find_group(G, g, (p * G.W + r) * G.K + e, &rows);
    *tail += rows % kK;
    *whole += rows / kK;
  }
}

// By the whole block, after build_groups.
__device__ void build_tails(const GroupParams& G, GroupTable& g, TailTable& tt) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int E = G.W * G.K, per = (E + nt - 1) / nt;
  const int x0 = min(tid * per, E), x1 = min(x0 + per, E);
  int sum = 0, whole, tail;
  for (int x = x0; x < x1; ++x) {
    expert_blocks(G, g, x, &whole, &tail);
    sum += (tail + kK - 1) / kK * kK;
  }
  int at = block_prefix(sum, g);
  for (int x = x0; x < x1; ++x) {
    expert_blocks(G, g, x, &whole, &tail);
    tt.first[x] = at;
    at += (tail + kK - 1) / kK * kK;
    if (x == E - 1) tt.first[E] = at;
  }
  __syncthreads();
}

// The packed remainders: a warp takes a packed row of dz and of x.  Memory
// bound: some 370 MB read and as many written in 116 us, 6.4 TB/s (32,768 rows
// as above).
struct TailParams {
  GroupParams g;
  const void* dz[kW];
  const void* x[kW];
  void* to_dz;
  void* to_x;
  int Z, D;
};

__global__ void __launch_bounds__(256) expert_tails_kernel(const __grid_constant__ TailParams P) {
  chain();
  __shared__ GroupTable g;
  __shared__ TailTable tt;
  if (!build_groups(P.g, g)) return;
  build_tails(P.g, g, tt);
  const int lane = threadIdx.x & 31, W = P.g.W, K = P.g.K, E = W * K;
  const int zv = P.Z / 8, xv = P.D / 8;  // 16-byte vectors of a row
  const int warps = gridDim.x * (blockDim.x / 32);
  const RowParts split(tt.first[E], warps, max(zv, xv));
  for (int unit = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; unit < tt.first[E] * split.parts;
       unit += warps) {
    const int row = unit / split.parts, part = unit - row * split.parts;
    int zi, z1, xi, x1;
    split.run(part, zv, &zi, &z1);
    split.run(part, xv, &xi, &x1);
    int lo = 0, hi = E;  // first[lo] <= row < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tt.first[mid] <= row)
        lo = mid;
      else
        hi = mid;
    }
    const int p = lo / K, e = lo - p * K;
    int in = row - tt.first[lo];
    long long from = -1;
    for (int r = 0; r < W && from < 0; ++r) {
      int rows;
      const long long first = find_group(P.g, g, (p * W + r) * K + e, &rows);
      const int tail = rows % kK;
      if (in < tail) from = first + (rows - tail) + in;
      in -= tail;
    }
    uint4* z = static_cast<uint4*>(P.to_dz) + (long long)row * zv;
    uint4* x = static_cast<uint4*>(P.to_x) + (long long)row * xv;
    const uint4* z0 = static_cast<const uint4*>(P.dz[p]) + from * zv;
    const uint4* x0 = static_cast<const uint4*>(P.x[p]) + from * xv;
#pragma unroll 4
    for (int i = zi + lane; i < z1; i += 32) z[i] = from < 0 ? make_uint4(0, 0, 0, 0) : z0[i];
#pragma unroll 4
    for (int i = xi + lane; i < x1; i += 32) x[i] = from < 0 ? make_uint4(0, 0, 0, 0) : x0[i];
  }
}

// A tile as the scheduler describes it.
struct GradSlot {
  int p, e, z, d;                     // peer, local expert, first row and column of d_w
  int blocks, last;                   // blocks of 64 rows; steps of 16 in the last
  int first[kW + 1], n[kW + 1];       // first row and blocks of each group, then of the packed rows
};

template <typename T>
__global__ void __launch_bounds__(kMmaThreads, 1) __cluster_dims__(2, 1, 1)
    expert_wgrad_kernel(const __grid_constant__ MmaParams P) {
  extern __shared__ unsigned char dynamic[];
  __shared__ GroupTable g;
  __shared__ TailTable tt;
  __shared__ GradSlot slots[kSlots];
  __shared__ Bars<kStages> b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t base = (smem_addr(dynamic) + 1023) & ~1023u;
  const uint32_t ring = smem_addr(&b.empty[0]);
  pair_begin(b, warp, 2, kEpilogueWarps + 1 + (rank == 0 ? 1 : 0));
  chain();
  const bool good = build_groups(P.g, g);
  if (good) build_tails(P.g, g, tt);
  const int W = P.g.W, K = P.g.K;
  const unsigned nz = (P.Z + kM - 1) / kM, nd = (P.D + kN - 1) / kN;
  const unsigned tiles = good ? (unsigned)(W * K) * nz * nd : 0;
  const unsigned pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  bool ok = true;
  unsigned i = 0;  // tiles so far

  if (warp == 3) {
    // --------------------------------------------------- scheduler --
    for (unsigned t = pair; t < tiles; t += pairs, ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_empty[sl]), ((i / kSlots) & 1) ^ 1, ring));
      if (!ok) break;
      GradSlot& slot = slots[sl];
      const unsigned pe = t / (nz * nd), in = t - pe * (nz * nd);
      const int p = pe / K, e = pe - p * K;
      int tail = 0, whole = 0;
      if (lane < W) {
        int rows;
        slot.first[lane] = (int)find_group(P.g, g, (p * W + lane) * K + e, &rows);
        slot.n[lane] = whole = rows / kK;
        tail = rows % kK;
      }
      tail = __reduce_add_sync(kAll, tail);
      whole = __reduce_add_sync(kAll, whole);
      if (lane == 0) {
        slot.first[W] = tt.first[pe];  // the packed rows
        slot.n[W] = (tail + kK - 1) / kK;
        slot.p = p;
        slot.e = e;
        slot.z = in / nd * kM;
        slot.d = in % nd * kN;
        slot.blocks = whole + (tail + kK - 1) / kK;
        slot.last = tail % kK == 0 ? 4 : (tail % kK + 15) / 16;
      }
      __syncwarp();
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_full[sl]));
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp == 0) {
    // ------------------------------------------------------ copies --
    // the CTA's 128 columns of dz and its up to 128 columns of x, in boxes of 64
    // columns x 64 rows
    const uint32_t full0 = map_to(smem_addr(&b.full[0]), 0);
    unsigned it = 0;
    for (unsigned t = pair; ok && t < tiles; t += pairs, ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring));
      if (!ok) break;
      const GradSlot& slot = slots[sl];
      const int p = slot.p;
      const uint32_t half = columns_of(P.D - slot.d) / 2;
      const bool two = half > 64;
      const unsigned bytes = two ? 4 * 8192 : 3 * 8192;
      const int z = slot.z + 128 * (int)rank, column = slot.d + (int)half * (int)rank;
      for (int r = 0; r <= W && ok; ++r) {  // the groups, then the packed rows
        const int n = slot.n[r], first = slot.first[r];
        const CUtensorMap* dz = r < W ? &P.weights[p] : &P.tail_dz;
        const CUtensorMap* x = r < W ? &P.rows[0][p] : &P.tail_x;
        for (int m = 0; m < n; ++m, ++it) {
          const unsigned s = it % kStages;
          ok = __all_sync(kAll, bar_wait(smem_addr(&b.empty[s]), ((it / kStages) & 1) ^ 1));
          if (!ok) break;
          if (elect_one()) {
            const uint32_t full = full0 + s * 8, at = base + s * kStageBytes;
            const int row = first + m * kK;
            bar_arrive_tx(full, bytes);
            tma_load(at, dz, z, row, 0, full);
            tma_load(at + 8192, dz, z + 64, row, 0, full);
            tma_load(at + kSideBytes, x, column, row, 0, full);
            if (two) tma_load(at + kSideBytes + 8192, x, column + 64, row, 0, full);
          }
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
    }
    if (lane == 0 && (!ok || !settle(b, it))) {
      note_error(P.g.status, A2AV_ERR_TIMEOUT);
      drain(b, rank, it);
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------- products --
    constexpr bool kBf16 = !__is_same(T, __half);
    const bool issuer = elect_one();
    const uint32_t tmem = __shfl_sync(kAll, b.tmem, 0);
    unsigned it = 0, n_tile = 0;
    for (unsigned t = pair; ok && t < tiles; t += pairs, ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring));
      if (!ok) break;
      const int blocks = slots[sl].blocks, last = slots[sl].last;
      const uint32_t idesc = product(kBf16, true, true, kM, columns_of(P.D - slots[sl].d));
      __syncwarp();
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
      if (blocks == 0) continue;
      const unsigned buf = n_tile & 1;
      const uint32_t d = tmem + buf * kN;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.acc_empty[buf]), ((n_tile >> 1) & 1) ^ 1, ring));
      if (!ok) break;
      fence_after_sync();
      ++n_tile;
      bool ready = false;
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kStages;
        if (!__all_sync(kAll, ready)) {
          ok = __all_sync(kAll, bar_wait(smem_addr(&b.full[s]), (it / kStages) & 1));
          if (!ok) break;
        }
        fence_after_sync();
        // (the next stage is looked at while this one's products are issued)
        const unsigned next = (it + 1) % kStages;
        ready = bar_test(smem_addr(&b.full[next]), ((it + 1) / kStages) & 1);
        const uint32_t at = base + s * kStageBytes;
        const uint64_t zd = operand(at, 8192), xd = operand(at + kSideBytes, 8192);
        const int steps = kb == blocks - 1 ? last : 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps)
            mma(d, zd + k * (2048 >> 4), xd + k * (2048 >> 4), idesc, kb > 0 || k > 0, issuer);
        mma_commit(smem_addr(&b.empty[s]), issuer);
      }
      if (ok) mma_commit(smem_addr(&b.acc_full[buf]), issuer);
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp >= 4) {
    // ---------------------------------------------------- epilogue --
    const int q = warp % 4, c0 = warp >= 8 ? 32 : 0;
    const uint32_t stage = base + kStages * kStageBytes + (warp - 4) * kStaging;
    const uint32_t empty0 = map_to(smem_addr(&b.acc_empty[0]), 0);
    // the address a lane gives for its row of the 8 x 8 blocks (below)
    const uint32_t put = stage + (((lane >> 3) & 1) * 8 + (lane & 7)) * kPitch + (lane >> 4) * 16;
    unsigned n_tile = 0;
    for (unsigned t = pair; ok && t < tiles; t += pairs, ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring));
      if (!ok) break;
      const int p = slots[sl].p, e = slots[sl].e, d0 = slots[sl].d;
      const int z0 = slots[sl].z + 128 * (int)rank + 32 * q;
      const bool any = slots[sl].blocks > 0;  // else the gradient is 0
      __syncwarp();
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
      const unsigned buf = n_tile & 1;
      const int columns = min(kN, P.D - d0);
      if (any) {
        ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.acc_full[buf]), (n_tile >> 1) & 1, ring));
        if (!ok) break;
        fence_after_sync();
        ++n_tile;
        if (c0 >= columns && lane == 0) bar_arrive_relaxed(empty0 + buf * 8);
      }
      T* out = static_cast<T*>(P.out[p]) + ((long long)e * P.Z + z0) * P.D;
      for (int c = c0; c < columns; c += 64) {
        float va[16] = {}, vb[16] = {};
        if (any) {
          const uint32_t at = b.tmem + buf * kN + c + ((uint32_t)(32 * q) << 16);
          tmem_load(at, va);
          tmem_load(at + (16u << 16), vb);
          tmem_load_wait();
          if (c + 64 >= columns) {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive_relaxed(empty0 + buf * 8);
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
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int z = lane / 4 + 8 * i, d = d0 + c + 8 * (lane % 4);
          if (z0 + z < P.Z && d < P.D) {
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(stage + z * kPitch + (lane % 4) * 16));
            *reinterpret_cast<uint4*>(out + (long long)z * P.D + d) = v;
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  }
  __syncwarp();
  pair_end(b, warp);
}

// ----------------------------------------------------------- host side --
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

// A gated expert's weights [K][2][N][D] as [K][N / 8][2][8][D]: a box has
// eight rows of the first half, their eight partners, the next eight...
bool encode_gated(CUtensorMap* m, const void* p, int dtype, long long D, long long N, long long K) {
  const cuuint64_t dims[5] = {(cuuint64_t)D, 8, 2, (cuuint64_t)N / 8, (cuuint64_t)K};
  const cuuint64_t strides[4] = {(cuuint64_t)D * 2, (cuuint64_t)(N * D) * 2, (cuuint64_t)D * 16,
                                 (cuuint64_t)(N * D) * 4};
  const cuuint32_t box[5] = {64, 8, 2, 8, 1}, steps[5] = {1, 1, 1, 1, 1};
  return encoder()(m, dtype == A2AV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   5, const_cast<void*>(p), dims, strides, box, steps,
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

int64_t a2av_expert_tail_rows(int W, int K, int64_t rows) {
  // at most 63 of each group, and zeros up to a multiple of 64 for each expert
  const int64_t groups = (int64_t)W * W * K, experts = (int64_t)W * K;
  const int64_t most = rows < groups * (kK - 1) ? rows : groups * (kK - 1);
  return rows == 0 ? 0 : most + experts * (kK - 1);
}

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
  if (direction == 2 && (long long)h->W * P.g.K * ((P.Z + kM - 1) / kM) * ((P.D + kN - 1) / kN) > kMaxCount)
    return false;
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
        made = encode(&M.rows[0][p], n_side, dtype, P.D, rows, 1, kK) &&
               encode(&M.weights[p], m_side, dtype, P.Z, rows, 1, kK);
    } else {
      // (no run of granules takes a box of twice the buffer's rows)
      for (int i = 0; i < kBoxes && made && rows > 0 && (i == 0 || (kGranule << i) < 2 * rows); ++i)
        made = encode(&M.rows[i][p], n_side, dtype, C, rows, 1, kGranule << i);
      made = made && (gated ? encode_gated(&M.weights[p], m_side, dtype, P.D, P.N, P.g.K)
                            : encode(&M.weights[p], m_side, dtype, P.D, P.Z, P.g.K,
                                     direction == 1 ? kK : 128));
    }
    if (!made) return false;
    M.out[p] = out;
    if (direction == 0) {
      M.bias[p] = P.bias[p];
      M.residual[p] = P.residual[p];
      M.pre[p] = P.pre[p];
    }
  }
  if (direction == 2) {
    if (!aligned_to(P.tails, 16)) return false;
    void* tail_x = static_cast<unsigned char*>(P.tails) + P.tail_rows * P.Z * 2;
    if (P.tail_rows > 0 && (!encode(&M.tail_dz, P.tails, dtype, P.Z, P.tail_rows, 1, kK) ||
                            !encode(&M.tail_x, tail_x, dtype, P.D, P.tail_rows, 1, kK)))
      return false;
    TailParams R;
    std::memset(&R, 0, sizeof(R));
    R.g = P.g;
    for (int p = 0; p < h->W; ++p) {
      R.dz[p] = P.dy[p];
      R.x[p] = P.x[p];
    }
    R.to_dz = P.tails;
    R.to_x = tail_x;
    R.Z = (int)P.Z;
    R.D = (int)P.D;
    *error = launch_chained(expert_tails_kernel, dim3(4 * h->sms), 256, 0, s, h->pdl, R);
    if (*error != cudaSuccess) return true;
  }
  const MmaKernel kernel = dtype == A2AV_BF16 ? mma_kernel_of<__nv_bfloat16>(direction, gated)
                                              : mma_kernel_of<__half>(direction, gated);
  *error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMmaSmem);
  if (*error != cudaSuccess) return true;
  *error = launch_chained(kernel, dim3(h->sms / 2 * 2), kMmaThreads,
                          kMmaSmem, s, h->pdl, M);
  return true;
}
