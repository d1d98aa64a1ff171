// experts_mx.cu -- the experts' products on packed rows and weights
// (a2av_expert_matmul_mx); the interface is in include/a2av_mx.h.
//
// The persistent kernel of CTA pairs that experts_mma.cu has for 16 bits, on the
// tensor cores' block-scaled products: a stage is again 128 bytes of 256 of an
// expert's features (the M side) and of up to 224 rows (the N side), which is 128
// or 256 values of the contraction, and four steps of products.  A step's scales
// have to be in TMEM, 32 rows to the lanes of a quarter and the next 32 in the next
// column, while in a packed row a block's scales follow one another.  So a warp for
// every 128 rows reads 16 bytes of scales of four rows a lane, which is a word or
// two for each of the next stages, puts words of the same blocks side by side (in
// its registers: no two lanes have to meet) into the stage, and the warp that issues
// the products copies them to TMEM before them.  The scales' columns are what a
// tile of 256 rows would need for its sums: 224 leave 32 columns behind each of the
// two tiles' sums, enough for the scales of one stage each.
//
// What it reaches: a decoding step's weights (256 rows for 64 gated experts, 7168 -> 2 x
// 2048, 1 GB of 4 bits) in 162 to 167 us, 90 % of the copy rate, 552 in 16 bits; 131,072
// Zipf-skewed rows of the same in 1.50 to 1.54 ms, 5.1 PFLOP/s (16 bits: 4.96 to 5.15 ms);
// 16,384 skewed rows, 2048 -> 7168, of 8 bits 276 to 309 us (467 to 490).
// What bounds it: shared memory.  A stage of 256 x 216 is written by the copies and
// read by the products once, 60 KB a CTA, which at 128 bytes a cycle is 0.25 us, and its products
// 0.27 us at 7.85 PFLOP/s (4 bits: four times the 16-bit rate measured, at which the tensor
// cores would be busy throughout); it takes 0.32 to 0.34, with the tensor pipe busy 56 to 59 % of
// the time.  With parts left out, of 360 us (4 bits, 32,768 rows, gated): the rows' copies cost 25 us, the
// weights' 17, storing the scales 14, copying them to TMEM 14; four stages instead of five
// 9.  A tile costs 1 to 1.5 us besides: its epilogue is not hidden behind fewer than some 14
// stages (64 -> 2048, a stage a tile, writes its results at 2.3 TB/s).
#include "experts_tile.cuh"
#include "mx_device.cuh"

namespace {

constexpr int kMxColumns = 224;       // most rows of a tile
constexpr int kTall = kMxColumns / kGranule;
constexpr int kMxStages = 5;
constexpr int kAccColumns = 256;      // columns between the two tiles' sums
constexpr int kScaleWarps = 3;        // 128 features, 128 rows and the other rows
constexpr int kAtom = 512;            // bytes of 128 rows' words of scales
constexpr int kMxThreads = 128 + 32 * (kEpilogueWarps + kScaleWarps);
constexpr int kAhead = 3;             // 16-byte pieces of a row's scales in flight, at most
constexpr int kHeld = kAhead * 128 * 16;  // of a scale warp's rows

// Words of scales that a stage has of each row.
template <int kFormat>
constexpr int kScaleWords = kFormat == A2AV_MXFP8 ? 1 : 2;
template <int kFormat>
constexpr int kScaleBytes = kScaleWords<kFormat> * kScaleWarps * kAtom;  // of a stage
template <int kFormat>
constexpr size_t kMxSmem = 1024 + (size_t)kMxStages * (kStageBytes + kScaleBytes<kFormat>) +
                           kEpilogueWarps * kStaging + kScaleWarps * kHeld;

struct MxParams {
  CUtensorMap rows[kBoxes][kW];  // [rows][bytes of values] in boxes of 1, 2 .. 16 granules
  CUtensorMap weights[kW];       // [K][Z][bytes of values]
  GroupParams g;
  const void* x[kW];
  const void* w[kW];
  const void* bias[kW];
  const void* residual[kW];
  void* out[kW];
  MxRow at;
  int F, Z;      // features of the result, rows of an expert's weights
  int act;
  int vector;    // results and residuals take vectors of 16 bytes
  int pairwise;  // gated weights come in one copy (their halves are whole eights)
};

// write_rows, or element by element where the rows take no vectors: a lane has one
// column of the staged rows, eight of them at a time.
template <typename T, int kPieces>
__device__ __forceinline__ void write_any(bool vector, uint32_t stage, T* to, const Slot& slot, int j,
                                          int f, int F, int lane) {
  if (vector) return write_rows<T, kPieces, kPieces>(stage, to, F, slot, j, f, F, 0, lane);
  constexpr int kValues = 8 * kPieces, kPer = 32 / kValues;  // columns, rows at a time
  const int c = lane % kValues;
  if (f + c >= F) return;
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    const int gr = j + g, n = slot.n[gr];
    unsigned short* at = reinterpret_cast<unsigned short*>(to) + (long long)slot.row[gr] * F + f + c;
#pragma unroll
    for (int i = 0; i < kGranule / kPer; ++i) {
      const int in = lane / kValues + kPer * i;
      unsigned short v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(stage + (kGranule * g + in) * kPitch + c * 2));
      if (in < n) at[(long long)in * F] = v;
    }
  }
}

// The rows that load_rows takes to registers, element by element into the staging.
template <typename T, int kPieces>
__device__ __forceinline__ void keep_elements(uint32_t stage, const T* from, const Slot& slot, int j, int f,
                                              int F, int lane) {
  constexpr int kValues = 8 * kPieces, kPer = 32 / kValues, kRows = 32 / kPer;
  const int c = lane % kValues;
  unsigned short v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = lane / kValues + kPer * i, gr = j + row / kGranule, in = row % kGranule;
    v[i] = 0;
    if (f + c < F && in < slot.n[gr])
      v[i] = reinterpret_cast<const unsigned short*>(from)[(long long)(slot.row[gr] + in) * F + f + c];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + (lane / kValues + kPer * i) * kPitch + c * 2), "h"(v[i])
                 : "memory");
}

template <typename T, int kFormat, bool kGated>
__global__ void __launch_bounds__(kMxThreads, 1) __cluster_dims__(2, 1, 1)
    expert_mx_kernel(const __grid_constant__ MxParams P) {
  extern __shared__ unsigned char dynamic[];
  __shared__ GroupTable g;
  __shared__ TileTable tt;
  __shared__ Slot slots[kSlots];
  __shared__ Bars<kMxStages> b;
  __shared__ unsigned long long filled[kMxStages];  // of the second CTA: its stage has its scales
  constexpr int kWords = kScaleWords<kFormat>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t base = (smem_addr(dynamic) + 1023) & ~1023u;
  const uint32_t scales = base + kMxStages * kStageBytes;  // of the stages, then the epilogue's staging
  const uint32_t ring = smem_addr(&b.empty[0]);
  constexpr int kTileF = kGated ? 128 : 256;  // features of the result per pair
  constexpr int kMyF = kTileF / 2;            // and per CTA
  if (threadIdx.x == 0)
    for (int s = 0; s < kMxStages; ++s) bar_init(smem_addr(&filled[s]), kScaleWarps);
  pair_begin(b, warp, 2 + kScaleWarps + 1, kEpilogueWarps + kScaleWarps + 2 + (rank == 0 ? 1 : 0));
  chain();
  const int nf = (P.F + kTileF - 1) / kTileF;
  const bool good = build_groups(P.g, g);
  if (good) build_tiles<kTall>(P.g, g, tt, nf);
  const long long tiles = good ? tt.first[P.g.W * P.g.K] + (long long)tt.singles * nf : 0;
  const unsigned pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int bytes = (int)P.at.values, blocks = (bytes + kLine - 1) / kLine;
  bool ok = true;
  unsigned i = 0;  // tiles so far

  if (warp == 3) {
    // --------------------------------------------------- scheduler --
    for (long long t; (t = tile_of(i, pair, pairs)) < tiles; ++i) {
      const unsigned sl = i % kSlots;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_empty[sl]), ((i / kSlots) & 1) ^ 1, ring));
      if (!ok) break;
      describe_tile<kTall>(P.g, g, tt, t, tiles, nf, kTileF, slots[sl], lane);
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
      const CUtensorMap* wm = &P.weights[p];
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kMxStages;
        ok = __all_sync(kAll, bar_wait(smem_addr(&b.empty[s]), ((it / kMxStages) & 1) ^ 1));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t full = full0 + s * 8;
          const uint32_t at = base + s * kStageBytes;
          const int c = kb * kLine;
          if (warp == 0) {
            bar_arrive_tx(full, kSideBytes + copies.bytes);
            if (!kGated) {
              tma_load(at, wm, c, f0, e, full);
            } else if (P.pairwise) {
              tma_load5(at, wm, c, 0, 0, f0 / 8, e, full);
            } else {
              for (int k = 0; k < 8; ++k) {
                tma_load(at + 2048 * k, wm, c, f0 + 8 * k, e, full);
                tma_load(at + 2048 * k + 1024, wm, c, P.F + f0 + 8 * k, e, full);
              }
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
    // (the whole warp goes through the loop, and a predicate has one lane issue)
    constexpr bool k4Bit = kFormat == A2AV_MXFP4;
    const bool issuer = elect_one();
    const uint32_t tmem = __shfl_sync(kAll, b.tmem, 0);
    unsigned it = 0;
    for (; ok && tile_of(i, pair, pairs) < tiles; ++i) {
      const unsigned sl = i % kSlots, buf = i & 1;
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (i / kSlots) & 1, ring) &&
                                bar_wait_tile(smem_addr(&b.acc_empty[buf]), ((i >> 1) & 1) ^ 1, ring));
      if (!ok) break;
      const int columns = (slots[sl].granules + 1) / 2 * 2 * kGranule;
      __syncwarp();
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
      const uint32_t idesc = product_scaled(k4Bit, kM, columns);
      const uint32_t d = tmem + buf * kAccColumns;
      fence_after_sync();
      bool ready = false;
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kMxStages;
        if (!__all_sync(kAll, ready)) {
          ok = __all_sync(kAll, bar_wait_filled(smem_addr(&b.full[s]), (it / kMxStages) & 1));
          if (!ok) break;
        }
        take_filled();  // (both CTAs' scales)
        fence_after_sync();
        // (the next stage is looked at while this one's products are issued)
        const unsigned next = (it + 1) % kMxStages;
        ready = bar_test_filled(smem_addr(&b.full[next]), ((it + 1) / kMxStages) & 1);
        // the stage's scales, in turn behind the one and the other tile's sums: a
        // column for every 32 rows, the features' words first
        const uint32_t sa = tmem + (it & 1) * kAccColumns + kMxColumns, sb = sa + 4 * kWords;
        const uint32_t from = scales + s * kScaleBytes<kFormat>;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t word = from + w * kScaleWarps * kAtom;
          tmem_copy(sa + 4 * w, scale_rows(word), issuer);
          tmem_copy(sb + 8 * w, scale_rows(word + kAtom), issuer);
          tmem_copy(sb + 8 * w + 4, scale_rows(word + 2 * kAtom), issuer && columns > 128);
        }
        const uint32_t at = base + s * kStageBytes;
        const uint64_t wd = operand(at, 16), xd = operand(at + kSideBytes, 16);
        // (the contraction's last block may have fewer steps of 32 bytes)
        const int left = bytes - kb * kLine, steps = left >= kLine ? 4 : (left + 31) / 32;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps)
            mma_scaled<k4Bit>(d, wd + k * (32 >> 4), xd + k * (32 >> 4),
                              with_scales(idesc, k4Bit ? k % 2 * 2 : k), sa + (k4Bit ? k / 2 * 4 : 0),
                              sb + (k4Bit ? k / 2 * 8 : 0), kb > 0 || k > 0, issuer);
        mma_commit(smem_addr(&b.empty[s]), issuer);
      }
      if (ok) mma_commit(smem_addr(&b.acc_full[buf]), issuer);
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp == 1) {
    // ------------------------------------ the second CTA's scales --
    // passed on to the first CTA, whose products read them (by the scale warps themselves
    // 131,072 rows of 4 bits take 1535 us, by this one 1502; without its fence 1490)
    const uint32_t full0 = map_to(smem_addr(&b.full[0]), 0);
    unsigned it = 0;
    for (; ok && tile_of(i, pair, pairs) < tiles; ++i)
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        const unsigned s = it % kMxStages;
        ok = __all_sync(kAll, bar_wait(smem_addr(&filled[s]), (it / kMxStages) & 1));
        if (!ok) break;
        if (lane == 0) bar_pass_filled(full0 + s * 8);
      }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp >= 4 + kEpilogueWarps) {
    // ------------------------------------------------------ scales --
    // a lane has rows lane, 32 + lane, 64 + lane and 96 + lane of the warp's 128;
    // pieces of 16 bytes of their scales come through a ring of the lane's own, the
    // next tile's behind this one's (no further: a slot three tiles on is described
    // when this tile is done)
    const int part = warp - 4 - kEpilogueWarps;
    const uint32_t into_bar = map_to(smem_addr(rank == 0 ? &b.full[0] : &filled[0]), rank);
    const uint32_t held = scales + kMxStages * kScaleBytes<kFormat> + kEpilogueWarps * kStaging +
                          part * kHeld + lane * 16;
    constexpr int kPer = 4 / kWords;  // stages that a piece lasts
    const int count = P.at.scales, pieces = (count + 15) / 16, lead = min(pieces, kAhead);
    const uint4* from[4];   // of the tile that is fetched; NULL: no such row
    unsigned fi = 0, it = 0, any = 0;  // that tile, stages, tiles with rows (a bit each)
    int fc = 0;             // the piece that is fetched next
    bool more = tile_of(0, pair, pairs) < tiles;
    uint32_t into = held, out_of = held;  // places in the ring
    const auto next_place = [&](uint32_t at) { return at == held + (kAhead - 1) * 2048 ? held : at + 2048; };
    const auto fetch = [&] {
      if (more) {
        if (fc == 0) {
          const unsigned sl = fi % kSlots;
          ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.slot_full[sl]), (fi / kSlots) & 1, ring));
          const Slot& slot = slots[sl];
          bool some = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = lane + 32 * k;
            const unsigned char* row = nullptr;
            if (!ok) {
            } else if (part == 0) {
              const int f = slot.f + kMyF * rank + (kGated ? r / 16 * 8 + r % 8 : r);
              const long long z = f + (kGated && r / 8 % 2 ? P.F : 0);
              if (f < P.F)
                row = static_cast<const unsigned char*>(P.w[slot.p]) +
                      ((long long)slot.e * P.Z + z) * P.at.bytes;
            } else {
              const int m = (part - 1) * 128 + r, gr = m / kGranule;
              if (m % kGranule < slot.n[gr])
                row = static_cast<const unsigned char*>(P.x[slot.p]) +
                      ((long long)slot.row[gr] + m % kGranule) * P.at.bytes;
            }
            from[k] = row == nullptr ? nullptr : reinterpret_cast<const uint4*>(row + P.at.values);
            some = some || row != nullptr;
          }
          const unsigned bit = 1u << (fi & 31);
          any = __any_sync(kAll, some) ? any | bit : any & ~bit;
          if (ok && lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // (zeros: nothing is read, but the address has to be one of 16 bytes all the same,
          // which weights are)
          const bool here = ok && from[k] != nullptr;
          copy_async(into + k * 512, here ? from[k] + fc : P.w[0], here ? 16 : 0);
        }
        into = next_place(into);
        if (++fc == pieces) {
          fc = 0;
          ++fi;
          more = ok && tile_of(fi, pair, pairs) < tiles;
        }
      }
      copy_async_commit();
    };
    for (int c = 0; c < lead; ++c) fetch();
    for (; ok && tile_of(i, pair, pairs) < tiles; ++i) {
      for (int c = 0; ok && c < pieces; ++c) {
        if (lead == 3)
          copy_async_wait<2>();
        else if (lead == 2)
          copy_async_wait<1>();
        else
          copy_async_wait<0>();
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                       : "r"(out_of + k * 512)
                       : "memory");
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (!ok || c * kPer + j >= blocks) continue;
          const unsigned s = it % kMxStages;
          ok = __all_sync(kAll, bar_wait(smem_addr(&b.empty[s]), ((it / kMxStages) & 1) ^ 1));
          if (!ok) continue;
          if (any >> (i & 31) & 1) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              const int word = j * kWords + w;
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = word == 0 ? v[k].x : word == 1 ? v[k].y : word == 2 ? v[k].z : v[k].w;
              // (what follows the scales is no scale: products with its zeros stay 0)
              const int valid = count - 16 * c - 4 * word;
              const uint32_t mask = valid >= 4 ? ~0u : valid <= 0 ? 0u : (1u << (8 * valid)) - 1;
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                               scales + s * kScaleBytes<kFormat> + (w * kScaleWarps + part) * kAtom + lane * 16),
                           "r"(x[0] & mask), "r"(x[1] & mask), "r"(x[2] & mask), "r"(x[3] & mask)
                           : "memory");
            }
            fence_async_shared();
          }
          __syncwarp();
          if (lane == 0) bar_arrive_filled(into_bar + s * 8);
          ++it;
        }
        out_of = next_place(out_of);
        if (ok) fetch();
      }
    }
    copy_async_wait<0>();
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  } else if (warp >= 4) {
    // ---------------------------------------------------- epilogue --
    // two warps share a quarter of the lanes, with every other 32 columns each
    const int q = warp % 4, c0 = warp >= 8 ? 32 : 0;
    const uint32_t stage = scales + kMxStages * kScaleBytes<kFormat> + (warp - 4) * kStaging;
    const uint32_t empty0 = map_to(smem_addr(&b.acc_empty[0]), 0);
    const bool vector = P.vector;
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
      const T* res = static_cast<const T*>(P.residual[p]);
      uint4 held[kPieces];  // of the residual
      if (res != nullptr && vector)
        load_rows<T, kPieces>(held, res, P.F, slot, c0 / kGranule, f, P.F, lane);
      ok = __all_sync(kAll, bar_wait_tile(smem_addr(&b.acc_full[buf]), (i >> 1) & 1, ring));
      if (!ok) break;
      fence_after_sync();
      if (c0 >= columns && lane == 0) bar_arrive_relaxed(empty0 + buf * 8);  // nothing to take
      for (int c = c0; c < columns; c += 64) {
        const int j = c / kGranule;
        const uint32_t at = b.tmem + buf * kAccColumns + c + ((uint32_t)(32 * q) << 16);
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
        apply_act(P.act, va);
        if (kGated) {
#pragma unroll
          for (int n = 0; n < 16; ++n) va[n] *= vb[n];
        } else {
          apply_act(P.act, vb);
        }
        if (res != nullptr) {
          if (vector) {
            keep_rows<kPieces>(stage, held, lane);
            load_rows<T, kPieces>(held, res, P.F, slot, j + 8, f, P.F, lane);
          } else {
            keep_elements<T, kPieces>(stage, res, slot, j, f, P.F, lane);
          }
          __syncwarp();
          add_block<T>(stage, 0, va, lane);
          if (!kGated) add_block<T>(stage, 32, vb, lane);
          __syncwarp();
        }
        stage_block<T>(stage, 0, va, lane);
        if (!kGated) stage_block<T>(stage, 32, vb, lane);
        __syncwarp();
        write_any<T, kPieces>(vector, stage, out, slot, j, f, P.F, lane);
        __syncwarp();
      }
      if (lane == 0) bar_arrive_here(smem_addr(&b.slot_empty[sl]));
    }
    if (!ok && lane == 0) note_error(P.g.status, A2AV_ERR_TIMEOUT);
  }
  __syncwarp();
  pair_end(b, warp);
}

// ----------------------------------------------------------- host side --
// Packed rows [depth][rows] in boxes of 128 bytes x box_rows.
bool encode(CUtensorMap* m, const void* p, const MxRow& at, long long rows, long long depth, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)at.values, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)at.bytes, (cuuint64_t)(at.bytes * rows)};
  const cuuint32_t box[3] = {kLine, (cuuint32_t)box_rows, 1}, steps[3] = {1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(p), dims, strides, box, steps,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A gated expert's weights [K][2][N] as [K][N / 8][2][8]: a box has eight rows of
// the first half, their eight partners, the next eight...
bool encode_gated(CUtensorMap* m, const void* p, const MxRow& at, long long N, long long K) {
  const cuuint64_t dims[5] = {(cuuint64_t)at.values, 8, 2, (cuuint64_t)N / 8, (cuuint64_t)K};
  const cuuint64_t strides[4] = {(cuuint64_t)at.bytes, (cuuint64_t)(N * at.bytes),
                                 (cuuint64_t)at.bytes * 8, (cuuint64_t)(2 * N * at.bytes)};
  const cuuint32_t box[5] = {kLine, 8, 2, 8, 1}, steps[5] = {1, 1, 1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(p), dims, strides, box, steps,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kFormat>
cudaError_t launch_mx(a2av_handle* h, const MxParams& M, bool gated, cudaStream_t s) {
  const auto kernel = gated ? expert_mx_kernel<T, kFormat, true> : expert_mx_kernel<T, kFormat, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kMxSmem<kFormat>);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3(h->sms / 2 * 2), kMxThreads, kMxSmem<kFormat>, s, h->pdl, M);
}

template <typename T>
cudaError_t launch_mx(a2av_handle* h, const MxParams& M, int format, bool gated, cudaStream_t s) {
  return format == A2AV_MXFP8 ? launch_mx<T, A2AV_MXFP8>(h, M, gated, s)
                              : launch_mx<T, A2AV_MXFP4>(h, M, gated, s);
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
  static_assert(sizeof(MxParams) <= 32764, "a kernel's parameters");
  if (encoder() == nullptr) return A2AV_ERR_CUDA;
  MxParams M;
  std::memset(&M, 0, sizeof(M));
  M.g = P.g;
  M.at = mx_row(P.D, format);
  if (P.Z * M.at.bytes >= (1LL << 40)) return A2AV_ERR_UNSUPPORTED;  // (a tensor map's strides)
  M.F = (int)P.N;
  M.Z = (int)P.Z;
  M.act = P.act;
  M.vector = P.N % 8 == 0;
  M.pairwise = P.N % 8 == 0;
  for (int p = 0; p < W; ++p) {
    const long long rows = rows_per_peer[p];
    bool made = true;
    // (no run of granules takes a box of twice the buffer's rows)
    for (int i = 0; i < kBoxes && made && rows > 0 && (i == 0 || (kGranule << i) < 2 * rows); ++i)
      made = encode(&M.rows[i][p], P.x[p], M.at, rows, 1, kGranule << i);
    made = made && (!P.gated      ? encode(&M.weights[p], P.w[p], M.at, P.Z, P.g.K, 128)
                    : M.pairwise ? encode_gated(&M.weights[p], P.w[p], M.at, P.N, P.g.K)
                                 : encode(&M.weights[p], P.w[p], M.at, P.Z, P.g.K, 8));
    if (!made) return A2AV_ERR_CUDA;
    M.x[p] = P.x[p];
    M.w[p] = P.w[p];
    M.bias[p] = P.bias[p];
    M.residual[p] = P.residual[p];
    M.out[p] = P.out[p];
    if (!aligned_to(P.out[p], 16) || !aligned_to(P.residual[p], 16)) M.vector = 0;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = shape->dtype == A2AV_BF16 ? launch_mx<__nv_bfloat16>(h, M, format, P.gated, s)
                                                  : launch_mx<__half>(h, M, format, P.gated, s);
  return e != cudaSuccess || cudaGetLastError() != cudaSuccess ? A2AV_ERR_CUDA : A2AV_OK;
}
