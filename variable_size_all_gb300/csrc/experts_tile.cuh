// experts_tile.cuh -- what the tensor-core kernels of the experts' products share:
// the tiles and their order, the copies that bring their rows, the pair's
// barriers, and the way of results between TMEM and the rows they belong to.
#pragma once

#include "experts.cuh"
#include "mma.cuh"

namespace {

constexpr int kM = 256;               // features of a pair's tile
constexpr int kLine = 128;            // bytes of a row that a stage has
constexpr int kSideBytes = 128 * kLine; // one operand's part of a stage in one CTA
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kGranule = 8;
constexpr int kTileGranules = 256 / kGranule;  // most that a tile can have
constexpr int kBoxes = 5;             // of 1, 2 .. 16 granules
constexpr int kSlots = 3;             // tiles the scheduler may be ahead
constexpr int kEpilogueWarps = 8;     // two for each quarter of the TMEM lanes
constexpr unsigned kTmemColumns = 512;
constexpr int kPitch = 80;            // bytes between staged rows: 8 of them hit all banks once
constexpr int kStaging = 32 * kPitch; // per epilogue warp

// ---------------------------------------------------------------- tiles --
// The copies that bring a CTA's half of a tile's granules.
struct Copies {
  int count;
  unsigned bytes;
  int row[kTileGranules / 2];
  int at[kTileGranules / 2];   // granules into the stage's N side
  int box[kTileGranules / 2];  // 2^box granules
};

// A tile as the scheduler (warp 3 of each CTA) describes it to the others.
struct Slot {
  int p, e;                // peer, local expert
  int f;                   // its first feature
  int granules;            // 1 .. 32
  int row[kTileGranules];  // each granule's first row in the peer's buffers
  int n[kTileGranules];    // and its rows, 0 past the last granule
  Copies copies;           // of this CTA
};

// The order of tiles.  Two kinds of experts: those of several tiles of rows,
// whose products are what takes time (their weights come from L2 after the
// first), and those whose rows fit one, which take as long as reading their
// weights does.  Each kind keeps its own order, and the two are dealt out
// evenly, so that at any time some pairs keep the tensor cores busy and others
// the memory.  (16,384 rows, Zipf-skewed over 64 experts, 2048 -> 7168: one kind
// after the other took the sum of both times.)
struct TileTable {
  int first[A2AV_MAX_DISPATCH_KEYS + 1];        // tiles of the first kind before each expert
  unsigned short single[A2AV_MAX_DISPATCH_KEYS];  // the experts of the second kind
  int singles;
};

// Number `t` of `tiles` dealt out of two kinds, `seconds` of the second: sets
// *index to its number within its kind, and returns whether that is the second.
__device__ __forceinline__ bool deal(long long t, long long tiles, long long seconds, int* index) {
  const long long before = t * seconds / tiles;
  const bool second = (t + 1) * seconds / tiles > before;
  *index = (int)(second ? before : t - before);
  return second;
}

// A pair's i-th tile: every pair takes one of each round, a place further each
// time (the kinds would else alternate in step with the pairs).
__device__ __forceinline__ long long tile_of(unsigned i, unsigned pair, unsigned pairs) {
  return (long long)i * pairs + (pair + i) % pairs;
}

// Rows of tiles that are taken together, for the sake of L2: a weight tile is
// read by this many pairs at about the same time.
constexpr int kBand = 8;

// Granules of a group of n rows (n up to 2^31 - 1).
__device__ __forceinline__ int granules_of(int n) {
  return (int)(((unsigned)n + kGranule - 1) / kGranule);
}

// Exclusive prefix sum of one value a thread over the block.
__device__ __forceinline__ int block_prefix(int x, GroupTable& g) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += v;
  }
  __syncthreads();
  if (lane == 31) g.warp_tiles[warp] = inc;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += (int)g.warp_tiles[w];
  return base + inc - x;
}

// By the whole block, after build_groups; `features`: tiles of a row of them;
// kTall: most granules of a tile.
template <int kTall>
__device__ void build_tiles(const GroupParams& G, GroupTable& g, TileTable& tt, int features) {
  const int tid = threadIdx.x, nt = blockDim.x, E = G.W * G.K, per = (E + nt - 1) / nt;
  const int x0 = min(tid * per, E), x1 = min(x0 + per, E);
  int tiles = 0, singles = 0;
  const auto tile_rows = [&](int x) {
    const int p = x / G.K, e = x - p * G.K;
    int granules = 0;
    for (int r = 0; r < G.W; ++r) {
      int rows;
      find_group(G, g, (p * G.W + r) * G.K + e, &rows);
      granules += granules_of(rows);
    }
    return (granules + kTall - 1) / kTall;
  };
  for (int x = x0; x < x1; ++x) {
    const int n = tile_rows(x);
    if (n == 1) ++singles;
    if (n > 1) tiles += n * features;
  }
  int at = block_prefix(tiles, g), single = block_prefix(singles, g);
  for (int x = x0; x < x1; ++x) {
    const int n = tile_rows(x);
    tt.first[x] = at;
    if (n == 1) tt.single[single++] = (unsigned short)x;
    if (n > 1) at += n * features;
    if (x == E - 1) {
      tt.first[E] = at;
      tt.singles = single;
    }
  }
  __syncthreads();
}

// Tile t, by a whole warp.
template <int kTall>
__device__ __forceinline__ void describe_tile(const GroupParams& G, const GroupTable& g,
                                              const TileTable& tt, long long t, long long tiles,
                                              int features, int tile_features, Slot& slot,
                                              int lane) {
  int at, lo;
  if (deal(t, tiles, (long long)tt.singles * features, &at)) {
    lo = tt.single[at / features];
    at %= features;
  } else {
    int hi = G.W * G.K;  // first[lo] <= at < first[hi]
    lo = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tt.first[mid] <= at)
        lo = mid;
      else
        hi = mid;
    }
    at -= tt.first[lo];
  }
  const int p = lo / G.K, e = lo - p * G.K;
  int rows = 0;
  long long first = 0;
  if (lane < G.W) first = find_group(G, g, (p * G.W + lane) * G.K + e, &rows);
  const int granules = granules_of(rows);
  int inc = granules;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += v;
  }
  const int total = __shfl_sync(kAll, inc, 31);
  // bands of kBand rows of tiles: down a band first, then along it
  // (its tiles have about the same number of granules: a tile of a few rows
  // costs half of a full one for its weights alone)
  const int row_tiles = (total + kTall - 1) / kTall;
  const int each = (total + row_tiles - 1) / row_tiles;
  const int band = at / (kBand * features), in = at - band * kBand * features;
  const int high = min(kBand, row_tiles - band * kBand), f = in / high;
  const int g0 = (band * kBand + in - f * high) * each, mine = g0 + lane;
  int r = 0;
  for (int i = 0; i < G.W - 1; ++i)
    if (__shfl_sync(kAll, inc, i) <= mine) r = i + 1;
  // rows of the group before this granule
  const int within = (int)((unsigned)(mine - __shfl_sync(kAll, inc - granules, r)) * kGranule);
  const int n = __shfl_sync(kAll, rows, r) - within;
  const long long row = __shfl_sync(kAll, first, r) + within;
  slot.row[lane] = (int)row;
  slot.n[lane] = lane < each && mine < total ? min(n, kGranule) : 0;
  if (lane == 0) {
    slot.p = p;
    slot.e = e;
    slot.f = f * tile_features;
    slot.granules = min(total - g0, each);
  }
}

// A CTA's half of a tile's granules as copies: a run of g consecutive granules
// takes the largest box of 2^b granules that it fills, and the same again so
// that it ends with the run (both bring the same bytes where they overlap).
// The half's last run takes one larger box instead where there is room: what
// that brings past the run is in no result.  So a run costs one or two copies;
// issuing them is what bounds tiles of many short groups.
__device__ __forceinline__ void plan_copies(Slot& slot, uint32_t rank) {
  Copies& c = slot.copies;
  const int half = (slot.granules + 1) / 2;
  const int j0 = rank == 0 ? 0 : half, j1 = rank == 0 ? half : slot.granules;
  unsigned granules = 0;
  int n = 0;
  for (int j = j0; j < j1;) {
    const int row = slot.row[j];
    int run = 1;
    while (j + run < j1 && (unsigned)slot.row[j + run] == (unsigned)row + kGranule * run) ++run;
    int box = 31 - __clz(run);
    if (j + run == j1 && (1 << box) < run && j - j0 + (2 << box) <= kTileGranules / 2) ++box;
    c.row[n] = row;
    c.at[n] = j - j0;
    c.box[n] = box;
    ++n;
    granules += 1u << box;
    if ((1 << box) < run) {
      const int by = run - (1 << box);
      c.row[n] = row + by * kGranule;
      c.at[n] = j - j0 + by;
      c.box[n] = box;
      ++n;
      granules += 1u << box;
    }
    j += run;
  }
  c.count = n;
  c.bytes = granules * 1024;
}

// ----------------------------------------------------------- the pair --
template <int kStages>
struct Bars {
  unsigned long long full[kStages];   // of the first CTA: what both CTAs bring has arrived
  unsigned long long empty[kStages];  // the products that read the stage are done
  unsigned long long acc_full[2];     // a tile's sums are complete
  unsigned long long acc_empty[2];    // of the first CTA: both CTAs have taken them
  unsigned long long slot_full[kSlots], slot_empty[kSlots];
  unsigned tmem;
};

// What the kernels share before and after their roles.  `fillers`: arrivals that
// fill a stage; `readers`: warps of this CTA that read the slots.
template <int kStages>
__device__ __forceinline__ void pair_begin(Bars<kStages>& b, int warp, int fillers, int readers) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(smem_addr(&b.full[s]), fillers);
      bar_init(smem_addr(&b.empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&b.acc_full[i]), 1);
      bar_init(smem_addr(&b.acc_empty[i]), 2 * kEpilogueWarps);
    }
    for (int i = 0; i < kSlots; ++i) {
      bar_init(smem_addr(&b.slot_full[i]), 1);
      bar_init(smem_addr(&b.slot_empty[i]), readers);
    }
    bar_init_done();
  }
  if (warp == 2) tmem_alloc(smem_addr(&b.tmem), kTmemColumns);
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
}

template <int kStages>
__device__ __forceinline__ void pair_end(Bars<kStages>& b, int warp) {
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 2) tmem_free(b.tmem, kTmemColumns);
}

// A bounded wait has run out: the copies still in flight (counted on the first
// CTA's barriers) are waited for, with a limit, before the block may leave.
template <int kStages>
__device__ __noinline__ void drain(const Bars<kStages>& b, uint32_t rank, unsigned issued) {
  if (rank != 0) return;
  for (unsigned i = 0; i < kStages && i < issued; ++i) {
    const unsigned at = issued - 1 - i;
    bar_wait(smem_addr(&b.full[at % kStages]), (at / kStages) & 1);
  }
}

// All copies are in: before the block leaves, the arrivals that the products
// still owe to this CTA's stages have to be there.
template <int kStages>
__device__ __forceinline__ bool settle(const Bars<kStages>& b, unsigned issued) {
  bool ok = true;
  for (unsigned i = 0; i < kStages && i < issued && ok; ++i) {
    const unsigned at = issued - 1 - i;
    ok = bar_wait(smem_addr(&b.empty[at % kStages]), (at / kStages) & 1);
  }
  return ok;
}

// ------------------------------------------------- rows of the results --
// The warp's 32 staged rows (four granules, from granule j of the slot) of
// kPieces x 16 bytes to the rows they stand for, `ld` apart; pieces past the
// first kSplit go `jump` elements further.
template <typename T, int kPieces, int kSplit>
__device__ __forceinline__ void write_rows(uint32_t stage, T* to, long long ld, const Slot& slot,
                                           int j, int f, int F, long long jump, int lane) {
  constexpr int kPer = 32 / kPieces;
  const int piece = lane % kPieces, within = piece % kSplit;
  if (f + 8 * within >= F) return;
  T* at = to + f + 8 * within + (piece >= kSplit ? jump : 0);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = lane / kPieces + kPer * i, gr = j + row / kGranule, in = row % kGranule;
    if (in < slot.n[gr]) {
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(stage + row * kPitch + piece * 16));
      *reinterpret_cast<uint4*>(at + (long long)(slot.row[gr] + in) * ld) = v;
    }
  }
}

// The other way, in two steps: rows into registers, and from there into the
// warp's staging (the loads are in flight while the sums are taken).
template <typename T, int kPieces>
__device__ __forceinline__ void load_rows(uint4 (&v)[kPieces], const T* from, long long ld,
                                          const Slot& slot, int j, int f, int F, int lane) {
  constexpr int kPer = 32 / kPieces;
  const int piece = lane % kPieces;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = lane / kPieces + kPer * i, gr = j + row / kGranule, in = row % kGranule;
    v[i] = make_uint4(0, 0, 0, 0);
    if (gr < kTileGranules && in < slot.n[gr] && f + 8 * piece < F)
      v[i] = *reinterpret_cast<const uint4*>(from + (long long)(slot.row[gr] + in) * ld + f + 8 * piece);
  }
}

template <int kPieces>
__device__ __forceinline__ void keep_rows(uint32_t stage, const uint4 (&v)[kPieces], int lane) {
  constexpr int kPer = 32 / kPieces;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                     stage + (lane / kPieces + kPer * i) * kPitch + lane % kPieces * 16),
                 "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w)
                 : "memory");
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

}  // namespace
