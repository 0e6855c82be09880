// Products grouped by expert (moe_grouped_gemm, moe_grouped_wgrad) on the
// tensor cores: tcgen05.mma kind::f16 on pairs of CTAs (cta_group::2), operands
// by tensor copies, FP32 accumulators in tensor memory.
//
// A pair computes tiles D [256 x up to 256].  The M side always is the side
// without ragged edges: the weights' output rows (forward), their columns
// (input gradient) or dw's rows (weight gradient); the ragged slots of a group
// are the N side of the first two, so a tile's width follows the group: a
// group of n slots is cut into ceil(n / 256) tiles of equal width (a multiple
// of 32), and the MMAs compute no more columns than that.  In the weight
// gradient the slots are the contraction.
//
//   mode     M (A operand)            N (B operand)     contraction
//   forward  w rows n, K-major        slots, K-major    K
//   SwiGLU   w rows, gate and up in alternating groups of 8 (a warp's lanes
//            0-7 and 16-23 hold gates, the eight lanes after each the ups)
//   dgrad    w columns k, M-major     slots, K-major    N
//   wgrad    dy columns n, M-major    x columns k, N-major   slots of the group
//
// Warps of each CTA: 0 issues A's tensor copies, 6 those of B (one thread
// issues a copy every ~0.1-0.2 us whatever its size, so a stage is one 16 KB
// copy of each), 1 (of the leader) the MMAs, 2-5 (and 7-10 in some modes)
// drain the accumulators, and 11 works out which tile comes next, up to four
// tiles ahead of the others (each role doing that for itself held up tiles that
// are only a few blocks long).  Two 256-column accumulators let the drain of
// one tile overlap the products of the next.  The CTAs are persistent: the
// tiles of all groups form one sequence, dealt round-robin to the pairs.
//
// What bounds it, and what it measures on one GB300 (BF16, bursts):
//  - many rows (8 experts of 8192, K 4096, N 2048): a block of 64 contraction
//    elements takes 0.30 us, of which 0.27 the MMAs and 0.24 the 32 KB that each
//    SM receives (about 135 GB/s at most); 1777 TFLOP/s forward, 1852 input
//    gradient, 1740 weight gradient;
//  - a training batch (288 experts of 228 rows): the weights' bytes; forward 854
//    us (6.6 TB/s), with SwiGLU and its inputs kept 885 us, input gradient 848
//    us; the weight gradient, 4.8 GB written, 1050 us (5.4 TB/s);
//  - few rows: the weights' bytes, see the few-slots path below.
#include <mutex>
#include <type_traits>

#include "tc_pair.cuh"
#include "train.cuh"

namespace moe {
namespace {

enum Mode { kForward, kSwiglu, kDgrad, kWgrad };

constexpr int kThreads = 384;

constexpr int kTileM = 256, kTileN = 256, kTileZ = 64;   // per pair; contraction elements per stage
constexpr int kABytes = 128 * kTileZ * 2;                // per CTA and stage
constexpr int kBBytes = 128 * kTileZ * 2;
constexpr int kMaxE = 2048;
// A warp's transposition of 16 columns (slots): 32 FP32 rows of one column in
// 128 bytes, padded so that the reads' 16-byte pieces meet different banks.
constexpr int kRowsPitch = 144, kRowsBytes = 16 * kRowsPitch;

template <Mode kMode> struct Cfg {
  static constexpr int kStages = kMode == kWgrad ? 5 : 6;   // of full size
  // the epilogue's transposition; the few-slots path's sums
  static constexpr int kStoreBytes = kMode == kWgrad ? 8 * 4096 : 8 * kRowsBytes;
  // Epilogue warps 2-5, and 7-10 where the drain has more to do than store: a
  // lane quarter's two warps take turns over the columns.  (In the plain
  // products eight warps beside the issuing ones cost 2.7% where the tensor
  // cores bound.)
  static constexpr int kEpiWarps = kMode == kWgrad || kMode == kSwiglu ? 8 : 4;
};
constexpr int kMaxStages = 9;
constexpr int kSumBuffers = 4;
constexpr int kQueue = 4;
constexpr int kFewGroups = 640;
constexpr int kFewWarps = 8, kFinishWarps = kThreads / 32 - kFewWarps;


struct Ctl {
  uint64_t full[kMaxStages];    // operands landed (the leader's counts both CTAs)
  uint64_t empty[kMaxStages];   // the stage's MMAs are done
  uint64_t tfull[2];            // accumulator complete
  uint64_t sfull[kSumBuffers], sempty[kSumBuffers];   // few slots: a unit's sums
  uint64_t tempty[2];           // (leader) accumulator drained by every epilogue warp of the pair
  uint64_t qfull[kQueue], qempty[kQueue];             // tile queue
  int4 queue[kQueue][2];
  uint32_t tmem_base;
  int abort_flag;
  uint32_t warp_sum[kThreads / 32];
  int warp_most[kThreads / 32];
  int most;                     // slots of the largest group
  uint32_t first[kMaxE + 1];    // tiles before each group
  union {
    int2 group[kFewGroups];       // few slots: (16 expert + slots - 1, first slot) of the groups that have any
    float weight[8][kTileN / 2];   // SwiGLU: route weights of the columns that a warp takes
  };
};

template <Mode kMode>
constexpr size_t smem_bytes() {
  return 1024 + static_cast<size_t>(Cfg<kMode>::kStages) * (kABytes + kBBytes) + Cfg<kMode>::kStoreBytes + sizeof(Ctl);
}
static_assert(smem_bytes<kForward>() <= 232448 && smem_bytes<kWgrad>() <= 232448, "shared memory budget");

struct Params {
  const int32_t* group_start;
  const int32_t* group_rows;
  const int32_t* route_ids;
  const float* route_weights;
  int32_t* status;
  const uint16_t* x;
  const uint16_t* w;
  uint16_t* y;
  uint16_t* pre;
  void* dw;        // wgrad
  int64_t ldx, ldy, ldpre, R;
  int rows;        // slots of the row buffers
  int E;
  int m;           // M extent of the products (2I for SwiGLU)
  int z;           // contraction extent (0 for wgrad: the group's slots)
  int n;           // wgrad: N extent
  uint32_t format; // 0 FP16, 1 BF16
  int accumulate;  // wgrad: add to dw, leave the dw of empty groups
  int late_tmem;    // take tensor memory only once the tiles are known to run
  int a_one, b_one; // an MN-major stage of A, B is one copy (its width a multiple of 64), else one per 64 columns
};

// The tensors of a launch.
struct Maps {
  CUtensorMap a;
  CUtensorMap b[3];    // K-major B: boxes of 32, 64 and 128 slots; wgrad: [0]
  CUtensorMap ag, bg;  // wgrad: single rows, for gather4
};

struct Tile {
  int e, m0;       // group, first row of the M side
  int n0, nt;      // first column of the N side, its width
  int s0, slots;   // the group's first slot and its slots
  int nkb;         // contraction blocks
};

// A group's slots; a group outside the buffer counts as empty.
__device__ __forceinline__ bool group_at(const Params& p, int e, int& s0, int& n) {
  s0 = p.group_start[e];
  n = p.group_rows[e];
  if (n == 0) return true;
  if (s0 < 0 || n < 0 || s0 > p.rows - n) {
    n = 0;
    return false;
  }
  return true;
}
template <Mode kMode>
__device__ __forceinline__ uint32_t tiles_of(const Params& p, int n) {
  const uint32_t mt = (p.m + kTileM - 1) / kTileM;
  if (kMode == kWgrad) return n == 0 && p.accumulate ? 0u : mt * ((p.n + kTileN - 1) / kTileN);
  return mt * ((n + kTileN - 1) / kTileN);
}

// Fills ctl->first (all threads).
template <Mode kMode>
__device__ __forceinline__ void count_tiles(const Params& p, Ctl* ctl) {
  const int per = (p.E + kThreads - 1) / kThreads;
  const int e0 = min(static_cast<int>(threadIdx.x) * per, p.E), e1 = min(e0 + per, p.E);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t sum = 0;
  int most = 0;
  bool bad = false;
  for (int e = e0; e < e1; ++e) {
    int s0, n;
    bad |= !group_at(p, e, s0, n);
    const uint32_t t = tiles_of<kMode>(p, n);
    ctl->first[e] = sum;
    sum += t;
    most = max(most, n);
  }
  if (bad && blockIdx.x == 0 && p.status) atomicOr(p.status, MOE_DEV_BAD_GROUP);
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    ctl->warp_sum[warp] = inc;
    ctl->warp_most[warp] = most;
  }
  __syncthreads();
  uint32_t base = inc - sum;
  for (int w = 0; w < warp; ++w) base += ctl->warp_sum[w];
  const uint32_t mt = (p.m + kTileM - 1) / kTileM;
  for (int e = e0; e < e1; ++e) {
    const uint32_t at = ctl->first[e] + base;
    ctl->first[e] = at;
    if (kMode == kForward || kMode == kSwiglu) {
      // (each group has mt tiles where this table is used)
      int s0, n;
      group_at(p, e, s0, n);
      if (n > 0 && at / mt < kFewGroups) ctl->group[at / mt] = make_int2(16 * e + min(n, 16) - 1, s0);
    }
  }
  if (threadIdx.x == kThreads - 1) {
    ctl->first[p.E] = base + sum;
    for (int w = 0; w < warp; ++w) most = max(most, ctl->warp_most[w]);
    ctl->most = most;
  }
}

// Walks a CTA pair's tiles in ascending order (a whole warp).  Each lane holds
// the table entries of one of 32 groups, so that most steps touch no memory.
template <Mode kMode>
struct Tiles {
  const Params& p;
  const Ctl* ctl;
  uint32_t tile, step, total;
  int base = 0;          // lane l holds group base + l
  uint32_t my_first = 0, my_past = 0;   // its tiles: [my_first, my_past)
  int my_s0 = 0, my_n = 0;
  int e = 0;             // group of `tile`

  __device__ __forceinline__ Tiles(const Params& p_, const Ctl* ctl_, uint32_t first, uint32_t step_)
      : p(p_), ctl(ctl_), tile(first), step(step_), total(ctl_->first[p_.E]) {
    load();
    find();
  }
  __device__ __forceinline__ bool done() const { return tile >= total; }
  __device__ __forceinline__ void load() {
    const int g = min(base + static_cast<int>(threadIdx.x % 32), p.E - 1);
    my_first = ctl->first[g];
    my_past = ctl->first[g + 1];
    group_at(p, g, my_s0, my_n);
  }
  __device__ __forceinline__ void find() {
    if (done()) return;
    // the first group whose tiles are not all before this one
    uint32_t past;
    while ((past = __ballot_sync(0xffffffffu, my_past > tile)) == 0) {
      base += 32;
      load();
    }
    e = base + __ffs(past) - 1;
  }
  __device__ __forceinline__ void next() {
    tile += step;
    find();
  }
  __device__ __forceinline__ Tile get() const {
    Tile t;
    const int n = __shfl_sync(0xffffffffu, my_n, e - base);
    t.e = e;
    t.s0 = __shfl_sync(0xffffffffu, my_s0, e - base);
    t.slots = n;
    const uint32_t local = tile - __shfl_sync(0xffffffffu, my_first, e - base);
    if (kMode == kWgrad) {
      const uint32_t nts = (p.n + kTileN - 1) / kTileN, m = local / nts;
      t.m0 = static_cast<int>(m * kTileM);
      t.n0 = static_cast<int>((local - m * nts) * kTileN);
      t.nt = min(kTileN, p.n - t.n0);
      t.nkb = (n + kTileZ - 1) / kTileZ;
    } else {
      t.nkb = (p.z + kTileZ - 1) / kTileZ;
      if (n <= kTileN) {
        t.m0 = static_cast<int>(local * kTileM);
        t.n0 = 0;
        t.nt = n;
        return t;
      }
      const uint32_t nts = (n + kTileN - 1) / kTileN, m = local / nts;
      const int width = static_cast<int>((n + nts - 1) / nts + 31) / 32 * 32;
      t.m0 = static_cast<int>(m * kTileM);
      t.n0 = static_cast<int>(local - m * nts) * width;
      t.nt = min(width, n - t.n0);
    }
    return t;
  }
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}
// Bounded wait while winding down: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  int dummy = 0;
  mbar_wait(bar, parity, &dummy);
}

// A place in the ring of stages.
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
};

// The queue's two sides.  A tile with nkb < 0 ends it.
template <Mode kMode>
__device__ __forceinline__ void publish_tiles(const Params& p, Ctl* ctl, uint32_t tile0, uint32_t step) {
  volatile int* abort_flag = &ctl->abort_flag;
  Tiles<kMode> tiles(p, ctl, tile0, step);
  for (uint32_t i = 0;; ++i) {
    const bool end = tiles.done();
    Tile t = {};
    t.nkb = -1;
    if (!end) {
      t = tiles.get();
      // every box, row and store of the tile follows from these
      if (!MOE_IN_BOUNDS(t.e >= 0 && t.e < p.E && t.m0 >= 0 && t.m0 < p.m && t.slots >= 0 && t.n0 >= 0 && t.nt > 0 &&
                         (t.slots == 0 || (t.s0 >= 0 && t.s0 <= p.rows - t.slots)) &&
                         t.n0 + t.nt <= (kMode == kWgrad ? p.n : t.slots))) {
        t = {};
        t.nt = 32;   // computes and stores nothing (wgrad: keeps clear of dw)
        t.m0 = p.m;
      }
    }
    const uint32_t q = i % kQueue;
    if (!warp_wait(smem_u32(&ctl->qempty[q]), ((i / kQueue) & 1u) ^ 1u, abort_flag)) return;
    if (threadIdx.x % 32 == 0) {
      ctl->queue[q][0] = make_int4(t.e, t.m0, t.n0, t.nt);
      ctl->queue[q][1] = make_int4(t.s0, t.slots, t.nkb, 0);
      mbar_arrive(smem_u32(&ctl->qfull[q]));
    }
    if (end) return;
    tiles.next();
  }
}
// The next tile; false at the end (or once a wait has run out).  kWarp: taken
// by a whole warp, else by one thread.
template <bool kWarp>
__device__ __forceinline__ bool take_tile(Ctl* ctl, uint32_t& i, Tile& t) {
  volatile int* abort_flag = &ctl->abort_flag;
  const uint32_t q = i % kQueue, parity = (i / kQueue) & 1u;
  ++i;
  const bool ok = kWarp ? warp_wait(smem_u32(&ctl->qfull[q]), parity, abort_flag)
                        : mbar_wait(smem_u32(&ctl->qfull[q]), parity, abort_flag);
  if (!ok) return false;
  const int4 a = ctl->queue[q][0], b = ctl->queue[q][1];
  t = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  if (kWarp) __syncwarp();
  if (!kWarp || threadIdx.x % 32 == 0) mbar_arrive(smem_u32(&ctl->qempty[q]));
  return t.nkb >= 0;
}

// Two values that this lane holds for columns c and c + 1 of its row, against
// the neighbour's: the even lane returns rows (lane, lane + 1) of column c,
// the odd lane rows (lane - 1, lane) of column c + 1.
template <typename T>
__device__ __forceinline__ uint32_t pair_rows(float v0, float v1, bool odd) {
  const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
  return odd ? Pack2<T>::store(got, v1) : Pack2<T>::store(v0, got);
}

// ---------------------------------------------------------------- few slots
//
// A decoding step's groups hold a slot or two, and its few tiles of 256 weight
// rows would keep few pairs busy.  The weights' bytes bound it: where no group
// has more than 16 slots (and no more than 640 groups have any), a unit is 16
// weight rows, whose contraction is split over 8, 4, 2 or 1 of a CTA's eight
// streaming warps (as many units run side by side as that leaves warps for).  A
// warp takes its blocks of 64 contraction elements through a ring of its own in
// shared memory (asynchronous 16-byte copies, 80-112 KB of weights in flight
// per SM, prefetched across units).  The other four warps add the sums, handed
// over through shared memory, so that no warp waits for another one's copies.
// (Loads into registers instead stalled at 17 GB/s per SM: beside this kernel's
// shared memory the L1 has room for few outstanding lines.)  The products are
// m16n8k16 MMAs with 8 or 16 slots as columns; as the order of the contraction
// is free, a lane's 16 contiguous bytes of a weight row serve as its A
// fragments of two MMAs, and the same 16 bytes of a slot's row as the B
// fragments.  One token through 9 of 257 experts (K 7168, N 512, SwiGLU): 16 us
// for 66 MB, of which about 3 are launch, tables and the first loads; 8 tokens
// 74 us (6.4 TB/s), 32 tokens 193 us (6.8 TB/s).
constexpr int kFewSlots = 16;

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes from global to shared memory, zeros where `bytes` is 0.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 load_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// kSlots: slots that a group has at most, 8 or 16.
template <int kSlots>
struct Few {
  static constexpr int kStages = kSlots == 8 ? 8 : 6;
  static constexpr int kStageBytes = (16 + kSlots) * 128;   // 16 weight rows and the slots: 64 elements each
  static constexpr int kSums = kFewWarps * kSlots * 16;     // the warps' sums
  static constexpr int kBuffers = kSlots == 8 ? kSumBuffers : kSumBuffers / 2;
  static_assert(kFewWarps * kStages * kStageBytes <= 6 * (kABytes + kBBytes), "the rings fit the operand stages");
  static_assert(kBuffers * kSums * 4 <= 8 * kRowsBytes, "the warps' sums");
};

// How the units are dealt: a unit of 16 weight rows is eight gates and their
// ups, or 16 rows in order; `side` units run side by side in a CTA, each on
// `split` warps.  The split is as wide as leaves a warp four blocks, or wider
// where the CTAs would not all have work.
template <Mode kMode>
struct FewUnits {
  int split, side, steps;   // steps: of `side` units, per group
  uint32_t total;           // steps of all groups
  __device__ __forceinline__ FewUnits(const Params& p, const Ctl* ctl) {
    const uint32_t groups = ctl->first[p.E] / ((p.m + kTileM - 1) / kTileM);
    const int units = (p.m + 15) / 16, nkb = (p.z + kTileZ - 1) / kTileZ;
    split = kFewWarps;
    while (split > 1 && nkb < 4 * split && groups * ((units * split + 15) / 16) >= gridDim.x) split /= 2;
    side = kFewWarps / split;
    steps = (units + side - 1) / side;
    total = groups * steps;
  }
};

// One of the eight streaming warps.
template <Mode kMode, typename T, int kSlots>
__device__ __forceinline__ void few_slots_stream(const Params& p, Ctl* ctl, uint8_t* ring, float* sums) {
  using F = Few<kSlots>;
  constexpr bool kGlu = kMode == kSwiglu;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &ctl->abort_flag;
  const FewUnits<kMode> f(p, ctl);
  const int nkb = (p.z + kTileZ - 1) / kTileZ;
  const int part = warp % f.split, side = warp / f.split;
  const int nst = part < nkb ? (nkb - part + f.split - 1) / f.split : 0;   // this warp's blocks of a unit
  const uint32_t base = smem_u32(ring) + warp * F::kStages * F::kStageBytes;

  // The copies run ahead: unit cu, block cb of it, into stage cs.
  uint32_t cu = blockIdx.x, cs = 0;
  int cb = 0;
  // this lane's 16-byte column of 4 rows, then of 2 slots, of each block
  const int chunk = lane % 8, sub = lane / 8;
  const uint16_t* cw[4];   // null: no such row
  const uint16_t* cx = nullptr;
  int cslots = 0;
  auto open = [&]() {
    if (cu >= f.total || nst == 0) return;
    int2 t = ctl->group[cu / f.steps];
    if (!MOE_IN_BOUNDS(t.x >= 0 && t.x / kFewSlots < p.E && t.y >= 0 && t.y <= p.rows - 1 - t.x % kFewSlots)) t = {0, 0};
    const int unit = static_cast<int>(cu % f.steps) * f.side + side;
    const uint16_t* we = p.w + static_cast<int64_t>(t.x / kFewSlots) * p.m * p.z;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * i + sub;
      const int r = kGlu ? 8 * unit + j % 8 : 16 * unit + j, top = kGlu ? p.m / 2 : p.m;
      cw[i] = r < top ? we + (static_cast<int64_t>(r) + (kGlu ? j / 8 * top : 0)) * p.z + 8 * chunk : nullptr;
    }
    cx = p.x + (static_cast<int64_t>(t.y) + sub) * p.ldx + 8 * chunk;
    cslots = t.x % kFewSlots + 1;
  };
  auto copy = [&]() {
    if (cu < f.total && nst > 0) {
      const int z = (part + cb * f.split) * kTileZ;
      const uint32_t st = base + cs * F::kStageBytes;
      const bool in = z + 8 * chunk < p.z;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * i + sub;
        const uint32_t dst = st + 128 * j + 16 * (chunk ^ (j & 7));
        copy16_async(dst, in && cw[i] ? cw[i] + z : p.w, in && cw[i] ? 16u : 0u);
      }
#pragma unroll
      for (int i = 0; i < kSlots / 4; ++i) {
        const int j = 4 * i + sub;
        if (j < cslots)
          copy16_async(st + 2048 + 128 * j + 16 * (chunk ^ (j & 7)), in ? cx + 4 * i * p.ldx + z : p.x, in ? 16u : 0u);
      }
      if (++cb == nst) {
        cb = 0;
        cu += gridDim.x;
        open();
      }
    }
    cs = cs + 1 == F::kStages ? 0 : cs + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  open();
  for (int i = 0; i < F::kStages - 1; ++i) copy();

  uint32_t s = 0, n = 0;
  for (uint32_t u = blockIdx.x; u < f.total; u += gridDim.x, ++n) {
    float d[kSlots / 8][4] = {};
    for (int b = 0; b < nst; ++b) {
      asm volatile("cp.async.wait_group %0;" ::"n"(F::kStages - 2) : "memory");
      __syncwarp();
      copy();   // into the stage read in the step before
      const uint32_t st = base + s * F::kStageBytes;
      const int g = lane / 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (columns 2 (lane % 4) + h: no two lanes of a quarter-warp share a bank)
        const uint32_t at = 128 * g + 16 * ((2 * (lane % 4) + h) ^ g);
        const uint4 a0 = load_shared16(st + at), a1 = load_shared16(st + 1024 + at);
#pragma unroll
        for (int c = 0; c < kSlots / 8; ++c) {
          const uint4 x = load_shared16(st + 2048 + 1024 * c + at);
          mma_16816<T>(d[c], a0.x, a1.x, a0.y, a1.y, x.x, x.y);
          mma_16816<T>(d[c], a0.z, a1.z, a0.w, a1.w, x.z, x.w);
        }
      }
      s = s + 1 == F::kStages ? 0 : s + 1;
      __syncwarp();
    }
    // sums[warp][slot][row]: weight rows lane / 4 and 8 on, slots 2 (lane % 4) and the next
    const uint32_t buf = n % F::kBuffers;
    if (!warp_wait(smem_u32(&ctl->sempty[buf]), ((n / F::kBuffers) & 1u) ^ 1u, abort_flag)) break;
    float* out = sums + buf * F::kSums + warp * kSlots * 16;
#pragma unroll
    for (int c = 0; c < kSlots / 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[(8 * c + 2 * (lane % 4) + (i & 1)) * 16 + lane / 4 + 8 * (i / 2)] = d[c][i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ctl->sfull[buf]));
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The finishing warps add the streaming warps' sums in order and write the
// results, each for every fourth of the units side by side.
template <Mode kMode, typename T, int kSlots>
__device__ __forceinline__ void few_slots_finish(const Params& p, Ctl* ctl, const float* sums) {
  using F = Few<kSlots>;
  constexpr bool kGlu = kMode == kSwiglu;
  constexpr int kMine = kSlots / 2;   // this lane's slots: lane / 16 + 0, 2, 4, ...
  const int lane = threadIdx.x % 32, row = lane % 16, turn = threadIdx.x / 32 - kFewWarps;
  volatile int* abort_flag = &ctl->abort_flag;
  const FewUnits<kMode> f(p, ctl);
  // route weights: ids two steps ahead, weights one (their loads follow one another)
  const bool weighted = kGlu && p.route_weights;
  int64_t id[kMine];
  float wt[kMine], next_wt[kMine];
  auto fetch_ids = [&](uint32_t u) {
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      id[c] = -1;
      if (!weighted || u >= f.total) continue;
      const int2 group = ctl->group[u / f.steps];
      const int slot = 2 * c + lane / 16;
      if (slot > group.x % kFewSlots) continue;
      id[c] = static_cast<int64_t>(group.y) + slot;
      if (!MOE_IN_BOUNDS(id[c] >= 0 && id[c] < p.rows)) id[c] = -1;
      if (p.route_ids && id[c] >= 0) id[c] = p.route_ids[id[c]];
    }
  };
  auto fetch_weights = [&](float (&w)[kMine]) {
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      w[c] = weighted ? 0.f : 1.f;
      if (id[c] >= 0 && (!p.route_ids || id[c] < p.R)) w[c] = p.route_weights[id[c]];
    }
  };
  fetch_ids(blockIdx.x);
  fetch_weights(wt);
  fetch_ids(blockIdx.x + gridDim.x);
  uint32_t n = 0;
  for (uint32_t u = blockIdx.x; u < f.total; u += gridDim.x, ++n) {
    const int2 group = ctl->group[u / f.steps];
    const int s0 = group.y;
    // (a group outside the buffer: no slot is written)
    const int slots = MOE_IN_BOUNDS(s0 >= 0 && s0 <= p.rows - 1 - group.x % kFewSlots) ? group.x % kFewSlots + 1 : 0;
    fetch_weights(next_wt);
    fetch_ids(u + 2 * gridDim.x);
    const uint32_t buf = n % F::kBuffers;
    if (!warp_wait(smem_u32(&ctl->sfull[buf]), (n / F::kBuffers) & 1u, abort_flag)) break;
    for (int side = turn; side < f.side; side += kFinishWarps) {
      const int unit = static_cast<int>(u % f.steps) * f.side + side;
      const float* in = sums + buf * F::kSums + side * f.split * kSlots * 16;
      float sum[kMine] = {};
      for (int w = 0; w < f.split; ++w)
#pragma unroll
        for (int c = 0; c < kMine; ++c) sum[c] += in[(w * kSlots + 2 * c + lane / 16) * 16 + row];
#pragma unroll
      for (int c = 0; c < kMine; ++c) {
        const int slot = 2 * c + lane / 16;
        const int64_t sl = static_cast<int64_t>(s0) + slot;
        const bool live = slot < slots;
        if (kGlu) {
          const float up = __shfl_down_sync(0xffffffffu, sum[c], 8);   // row + 8 of the same slot
          const int I = p.m / 2, i = 8 * unit + row % 8;
          if (live && i < I && p.pre)
            p.pre[sl * p.ldpre + (row < 8 ? i : I + i)] = static_cast<uint16_t>(Pack2<T>::store(sum[c], 0.f));
          if (live && i < I && row < 8)
            p.y[sl * p.ldy + i] =
                static_cast<uint16_t>(Pack2<T>::store(sum[c] * sigmoid_f32(sum[c]) * up * wt[c], 0.f));
        } else if (live && 16 * unit + row < p.m) {
          p.y[sl * p.ldy + 16 * unit + row] = static_cast<uint16_t>(Pack2<T>::store(sum[c], 0.f));
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ctl->sempty[buf]));
#pragma unroll
    for (int c = 0; c < kMine; ++c) wt[c] = next_wt[c];
  }
}

template <Mode kMode, typename T, int kSlots>
__device__ __forceinline__ void few_slots(const Params& p, Ctl* ctl, uint8_t* ring, float* sums) {
  if (threadIdx.x / 32 < kFewWarps)
    few_slots_stream<kMode, T, kSlots>(p, ctl, ring, sums);
  else
    few_slots_finish<kMode, T, kSlots>(p, ctl, sums);
}

// ---------------------------------------------------------------- tiles

// The route weights of the columns that a warp drains: 16 of every 32.
__device__ __forceinline__ void slot_weights(const Params& p, const Tile& t, int turn, float* out) {
  const int lane = threadIdx.x % 32;
  int64_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = 32 * i + lane, col = k / 16 * 32 + 16 * turn + k % 16;
    r[i] = col < t.nt ? static_cast<int64_t>(t.s0) + t.n0 + col : -1;
    if (!MOE_IN_BOUNDS(r[i] < p.rows)) r[i] = -1;
    if (r[i] >= 0 && p.route_ids) {
      r[i] = p.route_ids[r[i]];
      if (r[i] >= p.R) r[i] = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[32 * i + lane] = r[i] >= 0 ? p.route_weights[r[i]] : 0.f;
  __syncwarp();
}

template <Mode kMode, typename T, typename Out>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr bool kAmn = kMode == kDgrad || kMode == kWgrad;   // A stored along M
  constexpr bool kBmn = kMode == kWgrad;                      // B stored along N
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sA = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sC = sA + Cfg<kMode>::kStages * (kABytes + kBBytes);
  Ctl* ctl = reinterpret_cast<Ctl*>(sC + Cfg<kMode>::kStoreBytes);
  volatile int* abort_flag = &ctl->abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = pair::cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), 2 * Cfg<kMode>::kEpiWarps);
    }
    for (int b = 0; b < kSumBuffers; ++b) {
      mbar_init(smem_u32(&ctl->sfull[b]), kFewWarps);
      mbar_init(smem_u32(&ctl->sempty[b]), kFinishWarps);
    }
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(smem_u32(&ctl->qfull[q]), 1);
      // the producers, the leader's MMA issuer, the epilogue warps
      mbar_init(smem_u32(&ctl->qempty[q]), 2 + (rank == 0 ? 1 : 0) + Cfg<kMode>::kEpiWarps);
    }
    ctl->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b[0]);
  }
  // Tensor memory is taken while the group tables are still to be read, unless
  // the few-slots path, which has no use for it, is likely to run.
  if (!p.late_tmem && warp == 1) {
    pair::tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    pair::tmem_relinquish();
  }
  __syncwarp();
  pair::cluster_arrive();   // (waited for below: the peer's latency passes meanwhile)
  pdl_launch_dependents();
  pdl_wait();
  count_tiles<kMode>(p, ctl);
  tc_fence_before();
  __syncthreads();
  pair::cluster_wait();  // the peer's copies and arrivals target initialised barriers
  tc_fence_after();
  const uint32_t total = ctl->first[p.E];
  const uint32_t tile0 = blockIdx.x / 2, step = gridDim.x / 2;
  constexpr bool kFew = kMode == kForward || kMode == kSwiglu;
  // With more than 8 slots in a group the tiles are faster unless half of the
  // pairs would have none (24 groups of 9 slots, K 1160, N 712, 72 tiles: 11.9
  // us against 15.0; 14 of up to 9, K 5936, N 320, 28 tiles: 35 against 16).
  if (kFew && ctl->most <= (2 * total <= step ? kFewSlots : 8) &&
      total <= kFewGroups * static_cast<uint32_t>((p.m + kTileM - 1) / kTileM)) {
    if (ctl->most <= 8)
      few_slots<kMode, T, 8>(p, ctl, sA, reinterpret_cast<float*>(sC));
    else
      few_slots<kMode, T, 16>(p, ctl, sA, reinterpret_cast<float*>(sC));
    __syncthreads();
    if (threadIdx.x == 0 && ctl->abort_flag && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
    if (!p.late_tmem) {
      pair::cluster_sync();  // (tensor memory is given back by both CTAs together)
      if (warp == 1) pair::tmem_dealloc(ctl->tmem_base, 512);
    }
    return;
  }
  if (p.late_tmem) {
    if (warp == 1) {
      pair::tmem_alloc(smem_u32(&ctl->tmem_base), 512);
      pair::tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    pair::cluster_sync();
    tc_fence_after();
  }
  const uint32_t tmem_base = ctl->tmem_base;
  // Where no tile is wide, B's share of a stage is smaller and the ring longer:
  // few columns are soon multiplied, and it is the copies' latency that bounds
  // (24 groups of 65 slots, K 1160, N 712: a block every 0.33 us with 6 stages).
  const int bstage = kMode == kWgrad || ctl->most > 128 ? kBBytes : ctl->most > 64 ? kBBytes / 2 : kBBytes / 4;
  const int stages = kMode == kWgrad ? Cfg<kMode>::kStages : bstage == kBBytes ? 6 : bstage == kBBytes / 2 ? 8 : 9;
  uint8_t* sB = sA + stages * kABytes;
  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------ producers (A: warp 0, B: warp 6)
    const bool isA = warp == 0;
    const uint32_t lead_full0 = pair::mapa_shared(smem_u32(&ctl->full[0]), 0);
    Ring ring;
    bool ok = true;
    // lane 0 issues (wgrad's row-by-row copies: all lanes)
    constexpr bool kWarp = kMode == kWgrad;
    uint32_t next = 0;
    Tile t;
    while ((kWarp || lane == 0) && ok && take_tile<kWarp>(ctl, next, t)) {
      const int half = (t.nt + 31) / 32 * 16;               // N columns of each CTA
      const int chunks = (half + 63) / 64;                  // N-major B: 64-column boxes
      const int bsel = half <= 32 ? 0 : half <= 64 ? 1 : 2; // K-major B: box of 32, 64 or 128 slots
      const uint32_t bbytes = kBmn ? 8192u * (p.b_one ? 2 : chunks) : 4096u << bsel;
      const int arow = t.m0 + 128 * static_cast<int>(rank), bcol = t.n0 + static_cast<int>(rank) * half;
      // wgrad: a last block inside the buffer's first 64 slots cannot be a window that ends with the group
      const int last = kMode == kWgrad && t.slots % kTileZ && t.s0 + t.slots < kTileZ ? t.nkb - 1 : t.nkb;
      if (lane == 0) {
        for (int kb = 0; kb < last; ++kb, ring.next(stages)) {
          const int s = ring.s;
          if (!mbar_wait(smem_u32(&ctl->empty[s]), ring.phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full = lead_full0 + 8u * s;
          const uint32_t dst = smem_u32((isA ? sA : sB) + s * (isA ? kABytes : bstage));
          const int z = kb * kTileZ;
          if (isA && rank == 0) mbar_arrive_expect_tx(smem_u32(&ctl->full[s]), 2u * (kABytes + bbytes));
          if (kMode == kWgrad) {
            // a window of 64 slots that ends where the group does: the rest reads as zeros
            const int have = min(kTileZ, t.slots - z), w0 = kTileZ - have, start = t.s0 + z - w0;
            if (isA) {
              if (p.a_one)
                pair::load_4d(dst, &maps.a, full, 0, w0, arow / 64, start);
              else
                for (int j = 0; j < 2; ++j) pair::load_3d(dst + 8192u * j, &maps.a, full, arow + 64 * j, w0, start);
            } else if (p.b_one) {
              pair::load_4d(dst, &maps.b[0], full, 0, w0, bcol / 64, start);
            } else {
              for (int j = 0; j < chunks; ++j)
                pair::load_3d(dst + 8192u * j, &maps.b[0], full, bcol + 64 * j, w0, start);
            }
          } else if (!isA) {
            pair::load_2d(dst, &maps.b[bsel], full, z, t.s0 + bcol);
          } else if (kMode == kForward) {
            pair::load_3d(dst, &maps.a, full, z, arow, t.e);
          } else if (kMode == kSwiglu) {
            pair::load_5d(dst, &maps.a, full, z, 0, 0, arow / 16, t.e);
          } else if (p.a_one) {
            pair::load_4d(dst, &maps.a, full, 0, z, arow / 64, t.e);
          } else {
            for (int j = 0; j < 2; ++j) pair::load_3d(dst + 8192u * j, &maps.a, full, arow + 64 * j, z, t.e);
          }
        }
      }
      if (kWarp) {
        ring.s = __shfl_sync(0xffffffffu, ring.s, 0);
        ring.phase = __shfl_sync(0xffffffffu, ring.phase, 0);
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (kMode == kWgrad && last < t.nkb) {
        // row by row instead; row -1 reads as zeros
        const int s = ring.s, z = last * kTileZ;
        if (!ok || !warp_wait(smem_u32(&ctl->empty[s]), ring.phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t full = lead_full0 + 8u * s;
        const uint32_t dst = smem_u32((isA ? sA : sB) + s * (isA ? kABytes : kBBytes)) + (lane & 15) * 512u;
        if (isA && rank == 0 && lane == 0) mbar_arrive_expect_tx(smem_u32(&ctl->full[s]), 2u * (kABytes + bbytes));
        const int r0 = z + (lane & 15) * 4;
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = r0 + i < t.slots ? t.s0 + r0 + i : -1;
        const int j = lane / 16;   // 64-column box
        if (isA)
          pair::gather4(dst + 8192u * j, &maps.ag, full, arow + 64 * j, r[0], r[1], r[2], r[3]);
        else if (8192u * j < bbytes)
          pair::gather4(dst + 8192u * j, &maps.bg, full, bcol + 64 * j, r[0], r[1], r[2], r[3]);
        __syncwarp();
        ring.next(stages);
      }
    }
    // wind down: let the copies already issued (at most a ring's) land before
    // the CTA exits; a stage that has none under way has completed this phase
    if (!ok && lane == 0 && rank == 0)
      for (int j = 0; j < stages; ++j) {
        drain_wait(smem_u32(&ctl->full[ring.s]), ring.phase ^ 1u);
        ring.next(stages);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && lane == 0) {
      uint32_t done = 0, next = 0;
      Ring ring;
      // Descriptors of the first stage's first 16 contraction elements; the others'
      // differ in the address alone (its field is 14 bits of 16-byte units, which
      // no address of shared memory exceeds).  One thread issues everything, so
      // its few instructions per block are what narrow tiles cost.
      const uint64_t da = kAmn ? pair::sw128_mnmajor_desc(smem_u32(sA), 8192u) : sw128_kmajor_desc(smem_u32(sA));
      const uint64_t db = kBmn ? pair::sw128_mnmajor_desc(smem_u32(sB), 8192u) : sw128_kmajor_desc(smem_u32(sB));
      const uint32_t a_lo = static_cast<uint32_t>(da), a_hi = static_cast<uint32_t>(da >> 32);
      const uint32_t b_lo = static_cast<uint32_t>(db), b_hi = static_cast<uint32_t>(db >> 32);
      int last = -1;   // the last stage used, and its phase
      uint32_t last_phase = 0;
      bool ok = true;
      Tile t;
      while (ok && take_tile<false>(ctl, next, t)) {
        if (t.nkb == 0) continue;
        const uint32_t idesc = pair::idesc_f16(p.format, kAmn, kBmn, (t.nt + 31) / 32 * 32);
        const uint32_t tb = done & 1u, d = tmem_base + tb * kTileN;
        if (!mbar_wait(smem_u32(&ctl->tempty[tb]), ((done >> 1) & 1u) ^ 1u, abort_flag)) break;
        tc_fence_after();
        for (int kb = 0; kb < t.nkb; ++kb, ring.next(stages)) {
          const int s = ring.s;
          if (!mbar_wait(smem_u32(&ctl->full[s]), ring.phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = a_lo + s * (kABytes >> 4), b = b_lo + s * (bstage >> 4);
#pragma unroll
          for (int kk = 0; kk < kTileZ / 16; ++kk)
            pair::umma_f16(d, a + kk * (kAmn ? 128 : 2), a_hi, b + kk * (kBmn ? 128 : 2), b_hi, idesc,
                           kb > 0 || kk > 0 ? 1u : 0u);
          pair::umma_commit(smem_u32(&ctl->empty[s]));
          last = s;
          last_phase = ring.phase;
        }
        if (ok) {
          pair::umma_commit(smem_u32(&ctl->tfull[tb]));
          ++done;
        }
      }
      // no MMA may still be writing TMEM when it is released
      if (last >= 0) drain_wait(smem_u32(&ctl->empty[last]), last_phase);
    }
    __syncwarp();
  } else if (warp == 11) {
    publish_tiles<kMode>(p, ctl, tile0, step);
  } else if (warp < 6 || Cfg<kMode>::kEpiWarps == 8) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;   // the lanes of tensor memory that this warp may read
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    const int epi = warp < 6 ? warp - 2 : warp - 3, turn = warp < 6 ? 0 : 1;
    uint32_t done = 0, next = 0;
    bool ok = true;
    Tile t;
    while (ok && take_tile<true>(ctl, next, t)) {
      const uint32_t tb = done & 1u;
      // (fetched while the products still run)
      if (kMode == kSwiglu && p.route_weights) slot_weights(p, t, turn, ctl->weight[epi]);
      if (t.nkb > 0) {
        ok = warp_wait(smem_u32(&ctl->tfull[tb]), (done >> 1) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t acc = lanes + tb * kTileN;
      if (kMode == kForward || kMode == kDgrad) {
        // 32 columns (slots) at a time, neighbouring lanes' rows paired into
        // 4-byte stores (a transposition through shared memory, with 16-byte
        // stores, took 1.7% from products that the tensor cores bound)
        const bool odd = lane & 1;
        const int row = t.m0 + 128 * static_cast<int>(rank) + 32 * q + (lane & ~1);
        uint16_t* out = p.y + (static_cast<int64_t>(t.s0) + t.n0) * p.ldy + row;
        for (int c = 0; c < t.nt; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(acc + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t w = pair_rows<T>(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), odd);
            const int col = c + j + (odd ? 1 : 0);
            if (col < t.nt && row < p.m) *reinterpret_cast<uint32_t*>(out + col * p.ldy) = w;
          }
        }
      } else if (kMode == kSwiglu) {
        // 16 columns (slots) at a time through the warp's shared memory, then
        // 16-byte stores by two lanes a slot: eight gates and their ups each
        uint8_t* rows = sC + epi * kRowsBytes;
        const int I = p.m / 2, i = t.m0 / 2 + 64 * static_cast<int>(rank) + 16 * q + 8 * (lane & 1);
        const int64_t s0 = static_cast<int64_t>(t.s0) + t.n0;
        for (int c = 16 * turn; c < t.nt; c += 32) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(acc + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) *reinterpret_cast<uint32_t*>(rows + j * kRowsPitch + 4 * lane) = v[j];
          __syncwarp();
          const int col = c + lane / 2;
          if (col < t.nt && i < I) {
            const float4* in = reinterpret_cast<const float4*>(rows + lane / 2 * kRowsPitch + 64 * (lane & 1));
            const float4 ga = in[0], gb = in[1], ua = in[2], ub = in[3];
            const float g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
            const float u[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
            const float wt = p.route_weights ? ctl->weight[epi][c / 32 * 16 + lane / 2] : 1.f;
            float h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = g[j] * sigmoid_f32(g[j]) * u[j] * wt;
            *reinterpret_cast<uint4*>(p.y + (s0 + col) * p.ldy + i) = pack8<T>(h);
            if (p.pre) {
              uint16_t* pre = p.pre + (s0 + col) * p.ldpre + i;
              *reinterpret_cast<uint4*>(pre) = pack8<T>(g);
              *reinterpret_cast<uint4*>(pre + I) = pack8<T>(u);
            }
          }
          __syncwarp();
        }
      } else {
        // rows of dw, transposed through the warp's 4 KB of shared memory
        // (128-byte swizzle) into stores of whole 128-byte lines
        constexpr int kCols = 128 / sizeof(Out);   // columns of a line
        const int row0 = t.m0 + 128 * static_cast<int>(rank) + 32 * q;
        uint8_t* box = sC + epi * 4096;
        for (int c = kCols * turn; c < t.nt; c += 2 * kCols) {
#pragma unroll
          for (int h = 0; h < kCols / 32; ++h) {
            uint32_t v[32];
            if (t.nkb > 0) {
              tmem_ld_32x32b_x32(acc + c + 32 * h, v);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0u;
            }
            if (sizeof(Out) == 4) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(box + 128 * lane + 16 * (k ^ (lane & 7))) =
                    make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[8 * k + j]);
                *reinterpret_cast<uint4*>(box + 128 * lane + 16 * ((4 * h + k) ^ (lane & 7))) = pack8<T>(f);
              }
            }
          }
          __syncwarp();
          // eight lanes a row, four rows at a time
          const int chunk = lane % 8, col = t.n0 + c + chunk * static_cast<int>(16 / sizeof(Out));
          Out* out = static_cast<Out*>(p.dw) + (static_cast<int64_t>(t.e) * p.m + row0) * p.n + col;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + lane / 8;
            if (row0 + r < p.m && col < p.n) {
              uint4 v = *reinterpret_cast<const uint4*>(box + 128 * r + 16 * (chunk ^ (r & 7)));
              uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * p.n);
              if (sizeof(Out) == 4 && p.accumulate) {
                const uint4 old = *dst;
                v.x = __float_as_uint(__uint_as_float(old.x) + __uint_as_float(v.x));
                v.y = __float_as_uint(__uint_as_float(old.y) + __uint_as_float(v.y));
                v.z = __float_as_uint(__uint_as_float(old.z) + __uint_as_float(v.z));
                v.w = __float_as_uint(__uint_as_float(old.w) + __uint_as_float(v.w));
              }
              *dst = v;
            }
          }
          __syncwarp();
        }
      }
      if (t.nkb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 1)
            pair::mbar_arrive_cluster(pair::mapa_shared(smem_u32(&ctl->tempty[tb]), 0));
          else
            mbar_arrive(smem_u32(&ctl->tempty[tb]));
        }
        ++done;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  pair::cluster_sync();  // neither CTA leaves while the pair still touches its memory
  tc_fence_after();
  if (threadIdx.x == 0 && ctl->abort_flag && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
  if (warp == 1) pair::tmem_dealloc(tmem_base, 512);
}

// Launches the kernel with as many pairs as there can be tiles, at most as many
// as the GPU holds at once (a larger persistent grid would run a second wave).
template <Mode kMode, typename T, typename Out>
moe_status launch_grouped(int64_t most_tiles, const DeviceInfo& dev, cudaStream_t stream,
                          const Maps& maps, const Params& p) {
  constexpr auto kernel = grouped_kernel<kMode, T, Out>;
  constexpr size_t smem = smem_bytes<kMode>();
  static std::mutex mu;
  static int pairs[64] = {};
  int n;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (pairs[dev.device] == 0) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
          cudaSuccess)
        return MOE_ERR_CUDA;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(dev.sms / 2 * 2));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int fit = 0;
      if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess || fit < 1) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
      }
      pairs[dev.device] = fit;
    }
    n = pairs[dev.device];
  }
  if (most_tiles < n) n = static_cast<int>(most_tiles);
  MOE_CUDA_TRY(launch_pdl(kernel, dim3(2u * n), dim3(kThreads), smem, stream, 2, maps, p));
  return MOE_OK;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == MOE_TYPE_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
         : dtype == MOE_TYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
}
// Rows of `width` 16-bit elements, boxes of 64 elements (128 bytes) by `box_rows`.
bool rows_map(CUtensorMap* m, int dtype, const void* base, int64_t width, int64_t rows, int64_t ld, uint32_t box_rows) {
  return encode_tensor_map_2d_typed(m, map_type(dtype), base, static_cast<uint64_t>(width),
                                    static_cast<uint64_t>(rows), static_cast<uint64_t>(ld) * 2, 64, box_rows,
                                    CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}
// A dense [e, n, k] tensor.
bool weight_map(CUtensorMap* m, int dtype, const void* base, int64_t e, int64_t n, int64_t k, uint32_t box_k,
                uint32_t box_n) {
  const uint64_t eb = static_cast<uint64_t>(type_bytes(dtype));
  const uint64_t dims[3] = {static_cast<uint64_t>(k), static_cast<uint64_t>(n), static_cast<uint64_t>(e)};
  const uint64_t strides[2] = {dims[0] * eb, dims[0] * dims[1] * eb};
  const uint32_t box[3] = {box_k, box_n, 1};
  return encode_tensor_map(m, map_type(dtype), 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ==
         CUDA_SUCCESS;
}

// Windows of 64 rows: row i of the window that starts at row j is row i + j,
// and rows past the window read as zeros.  A block of a group's last rows is
// the end of the window that ends with the group.  Boxes of 64 columns, or of
// two such boxes one after the other (`one`; the width is a multiple of 64).
bool window_map(CUtensorMap* m, int dtype, const void* base, int64_t width, int64_t rows, int64_t ld, bool one) {
  const uint64_t row = static_cast<uint64_t>(ld) * 2, starts = static_cast<uint64_t>(rows > 64 ? rows - 63 : 1);
  const uint64_t high = static_cast<uint64_t>(rows < 64 ? rows : 64);
  if (one) {
    const uint64_t dims[4] = {64, high, static_cast<uint64_t>(width) / 64, starts};
    const uint64_t strides[3] = {row, 128, row};
    const uint32_t box[4] = {64, 64, 2, 1};
    return encode_tensor_map(m, map_type(dtype), 4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ==
           CUDA_SUCCESS;
  }
  const uint64_t dims[3] = {static_cast<uint64_t>(width), high, starts};
  const uint64_t strides[2] = {row, row};
  const uint32_t box[3] = {64, 64, 1};
  return encode_tensor_map(m, map_type(dtype), 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ==
         CUDA_SUCCESS;
}

bool ok_sizes(int64_t rows, int E, int N, int K) {
  return rows >= 0 && rows < (int64_t(1) << 31) && E >= 1 && E <= 2048 && N >= 8 && N % 8 == 0 && K >= 8 && K % 8 == 0 &&
         static_cast<int64_t>(N) * K <= kMostElements / E;
}
bool ok_stride(int64_t ld, int64_t width) { return ld % 8 == 0 && ld >= width && ld <= kMostElements; }

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_grouped_gemm(const moe_grouped_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  if (!is_half_type(a->dtype)) return MOE_ERR_DTYPE;
  const bool fwd = a->direction == MOE_GROUPED_FORWARD, glu = a->epilogue == MOE_GROUPED_SWIGLU;
  if ((!fwd && a->direction != MOE_GROUPED_INPUT_GRADIENT) || (!glu && a->epilogue != MOE_GROUPED_PLAIN) ||
      (glu && (!fwd || a->N % 16)) || !ok_sizes(a->rows, a->E, a->N, a->K) || a->R < 0)
    return MOE_ERR_SHAPE;
  const int64_t in = fwd ? a->K : a->N, out = fwd ? (glu ? a->N / 2 : a->N) : a->K;
  const bool pre = glu && a->pre;
  if (!ok_stride(a->ldx, in) || !ok_stride(a->ldy, out) || (pre && !ok_stride(a->ldpre, a->N))) return MOE_ERR_SHAPE;
  if (a->rows == 0) return MOE_OK;
  if (!a->x || !a->w || !a->y || !a->group_start || !a->group_rows) return MOE_ERR_NULL;
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned16(a->y) || (pre && !aligned16(a->pre)) ||
      !aligned4(a->group_start, a->group_rows, a->device_status) || (glu && !aligned4(a->route_ids, a->route_weights)))
    return MOE_ERR_ALIGN;
  const Rows rx{a->x, a->rows, a->ldx, in}, ry{a->y, a->rows, a->ldy, out}, rp{a->pre, pre ? a->rows : 0, a->ldpre, a->N};
  const Rows rw{a->w, 1, 0, static_cast<int64_t>(a->E) * a->N * a->K};   // (one row)
  if (overlap(ry, rx, 2) || overlap(ry, rw, 2) || overlap(rp, rx, 2) || overlap(rp, rw, 2) || overlap(rp, ry, 2))
    return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (dev.major != 10 || dev.minor != 3) return MOE_ERR_DEVICE;
  const void* ptrs[] = {a->x, a->w, a->y, pre ? a->pre : nullptr, a->group_start, a->group_rows,
                        glu ? a->route_ids : nullptr, glu ? a->route_weights : nullptr, a->device_status};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  Params p = {};
  p.group_start = a->group_start;
  p.group_rows = a->group_rows;
  p.route_ids = glu && a->route_weights ? a->route_ids : nullptr;
  p.route_weights = glu ? a->route_weights : nullptr;
  p.status = a->device_status;
  p.x = a->x;
  p.w = a->w;
  p.ldx = a->ldx;
  p.y = a->y;
  p.pre = pre ? a->pre : nullptr;
  p.ldy = a->ldy;
  p.ldpre = a->ldpre;
  p.R = a->R;
  p.rows = static_cast<int>(a->rows);
  p.E = a->E;
  p.m = fwd ? a->N : a->K;
  p.z = fwd ? a->K : a->N;
  p.format = a->dtype == MOE_TYPE_BF16 ? 1u : 0u;
  Maps maps;
  bool ok = true;
  for (int i = 0; i < 3; ++i) ok = ok && rows_map(&maps.b[i], a->dtype, a->x, in, a->rows, a->ldx, 32u << i);
  const uint64_t K = static_cast<uint64_t>(a->K), N = static_cast<uint64_t>(a->N), E = static_cast<uint64_t>(a->E);
  if (glu) {
    // rows 8 i + j of the gate, then of the up half, j < 8
    const uint64_t dims[5] = {K, 8, 2, N / 16, E};
    const uint64_t strides[4] = {2 * K, N * K, 16 * K, 2 * N * K};
    const uint32_t box[5] = {64, 8, 2, 8, 1};
    ok = ok && encode_tensor_map(&maps.a, map_type(a->dtype), 5, a->w, dims, strides, box,
                                 CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
  } else if (!fwd && a->K % 64 == 0) {
    // two 64-column boxes as one copy
    p.a_one = 1;
    const uint64_t dims[4] = {64, N, K / 64, E};
    const uint64_t strides[3] = {2 * K, 128, 2 * N * K};
    const uint32_t box[4] = {64, 64, 2, 1};
    ok = ok && encode_tensor_map(&maps.a, map_type(a->dtype), 4, a->w, dims, strides, box,
                                 CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
  } else {
    ok = ok && weight_map(&maps.a, a->dtype, a->w, a->E, a->N, a->K, 64, fwd ? 128 : 64);
  }
  if (!ok) return MOE_ERR_CUDA;
  maps.ag = maps.bg = maps.a;  // not used
  const int64_t mt = ceil_div(p.m, kTileM);
  const int64_t groups = a->E < a->rows ? a->E : a->rows;
  int64_t most = mt * (ceil_div(a->rows, kTileN) + groups);
  // (0.6 us either way: at 144 slots for 9 groups of one, at 1560 for 24 of 65)
  p.late_tmem = fwd && a->rows <= 2 * kFewSlots * groups ? 1 : 0;
  // (the few-slots path has a unit of 16 rows for each CTA)
  if (fwd && most < ceil_div(p.m, 32) * groups) most = ceil_div(p.m, 32) * groups;
  const bool bf = a->dtype == MOE_TYPE_BF16;
  if (glu)
    return bf ? launch_grouped<kSwiglu, __nv_bfloat16, __nv_bfloat16>(most, dev, stream, maps, p)
              : launch_grouped<kSwiglu, __half, __half>(most, dev, stream, maps, p);
  if (fwd)
    return bf ? launch_grouped<kForward, __nv_bfloat16, __nv_bfloat16>(most, dev, stream, maps, p)
              : launch_grouped<kForward, __half, __half>(most, dev, stream, maps, p);
  return bf ? launch_grouped<kDgrad, __nv_bfloat16, __nv_bfloat16>(most, dev, stream, maps, p)
            : launch_grouped<kDgrad, __half, __half>(most, dev, stream, maps, p);
}

moe_status moe_grouped_wgrad(const moe_grouped_wgrad_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  if (!is_half_type(a->dtype) || (a->dw_dtype != a->dtype && a->dw_dtype != MOE_TYPE_FP32)) return MOE_ERR_DTYPE;
  if (a->accumulate && a->dw_dtype != MOE_TYPE_FP32) return MOE_ERR_DTYPE;
  if (!ok_sizes(a->rows, a->E, a->N, a->K) || !ok_stride(a->lddy, a->N) || !ok_stride(a->ldx, a->K)) return MOE_ERR_SHAPE;
  if (!a->dw || !a->group_start || !a->group_rows || (a->rows > 0 && (!a->dy || !a->x))) return MOE_ERR_NULL;
  if (!aligned16(a->dy) || !aligned16(a->x) || !aligned16(a->dw) ||
      !aligned4(a->group_start, a->group_rows, a->device_status))
    return MOE_ERR_ALIGN;
  const int64_t bd = static_cast<int64_t>(type_bytes(a->dw_dtype)) * a->E * a->N * a->K;
  if (overlap(a->dw, bd, a->dy, extent_bytes(a->rows, a->lddy, a->N, 2)) ||
      overlap(a->dw, bd, a->x, extent_bytes(a->rows, a->ldx, a->K, 2)))
    return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (dev.major != 10 || dev.minor != 3) return MOE_ERR_DEVICE;
  const void* ptrs[] = {a->dy, a->x, a->dw, a->group_start, a->group_rows, a->device_status};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  Params p = {};
  p.group_start = a->group_start;
  p.group_rows = a->group_rows;
  p.status = a->device_status;
  p.rows = static_cast<int>(a->rows);
  p.E = a->E;
  p.m = a->N;
  p.n = a->K;
  p.format = a->dtype == MOE_TYPE_BF16 ? 1u : 0u;
  p.accumulate = a->accumulate ? 1 : 0;
  p.dw = a->dw;
  // without slots every group is empty and nothing is read: any address will do
  const void* dy = a->rows > 0 ? a->dy : static_cast<const uint16_t*>(a->dw);
  const void* x = a->rows > 0 ? a->x : static_cast<const uint16_t*>(a->dw);
  const int64_t rows = a->rows > 0 ? a->rows : 1;
  p.a_one = a->N % 64 == 0;
  p.b_one = a->K % 128 == 0;   // (each CTA's half then starts and ends at a multiple of 64)
  Maps maps;
  if (!window_map(&maps.a, a->dtype, dy, a->N, rows, a->lddy, p.a_one) ||
      !window_map(&maps.b[0], a->dtype, x, a->K, rows, a->ldx, p.b_one) ||
      !rows_map(&maps.ag, a->dtype, dy, a->N, rows, a->lddy, 1) ||
      !rows_map(&maps.bg, a->dtype, x, a->K, rows, a->ldx, 1))
    return MOE_ERR_CUDA;
  maps.b[1] = maps.b[2] = maps.b[0];  // not used
  const int64_t most = static_cast<int64_t>(a->E) * ceil_div(p.m, kTileM) * ceil_div(p.n, kTileN);
  const bool bf = a->dtype == MOE_TYPE_BF16;
  if (a->dw_dtype == MOE_TYPE_FP32)
    return bf ? launch_grouped<kWgrad, __nv_bfloat16, float>(most, dev, stream, maps, p)
              : launch_grouped<kWgrad, __half, float>(most, dev, stream, maps, p);
  return bf ? launch_grouped<kWgrad, __nv_bfloat16, __nv_bfloat16>(most, dev, stream, maps, p)
            : launch_grouped<kWgrad, __half, __half>(most, dev, stream, maps, p);
}

}  // extern "C"

MOE_BOUNDS_TU()
