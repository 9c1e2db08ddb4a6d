// expert_product.cu -- the per-expert products of a training step on the
// 5th-generation tensor cores. The rows of expert e are the sorted pairs
// p = offsets[e] .. offsets[e+1]-1; every output element is one fp32
// accumulation over its whole K axis, in increasing order, rounded once, the
// same whatever other rows there are (no split of K by the number of tiles):
//
//   forward   out[p, o] = sum_i a[p, i] * w[e, o, i]     a [P, n_in],  w [E, n_out, n_in]
//   rows' gradient
//             out[p, i] = sum_o a[p, o] * w[e, o, i]     a [P, n_out]
//   weights' gradient
//             dw[e, o, i] = sum_{p of e} dy[p, o] * a[p, i]
//
// Two CTAs of a cluster (one TPC) compute one 256 x 256 tile with
// cta_group::2: each stages 128 rows of the M operand and half of the N
// operand (32 KB per 64-deep K step), two thirds of the bytes that two separate
// 128 x 256 tiles would bring from L2. M is the feature axis, so its tiles
// are always full; N is the expert's rows in the first two forms (the MMA
// width follows the rows left, in steps of 32), the input features in the
// third.
//
// Operands come by TMA in 128-byte swizzled boxes of 64 elements. Where the
// K axis is the contiguous one in memory (forward: both; rows' gradient: a)
// the box is K-major; where it is the row axis (the weights in the rows'
// gradient, both operands of the weights' gradient) the box is MN-major and
// the MMA reads it transposed, so nothing is ever transposed in memory.
//
// The tensor cores align each product to the running sum and cut it off there,
// so a long run drifts towards zero: up to 2^-23 of the running sum per row in
// the worst case (5e-9 to 1e-8 of the sum per row for positive terms, measured).
// An fp32 weights' gradient is therefore summed in segments of K (kSegment),
// the first one stored, the others added by the TMA in L2, by the same thread
// one after the other. A bf16 gradient is summed in runs of kLongRun, which are
// added up in fp32 in TMEM and rounded once: 2^15 rows cannot drift further
// than half a step of bf16 (2^-8). The other two forms are one run (K at most
// 2^14).
//
// In the weights' gradient K is the expert's own rows. Whole groups of 16 rows
// (one MMA's K) go through the stages; groups that reach into the next expert's
// rows are not issued. The last 1 to 15 rows of an expert come as a box of 16
// rows of their own, whose other rows (the next expert's, or anything behind
// the last one) a warp of each CTA zeroes in both operands before the MMA may
// read them. The box is fetched when the tile's first stage is, so that neither
// the zeros nor their publication to the other CTA (a release at cluster scope,
// 4-5% of an fp32 gradient when it sat in the last stage) is waited for.
//
// Warp roles: 0..3 epilogue (TMEM -> registers -> global), 4 TMA producer,
// 5 TMEM allocation and, in the leader CTA, the MMA issuer, 6 the tail's
// zero writer. Persistent; two TMEM accumulators of 256 columns, so a tile's
// epilogue overlaps the next tile's MMAs. Every wait is bounded.
//
// Measured under the power cap (990 W, the state of a training step), 4096 x
// 4096: forward and rows' gradient of one expert x 32768 rows 814 us (1351
// TFLOP/s; cuBLAS 1371), of 48 experts x 683 rows, with 1.6 GB of weights to
// stream, 980 us (1122; 704 columns of MMA for 683 rows); fp32 weights' gradient
// there 1290 us (3.2 GB written), bf16 1084 us. Not capped, 8 experts x 4096
// rows: 692 us (1588) and 713 us. 333 rows: 246 us for the 1.6 GB of weights.
//
// What made the difference: expect_tx and waits without cluster-scope release
// and acquire (1693 -> 916 us for 48 x 683 rows); whole sectors and TMA stores
// in the epilogue (fp32 gradient 2154 -> 1207 us); warp-uniform issuing (8 x
// 4096 rows 756 -> 692 us, their weights' gradient 835 -> 713 us). What did not:
// bringing weights into L2 ahead (900 -> 995 us: the copies' issue rate is what
// it costs), eight epilogue warps (no faster), 32-byte stores straight from the
// lanes (to 30% slower with few rows per expert), coalesced stores from shared
// memory instead of TMA stores and eviction hints on those (no faster), nine
// smaller steps in flight for few rows (no faster). The fp32 weights' gradient
// is slower for its stores: 12 experts x 683 rows take 289 us, 209 without
// them, 196 without the epilogue (tensor pipe 53% busy, DRAM 2.8 TB/s; forward
// 90%). Where a store waits (DRAM, the L2 port, the staging boxes) is not known.
#include <algorithm>

#include "common.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kTileM = 256;  // features per CTA pair
constexpr int kTileN = 256;
// K steps in flight: the weights' gradient gives one up for its tails and a third store box per warp.
__host__ __device__ constexpr int stages(bool wgrad) { return wgrad ? 5 : 6; }
// N tiles of an expert that are in flight together, against all of its M tiles in turn: with all N tiles innermost,
// one expert of 32768 rows re-read its rows from HBM for every M tile (then 1166 us under the power cap, 879 us in
// bands of 8, 864 in bands of 4; the weights' gradient is 1% faster in bands of 8).
constexpr int kBand = 8;
constexpr uint32_t kOpBytes = 128 * 128;          // one operand's half tile: 128 x 64 bf16
constexpr uint32_t kStageBytes = 2 * kOpBytes;    // [M operand][N operand]
constexpr int kThreads = 224;
__host__ __device__ constexpr int barriers(bool wgrad) { return 2 * stages(wgrad) + 10; }
// K steps summed in TMEM before an fp32 gradient goes out. Over 16384 rows in one run it was 1.9e-5 off (2-norm, terms
// of both signs), over 65536 rows 7.6e-5. In segments of 14 steps (896 rows) the error does not grow with the rows:
// 6.5e-7 (terms of both signs), or 1.5e-6 low (positive terms), where fp32 multiply-adds have 1.9e-7. Time at 8192
// rows, 4096 x 4096: 238 us in one run, 252 us in segments of 32 steps, 272 us of 16, 286 us of 14, 326 us of 8.
constexpr int kSegment = 14;
// K steps of one run of a bf16 gradient (32768 rows). Without it, positive terms over 65536 rows came out 6.5e-4 low,
// over 524288 rows 3.2e-3, over 2097152 rows 1.2e-2. The sum of the runs so far stays in one accumulator while the
// other takes the next run; the MMA waits while the epilogue adds it (one expert of 131072 rows, 4096 x 4096: 3590 us,
// 3660 us in one run, within each other's noise). Experts of up to 32768 rows are one run.
constexpr int kLongRun = 512;
constexpr uint32_t kBoxBytes = 64 * 128;          // MN-major box: 64 K rows x 64 elements
constexpr uint32_t kStoreBox = 32 * 128;          // one warp's store box: 32 rows x 128 bytes
constexpr uint32_t kPieceBytes = 32 * 256;        // 32 rows x 128 features
// Output staging: kBoxes store boxes per epilogue warp (weights' gradient), or two pieces.
constexpr int kBoxes = 3;
__host__ __device__ constexpr uint32_t staging_bytes(bool wgrad) {
  return wgrad ? 4 * kBoxes * kStoreBox : 2 * kPieceBytes;
}
constexpr uint32_t kTailBox = 16 * 128;           // weights' gradient: 16 rows x 64 elements
constexpr uint32_t kTailBytes = 4 * kTailBox;     // two boxes of the M operand, two of the N operand

enum Form { kForward = 0, kRowGrad = 1, kWeightGrad = 2 };

// ------------------------------------------------------- cluster helpers --
__device__ __forceinline__ void named_bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The shared::cluster address of `addr` (this CTA's offset) in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void remote_arrive(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// With the writes of this thread's CTA before it, for an MMA that reads them from the other one.
__device__ __forceinline__ void remote_publish(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Bounded wait for what remote_publish released.
__device__ __forceinline__ bool wait_published(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
}

// Relaxed: it publishes no data of this thread (the copies' bytes order themselves).
__device__ __forceinline__ void remote_expect_tx(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar),
               "r"(bytes)
               : "memory");
}

// TMA load into this CTA's shared memory; the bytes complete on a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* map, uint32_t cluster_bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(cluster_bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// One lane of a warp that is here together; the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// A value that all lanes hold, for the compiler to know it.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One arrival on `bar` in both CTAs once this thread's MMAs so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// MN-major operand in 128-byte swizzled boxes of K rows x 64 elements: groups
// of 8 K rows 1024 bytes apart (stride byte offset), the next 64 elements one
// box further (leading byte offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t box_bytes) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(box_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// TMA store of one box of this CTA's shared memory; kAdd: fp32 add in place.
template <bool kAdd>
__device__ __forceinline__ void tma_store_2d(const void* map, uint32_t src, int c0, int c1) {
  if (kAdd)
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
                 "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The two TMEM accumulators as the MMA warp and the epilogue walk them, in step. A tile takes them in turn, one per
// segment, except where it carries its sum: then the first segment's holds the sum and the others all use the other.
struct Accumulators {
  int next = 0;
  uint32_t phases = 0;  // bit b: parity of the uses of accumulator b
  __device__ int of(int seg, bool carry) const { return carry && seg > 0 ? next ^ 1 : next; }
  __device__ uint32_t phase(int b) const { return (phases >> b) & 1u; }
  __device__ void used(int b) { phases ^= 1u << b; }
};

struct Tile {
  int e, m0, row0, rows, n0, n;  // n0, n: first column and width of the N axis (weights' gradient: input features)
};

// The sorted rows [begin, end) of one expert as `offsets` has them.
struct Rows {
  int begin, end;
  // No rows in place of a range that is not inside [0, P].
  __device__ Rows within(int P, int* status) const {
    if (begin >= 0 && end >= begin && end <= P) return *this;
    flag_status(status, MOE_DEV_BAD_INDEX);
    return Rows{0, 0};
  }
};

__device__ __forceinline__ Rows expert_rows(const int32_t* __restrict__ offsets, int e) {
  return Rows{__ldg(offsets + e), __ldg(offsets + e + 1)};
}

}  // namespace

template <int FORM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_product_kernel(const __grid_constant__ ProductMaps maps, const ProductArgs a) {
  constexpr bool kWG = FORM == kWeightGrad;
  constexpr bool kMmn = FORM != kForward;  // the M operand is MN-major
  constexpr bool kNmn = kWG;               // so is the N operand
  constexpr int kStages = stages(kWG);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int m_tiles = (a.m_total + kTileM - 1) / kTileM;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t staging = base + kStages * kStageBytes;  // 1024-byte aligned, as are the tails
  const uint32_t tails = staging + staging_bytes(kWG);
  const uint32_t bars = tails + (kWG ? 2 * kTailBytes : 0);
  auto full = [&](int s) { return bars + 8u * s; };  // in the leader CTA; one arrival per CTA and the bytes of both
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto tfull = [&](int b) { return bars + 8u * (2 * kStages + b); };
  auto tempty = [&](int b) { return bars + 8u * (2 * kStages + 2 + b); };  // in the leader CTA
  // tail boxes: landed (before the zeros), ready (in the leader CTA; one arrival per CTA), free
  auto tail_landed = [&](int b) { return bars + 8u * (2 * kStages + 4 + b); };
  auto tail_ready = [&](int b) { return bars + 8u * (2 * kStages + 6 + b); };
  auto tail_free = [&](int b) { return bars + 8u * (2 * kStages + 8 + b); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * barriers(kWG));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* ep_abort = reinterpret_cast<volatile int*>(tmem_slot + 2);  // written by epilogue warps only
  // not in kWG: [E + 1] N tiles before each expert, [E] its first row, [E] its rows
  int* prefix = reinterpret_cast<int*>(tmem_slot + 4);
  int *first_row = prefix + a.E + 1, *n_rows = first_row + a.E;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 2);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), 8);  // four epilogue warps of each CTA
      mbar_init(tail_landed(b), 1);
      mbar_init(tail_ready(b), 2);
      mbar_init(tail_free(b), 1);
    }
    *abort_flag = 0;
    *ep_abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc2(smem_u32(tmem_slot), 512);
  if (!kWG && warp == 6) {
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      int nt = 0;
      if (e0 + lane < a.E) {
        const Rows r = expert_rows(a.offsets, e0 + lane).within(a.P, a.status);
        first_row[e0 + lane] = r.begin;
        n_rows[e0 + lane] = r.end - r.begin;
        nt = (r.end - r.begin + kTileN - 1) / kTileN;
      }
      int incl = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e0 + lane < a.E) prefix[e0 + lane] = run + incl - nt;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) prefix[a.E] = run;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const uint32_t tmem_u = (uint32_t)uniform((int)tmem), base_u = (uint32_t)uniform((int)base);

  const int n_tiles_w = (a.n_total + kTileN - 1) / kTileN;  // kWG: N tiles of one expert
  const int total = kWG ? a.E * m_tiles * n_tiles_w : prefix[a.E] * m_tiles;
  // kWG: the raw rows of a tile's expert are read one tile ahead, so that no role waits for them between tiles.
  const int per_expert = m_tiles * n_tiles_w;
  auto ahead = [&](int tile) { return kWG && tile < total ? expert_rows(a.offsets, tile / per_expert) : Rows{0, 0}; };
  // Tile r of an expert with nti N tiles: bands of kBand N tiles, M tiles within a band, the band's N tiles innermost,
  // so that the tiles in flight (one per CTA pair) share their operands in both directions.
  auto raster = [&](int r, int nti, int& mt, int& nt) {
    const int band = r / (kBand * m_tiles);
    const int width = min(kBand, nti - band * kBand);
    const int q = r - band * kBand * m_tiles;
    mt = q / width;
    nt = band * kBand + q - mt * width;
  };
  auto decode = [&](int tile, const Rows& raw) {
    Tile t;
    if (kWG) {
      t.e = tile / per_expert;
      int mt, nt;
      raster(tile - t.e * per_expert, n_tiles_w, mt, nt);
      t.m0 = mt * kTileM;
      t.n0 = nt * kTileN;
      t.n = min(kTileN, a.n_total - t.n0);
      const Rows rows = raw.within(a.P, a.status);
      t.row0 = rows.begin;
      t.rows = rows.end - rows.begin;
    } else {
      int lo = 0, hi = a.E;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] * m_tiles <= tile) lo = mid;
        else hi = mid;
      }
      int mt, nt;
      raster(tile - prefix[lo] * m_tiles, prefix[lo + 1] - prefix[lo], mt, nt);
      t.e = lo;
      t.m0 = mt * kTileM;
      t.row0 = first_row[lo] + nt * kTileN;
      t.rows = min(kTileN, n_rows[lo] - nt * kTileN);
      t.n0 = 0;
      t.n = (t.rows + 31) & ~31;
    }
    return t;
  };
  // An fp32 gradient over many rows is summed in segments of at most kSegment K steps: the first is stored, the others
  // are added in L2.
  // A bf16 one carries its sum from one long run to the next.
  auto segments = [&](int KB) {
    const int longest = a.out_f32 ? kSegment : kLongRun;
    return kWG && KB > longest ? (KB + longest - 1) / longest : 1;
  };
  auto carries = [&](int nseg) { return kWG && !a.out_f32 && nseg > 1; };
  auto k_steps = [&](const Tile& t) { return kWG ? (t.rows + 48) / 64 : a.k_total / 64; };  // steps with a whole group
  auto tail_rows = [&](const Tile& t) { return kWG ? t.rows & 15 : 0; };

  if (warp == 4) {
    // -------------------------------------------------------------- producer (warp-uniform, as the MMA issuer below)
    const int n_all = uniform(total);
    int issued = 0, n_tails = 0;
    bool ok = true;
    Rows raw = ahead(cluster);
    for (int tile = cluster; ok && tile < n_all && !uniform(*abort_flag); tile += n_clusters) {
      const Tile t = decode(tile, raw);
      raw = ahead(tile + n_clusters);
      const int KB = uniform(k_steps(t)), tail = uniform(tail_rows(t));
      const int half = uniform(t.n / 2);  // this CTA's part of the N operand
      const int mrow = uniform(t.m0 + (int)rank * 128), ncol = uniform(t.n0 + (int)rank * half);
      const int row0 = uniform(t.row0), wrow = uniform(t.e * (FORM == kForward ? a.m_total : a.k_total));
      if (tail) {
        const int b = n_tails & 1;
        ok = n_tails < 2 || __all_sync(0xffffffffu, mbar_wait(tail_free(b), ((n_tails >> 1) - 1) & 1));
        if (!ok) break;
        ++n_tails;
        if (elect_one()) {
          const uint32_t at = tails + b * kTailBytes, bar = map_rank(tail_landed(b), rank);
          const int row = row0 + (t.rows & ~15);
          mbar_arrive_expect_tx(tail_landed(b), (2 + half / 64) * kTailBox);
          tma_load_pair(at, &maps.n[2], bar, mrow, row);
          tma_load_pair(at + kTailBox, &maps.n[2], bar, mrow + 64, row);
          for (int j = 0; j < half / 64; ++j)
            tma_load_pair(at + (2 + j) * kTailBox, &maps.n[1], bar, ncol + 64 * j, row);
        }
        __syncwarp();
      }
      // K-major N operand: one box of 16, 32, 64 or 128 rows
      const int bi = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
      const uint32_t bytes = kOpBytes + (kNmn ? (uint32_t)(half / 64) * kBoxBytes : (16u << bi) * 128u);
      for (int kb = 0; kb < KB; ++kb, ++issued) {
        const int s = issued % kStages;
        ok = issued < kStages || __all_sync(0xffffffffu, mbar_wait(empty(s), ((issued / kStages) - 1) & 1));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t sa = base_u + s * kStageBytes, sb = sa + kOpBytes;
          const uint32_t bar = map_rank(full(s), 0);
          remote_expect_tx(bar, bytes);
          if (FORM == kForward) {
            tma_load_pair(sa, &maps.m, bar, kb * 64, wrow + mrow);
          } else {
            const int row = (kWG ? row0 : wrow) + kb * 64;
            tma_load_pair(sa, &maps.m, bar, mrow, row);
            tma_load_pair(sa + kBoxBytes, &maps.m, bar, mrow + 64, row);
          }
          if (kNmn) {
            for (int j = 0; j < half / 64; ++j)
              tma_load_pair(sb + j * kBoxBytes, &maps.n[0], bar, ncol + 64 * j, row0 + kb * 64);
          } else {
            tma_load_pair(sb, &maps.n[bi], bar, kb * 64, row0 + ncol);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      flag_status(a.status, MOE_DEV_TIMEOUT);
    }
    // copies of the pair have landed before the leader goes on to the last cluster barrier
    if (rank == 0)
      for (int g = issued - kStages < 0 ? 0 : issued - kStages; g < issued; ++g)
        mbar_wait(full(g % kStages), (g / kStages) & 1);
    for (int g = n_tails - 2 < 0 ? 0 : n_tails - 2; g < n_tails; ++g) mbar_wait(tail_landed(g & 1), (g >> 1) & 1);
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the steps and one lane issues: warp-uniform code keeps descriptors in uniform registers,
    // without a move to them before each MMA.
    if (rank == 0) {
      int consumed = 0, n_tails = 0;
      Accumulators acc;
      const int n_all = uniform(total);
      Rows raw = ahead(cluster);
      for (int tile = cluster; tile < n_all; tile += n_clusters) {
        const Tile t = decode(tile, raw);
        raw = ahead(tile + n_clusters);
        const int rows = uniform(t.rows);
        if (rows == 0) continue;  // an expert without rows: the epilogue writes zeros
        const int KB = uniform(k_steps(t)), nseg = uniform(segments(KB)), tail = uniform(tail_rows(t));
        const uint32_t idesc =
            instr_desc(256, uniform(t.n), 1u) | (kMmn ? 1u << 15 : 0u) | (kNmn ? 1u << 16 : 0u);
        const bool carry = carries(nseg);
        bool ok = true;
        for (int seg = 0; ok && seg < nseg; ++seg) {
          const int buf = acc.of(seg, carry);
          ok = __all_sync(0xffffffffu, mbar_wait(tempty(buf), acc.phase(buf) ^ 1u));  // passes before the first use
          acc.used(buf);
          if (!carry || seg == nseg - 1) acc.next ^= 1;
          tc_fence_after();
          const uint32_t d = tmem_u + buf * kTileN;
          const int kb0 = KB * seg / nseg, kb1 = KB * (seg + 1) / nseg;
          uint32_t accumulate = 0;
          for (int kb = kb0; ok && kb < kb1; ++kb, ++consumed) {
            const int s = consumed % kStages;
            if (!__all_sync(0xffffffffu, mbar_wait(full(s), (consumed / kStages) & 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = base_u + s * kStageBytes, sb = sa + kOpBytes;
            const int ks = kWG ? min(4, (rows - kb * 64) >> 4) : 4;  // whole groups of this step
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint64_t ad =
                    kMmn ? sw128_mnmajor_desc(sa + k * 2048, kBoxBytes) : sw128_kmajor_desc(sa + k * 32);
                const uint64_t bd =
                    kNmn ? sw128_mnmajor_desc(sb + k * 2048, kBoxBytes) : sw128_kmajor_desc(sb + k * 32);
                if (!kWG || k < ks) mma_pair(d, ad, bd, idesc, k > 0 ? 1u : accumulate);
              }
              commit_pair(empty(s));
            }
            __syncwarp();
            accumulate = 1;
          }
          if (ok && seg == nseg - 1 && tail) {
            const int b = n_tails & 1;
            ok = __all_sync(0xffffffffu, wait_published(tail_ready(b), (n_tails >> 1) & 1));
            ++n_tails;
            if (ok) {
              tc_fence_after();
              const uint32_t at = tails + b * kTailBytes;
              if (elect_one()) {
                mma_pair(d, sw128_mnmajor_desc(at, kTailBox), sw128_mnmajor_desc(at + 2 * kTailBox, kTailBox), idesc,
                         accumulate);
                commit_pair(tail_free(b));
              }
              __syncwarp();
            }
          }
          if (elect_one()) commit_pair(tfull(buf));
          __syncwarp();
        }
        if (!ok) {
          if (lane == 0) {
            *abort_flag = 1;
            flag_status(a.status, MOE_DEV_TIMEOUT);
          }
          break;
        }
      }
    }
  } else if (warp == 6) {
    // ---------------------------------------------------- zeros of the tails
    if (kWG) {
      int n_tails = 0;
      Rows raw = ahead(cluster);
      for (int tile = cluster; tile < total; tile += n_clusters) {
        const Tile t = decode(tile, raw);
        raw = ahead(tile + n_clusters);
        const int rem = tail_rows(t);
        if (rem == 0) continue;
        const int b = n_tails & 1;
        // every lane waits itself: each writes over bytes that the copy brought
        const int ok = __all_sync(0xffffffffu, mbar_wait(tail_landed(b), (n_tails >> 1) & 1));
        ++n_tails;
        if (!ok) {
          if (lane == 0) {
            *abort_flag = 1;
            flag_status(a.status, MOE_DEV_TIMEOUT);
          }
          break;
        }
        const int boxes = 2 + t.n / 128;  // M operand, then this CTA's part of the N operand
        uint8_t* at = gbase + (tails - base) + b * kTailBytes + rem * 128;
        for (int x = 0; x < boxes; ++x)
          for (int v = lane; v < (16 - rem) * 8; v += 32)
            *reinterpret_cast<uint4*>(at + x * kTailBox + v * 16) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) remote_publish(map_rank(tail_ready(b), 0));
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    Accumulators acc;
    int piece = 0;  // staged pieces so far
    bool gave_up = false;
    Rows raw = ahead(cluster);
    for (int tile = cluster; tile < total && !gave_up; tile += n_clusters) {
      const Tile t = decode(tile, raw);
      raw = ahead(tile + n_clusters);
      const bool any = t.rows > 0;
      if (!any && a.accumulate) continue;  // nothing to add
      const bool in_m = t.m0 + (int)rank * 128 < a.m_total;  // CTA-uniform
      const int nseg = segments(k_steps(t));
      const bool carry = carries(nseg);
      const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
      for (int seg = 0; seg < nseg && !gave_up; ++seg) {
        const int buf = acc.of(seg, carry);
        const uint32_t tl = tmem + buf * kTileN + lanes, held = tmem + (buf ^ 1) * kTileN + lanes;  // held: with carry
        if (any) {
          if (lane == 0 && !mbar_wait(tfull(buf), acc.phase(buf))) *ep_abort = 1;
          named_bar_sync(2, 128);  // the four warps leave the loop together or not at all
          if (*ep_abort) {
            if (lane == 0) {
              *abort_flag = 1;
              flag_status(a.status, MOE_DEV_TIMEOUT);
            }
            gave_up = true;
            break;
          }
          tc_fence_after();
          acc.used(buf);
          if (!carry || seg == nseg - 1) acc.next ^= 1;
        }
        if (carry && seg < nseg - 1) {  // this run joins the sum of those before it
          if (seg == 0) continue;
          if (in_m) {
#pragma unroll 1
            for (int c = 0; c < t.n; c += 32) {
              uint32_t v[32], sum[32];
              tmem_ld32(tl + c, v);
              tmem_ld32(held + c, sum);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q)
                sum[q] = __float_as_uint(__uint_as_float(sum[q]) + __uint_as_float(v[q]));
              tmem_st32(held + c, sum);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(map_rank(tempty(buf), 0));
          continue;
        }
        const bool joins = kWG && seg > 0 && !carry;  // adds to the segments stored before it
        const bool add = joins || (kWG && a.accumulate);
        // what this warp stored of the last segment is in place before it adds to it
        if (joins && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (in_m) {
          const int cols = kWG ? t.n : t.rows;
          // columns per step: a 128-byte store box of the output type, or 32 rows of the output
          const int step = kWG && !a.out_f32 ? 64 : 32;
#pragma unroll 1
          for (int c = 0; c < cols; c += step, ++piece) {
            uint32_t v[32];
            auto load = [&](int at) {
              if (any) {
                tmem_ld32(tl + at, v);
                tmem_wait_ld();
                if (carry) {  // the last run and the sum of the others
                  uint32_t sum[32];
                  tmem_ld32(held + at, sum);
                  tmem_wait_ld();
#pragma unroll
                  for (int q = 0; q < 32; ++q)
                    v[q] = __float_as_uint(__uint_as_float(sum[q]) + __uint_as_float(v[q]));
                }
              } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = 0u;
              }
            };
            if (kWG) {
              // this lane's 128-byte row of the box, 16-byte chunks swizzled as the store expects them
              const uint32_t at = staging + (warp * kBoxes + piece % kBoxes) * kStoreBox;
              uint8_t* row = gbase + (at - base) + lane * 128;
              // the box is free again
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBoxes - 1) : "memory");
              __syncwarp();
              if (a.out_f32) {
                load(c);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  *reinterpret_cast<uint4*>(row + ((q ^ (lane & 7)) << 4)) =
                      make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
              } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  load(c + half * 32);
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4*>(row + (((half * 4 + q) ^ (lane & 7)) << 4)) =
                        make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                                   pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
                }
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) {
                const int r = t.e * a.m_total + t.m0 + (int)rank * 128 + warp * 32;
                if (add) tma_store_2d<true>(&maps.out, at, t.n0 + c, r);
                else tma_store_2d<false>(&maps.out, at, t.n0 + c, r);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
              }
            } else {
              // The accumulator holds features in lanes and rows in columns: the four warps turn 32 rows x 128
              // features round in shared memory, then write whole 256-byte pieces of each row (64-byte pieces
              // straight from the lanes took three times as long at K = 512).
              uint8_t* buf32 = gbase + (staging - base) + (piece & 1) * kPieceBytes;
              load(c);
#pragma unroll
              for (int q = 0; q < 32; ++q)
                *reinterpret_cast<__nv_bfloat16*>(buf32 + q * 256 + (warp * 32 + lane) * 2) =
                    __float2bfloat16_rn(__uint_as_float(v[q]));
              named_bar_sync(1, 128);  // also: everyone is done reading the piece before last
              __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + t.m0 + rank * 128;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int q = warp * 8 + i * 2 + (lane >> 4), ch = lane & 15;
                if (c + q < cols)
                  *reinterpret_cast<uint4*>(out + (size_t)(t.row0 + c + q) * a.m_total + ch * 8) =
                      *reinterpret_cast<const uint4*>(buf32 + q * 256 + ch * 16);
              }
            }
          }
        }
        if (any) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            remote_arrive(map_rank(tempty(buf), 0));
            if (carry) remote_arrive(map_rank(tempty(buf ^ 1), 0));
          }
        }
      }
    }
    // the stores have read their boxes and reached global memory before the CTA goes
    if (kWG && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs are done with each other's barriers and with TMEM
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

namespace {
template <int FORM>
cudaError_t launch_form(const ProductMaps& maps, const ProductArgs& a, long long max_tiles, int num_sms,
                        cudaStream_t s) {
  constexpr bool kWG = FORM == kWeightGrad;
  // 226 KB at most (a CTA may have 227)
  const size_t smem = 1024 + (size_t)stages(kWG) * kStageBytes + staging_bytes(kWG) + (kWG ? 2 * kTailBytes : 0) +
                      8 * barriers(kWG) + 16 + (kWG ? 0 : 4 * (3 * (size_t)a.E + 1));
  // The limit belongs to the kernel, not to the call: one by this call's E could be lowered by another thread, for a
  // layer of fewer experts, before the launch below.
  constexpr int kMostSmem = 227 * 1024;
  const cudaError_t err = cudaFuncSetAttribute(expert_product_kernel<FORM>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (err != cudaSuccess) return err;
  const long long clusters = std::max(1LL, std::min<long long>(num_sms / 2, max_tiles));
  expert_product_kernel<FORM><<<dim3((unsigned)(2 * clusters)), dim3(kThreads), smem, s>>>(maps, a);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_expert_product(int form, const ProductMaps& maps, const ProductArgs& a, int num_sms,
                                  cudaStream_t s) {
  const long long m_tiles = (a.m_total + kTileM - 1) / kTileM;
  const long long rows_tiles = (a.P + kTileN - 1) / kTileN + std::min(a.E, a.P);
  if (form == kForward) return launch_form<kForward>(maps, a, rows_tiles * m_tiles, num_sms, s);
  if (form == kRowGrad) return launch_form<kRowGrad>(maps, a, rows_tiles * m_tiles, num_sms, s);
  return launch_form<kWeightGrad>(maps, a, (long long)a.E * m_tiles * ((a.n_total + kTileN - 1) / kTileN), num_sms,
                                  s);
}

}  // namespace moe
