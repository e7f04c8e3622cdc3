// mrs_experts.cu -- the experts' products of MXFP4 rows and weights, driven by the sort step.
//
// For every row p of the sorted list that is a route r = sorted_token_ids[p] (r < T * topk), with
// e the owner of its block:
//   out[r, n] = w_p * sum over k of X[row(r), k] W[e, n, k],   row(r) = r, or r / topk
// X and W are E2M1 codes with one E8M0 scale per 32 columns; sums are fp32, the row's weight
// (1 without weights) is applied in fp32, and the result is rounded once to the output type.
//
// One tile is up to 128 rows of one expert (the M side of the tensor-core product, 128 lanes of
// tensor memory) by BN = 96, 128, 192 or 256 outputs (the N side).  Blocks of more rows are cut;
// neighbouring blocks of fewer rows that have the same expert share a tile: the list is taken in
// windows of at most 128 rows and 32 blocks, and a tile is a run of one expert's blocks in a
// window (block_m = 16, 4024 tokens, 191 experts, 1984 -> 656: a quarter of the time).  Rows on the
// lanes make a unit of few rows the work of few storing warps; a block of 16 rows costs the tensor
// core as much as one of 128, which it has time for: such calls wait for the weights.  A persistent
// CTA per SM takes units round robin, a unit being one tile, or for short rows several output tiles
// of one block; neighbours share a block's rows and an expert's weights in L2.
//
// Steps of 256 columns (128 bytes a row) go through two rings of shared-memory slots, one of rows
// and one of weights; a unit of several tiles keeps its rows' slots until its last tile.  The
// warps of a CTA each have one task:
//   0      copies the weights (a tensor copy, in the 128-byte swizzle that the tensor core reads)
//   1      copies a step's scales to tensor memory and issues four products of 64 columns; the
//          tensor core applies the scales and adds into fp32 in tensor memory
//   4-7    a finished tile from tensor memory to the output rows, while the next one is computed
//          (two accumulators, one of 256 outputs; eight warps, four per accumulator, took 204 us
//          where four took 198 at T = 512, 3584 -> 768)
//   8-11   the rows, 16 bytes a thread into the same swizzle, and their scales, all copies that
//          arrive on the slot's barrier themselves; where one warp or two hold the rows, the others
//          take steps of their own
//   12-15  the weights' scales, a step a warp in turn
// Scales go from row-major bytes to the order that tensor memory wants: row r of 128 on lane
// r % 32, word r / 32 of 4 scales.  (A warp works through a step in 600 to 900 clocks whatever
// there is to do, so taking turns is what keeps a single token's 14 steps short: 10.6 us before,
// 9.1 so.)
//
// What bounds it: an SM takes in at most 38 bytes a clock (measured, tensor copies, thread copies
// and multicast alike, on one SM and on all), so a step of 128 x 128 costs 890 clocks and its
// products 260; hence the wider tile, and rows that stay.  Few tokens are bound by HBM, which
// gives an SM 23 bytes a clock: 202 us at T = 512, 3584 -> 768, 1.32 GB at 6.5 TB/s.  Short rows are
// bound by both ways of an SM's traffic, 287 us at T = 8192, 384 -> 3584, 215 without the stores.
// Many tokens of few experts are bound by what an SM takes in: T = 8192, E = 64, 7168 -> 2048 takes
// 571 us, and 674 with tiles of 192 outputs.  (256 rows by 192 outputs, two products a step on the
// same weights, take in a fifth less for the same work but leave three slots for rows and twice the
// outputs to store between tiles: 658 us, 580 without the stores.)
//
// Each task has the list entries of the next unit in flight.  Every wait is bounded; a wait that
// gives up ends its warp's task with the status bit set, and the CTA leaves once nothing of its own
// is in flight.
#include <type_traits>

#include <cuda_bf16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_tc.cuh"

namespace mrs {

struct ExpertsArgs {
  const unsigned char *xc, *xs, *ws;  // rows, their scales, the weights' scales
  const int32_t* sid;
  const float* sw;  // or null
  const int32_t* eid;
  const int32_t* npp;
  int32_t* status;  // or null: g_experts_status
  void* out;
  unsigned long long wait_limit_ns;
  int routes, topk, per_route;
  int E, K, N, B, log2B, scols, max_rows;
  int group;        // blocks of a window; 1: every block by itself, in `subs` parts
  int span, subs;   // rows of a window or part (<= 128)
  int ntile;        // tiles along the outputs
  int chunk;        // tiles of a unit (the last of a block may have fewer)
  int nchunk;       // units along the outputs
  int ksteps;       // steps of 256 columns
  int wide_scales;  // the weights' scale rows start on 8 bytes
};

constexpr int kExpThreads = 512;  // warps 2 and 3 are idle: a warp reads the lanes of its number mod 4
constexpr int kExpRows = 128;     // lanes of a tile: rows of a block
constexpr int kStepBytes = 128;   // bytes of a row per step
constexpr int kTmemCols = 512;

// Bits of the calls on this device that bring no workspace.
static __device__ int32_t g_experts_status;

__device__ __forceinline__ void report(const ExpertsArgs& a, int bit) {
  atomicOr(a.status != nullptr ? a.status : &g_experts_status, bit);
}

__global__ void mrs_experts_status_kernel(int32_t* dst, int clear) {
  *dst = clear ? atomicExch(&g_experts_status, 0) : *const_cast<volatile int32_t*>(&g_experts_status);
}

// Slots of both rings and the places of everything, for tiles of BN outputs.
template <int BN>
struct ExpertsShape {
  static constexpr int kAtoms = (BN + 127) / 128;             // scales come for 128 rows at a time
  static constexpr int kX = kExpRows * kStepBytes;            // rows of a slot
  static constexpr int kXSlot = kX + 2 * 512;                 // and their scales
  static constexpr int kW = BN * kStepBytes;
  static constexpr int kWSlot = kW + 2 * 512 * kAtoms;
  // what fits in 227 KB (five slots of 192 would, and take 311 us for T = 8192, 384 -> 3584, where
  // four take 297)
  static constexpr int kSlots = BN == 96 ? 7 : (BN == 128 ? 6 : 4);
  static constexpr int kStoreBytes = 32 * (BN == 96 ? 64 : 128);  // of a storing warp
  static constexpr size_t kSmem =
      static_cast<size_t>(kSlots) * (kXSlot + kWSlot) + 4 * kStoreBytes + 1024;
  static_assert(kSmem + 512 <= 227 * 1024, "");
  // tensor memory: the accumulators, then the scales of each slot
  static constexpr int kAcc = BN == 256 ? 1 : 2;
  static constexpr int kXScales = kAcc * BN;
  static constexpr int kWScales = kXScales + 8 * kSlots;
  static_assert(kWScales + 8 * kAtoms * kSlots <= kTmemCols, "");
};

// A unit of the list: run `slot` of a window (the run of blocks that starts at the window's block
// `slot`, if one does), or a block's part, by some output tiles.  The expert ids it depends on are
// in flight until resolve().  Runs are numbered after windows: the first runs of all windows, which
// there always are, spread evenly over the CTAs.
template <bool kWindows>
struct ExpertsUnit {
  int it, p0, n0, tiles, slot, blocks;  // blocks: of the window that there are
  int id;    // of the window's block `lane`
  int e, rows;
  bool lead;
  __device__ __forceinline__ void at(const ExpertsArgs& a, int i, int units, int windows,
                                     int total_blocks, int bn) {
    it = i;
    const int per = max(windows * a.nchunk, 1);
    const int run = kWindows ? i / per : 0;
    slot = min(run, 31);  // (past the last unit it means nothing)
    // (a division takes longer than a step of the ring; mostly there is nothing to divide by)
    const int q = i - run * per, b = a.nchunk == 1 ? q : q / a.nchunk;
    const int first = (q - b * a.nchunk) * a.chunk;
    n0 = first * bn;
    tiles = min(a.chunk, a.ntile - first);
    id = -1;
    if constexpr (kWindows) {
      const int lane = threadIdx.x & 31, b0 = b * a.group;
      p0 = (b0 + slot) * a.B;
      blocks = min(a.group, total_blocks - b0);
      if (i < units && lane < blocks) id = __ldg(a.eid + b0 + lane);
    } else {
      p0 = b * a.span;
      blocks = 1;
      if (i < units) id = __ldg(a.eid + (a.subs == 1 ? b : b / a.subs));
    }
  }
  __device__ __forceinline__ void resolve(const ExpertsArgs& a, int units) {
    if constexpr (kWindows) {
      const int lane = threadIdx.x & 31;
      e = __shfl_sync(kFull, id, slot);
      const int before = __shfl_sync(kFull, id, max(slot - 1, 0));
      lead = it < units && slot < blocks && (slot == 0 || before != e);
      const unsigned same = __ballot_sync(kFull, id == e && lane < blocks) >> slot;
      rows = (same == ~0u ? 32 : __ffs(~same) - 1) * a.B;
    } else {
      e = id;
      lead = it < units;
      rows = a.span;
    }
  }
  __device__ __forceinline__ bool valid(const ExpertsArgs& a) const {
    return lead && e >= 0 && e < a.E;
  }
  // Entry i behind the unit's first row (-1: none that could be the unit's).
  __device__ __forceinline__ int entry(const ExpertsArgs& a, int i, int units, int total_rows) const {
    return (it < units && i < a.span && p0 + i < total_rows) ? __ldg(a.sid + p0 + i) : -1;
  }
};

// A place in a ring of S slots, and the parity of its round.
template <int S>
struct RingPlace {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void skip(int steps) {
    const int to = slot + steps;
    phase ^= static_cast<uint32_t>(to / S) & 1u;
    slot = to % S;
  }
  __device__ __forceinline__ void advance() {
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// Scales of one row of weights for step `ks`; zeros past the row's end.  Nothing here looks at what
// it loads: a use would wait for it.
__device__ __forceinline__ uint2 load_scales(const unsigned char* row, int ks, const ExpertsArgs& a) {
  const int at = 8 * ks, left = a.K / 32 - at;
  if (a.wide_scales) return __ldg(reinterpret_cast<const uint2*>(row + at));
  const uint32_t* p = reinterpret_cast<const uint32_t*>(row + at);
  return make_uint2(__ldg(p), left > 4 ? __ldg(p + 1) : 0u);
}

// Mask of the first `left` bytes of four scales: what lies behind a row's K / 32 scales is
// padding, and its columns' products of zeros have to meet a finite scale.
__device__ __forceinline__ uint32_t scale_mask(int left) {
  return left >= 4 ? ~0u : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
}

__device__ __forceinline__ void store_shared(uint32_t dst, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Where the scales of row r of 128 start in a step's 512 bytes.
__device__ __forceinline__ uint32_t scale_place(int r) { return 16 * (r & 31) + 4 * (r >> 5); }

template <int BN, bool kWindows, class Out>
__global__ void __launch_bounds__(kExpThreads, 1)
    mrs_experts_kernel(const __grid_constant__ CUtensorMap wmap, const ExpertsArgs a) {
  using Sh = ExpertsShape<BN>;
  constexpr int S = Sh::kSlots;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned long long xfull_s[S], xfree_s[S], wfull_s[S], wfree_s[S], acc_full_s[2],
      acc_free_s[2], done_s;
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // the operands' tiles first: each starts on 1024 bytes
  const uint32_t xbase = base, wbase = base + S * Sh::kX;
  const uint32_t xscales = wbase + S * Sh::kW, wscales = xscales + S * 1024;
  const uint32_t stores = wscales + S * 1024 * Sh::kAtoms;
  const unsigned long long limit = a.wait_limit_ns;
  const int copiers = (a.span + 31) / 32;  // warps that hold a window's rows: 1, 2 or 4
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&xfull_s[s], 32 * copiers);  // every copying thread
      mbar_init(&xfree_s[s], 1);
      mbar_init(&wfull_s[s], 1 + 1);  // the weights' copy, and the warp with its scales
      mbar_init(&wfree_s[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_s[b], 1);
      mbar_init(&acc_free_s[b], 4);
    }
    mbar_init(&done_s, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_s, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  pdl_wait();

  // one block a window: the first unit's list entries do not wait for the list's length
  const int step = gridDim.x;
  ExpertsUnit<kWindows> t, n;
  // of warps 4-7 (a quarter of the lanes each) and 8-11
  const int my_row = 32 * (warp < 8 ? warp & 3 : (warp - 8) & (copiers - 1)) + lane;
  int entry = -1;
  if constexpr (!kWindows) {
    const int most = (a.max_rows >> a.log2B) * a.subs * a.nchunk;
    t.at(a, blockIdx.x, most, 0, 0, BN);
    if (warp >= 4 && warp < 12) entry = t.entry(a, my_row, most, a.max_rows);
  }
  const int blocks = min(max(__ldg(a.npp), 0), a.max_rows) >> a.log2B, rows = blocks << a.log2B;
  const int windows =  // group and block_m are powers of two
      kWindows ? (blocks + a.group - 1) >> (__ffs(a.group) - 1) : blocks * a.subs;
  const int units = (kWindows ? a.group : 1) * windows * a.nchunk;
  if constexpr (kWindows) {
    t.at(a, blockIdx.x, units, windows, blocks, BN);
    if (warp >= 4 && warp < 12) entry = t.entry(a, my_row, units, rows);
  }
  auto look = [&](ExpertsUnit<kWindows>& q, int i) { q.at(a, i, units, windows, blocks, BN); };
  // bytes of the last step's scales that are scales
  const int tail = a.K / 32 - 8 * (a.ksteps - 1);
  const uint32_t tail0 = scale_mask(tail), tail1 = scale_mask(tail - 4);
  bool ok = true;
  RingPlace<S> x, w;

  // Tasks that wait for every step do it without agreeing on the outcome (a vote takes 80 clocks):
  // one thread works alone, or each lane for itself until the unit ends.
  if (warp == 0) {
    long long issued = 0;
    for (; ok && t.it < units; t = n) {
      look(n, t.it + step);
      t.resolve(a, units);
      if (!t.valid(a)) {
        if (t.lead && lane == 0) report(a, MOE_RS_DEVICE_BAD_EXPERT_ID);
        continue;
      }
      const int steps = t.tiles * a.ksteps;
      if (elect_one()) {
        RingPlace<S> at = w;
        for (int c = 0; ok && c < t.tiles; ++c) {
          for (int ks = 0; ks < a.ksteps; ++ks) {
            ok = thread_wait(&wfree_s[at.slot], at.phase ^ 1u, limit);
            if (!ok) break;
            mbar_expect(&wfull_s[at.slot], Sh::kW);
            tma_load_3d(wbase + at.slot * Sh::kW, &wmap, ks * kStepBytes, t.n0 + c * BN, t.e,
                        &wfull_s[at.slot]);
            ++issued;
            at.advance();
          }
        }
        if (!ok) {
          // a copy still on its way must land before the CTA leaves; the phase it completes may be
          // missing other arrivals, so this waits for what has no one to take it any more
          for (long long q = issued > S ? issued - S : 0; q < issued; ++q)
            thread_wait(&wfull_s[q % S], static_cast<uint32_t>(q / S) & 1u, kWaitLimitNs);
        }
      }
      ok = __all_sync(kFull, ok);
      w.skip(steps);
    }
  } else if (warp == 1) {
    int buf = 0;
    uint32_t acc_phase = 0;
    bool any = false;
    for (; ok && t.it < units; t = n) {
      look(n, t.it + step);
      t.resolve(a, units);
      if (!t.valid(a)) continue;
      any = true;
      if (elect_one()) {
        RingPlace<S> xs, at = w;
        int to = buf;
        uint32_t to_phase = acc_phase;
        for (int c = 0; ok && c < t.tiles; ++c) {
          ok = thread_wait(&acc_free_s[to], to_phase ^ 1u, limit);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + to * BN;
          xs = x;  // every tile of the unit takes the same rows
          for (int ks = 0; ks < a.ksteps; ++ks) {
            ok = (c > 0 || thread_wait(&xfull_s[xs.slot], xs.phase, limit)) &&
                 thread_wait(&wfull_s[at.slot], at.phase, limit);
            if (!ok) break;
            tc_fence_after();
            if (c == 0) fence_proxy_async_smem();  // the rows were written by threads
            const uint32_t xsc = xscales + xs.slot * 1024;
            const uint32_t wsc = wscales + at.slot * (1024 * Sh::kAtoms);
            const uint32_t tx = tmem + Sh::kXScales + xs.slot * 8;
            const uint32_t tw = tmem + Sh::kWScales + at.slot * (8 * Sh::kAtoms);
            const uint64_t dx = desc_rows128(xbase + xs.slot * Sh::kX);
            const uint64_t dw = desc_rows128(wbase + at.slot * Sh::kW);
            const int parts = (a.K - 256 * ks + 63) >> 6;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (c == 0) tc_copy_scales(tx + 4 * g, desc_scales(xsc + 512 * g));
#pragma unroll
              for (int q = 0; q < Sh::kAtoms; ++q)
                tc_copy_scales(tw + 4 * (Sh::kAtoms * g + q),
                               desc_scales(wsc + 512 * (Sh::kAtoms * g + q)));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q < parts)  // else columns past K
                // 32 bytes further along the swizzled rows: 2 units of 16
                tc_mma_mxf4(d, dx + 2 * q, dw + 2 * q, mxf4_word(kExpRows, BN, (q & 1) * 2),
                            tx + 4 * (q >> 1), tw + 4 * Sh::kAtoms * (q >> 1), ks > 0 || q > 0);
            tc_commit(&wfree_s[at.slot]);
            if (c + 1 == t.tiles) tc_commit(&xfree_s[xs.slot]);
            if (ks + 1 == a.ksteps) tc_commit(&acc_full_s[to]);
            xs.advance();
            at.advance();
          }
          if (++to == Sh::kAcc) {
            to = 0;
            to_phase ^= 1u;
          }
        }
      }
      ok = __all_sync(kFull, ok);
      x.skip(a.ksteps);
      w.skip(t.tiles * a.ksteps);
      acc_phase ^= static_cast<uint32_t>((buf + t.tiles) / Sh::kAcc) & 1u;
      buf = (buf + t.tiles) % Sh::kAcc;
    }
    // nothing of the tensor core may be in flight when tensor memory is given back
    if (any) {
      if (elect_one()) tc_commit(&done_s);
      __syncwarp();
      warp_wait(&done_s, 0, kWaitLimitNs);
    }
  } else if (warp >= 4 && warp < 8) {
    int buf = 0;
    uint32_t acc_phase = 0;
    for (; ok && t.it < units; t = n) {
      look(n, t.it + step);
      const int r = entry;
      entry = n.entry(a, my_row, units, rows);
      t.resolve(a, units);
      if (!t.valid(a)) continue;
      const bool used = 32 * (warp & 3) < t.rows;
      const bool put = my_row < t.rows && r >= 0 && r < a.routes;
      const float by = (a.sw != nullptr && put) ? __ldg(a.sw + t.p0 + my_row) : 1.0f;
      // 64 or 128 bytes of a row are stored side by side, 16 by each of kLanes lanes
      constexpr int kLine = BN > 96 && sizeof(Out) == 2 ? 128 : 64, kLanes = kLine / 16;
      const int piece = lane % kLanes;
      int line[kLanes];  // routes of the rows that this lane stores parts of
#pragma unroll
      for (int i = 0; i < kLanes; ++i)
        line[i] = __shfl_sync(kFull, put ? r : -1, 32 / kLanes * i + lane / kLanes);
      for (int tile = 0; tile < t.tiles; ++tile) {
        ok = warp_wait(&acc_full_s[buf], acc_phase, limit);
        if (!ok) break;
        if (used) {
          tc_fence_after();
          const uint32_t src = tmem + buf * BN + (static_cast<uint32_t>(32 * (warp - 4)) << 16);
          const int n0 = t.n0 + tile * BN, left = a.N - n0;  // left: a multiple of 8
          // A lane holds a row; a line's bytes of each row go through shared memory so that
          // neighbouring lanes store them side by side.  (T = 8192, 384 -> 3584, us: 411 where a
          // lane stored 32 bytes of its row, 297 with 64 bytes a row, 287 with 128; one token
          // and 32-bit outputs are faster with 64.)  The outputs are marked as the first to leave
          // L2, which the weights want for themselves (1%).
          constexpr int kCols = 64 / sizeof(Out), kPiece = 16 / sizeof(Out);
          const uint32_t to = stores + (warp - 4) * Sh::kStoreBytes;
          auto place = [&](int row, int p) {  // 16 bytes, spread over the banks
            return to + kLine * row + 16 * (p ^ (kLine == 128 ? row & 7 : (row >> 1) & 3));
          };
          // the next 32 columns are on their way while these are stored (columns past the
          // outputs are read, as zeros, and not stored)
          uint32_t ahead[2][32];
          tmem_load32(src, ahead[0]);
#pragma unroll
          for (int c0 = 0; c0 < BN; c0 += 32) {
            uint32_t(&v)[32] = ahead[(c0 / 32) & 1];
            tmem_wait(v);
            if (c0 + 32 < BN) tmem_load32(src + c0 + 32, ahead[(c0 / 32 + 1) & 1]);
            if constexpr (sizeof(Out) == 4) {
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(by * __uint_as_float(v[c]));
            } else {
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(by * __uint_as_float(v[2 * c]),
                                                               by * __uint_as_float(v[2 * c + 1]));
                v[c] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
            // pieces of the line that are there already
            const int had = kLine == 128 ? (c0 & 32) / 8 : 0;
#pragma unroll
            for (int part = 0; part < (kLine == 128 ? 1 : 32 / kCols); ++part) {
              const uint32_t* q = v + 16 * part;
              if (had == 0) __syncwarp();  // what was there has been read
#pragma unroll
              for (int c = 0; c < 4; ++c)
                store_shared(place(lane, had + c), q[4 * c], q[4 * c + 1], q[4 * c + 2],
                             q[4 * c + 3]);
              if (had + 4 < kLanes && c0 + 32 < BN) continue;  // the line is not full
              __syncwarp();
              const int col = c0 - 8 * had + kCols * part + kPiece * piece;
              const bool mine = col < left && piece < had + 4;
#pragma unroll
              for (int i = 0; i < kLanes; ++i) {
                uint32_t w[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(place(32 / kLanes * i + lane / kLanes, piece))
                             : "memory");
                if (line[i] >= 0 && mine)
                  __stcs(reinterpret_cast<uint4*>(static_cast<Out*>(a.out) +
                                                  static_cast<size_t>(line[i]) * a.N + n0 + col),
                         make_uint4(w[0], w[1], w[2], w[3]));
              }
            }
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_free_s[buf]);
        if (++buf == Sh::kAcc) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // a warp copies rows w32 .. w32 + 31 of the unit, four rows (8 lanes each) at a time, and lane l
    // the scales of row w32 + l, in every turns-th step
    const int w32 = my_row - lane, turns = 4 / copiers, turn = (warp - 8) / copiers;
    int now = 0;  // whose step it is (at most 4 steps lie between two of a warp: less than a ring)
    static_assert(S >= 4, "");
    const int chunk = lane & 7, sub4 = lane >> 3;
    const size_t half = static_cast<size_t>(a.K / 2);
    // row 4 j + sub4 of the warp: two swizzles, for even and odd j
    const uint32_t place = xbase + (w32 + sub4) * kStepBytes;
    const uint32_t even = place + 16 * (chunk ^ sub4), odd = place + 16 * (chunk ^ (sub4 + 4));
    const uint32_t scale_at = xscales + scale_place(my_row);
    for (; ok && t.it < units; t = n) {
      look(n, t.it + step);
      const int r = entry;
      entry = n.entry(a, my_row, units, rows);
      t.resolve(a, units);
      if (!t.valid(a)) continue;
      const int src = my_row < t.rows && r >= 0 && r < a.routes
                          ? (a.per_route ? r : r / a.topk) : -1;
      // rows that are no route keep the codes that were there, in rows that are not stored, and
      // get scales of zero bytes
      const unsigned char* scales = a.xs + static_cast<size_t>(max(src, 0)) * a.scols;
      const unsigned char* from[8];
      unsigned has = 0u;
      const int mine = min(t.rows - w32, 32);  // rows of this warp, 0 or fewer: none
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int s = __shfl_sync(kFull, src, 4 * j + sub4);
        from[j] = a.xc + static_cast<size_t>(max(s, 0)) * half + 16 * chunk;
        has |= s >= 0 ? 1u << j : 0u;
      }
      for (int ks = 0; ks < a.ksteps; ++ks) {
        if (now == turn) {
          ok = thread_wait(&xfree_s[x.slot], x.phase ^ 1u, limit);
          if (!ok) break;  // this lane; the others follow below
          const uint32_t dst = x.slot * Sh::kX;
          // (columns past K keep what was there too: they meet weights that read as zero)
          const unsigned live = ks * kStepBytes + 16 * chunk < a.K / 2 ? has : 0u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (4 * j >= mine) break;
            if ((live >> j) & 1u)
              copy16(dst + ((j & 1) ? odd : even) + 512 * j,
                     from[j] + static_cast<size_t>(ks) * kStepBytes);
          }
          const int left = src < 0 ? 0 : a.K / 32 - 8 * ks;  // scales from this step on
          const unsigned char* q = scales + (left > 0 ? 8 * ks : 0);
          copy4(scale_at + x.slot * 1024, q, min(max(left, 0), 4));
          copy4(scale_at + x.slot * 1024 + 512, left > 4 ? q + 4 : q, min(max(left - 4, 0), 4));
          copy_arrive(&xfull_s[x.slot]);
        }
        if (++now == turns) now = 0;
        x.advance();
      }
      ok = __all_sync(kFull, ok);
    }
    copy_wait_all();
  } else if (warp >= 12) {
    // Steps go to the four warps in turn, and a warp loads its next step's scales before it hands on
    // the last one's.  Lane l has the rows l + 32 r.  (A slot's barrier only tells odd rounds from
    // even ones: a warp may ask for a round only once the one two back is over, which its own step
    // four back vouches for in a ring of four or more.)
    static_assert(S >= 4, "");
    constexpr int kR = BN / 32;  // rows of a lane
    constexpr int kWords = 4 * Sh::kAtoms;
    const int me = warp - 12;
    int at = 0;  // steps so far, all warps' together
    bool have = false, have_last = false;
    RingPlace<S> had;
    uint2 cur[kR], nx[kR];
    auto hand_on = [&] {
      if (!have) return;
      // (a lane whose wait gave up goes along, without waiting again, until the tile ends)
      ok = ok && thread_wait(&wfree_s[had.slot], had.phase ^ 1u, limit);
      const uint32_t dst = wscales + had.slot * (1024 * Sh::kAtoms) + 16 * lane;
      const uint32_t keep0 = have_last ? tail0 : ~0u, keep1 = have_last ? tail1 : ~0u;
      uint32_t w0[kWords], w1[kWords];
#pragma unroll
      for (int r = 0; r < kWords; ++r) {
        w0[r] = r < kR ? cur[r < kR ? r : 0].x & keep0 : 0u;
        w1[r] = r < kR ? cur[r < kR ? r : 0].y & keep1 : 0u;
      }
      if (ok) {
#pragma unroll
        for (int q = 0; q < Sh::kAtoms; ++q) {
          store_shared(dst + 512 * q, w0[4 * q], w0[4 * q + 1], w0[4 * q + 2], w0[4 * q + 3]);
          store_shared(dst + 512 * (Sh::kAtoms + q), w1[4 * q], w1[4 * q + 1], w1[4 * q + 2],
                       w1[4 * q + 3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&wfull_s[had.slot]);
    };
    for (; ok && t.it < units; t = n) {
      look(n, t.it + step);
      t.resolve(a, units);
      if (!t.valid(a)) continue;
      for (int c = 0; ok && c < t.tiles; ++c) {
        const int o = t.n0 + c * BN + lane;
        const unsigned char* p = a.ws + (static_cast<size_t>(t.e) * a.N + o) * a.scols;
        for (int ks = 0; ks < a.ksteps; ++ks) {
          if ((at++ & 3) == me) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              nx[r] = make_uint2(0u, 0u);
              if (o + 32 * r < a.N)
                nx[r] = load_scales(p + static_cast<size_t>(32 * r) * a.scols, ks, a);
            }
            hand_on();
#pragma unroll
            for (int r = 0; r < kR; ++r) cur[r] = nx[r];
            had = w;
            have = true;
            have_last = ks + 1 == a.ksteps;
          }
          w.advance();
        }
        ok = __all_sync(kFull, ok);
      }
    }
    if (ok) hand_on();
    ok = __all_sync(kFull, ok);
  }
  if (!ok && lane == 0) report(a, MOE_RS_DEVICE_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, kTmemCols);
}

// ------------------------------------------------------------------------------ host side
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// The weights: `outs` rows of `row` bytes for each of E experts; the copied box is 128 bytes of
// `tile` rows of one expert (rows past the last and bytes past the row's end read as zero).
bool encode_weights(CUtensorMap* map, const void* p, size_t row, size_t outs, size_t E, int tile) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {row, outs, E};
  const cuuint64_t strides[2] = {row, row * outs};
  const cuuint32_t box[3] = {kStepBytes, static_cast<cuuint32_t>(tile), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool kWindows, class Out>
cudaError_t launch_experts(const CUtensorMap& wmap, const ExpertsArgs& a, int grid,
                           cudaStream_t st) {
  auto* k = mrs_experts_kernel<BN, kWindows, Out>;
  constexpr size_t smem = ExpertsShape<BN>::kSmem;
  static SmemGrant granted;
  const cudaError_t err = grant_smem(reinterpret_cast<const void*>(k), smem, granted);
  if (err != cudaSuccess) return err;
  return launch_pdl(k, dim3(grid), dim3(kExpThreads), smem, st, wmap, a);
}

// Tile width and units of a call.  Blocks below 128 rows go in windows where some expert can have
// more than one (more routes than a block holds).  `rowtiles` counts row tiles at most: parts of
// blocks, or with windows one per 128 routes and expert.  An SM's time for a tile goes by the bytes
// it takes in, its rows and BN weights, so the width is the one with the smallest product of rounds
// and bytes.  Rows of at most half a ring's steps stay for several tiles once every SM has work for
// eight rounds without that (us with and without: T = 8192, E = 896, 384 -> 3584 307 505; T = 2048
// 149 243; T = 3000, E = 700, 256 -> 640 48 65; T = 2048, E = 64, 384 -> 3584 42 51.  Four rounds,
// where eight leave one or two tiles a unit: T = 1000, E = 128, 512 -> 2048 26 for 31).  Tiles of 256
// outputs leave room for one accumulator, so that a tile is stored before the next one's products;
// they are for rows that do not stay, whose copies cover most of that (T = 8192, E = 64, outs = 2048,
// us with and without them: 83 63 at 512 columns, 101 119 at 768, 118 140 at 1024, 182 223 at 2048).
struct ExpertsPlan {
  int group, span, subs;
  int bn, ntile, chunk, nchunk, ksteps;
};
ExpertsPlan experts_plan(int64_t blocks, int64_t routes, int E, int B, int outs, int cols,
                         int sms) {
  ExpertsPlan p{};
  p.group = B >= kExpRows || routes <= B ? 1 : (kExpRows / B < 32 ? kExpRows / B : 32);
  p.span = p.group > 1 ? p.group * B : (B < kExpRows ? B : kExpRows);
  p.subs = p.group > 1 ? 1 : B / p.span;
  int64_t rowtiles = blocks * p.subs;
  if (p.group > 1) {
    const int64_t runs = routes / p.span + (routes < E ? routes : E);
    rowtiles = rowtiles < runs ? rowtiles : runs;
  }
  auto cost = [&](int bn) {
    const int64_t tiles = rowtiles * ((outs + bn - 1) / bn);
    return (tiles + sms - 1) / sms * (p.span + bn);
  };
  p.bn = 128;
  if (cost(192) < cost(p.bn)) p.bn = 192;
  if (cost(96) < cost(p.bn)) p.bn = 96;
  p.ksteps = (cols + 255) / 256;
  if (2 * p.ksteps > ExpertsShape<256>::kSlots && cost(256) < cost(p.bn)) p.bn = 256;
  p.ntile = (outs + p.bn - 1) / p.bn;
  p.chunk = 1;
  const int slots = p.bn == 96    ? ExpertsShape<96>::kSlots
                    : p.bn == 128 ? ExpertsShape<128>::kSlots
                    : p.bn == 192 ? ExpertsShape<192>::kSlots
                                  : ExpertsShape<256>::kSlots;
  if (2 * p.ksteps <= slots) {
    const int64_t each = rowtiles * p.ntile / (8 * static_cast<int64_t>(sms));
    p.chunk = each < 1 ? 1 : (each > p.ntile ? p.ntile : static_cast<int>(each));
  }
  p.nchunk = (p.ntile + p.chunk - 1) / p.chunk;
  p.chunk = (p.ntile + p.nchunk - 1) / p.nchunk;
  return p;
}

}  // namespace
}  // namespace mrs

using namespace mrs;

extern "C" {

size_t moe_experts_mxfp4_workspace_bytes(int T, int E, int topk, int block_m) {
  if (T < 0 || E < 1 || E > kMaxExperts || topk < 1 || topk > kMaxTopk || block_m < 1 ||
      block_m > 1024 || (block_m & (block_m - 1)) != 0)
    return 0;
  return 256;
}

int moe_experts_mxfp4(const uint8_t* x_codes, const uint8_t* x_scales, int x_per_route,
                      const uint8_t* w_codes, const uint8_t* w_scales, int T, int E, int topk,
                      int cols, int outs, int block_m, const int32_t* sorted_token_ids,
                      const float* sorted_weights, const int32_t* expert_ids,
                      const int32_t* num_tokens_post_pad, void* out, int out_dtype,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (T < 0) return MOE_RS_ERR_BAD_TOKENS;
  if (E < 1 || E > kMaxExperts) return MOE_RS_ERR_BAD_EXPERTS;
  if (topk < 1 || topk > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  const size_t need = moe_experts_mxfp4_workspace_bytes(T, E, topk, block_m);
  if (need == 0) return MOE_RS_ERR_BAD_BLOCK_M;
  const int scols = moe_mxfp4_scale_cols(cols);
  if (scols == 0 || outs < 8 || outs > MOE_RS_MXFP4_MAX_OUTS || outs % 8 != 0)
    return MOE_RS_ERR_BAD_COLS;
  if (out_dtype != MOE_RS_BF16 && out_dtype != MOE_RS_FP32) return MOE_RS_ERR_BAD_DTYPE;
  if (static_cast<int64_t>(T) * topk > INT32_MAX ||
      static_cast<int64_t>(moe_sort_max_padded(T, E, topk, block_m)) > INT32_MAX)
    return MOE_RS_ERR_OVERFLOW;
  const bool own_word = !workspace && workspace_bytes == 0;
  if (!own_word && (!workspace || workspace_bytes < need)) return MOE_RS_ERR_WORKSPACE;
  if (T == 0) return MOE_RS_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !sorted_token_ids || !expert_ids ||
      !num_tokens_post_pad || !out)
    return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 4) ||
      !aligned(w_scales, 4) || !aligned(sorted_token_ids, 4) || !aligned(sorted_weights, 4) ||
      !aligned(expert_ids, 4) || !aligned(num_tokens_post_pad, 4) || !aligned(out, 16) ||
      !aligned(workspace, 16))
    return MOE_RS_ERR_MISALIGNED;
  const size_t routes = static_cast<size_t>(T) * topk;
  const size_t xrows = x_per_route ? routes : static_cast<size_t>(T);
  const size_t wrows = static_cast<size_t>(E) * outs;
  const size_t P = moe_sort_max_padded(T, E, topk, block_m);
  const Span outs_s[] = {span(out, routes * outs * (out_dtype == MOE_RS_FP32 ? 4 : 2)),
                         span(workspace, workspace_bytes)};
  const Span ins[] = {span(x_codes, xrows * (cols / 2)),
                      span(x_scales, xrows * scols),
                      span(w_codes, wrows * (cols / 2)),
                      span(w_scales, wrows * scols),
                      span(sorted_token_ids, 4 * P),
                      span(sorted_weights, sorted_weights ? 4 * P : 0),
                      span(expert_ids, 4 * (P / block_m)),
                      span(num_tokens_post_pad, 4)};
  if (any_alias(outs_s, 2, ins, 8)) return MOE_RS_ERR_ALIAS;
  const bool f32 = out_dtype == MOE_RS_FP32;
  const int64_t blocks = static_cast<int64_t>(P / block_m);
  // units: every part of 128 rows and every tile of outputs, windows of 32 blocks rounded up
  if ((blocks * ((block_m + kExpRows - 1) / kExpRows) + 32) * ((outs + 95) / 96) > INT32_MAX / 2)
    return MOE_RS_ERR_OVERFLOW;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  const ExpertsPlan p =
      experts_plan(blocks, static_cast<int64_t>(routes), E, block_m, outs, cols, sms);
  ExpertsArgs a{};
  a.xc = x_codes;
  a.xs = x_scales;
  a.ws = w_scales;
  a.sid = sorted_token_ids;
  a.sw = sorted_weights;
  a.eid = expert_ids;
  a.npp = num_tokens_post_pad;
  a.status = static_cast<int32_t*>(workspace);
  a.out = out;
  a.routes = static_cast<int>(routes);
  a.topk = topk;
  a.per_route = x_per_route != 0;
  a.E = E;
  a.K = cols;
  a.N = outs;
  a.B = block_m;
  while ((1 << a.log2B) < block_m) ++a.log2B;
  a.scols = scols;
  a.max_rows = static_cast<int>(P);
  a.wait_limit_ns = debug_wait_limit_ns();
  a.group = p.group;
  a.span = p.span;
  a.subs = p.subs;
  a.ntile = p.ntile;
  a.chunk = p.chunk;
  a.nchunk = p.nchunk;
  a.ksteps = p.ksteps;
  a.wide_scales = scols % 8 == 0 && aligned(w_scales, 8);
  CUtensorMap wmap;
  if (!encode_weights(&wmap, w_codes, cols / 2, outs, E, p.bn)) return MOE_RS_ERR_LAUNCH;
  const int64_t units = (p.group > 1 ? (blocks + p.group - 1) / p.group * p.group
                                     : blocks * p.subs) * p.nchunk;
  const int grid = units < sms ? static_cast<int>(units) : sms;
  auto go = [&](auto n) {
    constexpr int BN = decltype(n)::value;
    if (p.group > 1)
      return f32 ? launch_experts<BN, true, float>(wmap, a, grid, stream)
                 : launch_experts<BN, true, __nv_bfloat16>(wmap, a, grid, stream);
    return f32 ? launch_experts<BN, false, float>(wmap, a, grid, stream)
               : launch_experts<BN, false, __nv_bfloat16>(wmap, a, grid, stream);
  };
  return launch_status(p.bn == 96    ? go(std::integral_constant<int, 96>{})
                       : p.bn == 128 ? go(std::integral_constant<int, 128>{})
                       : p.bn == 192 ? go(std::integral_constant<int, 192>{})
                                     : go(std::integral_constant<int, 256>{}));
}

int moe_experts_mxfp4_plan(int T, int E, int topk, int cols, int outs, int block_m, int sms,
                           int32_t* plan) {
  if (T < 1) return MOE_RS_ERR_BAD_TOKENS;
  if (E < 1 || E > kMaxExperts) return MOE_RS_ERR_BAD_EXPERTS;
  if (topk < 1 || topk > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  if (moe_experts_mxfp4_workspace_bytes(T, E, topk, block_m) == 0) return MOE_RS_ERR_BAD_BLOCK_M;
  if (moe_mxfp4_scale_cols(cols) == 0 || outs < 8 || outs > MOE_RS_MXFP4_MAX_OUTS || outs % 8 != 0)
    return MOE_RS_ERR_BAD_COLS;
  if (sms < 1 || static_cast<int64_t>(T) * topk > INT32_MAX) return MOE_RS_ERR_OVERFLOW;
  if (!plan) return MOE_RS_ERR_NULL_POINTER;
  const int64_t blocks = static_cast<int64_t>(moe_sort_max_padded(T, E, topk, block_m) / block_m);
  const ExpertsPlan p =
      experts_plan(blocks, static_cast<int64_t>(T) * topk, E, block_m, outs, cols, sms);
  const int32_t v[] = {p.bn, p.group, p.subs, p.ntile, p.chunk, p.nchunk, p.ksteps};
  for (int i = 0; i < 7; ++i) plan[i] = v[i];
  return MOE_RS_OK;
}

int moe_experts_mxfp4_status(int32_t* dst, int clear, cudaStream_t stream) {
  if (!dst) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(dst, 4)) return MOE_RS_ERR_MISALIGNED;
  mrs_experts_status_kernel<<<1, 1, 0, stream>>>(dst, clear != 0);
  return launch_status(cudaGetLastError());
}

}  // extern "C"
