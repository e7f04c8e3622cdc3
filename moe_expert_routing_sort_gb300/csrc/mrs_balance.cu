// mrs_balance.cu -- the balance loss of a router with its per-expert counts, and the gradient
// of the routing weights and of that loss to the router logits.
//
// x = float(bf16 logit); S sequences of consecutive tokens, n_i tokens in sequence i:
//   p_te    = softmax(x_t)_e, or sigmoid(x_te) / sum over e of sigmoid(x_te)
//   c_ie    = routes of sequence i that go to expert e
//   P_ie    = mean of p_te over the sequence
//   loss    = coef / S * sum_i sum_e (E c_ie / (K n_i)) P_ie
// The counts are constants of the gradient: with g_ie = grad_loss coef E c_ie / (S K n_i^2),
//   softmax  dx_e = p_e (g_e - sum p g)        sigmoid  dx_e = p_e (1 - s_e) (g_e - sum p g)
// and the routing weights w_k = R u_k / sum u (u = sigmoid or exp of the routed logits) add, at
// the routed experts,    R q_k (gw_k - sum q gw), q = u / sum u      (times 1 - s_k for sigmoid).
//
// Both passes read the logits once.  A row belongs to a group of W warps (W = ceil(E / 1024), or
// ceil(E / 512) for rows that do not start on 16 bytes), each lane holding up to 32 of its columns
// in registers, the same columns for every row: the row sums are warp shuffles (and one exchange
// through shared memory when W > 1), and the column sums of the loss stay in registers for 64 rows
// (about the square root of a longer stretch) or until the sequence or the CTA's token range ends.
// A softmax row needs one reduction: every lane takes exponentials against its own maximum and the
// reduction joins (maximum, sum) pairs.  Each lane copies its own columns of the next rows to shared
// memory in the background (kDepth rows, 96 KB on their way per SM; one row ahead in registers,
// 16 KB, left the memory idle: T = 8192, E = 896 16.7 us, 14.8 with the ring) and reads back only
// what it copied, so no wait is shared.  All sums are fp32 in an order fixed by the shape: results
// are the same bits every call.
//
// What it takes now: the loss 14.2 us at T = 8192, E = 896 (two kernels; 2.3 us of bytes) and 37 at
// T = 16384, E = 4096 (19.9 of bytes; 71% of the issue slots), the gradient 12.2 us at T = 8192,
// E = 896 (4.5 of bytes; half of the slots, the rest is the first rows' way in).
//
// Partial column sums: CTA b of the first kernel and sequence i meet in at most one stretch of
// tokens; it writes its sums to slot b + i (a monotone walk through (b, i): no two stretches
// share a slot), and the second kernel adds the slots of each sequence in CTA order.  A call of
// few tokens is one CTA, which writes the results itself.
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_tc.cuh"

namespace mrs {

constexpr int kBalThreads = 512;
constexpr int kJoinThreads = 256;
constexpr int kDepth = 4;          // rows of a lane in flight, the one it works on among them
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxCtas = 256;
constexpr int kIdsAhead = 4;       // routes of a thread loaded ahead of a stretch's rows
constexpr int kSumRows = 64;       // rows whose sum stays in registers, at least
constexpr int kSoloRows = 4;       // rows per group up to which one CTA takes the call
constexpr int kSoloSeqs = 8;
constexpr int kBalMaxJoin = 1024;  // CTAs of the second kernel
constexpr float kLog2e = 1.4426950408889634f;
// Below every finite bf16 and itself finite: maxima start here, so that a column of -inf gives a
// term of exp(-inf) = 0 whatever the others hold, and a row of the type's lowest value is even.
constexpr float kLowest = -3.402823466e38f;
// Finite logits further out than this count as this in a softmax: up to here the rounding of
// m log2 e (below) is a factor of at most 2^3 that cancels, not one that overflows.
constexpr float kFarLogit = 67108864.0f;  // 2^26

struct BalanceArgs {
  const uint16_t* logits;
  const int32_t* ids;
  const int32_t* offsets;  // [S + 1], or null: one sequence of all T tokens
  int T, E, K, S, W;       // W: warps per row
  int tpc;                 // tokens per CTA
  int solo;                // one CTA writes the results, no second kernel
  float coef;
  float* loss;
  int32_t* counts;
  float* mean;
  float* psum;      // [ctas + S][E] slots
  int32_t* csum;    // [ctas + S][E]
  float* partial;   // [kBalMaxJoin]
  unsigned* ticket;
};

struct RouteBackwardArgs {
  const uint16_t* logits;
  const int32_t* ids;
  const float* gw;         // [T, K] or null
  const float* gl;         // [1] or null
  const int32_t* counts;   // [S, E] (null with gl)
  const int32_t* offsets;
  int T, E, K, S, W, tpc;
  int wide_counts;         // counts start on 16 bytes
  float R, coef;
  void* out;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Borders of the sequences, kept inside [0, T] whatever the array holds.
__device__ __forceinline__ int seq_border(const int32_t* o, int i, int T) {
  return o == nullptr ? (i == 0 ? 0 : T) : min(max(__ldg(o + i), 0), T);
}

// First sequence that ends behind token t (S if none does); all lanes of a warp.  32 borders are
// looked at together, so a packed batch takes one load's time and 65536 sequences four.
__device__ __forceinline__ int seq_behind(const int32_t* o, int S, int T, int t) {
  if (o == nullptr) return t < T ? 0 : 1;
  int lo = 0, n = S;  // the answer lies in [lo, lo + n]
  const int lane = threadIdx.x & 31;
  while (n > 0) {
    const int each = (n + 31) / 32, i = lo + min((lane + 1) * each, n) - 1;
    const unsigned behind = __ballot_sync(kFull, seq_border(o, i + 1, T) > t);
    if (behind == 0u) return lo + n;
    const int first = __ffs(behind) - 1;  // sequence lo + (first + 1) each - 1 ends behind t
    lo += first * each;
    n = min(each - 1, n - 1 - first * each);
    n = n < 0 ? 0 : n;
  }
  return lo;
}

// The largest and the most negative of a lane's logits, two bf16 patterns a word: among signed
// numbers a positive pattern, among unsigned ones a negative pattern is the larger the further it is
// from zero.
struct Extremes {
  uint32_t up, down;
  __device__ __forceinline__ void add(uint32_t a, uint32_t b) {
    up = __vimax3_s16x2(up, a, b);
    down = __vimax3_u16x2(down, a, b);
  }
  // Any beyond 7.5, where 1 / (1 + e^-x) is too near 1 to be taken from it.
  __device__ __forceinline__ bool high() const {
    return max(static_cast<int>(up << 16), static_cast<int>(up & 0xffff0000u)) > 0x40f00000;
  }
  // Any at or below -43, where a product of two 1 + e^-x could leave the range.
  __device__ __forceinline__ bool low() const {
    return max(down << 16, down & 0xffff0000u) >= 0xc22c0000u;
  }
};

// Rows of a lane on their way: the lane's columns of row `row`, `step` rows after the one before.
// kVec: 16-byte vectors of 8 columns, vector v of the lane being vector v * lanes + lane of the
// row, copied to shared memory (ring: 16 bytes per vector, thread and slot); else single columns
// i * lanes + lane, one row ahead in registers.  Columns past E read as -inf, a term of zero; for
// sigmoids in vectors as -40, which keeps their lanes on the short way, and their terms are left
// out of the row's sum.
template <int NC, bool kVec, bool kSoftmax>
struct RowStream {
  static constexpr int NV = NC / 8;
  static constexpr uint32_t kPast = kSoftmax ? 0xff80ff80u : 0xc220c220u;
  uint32_t next[kVec ? 1 : NC];
  uint32_t ring, slot;     // slot: bytes into the ring of the row that is taken next
  const uint16_t* from;    // the lane's first column of the row that is fetched next
  int row;                 // and its number

  __device__ __forceinline__ void fetch(int E, int hi, int lane, int lanes, uint32_t to) {
    if constexpr (kVec) {
      if (row < hi) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (8 * (v * lanes + lane) < E)
            copy16(to + 16 * kBalThreads * v, from + 8 * v * lanes);
      }
      copy_close();  // a group per row, empty past the last, so that the count below holds
    } else if (row < hi) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        next[i] = i * lanes + lane < E ? static_cast<uint32_t>(__ldg(from + i * lanes)) << 16
                                       : 0xff800000u;
    }
  }
  // Starts with rows first, first + step, ... below hi.
  __device__ __forceinline__ void open(const uint16_t* logits, int E, int first, int step, int hi,
                                       int lane, int lanes, uint32_t ring_base) {
    ring = ring_base;
    slot = 0;
    row = first;
    from = logits + static_cast<size_t>(first) * E + (kVec ? 8 : 1) * lane;
#pragma unroll
    for (int d = 0; d < (kVec ? kDepth - 1 : 1); ++d) {
      fetch(E, hi, lane, lanes, ring + 16 * kBalThreads * NV * d);
      row += step;
      from += static_cast<size_t>(step) * E;
    }
  }
  // The values of the next row, whose successors keep coming.  (Sigmoids: their extremes too.)
  __device__ __forceinline__ void take(int E, int step, int hi, int lane, int lanes,
                                       float (&x)[NC], Extremes& ext) {
    constexpr uint32_t kRow = 16 * kBalThreads * NV;
    ext.up = ext.down = 0u;
    if constexpr (kVec) {
      fetch(E, hi, lane, lanes, ring + (slot == 0 ? (kDepth - 1) * kRow : slot - kRow));
      copy_wait<kDepth - 1>();
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        uint32_t q[4] = {kPast, kPast, kPast, kPast};
        if (8 * (v * lanes + lane) < E)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                       : "r"(ring + slot + 16 * kBalThreads * v)
                       : "memory");
        if constexpr (!kSoftmax) {
          ext.add(q[0], q[1]);
          ext.add(q[2], q[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * v + 2 * j] = __uint_as_float(q[j] << 16);
          x[8 * v + 2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
        }
      }
      slot = slot == (kDepth - 1) * kRow ? 0 : slot + kRow;
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) x[i] = __uint_as_float(next[i]);
      if constexpr (!kSoftmax) {
#pragma unroll
        for (int i = 0; i < NC; i += 2) ext.add(next[i], next[i + 1]);
      }
      fetch(E, hi, lane, lanes, 0);
    }
    row += step;
    from += static_cast<size_t>(step) * E;
  }
};

template <int NC, bool kVec>
__device__ __forceinline__ unsigned vectors_past(int E, int lane, int lanes) {
  unsigned p = 0u;
#pragma unroll
  for (int v = 0; kVec && v < NC / 8; ++v) p |= 8 * (v * lanes + lane) >= E ? 1u << v : 0u;
  return p;
}

// Shared memory of the loss: the ring, then NC floats per thread.  (The gradient takes the ring.)
template <int NC, bool kVec>
__host__ __device__ constexpr size_t row_smem() {
  return (kVec ? 16ull * kBalThreads * kDepth * (NC / 8) : 0ull) +
         sizeof(float) * kBalThreads * NC;
}

// Column of a lane's element i (may be >= E).
template <bool kVec>
__device__ __forceinline__ int column_of(int i, int lane, int lanes) {
  return kVec ? 8 * ((i >> 3) * lanes + lane) + (i & 7) : i * lanes + lane;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Groups of W warps in a CTA.  A group of several warps (8 groups at most) has a hardware barrier of
// its own beside the CTA's.
__host__ __device__ constexpr int groups_of(int W) { return kBalWarps / W; }

// A sigmoid (of 7.6) from which 1 - s is not taken as it stands: what s was rounded by, 2^-24, would
// be 2^-13 of the difference and more, until at a logit of 17 nothing is left of it.
constexpr float kHighSigmoid = 0.9995f;
// 1 - s of the sigmoid s of x.
__device__ __forceinline__ float one_less(float s, float x) {
  return s > kHighSigmoid ? s * ex2(-kLog2e * x) : 1.0f - s;
}

// Barrier of the W warps of group `grp`.
__device__ __forceinline__ void group_sync(int grp, int W) {
  asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(32 * W) : "memory");
}

// Sigmoids in place.  One reciprocal serves two, 1 / (a b) times the other, unless a product of
// two denominators could leave the range.
template <int NC>
__device__ __forceinline__ void sigmoids(float (&x)[NC], const Extremes& ext) {
  if (!ext.low()) {
#pragma unroll
    for (int i = 0; i < NC; i += 2) {
      const float e0 = 1.0f + ex2(-kLog2e * x[i]), e1 = 1.0f + ex2(-kLog2e * x[i + 1]);
      const float r = rcp(e0 * e1);
      x[i] = r * e1;
      x[i + 1] = r * e0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) x[i] = rcp(1.0f + ex2(-kLog2e * x[i]));
  }
}

// Scores of one row in place, and the row's sums.  On return x holds the terms u_e of the lane
// (scaled by a factor of its own for softmax), `scale` turns a term into a probability, and
// `dot` is sum over e of p_e g_e (kDot); 2^(x log2 e - `top`) `inv` is any column's
// probability in a softmax.  xchg: [2][W] float4 of the group, buffer `buf`; bit v of
// `past`: the lane's v-th vector of 8 columns lies past E.
// A softmax lane takes 2^(x log2 e - m), m its own maximum times log2 e as rounded, and the
// reduction rescales by differences of those same m: nothing is lost to the rounding of m.
// (Two values per instruction, .f32x2, was tried: packing the exponentials cost what it saved.)
template <int NC, bool kSoftmax, bool kDot>
__device__ __forceinline__ void row_terms(float (&x)[NC], const Extremes& ext,
                                          const float (&g)[kDot ? NC : 1], unsigned past, int W,
                                          int grp, int gw, float4* xchg, int buf, float& scale,
                                          float& dot, float& top, float& inv) {
  float m = 0.0f;
  if constexpr (kSoftmax) {
    float m0 = kLowest, m1 = kLowest;
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      m0 = max3(m0, x[i], x[i + 1]);
      m1 = max3(m1, x[i + 2], x[i + 3]);
    }
    m = fmaxf(m0, m1);
    if (!(fabsf(m) <= kFarLogit)) {  // also lanes of -inf alone
      m = fminf(fmaxf(m, -kFarLogit), kFarLogit);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        x[i] = x[i] == -INFINITY ? x[i] : fminf(fmaxf(x[i], -kFarLogit), kFarLogit);
    }
    m *= kLog2e;
#pragma unroll
    for (int i = 0; i < NC; ++i) x[i] = ex2(fmaf(x[i], kLog2e, -m));
  } else {
    sigmoids<NC>(x, ext);
  }
  float sum = 0.0f, d4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < NC / 8; ++v) {
    float s0 = x[8 * v], s1 = x[8 * v + 1];
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
      s0 += x[8 * v + i];
      s1 += x[8 * v + i + 1];
    }
    if (kSoftmax || ((past >> v) & 1u) == 0u) sum += s0 + s1;
  }
  if constexpr (kDot) {
#pragma unroll
    for (int i = 0; i < NC; ++i) d4[i & 3] = fmaf(x[i], g[i], d4[i & 3]);
  }
  float sg = (d4[0] + d4[1]) + (d4[2] + d4[3]);
  float f = 1.0f;  // the lane's factor
  if constexpr (kSoftmax) {
    const float M = warp_max(m);
    f = ex2(m - M);
    sum *= f;
    sg *= f;
    m = M;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, d);
    if constexpr (kDot) sg += __shfl_xor_sync(kFull, sg, d);
  }
  if (W > 1) {
    float4* slot = xchg + buf * W;
    if ((threadIdx.x & 31) == 0) slot[gw] = make_float4(m, sum, sg, 0.0f);
    group_sync(grp, W);
    float M = m;
    if constexpr (kSoftmax)
      for (int w = 0; w < W; ++w) M = fmaxf(M, slot[w].x);
    sum = 0.0f;
    sg = 0.0f;
    for (int w = 0; w < W; ++w) {
      const float4 q = slot[w];
      const float r = kSoftmax ? ex2(q.x - M) : 1.0f;
      sum = fmaf(q.y, r, sum);
      if constexpr (kDot) sg = fmaf(q.z, r, sg);
    }
    if constexpr (kSoftmax) f *= ex2(m - M);
    m = M;
  }
  top = m;
  inv = sum > 0.0f ? rcp(sum) : 0.0f;
  scale = f * inv;
  dot = sg * inv;
}

// ------------------------------------------------------------------------------ the loss
template <int NC, bool kVec, bool kSoftmax, int kW>
__global__ void __launch_bounds__(kBalThreads, 1) mrs_balance_rows_kernel(const BalanceArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float4 xchg_s[kBalWarps][2];
  float* red = reinterpret_cast<float*>(smem + row_smem<NC, kVec>()) - kBalThreads * NC;
  int* hist = reinterpret_cast<int*>(smem + row_smem<NC, kVec>());  // [E]
  const int tid = threadIdx.x, warp = tid >> 5, W = kW > 0 ? kW : a.W, E = a.E;
  const int grp = warp / W, gw = warp - grp * W, groups = groups_of(W);
  const int lanes = 32 * W, lane = 32 * gw + (tid & 31);
  const bool idle = grp >= groups;  // a W that does not divide the warps leaves some without a group
  float4* xchg = &xchg_s[0][0] + grp * 2 * W;
  const uint32_t ring = smem_u32(smem) + 16 * tid;
  const unsigned past = vectors_past<NC, kVec>(E, lane, lanes);
  for (int e = tid; e < E; e += kBalThreads) hist[e] = 0;
  pdl_wait();
  pdl_trigger();  // only now: the second kernel reads the call's inputs before this one ends
  if (blockIdx.x == 0 && tid == 0 && !a.solo) *a.ticket = 0u;
  __syncthreads();

  const int t0 = min(static_cast<int>(blockIdx.x) * a.tpc, a.T);
  const int t1 = min(a.T - t0, a.tpc) + t0;
  float g0[1] = {0.0f};
  float loss = 0.0f;  // solo: this thread's experts
  int t = t0;
  int i = a.solo ? 0 : seq_behind(a.offsets, a.S, a.T, t0);
  bool again = false;
  while (i < a.S && (t < t1 || a.solo)) {
    const int lo_i = seq_border(a.offsets, i, a.T), hi_i = seq_border(a.offsets, i + 1, a.T);
    const int lo = max(lo_i, t), hi = min(hi_i, t1);
    if (hi <= lo) {
      if (a.solo) {
        for (int e = tid; e < E; e += kBalThreads) {
          a.counts[static_cast<size_t>(i) * E + e] = 0;
          a.mean[static_cast<size_t>(i) * E + e] = 0.0f;
        }
      } else if (lo_i >= t1) {
        break;
      }
      ++i;  // mostly one empty sequence; else past any number of them
      if (again && !a.solo) i = max(i, seq_behind(a.offsets, a.S, a.T, lo));
      again = true;
      continue;
    }
    again = false;
    t = hi;
    RowStream<NC, kVec, kSoftmax> rows;
    int row = lo + grp;
    if (!idle) rows.open(a.logits, E, row, groups, hi, lane, lanes, ring);
    // the stretch's routes: loaded now, counted after the rows
    const size_t r1 = static_cast<size_t>(hi) * a.K;
    size_t r = static_cast<size_t>(lo) * a.K + tid;
    int id[kIdsAhead];
#pragma unroll
    for (int q = 0; q < kIdsAhead; ++q, r += kBalThreads) id[q] = r < r1 ? __ldg(a.ids + r) : -1;
    if (!idle && row < hi) {
      float* mine = red + static_cast<size_t>(grp) * lanes * NC;
      // Sums of up to `each` rows, then the sum of those: about 2 sqrt(rows) additions deep and not
      // one per row, which for 7000 rows of equal terms is off by up to 2^-11.
      int each = kSumRows;
      while (static_cast<long long>(each) * each * groups < hi - lo) each *= 2;
      for (int buf = 0, part = 0; row < hi; ++part) {
        float acc[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c] = 0.0f;
        for (int q = 0; q < each && row < hi; ++q, row += groups, buf ^= 1) {
          float x[NC], scale, dot, top, inv;
          Extremes ext;
          rows.take(E, groups, hi, lane, lanes, x, ext);
          row_terms<NC, kSoftmax, false>(x, ext, g0, past, W, grp, gw, xchg, buf, scale, dot, top, inv);
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[c] = fmaf(x[c], scale, acc[c]);
        }
#pragma unroll
        for (int c = 0; c < NC; c += kVec ? 4 : 1) {
          float* to = mine + column_of<kVec>(c, lane, lanes);
          if constexpr (kVec) {
            float4* to4 = reinterpret_cast<float4*>(to);
            const float4 had = part > 0 ? *to4 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            *to4 = make_float4(had.x + acc[c], had.y + acc[c + 1], had.z + acc[c + 2],
                               had.w + acc[c + 3]);
          } else {
            *to = part > 0 ? *to + acc[c] : acc[c];
          }
        }
      }
    }
    auto count = [&](int e) {
      if (e >= 0 && e < E) atomicAdd(hist + e, 1);  // integers: any order, the same sum
    };
#pragma unroll
    for (int q = 0; q < kIdsAhead; ++q) count(id[q]);
    for (; r < r1; r += kBalThreads) count(__ldg(a.ids + r));
    copy_wait_all();
    __syncthreads();
    const int had = min(groups, hi - lo);  // groups with a row of the stretch
    const size_t slot = static_cast<size_t>(a.solo ? i : blockIdx.x + i) * E;
    const float n = static_cast<float>(hi - lo);
    for (int e = tid; e < E; e += kBalThreads) {
      float s = red[e];
#pragma unroll 4
      for (int q = 1; q < had; ++q) s += red[static_cast<size_t>(q) * lanes * NC + e];
      const int c = hist[e];
      hist[e] = 0;
      if (a.solo) {
        const float mean = s / n;
        a.counts[slot + e] = c;
        a.mean[slot + e] = mean;
        loss += static_cast<float>(c) * mean / n;
      } else {
        a.psum[slot + e] = s;
        a.csum[slot + e] = c;
      }
    }
    __syncthreads();
    ++i;
  }
  if (a.solo) {
    loss = warp_sum(loss);
    if ((tid & 31) == 0) red[warp] = loss;
    __syncthreads();
    if (warp == 0) {
      loss = warp_sum(tid < kBalWarps ? red[tid] : 0.0f);
      if (tid == 0) *a.loss = loss * (a.coef * a.E / (static_cast<float>(a.K) * a.S));
    }
  }
}

// Joins the slots: CTA (bx, by) takes 32 experts of the sequences by, by + gridDim.y, ...; warp w
// the slots w, w + 8, ... of a sequence.  The last CTA to finish adds the loss.  (In fp64 its few
// divisions took 4 us.  Its terms are all of one sign, and a thread's sum over sequences is
// compensated: against 64 bits the losses of T = 64 to 16384 measured within 2e-7.)
__global__ void __launch_bounds__(kJoinThreads) mrs_balance_join_kernel(const BalanceArgs a) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float ps[2][kWarps][32];
  __shared__ int cs[2][kWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int e = blockIdx.x * 32 + lane;
  // the borders are inputs: the first kernel started after they were written
  int lo = seq_border(a.offsets, blockIdx.y, a.T), hi = seq_border(a.offsets, blockIdx.y + 1, a.T);
  pdl_trigger();
  pdl_wait();
  float loss = 0.0f, lost = 0.0f;  // a sum of up to 8192 sequences, and what its roundings left out
  int buf = 0;
  for (int i = blockIdx.y; i < a.S; i += gridDim.y, buf ^= 1) {
    float p = 0.0f;
    int c = 0;
    if (hi > lo && e < a.E) {
      const int b0 = lo / a.tpc + warp, b1 = (hi - 1) / a.tpc;
      const size_t at = static_cast<size_t>(i) * a.E + e;
#pragma unroll 8
      for (int b = b0; b <= b1; b += kWarps) {
        p += a.psum[at + static_cast<size_t>(b) * a.E];
        c += a.csum[at + static_cast<size_t>(b) * a.E];
      }
    }
    ps[buf][warp][lane] = p;
    cs[buf][warp][lane] = c;
    __syncthreads();
    if (warp == 0 && e < a.E) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        p += ps[buf][w][lane];
        c += cs[buf][w][lane];
      }
      const float n = static_cast<float>(max(hi - lo, 1));
      const float mean = p / n;
      const size_t at = static_cast<size_t>(i) * a.E + e;
      a.counts[at] = c;
      a.mean[at] = mean;
      const float add = static_cast<float>(c) * mean / n - lost, sum = loss + add;
      lost = (sum - loss) - add;
      loss = sum;
    }
    lo = seq_border(a.offsets, min(i + static_cast<int>(gridDim.y), a.S), a.T);
    hi = seq_border(a.offsets, min(i + static_cast<int>(gridDim.y) + 1, a.S), a.T);
  }
  if (warp != 0) return;
  // this CTA's part of the loss, then everybody's
  const int ctas = gridDim.x * gridDim.y;
  loss = warp_sum(loss);
  int last = 0;
  if (lane == 0) {
    a.partial[blockIdx.y * gridDim.x + blockIdx.x] = loss;
    unsigned before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(a.ticket)
                 : "memory");
    last = before == static_cast<unsigned>(ctas - 1) ? 1 : 0;
  }
  if (__shfl_sync(kFull, last, 0) == 0) return;
  __syncwarp();  // (a shuffle orders no memory: the other lanes' reads come behind the ticket)
  float s = 0.0f;
  for (int q = lane; q < ctas; q += 32) s += __ldcg(a.partial + q);
  s = warp_sum(s);
  if (lane == 0) *a.loss = s * (a.coef * a.E / (static_cast<float>(a.K) * a.S));
}

// -------------------------------------------------------------------------- the gradient
template <int NC, bool kVec, bool kSoftmax, int kW, class Out>
__global__ void __launch_bounds__(kBalThreads, 1)
    mrs_route_backward_kernel(const RouteBackwardArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float4 xchg_s[kBalWarps][2];
  const int tid = threadIdx.x, warp = tid >> 5, wl = tid & 31;
  const int W = kW > 0 ? kW : a.W, E = a.E, K = a.K;
  const int grp = warp / W, gw = warp - grp * W, groups = groups_of(W);
  const int lanes = 32 * W, lane = 32 * gw + wl;
  float4* xchg = &xchg_s[0][0] + grp * 2 * W;
  const uint32_t ring = smem_u32(smem) + 16 * tid;
  const unsigned past = vectors_past<NC, kVec>(E, lane, lanes);
  pdl_trigger();
  if (grp >= groups) return;  // a W that does not divide the warps leaves some without a group
  pdl_wait();
  const bool dense = a.gl != nullptr, sparse = a.gw != nullptr;
  const float gl = dense ? __ldg(a.gl) : 0.0f;

  const int t0 = min(static_cast<int>(blockIdx.x) * a.tpc, a.T);
  const int t1 = min(a.T - t0, a.tpc) + t0;
  int i = seq_behind(a.offsets, a.S, a.T, t0);
  int buf = 0;
  for (int t = t0; t < t1;) {
    // the next stretch: a part of sequence i, or tokens of none (no balance term)
    int hi = t1;
    bool in_seq = false;
    int lo_i = 0, hi_i = 0;
    for (bool again = false; i < a.S; again = true) {
      lo_i = seq_border(a.offsets, i, a.T);
      hi_i = seq_border(a.offsets, i + 1, a.T);
      if (hi_i > t && hi_i > lo_i) break;
      ++i;  // mostly the next one; else past any number of empty ones
      if (again) i = max(i, seq_behind(a.offsets, a.S, a.T, max(t, lo_i)));
    }
    if (i < a.S) {
      in_seq = lo_i <= t;
      hi = min(t1, in_seq ? hi_i : lo_i);
    }
    float g[NC], f = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) g[c] = 0.0f;
    const int32_t* counts = a.counts;
    int even = 0;
    if (dense && in_seq) {
      const float n = static_cast<float>(hi_i - lo_i);
      // sum p = 1, so any number may be taken off the counts: that of an even router, for what an
      // almost even one has left is little beside its counts
      even = static_cast<int>(static_cast<float>(K) * n / E);
      f = gl * (a.coef / a.S) * (static_cast<float>(E) / K) / n / n;
      counts += static_cast<size_t>(i) * E;
      if (kVec && a.wide_counts) {
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const int e = column_of<kVec>(c, lane, lanes);
          if (e >= E) continue;
          const int4 q = __ldg(reinterpret_cast<const int4*>(counts + e));
          g[c] = f * static_cast<float>(q.x - even);
          g[c + 1] = f * static_cast<float>(q.y - even);
          g[c + 2] = f * static_cast<float>(q.z - even);
          g[c + 3] = f * static_cast<float>(q.w - even);
        }
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int e = column_of<kVec>(c, lane, lanes);
          if (e < E) g[c] = f * static_cast<float>(__ldg(counts + e) - even);
        }
      }
    }
    RowStream<NC, kVec, kSoftmax> rows;
    int row = t + grp;
    int next_id = -1;
    float next_gw = 0.0f;
    auto fetch = [&](int r) {
      if (sparse && wl < K && r < hi) {
        next_id = __ldg(a.ids + static_cast<size_t>(r) * K + wl);
        next_gw = __ldg(a.gw + static_cast<size_t>(r) * K + wl);
      }
    };
    rows.open(a.logits, E, row, groups, hi, lane, lanes, ring);
    fetch(row);
    for (; row < hi; row += groups) {
      const uint16_t* xr = a.logits + static_cast<size_t>(row) * E;
      float x[NC];
      int id = next_id;
      float wg = next_gw;
      const bool valid = sparse && wl < K && id >= 0 && id < E;
      const float xk = valid ? bf16_bits_to_float(__ldg(xr + id)) : -INFINITY;
      const float gk = valid && f != 0.0f ? f * static_cast<float>(__ldg(counts + id) - even) : 0.0f;
      fetch(row + groups);
      Extremes ext;
      rows.take(E, groups, hi, lane, lanes, x, ext);
      float scale = 0.0f, dot = 0.0f, top = 0.0f, inv = 0.0f;
      if (dense) {
        row_terms<NC, kSoftmax, true>(x, ext, g, past, W, grp, gw, xchg, buf, scale, dot, top, inv);
        buf ^= 1;
        if (!kSoftmax && ext.high()) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float p = x[c] * scale;
            float q = fmaf(-p, x[c], p);
            if (x[c] > kHighSigmoid)
              q = p * one_less(x[c], bf16_bits_to_float(__ldg(xr + column_of<kVec>(c, lane, lanes))));
            x[c] = q * (g[c] - dot);
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float p = x[c] * scale;
            x[c] = (kSoftmax ? p : fmaf(-p, x[c], p)) * (g[c] - dot);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) x[c] = 0.0f;
      }
      Out* out = static_cast<Out*>(a.out) + static_cast<size_t>(row) * E;
      if constexpr (kVec) {
#pragma unroll
        for (int v = 0; v < NC / 8; ++v) {
          const int c = 8 * (v * lanes + lane);
          if (c >= E) continue;
          const float* y = x + 8 * v;
          if constexpr (sizeof(Out) == 4) {
            float4* o = reinterpret_cast<float4*>(out + c);
            o[0] = make_float4(y[0], y[1], y[2], y[3]);
            o[1] = make_float4(y[4], y[5], y[6], y[7]);
          } else {
            // bf16 gradients: one rounding of the fp32 sum
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
              w[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int e = c * lanes + lane;
          if (e >= E) continue;
          if constexpr (sizeof(Out) == 4) out[e] = x[c];
          else out[e] = __float2bfloat16_rn(x[c]);
        }
      }
      if (sparse) {
        // Every warp of the group works the K routes out, lane k route k, and writes those in its
        // columns: the whole gradient there, its balance term taken anew from the row's sums, over
        // the one that the column's lane has just written.
        if (!valid) wg = 0.0f;
        float u, s = 0.0f, less = 1.0f;
        const float m = fmaxf(warp_max(xk), kLowest);
        // The weights' sum is constant, so their gradients count from any one of them: from the
        // largest weight's, so that a route that holds nearly all has the others' small part as it
        // is and not as a difference (a token's only route: 0, where u rcp(u) is not quite 1).
        wg -= __shfl_sync(kFull, wg, (__ffs(__ballot_sync(kFull, xk == m)) - 1) & 31);
        if (kSoftmax) {
          u = ex2((xk - m) * kLog2e);
        } else {
          u = s = rcp(1.0f + ex2(-kLog2e * xk));  // 0 for a route that is none
          less = one_less(s, xk);
        }
        const float su = warp_sum(u);
        const float q = su > 0.0f ? u * rcp(su) : 0.0f;
        const float mean = warp_sum(q * wg);
        float d = a.R * q * (wg - mean) * less;
        // an expert named twice: the lowest lane takes the sum, in slot order
        const int key = valid ? id : -1 - wl;
        const unsigned same = __match_any_sync(kFull, key);
        if (__any_sync(kFull, (same & (same - 1u)) != 0u)) {
          float all = 0.0f;
          for (int l = 0; l < 32; ++l) {
            const float o = __shfl_sync(kFull, d, l);
            if ((same >> l) & 1u) all += o;
          }
          d = all;
        }
        const int owner = kVec ? (id >> 3) % lanes : id % lanes;
        const float xc = fminf(fmaxf(xk, -kFarLogit), kFarLogit);
        // (without the loss there are no sums to take the power against: it could leave the range)
        const bool none = !dense || xk == -INFINITY;
        const float p = kSoftmax ? (none ? 0.0f : ex2(fmaf(xc, kLog2e, -top)) * inv) : s * inv;
        d = fmaf(p * less, gk - dot, d);
        __syncwarp();  // the row's own stores come first
        if (valid && (same & lanemask_lt(wl)) == 0u && (owner >> 5) == gw) {
          if constexpr (sizeof(Out) == 4) out[id] = d;
          else out[id] = __float2bfloat16_rn(d);
        }
      }
    }
    copy_wait_all();  // the groups past the last row are empty
    t = hi;
  }
}

// ------------------------------------------------------------------------------ host side
namespace {

// Warps per row, columns per lane and the kind of loads for E experts.  16-byte loads need rows
// that start on 16 bytes (E a multiple of 8); without them a lane's next row is in registers, and
// more than 16 columns would not fit there.  (The widest calls fill 71% of the issue slots, a third
// of them per row and not per column: twice the warps with half the columns took T = 16384, E = 4096
// from 45 to 50 us.)
struct RowPlan {
  int W, NC;
  bool vec;
};
RowPlan row_plan(int E) {
  RowPlan p{};
  p.vec = E % 8 == 0;
  p.W = p.vec ? (E + 1023) / 1024 : (E + 511) / 512;
  const int per = p.vec ? (E / 8 + 32 * p.W - 1) / (32 * p.W) * 8 : (E + 32 * p.W - 1) / (32 * p.W);
  p.NC = per <= 8 ? 8 : (per <= 16 ? 16 : 32);
  return p;
}

// Tokens per CTA: one row per group of warps until every SM has a CTA.
int tokens_per_cta(int T, int W, int sms) {
  const int groups = groups_of(W);
  int ctas = sms < kBalMaxCtas ? sms : kBalMaxCtas;
  const int most = (T + groups - 1) / groups;
  if (most < ctas) ctas = most;
  return (T + ctas - 1) / ctas;
}

struct BalanceLayout {
  size_t ticket, partial, psum, csum, total;
};
// The largest number of CTAs of any device bounds the slots.
BalanceLayout balance_layout(int T, int E, int S) {
  const size_t most = static_cast<size_t>(T) < kBalMaxCtas ? static_cast<size_t>(T) : kBalMaxCtas;
  const size_t slots = (most + static_cast<size_t>(S)) * static_cast<size_t>(E);
  BalanceLayout l{};
  l.partial = 16;
  l.psum = l.partial + sizeof(float) * kBalMaxJoin;
  l.csum = align16(l.psum + sizeof(float) * slots);
  l.total = align16(l.csum + sizeof(int32_t) * slots);
  return l;
}

int check_router(int T, int E, int K, int S) {
  if (T < 0) return MOE_RS_ERR_BAD_TOKENS;
  if (E < 1 || E > kMaxExperts) return MOE_RS_ERR_BAD_EXPERTS;
  if (K < 1 || K > kMaxTopk || K > E) return MOE_RS_ERR_BAD_TOPK;
  if (S < 1 || S > MOE_RS_MAX_SEQUENCES) return MOE_RS_ERR_BAD_SEQUENCES;
  // (row numbers run a few rows past T)
  if (static_cast<int64_t>(T) * K > INT32_MAX || T > INT32_MAX - (1 << 16))
    return MOE_RS_ERR_OVERFLOW;
  return MOE_RS_OK;
}

template <int NC, bool kVec, int kW>
cudaError_t launch_balance(const BalanceArgs& a, bool softmax, int ctas, cudaStream_t st) {
  auto* k = softmax ? mrs_balance_rows_kernel<NC, kVec, true, kW>
                    : mrs_balance_rows_kernel<NC, kVec, false, kW>;
  const size_t smem = row_smem<NC, kVec>() + sizeof(int) * static_cast<size_t>(a.E);
  static SmemGrant granted[2];
  const cudaError_t err =
      grant_smem(reinterpret_cast<const void*>(k),
                 row_smem<NC, kVec>() + sizeof(int) * kMaxExperts, granted[softmax]);
  if (err != cudaSuccess) return err;
  return launch_pdl(k, dim3(ctas), dim3(kBalThreads), smem, st, a);
}

template <int NC, bool kVec, int kW, class Out>
cudaError_t launch_backward(const RouteBackwardArgs& a, bool softmax, int ctas, cudaStream_t st) {
  auto* k = softmax ? mrs_route_backward_kernel<NC, kVec, true, kW, Out>
                    : mrs_route_backward_kernel<NC, kVec, false, kW, Out>;
  const size_t smem = row_smem<NC, kVec>() - sizeof(float) * kBalThreads * NC;  // the ring alone
  static SmemGrant granted[2];
  const cudaError_t err =
      grant_smem(reinterpret_cast<const void*>(k), smem, granted[softmax]);
  if (err != cudaSuccess) return err;
  return launch_pdl(k, dim3(ctas), dim3(kBalThreads), smem, st, a);
}

// The kernels' instances: 8, 16 or 32 columns per lane in vectors, more than one warp a row only
// with 32; 8 or 16 without, any number of warps.
template <class Go>
cudaError_t with_plan(const RowPlan& p, Go go) {
  using std::integral_constant;
  using N8 = integral_constant<int, 8>;
  using N16 = integral_constant<int, 16>;
  using N32 = integral_constant<int, 32>;
  using Any = integral_constant<int, 0>;
  using W1 = integral_constant<int, 1>;
  if (!p.vec)
    return p.NC == 8 ? go(N8{}, std::false_type{}, Any{}) : go(N16{}, std::false_type{}, Any{});
  if (p.W == 2) return go(N32{}, std::true_type{}, integral_constant<int, 2>{});
  if (p.W == 3) return go(N32{}, std::true_type{}, integral_constant<int, 3>{});
  if (p.W == 4) return go(N32{}, std::true_type{}, integral_constant<int, 4>{});
  return p.NC == 8    ? go(N8{}, std::true_type{}, W1{})
         : p.NC == 16 ? go(N16{}, std::true_type{}, W1{})
                      : go(N32{}, std::true_type{}, W1{});
}

}  // namespace
}  // namespace mrs

using namespace mrs;

extern "C" {

size_t moe_balance_workspace_bytes(int T, int E, int n_seq) {
  if (check_router(T, E, 1, n_seq)) return 0;
  return balance_layout(T, E, n_seq).total;
}

int moe_balance_loss(const void* logits_bf16, const int32_t* topk_ids, const int32_t* seq_offsets,
                     int T, int E, int topk, int n_seq, int softmax, float coef, float* loss,
                     int32_t* counts, float* mean_probs, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  int rc = check_router(T, E, topk, n_seq);
  if (rc) return rc;
  if (!std::isfinite(coef)) return MOE_RS_ERR_BAD_SCALE;
  if (!seq_offsets && n_seq != 1) return MOE_RS_ERR_BAD_SEQUENCES;
  if (!workspace) return MOE_RS_ERR_WORKSPACE;
  if (!loss || !counts || !mean_probs || (T > 0 && (!logits_bf16 || !topk_ids)))
    return MOE_RS_ERR_NULL_POINTER;
  const BalanceLayout l = balance_layout(T, E, n_seq);
  if (workspace_bytes < l.total) return MOE_RS_ERR_WORKSPACE;
  if (!aligned(workspace, 16) || !aligned(loss, 4) || !aligned(counts, 4) ||
      !aligned(mean_probs, 4) || !aligned(seq_offsets, 4) ||
      (T > 0 && (!aligned(logits_bf16, 16) || !aligned(topk_ids, 4))))
    return MOE_RS_ERR_MISALIGNED;
  const size_t SE = static_cast<size_t>(n_seq) * E;
  const Span outs[] = {span(loss, 4), span(counts, 4 * SE), span(mean_probs, 4 * SE),
                       span(workspace, workspace_bytes)};
  const Span ins[] = {span(logits_bf16, 2 * static_cast<size_t>(T) * E),
                      span(topk_ids, 4 * static_cast<size_t>(T) * topk),
                      span(seq_offsets, seq_offsets ? 4 * (static_cast<size_t>(n_seq) + 1) : 0)};
  if (any_alias(outs, 4, ins, 3)) return MOE_RS_ERR_ALIAS;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  const RowPlan p = row_plan(E);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  BalanceArgs a{};
  a.logits = static_cast<const uint16_t*>(logits_bf16);
  a.ids = topk_ids;
  a.offsets = seq_offsets;
  a.T = T;
  a.E = E;
  a.K = topk;
  a.S = n_seq;
  a.W = p.W;
  const int groups = groups_of(p.W);
  a.solo = T <= kSoloRows * groups && n_seq <= kSoloSeqs;
  a.tpc = a.solo || T == 0 ? (T > 0 ? T : 1) : tokens_per_cta(T, p.W, sms);
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.mean = mean_probs;
  a.ticket = reinterpret_cast<unsigned*>(ws);
  a.partial = reinterpret_cast<float*>(ws + l.partial);
  a.psum = reinterpret_cast<float*>(ws + l.psum);
  a.csum = reinterpret_cast<int32_t*>(ws + l.csum);
  const int ctas = T > 0 ? (T + a.tpc - 1) / a.tpc : 1;
  const cudaError_t err = with_plan(p, [&](auto nc, auto vec, auto w) {
    return launch_balance<decltype(nc)::value, decltype(vec)::value, decltype(w)::value>(
        a, softmax != 0, ctas, stream);
  });
  if (err != cudaSuccess || a.solo) return launch_status(err);
  const int gx = (E + 31) / 32;
  int gy = kBalMaxJoin / gx < 8 ? 8 : kBalMaxJoin / gx;  // gx <= 128
  if (gy > n_seq) gy = n_seq;
  return launch_status(
      launch_pdl(mrs_balance_join_kernel, dim3(gx, gy), dim3(kJoinThreads), 0, stream, a));
}

int moe_route_backward(const void* logits_bf16, const int32_t* topk_ids, const float* grad_weights,
                       const float* grad_loss, const int32_t* counts, const int32_t* seq_offsets,
                       int T, int E, int topk, int n_seq, int softmax, float routed_scale,
                       float coef, void* grad_logits, int grad_dtype, cudaStream_t stream) {
  int rc = check_router(T, E, topk, n_seq);
  if (rc) return rc;
  if (grad_dtype != MOE_RS_BF16 && grad_dtype != MOE_RS_FP32) return MOE_RS_ERR_BAD_DTYPE;
  if (!std::isfinite(coef) || !std::isfinite(routed_scale)) return MOE_RS_ERR_BAD_SCALE;
  if (!seq_offsets && n_seq != 1) return MOE_RS_ERR_BAD_SEQUENCES;
  if (T == 0) return MOE_RS_OK;
  if (!logits_bf16 || !grad_logits || (grad_weights && !topk_ids) || (grad_loss && !counts))
    return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(logits_bf16, 16) || !aligned(grad_logits, 16) || !aligned(topk_ids, 4) ||
      !aligned(grad_weights, 4) || !aligned(grad_loss, 4) || !aligned(counts, 4) ||
      !aligned(seq_offsets, 4))
    return MOE_RS_ERR_MISALIGNED;
  const size_t TE = static_cast<size_t>(T) * E, TK = static_cast<size_t>(T) * topk;
  const Span outs[] = {span(grad_logits, (grad_dtype == MOE_RS_FP32 ? 4 : 2) * TE)};
  const Span ins[] = {span(logits_bf16, 2 * TE),
                      span(topk_ids, topk_ids ? 4 * TK : 0),
                      span(grad_weights, grad_weights ? 4 * TK : 0),
                      span(grad_loss, grad_loss ? 4 : 0),
                      span(counts, counts ? 4 * static_cast<size_t>(n_seq) * E : 0),
                      span(seq_offsets, seq_offsets ? 4 * (static_cast<size_t>(n_seq) + 1) : 0)};
  if (any_alias(outs, 1, ins, 6)) return MOE_RS_ERR_ALIAS;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  const RowPlan p = row_plan(E);
  RouteBackwardArgs a{};
  a.logits = static_cast<const uint16_t*>(logits_bf16);
  a.ids = topk_ids;
  a.gw = grad_weights;
  a.gl = grad_loss;
  a.counts = counts;
  a.offsets = seq_offsets;
  a.T = T;
  a.E = E;
  a.K = topk;
  a.S = n_seq;
  a.W = p.W;
  a.tpc = tokens_per_cta(T, p.W, sms);
  a.wide_counts = aligned(counts, 16);
  a.R = routed_scale;
  a.coef = coef;
  a.out = grad_logits;
  const int ctas = (T + a.tpc - 1) / a.tpc;
  const bool sm = softmax != 0, f32 = grad_dtype == MOE_RS_FP32;
  return launch_status(with_plan(p, [&](auto nc, auto vec, auto w) {
    constexpr int NC = decltype(nc)::value, kW = decltype(w)::value;
    constexpr bool V = decltype(vec)::value;
    return f32 ? launch_backward<NC, V, kW, float>(a, sm, ctas, stream)
               : launch_backward<NC, V, kW, __nv_bfloat16>(a, sm, ctas, stream);
  }));
}

}  // extern "C"
