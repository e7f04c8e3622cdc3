// mrs_product.cu -- the experts' products in 16 and 8 bits, driven by the sort step, and the
// gradient of their rows.
//
// For every route r of the sorted list, with e the owner of its block:
//   out[r, m] = w_r * sx_row * sw_em * sum over k of X[row, k] A_e[m, k]
// A_e is W[e] (m an output, k a column), or for the rows' gradient its transpose (m a column, k an
// output).  Sums are fp32; the row's weight, its scale and the output's scale are applied in fp32,
// and the result is rounded once.
//
// A pair of CTAs computes tiles of 256 m by up to 256 (or 64) rows of one expert.  m, which is
// regular and long, is on the 256 lanes of both tensor memories, the ragged rows are the product's
// N, which goes in steps of 32: an expert's last rows cost what they are, not a whole tile.  Each
// CTA brings 128 m and half of the rows into shared memory, 128 bytes of each a step, so that a
// byte of either operand serves twice the products that it would in one CTA.  Rows are copied by
// threads: tensor copies that gather four rows take their warp 100 to 400 clocks each (T = 8192,
// E = 64, 7168 -> 2048: 1600 us with four warps of them, 1380 with four warps of thread copies).
//
// The warps of a CTA each have one task:
//   0      copies of a step's weights
//   1      the list: rows, routes and factors of the next units into a ring in shared memory
//   2      in the first CTA of a pair the products; both CTAs' copies are counted on its barriers
//   4-11   finished tiles from tensor memory to the output rows, while the next one is computed
//   12-15  copies of a step's rows; 3 says when those that threads write are there
// Every wait is bounded; one that gives up ends its warp's task with the status bit set.  The CTAs
// of a pair leave together.
//
// The sums are the tensor core's: it keeps fp32 and cuts where an addition would round, so that they
// come out low, by 1.0e-6 of their size over 1024 columns, 4.4e-6 over 4096 and 1.9e-5 over 16384.
//
// Bound by the weights' bytes where an expert has few rows (T = 512, E = 896, 3584 -> 768, 16 bits:
// 720 us, the floor of 729 at the rate of a copy; 8 bits 388 of 365) and by the tensor cores where it has
// many: T = 8192, E = 64, topk = 8, 7168 -> 2048 in 1150 to 1340 us, cool and warm, up to 84 % of the tensor
// cores' clocks; a library product of the same size in one piece takes 996 at the rate of a short run and
// 1116 at that of a long one, where power holds the clock.  In 8 bits 600 to 650 us, of 498.  Short contractions (8192 skewed tokens, E = 896,
// 384 -> 3584 in 8 bits, 430 us of 329) wait for the warps that store: three steps of products are
// 130 KB of output.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mrs_product.cuh"
#include "mrs_rows.cuh"

namespace mrs {

// ------------------------------------------------------------------------ the row tiles
// Cuts the list into tiles: kThreads threads of a CTA, start [E + 1] and used [E] its shared memory,
// meet a word for each warp.  put(i, expert, first row, rows) gets tile i; returns how many there are.
template <int kThreads, class Put>
__device__ __forceinline__ int cut_list(const ListArgs& a, int* start, int* used, int* meet,
                                        int32_t* status, Put&& put) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (the first owners are on their way together with the list's length)
  const bool holds = tid < a.max_rows >> a.log2B;
  const int owner = holds ? __ldg(a.eid + tid) : 0, previous = holds && tid > 0 ? __ldg(a.eid + tid - 1) : -1;
  const int blocks = min(max(__ldg(a.npp), 0), a.max_rows) >> a.log2B;
  for (int e = tid; e <= a.E; e += kThreads) start[e] = blocks;
  __syncthreads();
  bool bad = false;
  auto look = [&](int b, int e, int before) {
    if (e < 0 || e >= a.E || e < before) bad = true;
    else if (e != before) start[e] = b;
  };
  if (tid < blocks) look(tid, owner, previous);
#pragma unroll 4
  for (unsigned b = tid + kThreads; b < static_cast<unsigned>(blocks); b += kThreads)
    look(b, __ldg(a.eid + b), __ldg(a.eid + b - 1));
  if (__syncthreads_or(bad) && tid == 0) atomicOr(status, MOE_RS_DEVICE_BAD_EXPERT_ID);
  // an expert without a run starts where the next one does: the least start from it on (which is
  // in order whatever the list holds)
  const int each = (a.E + kThreads - 1) / kThreads, e0 = min(tid * each, a.E), e1 = min(e0 + each, a.E);
  int least = blocks;
  for (int e = e0; e < e1; ++e) least = min(least, start[e]);
  int after = least;  // of the warp's threads from this one on
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_down_sync(kFull, after, o);
    if (lane + o < 32) after = min(after, v);
  }
  if (lane == 0) meet[warp] = after;
  int next = __shfl_down_sync(kFull, after, 1);
  if (lane == 31) next = blocks;
  __syncthreads();
  for (int w = warp + 1; w < kWarps; ++w) next = min(next, meet[w]);
  for (int e = e1 - 1; e >= e0; --e) start[e] = next = min(next, start[e]);
  __syncthreads();
  // rows of each run; where asked for, up to its last route: routes come first in its last block
  for (int e = tid; e < a.E; e += kThreads) {
    const int p0 = start[e] * a.B, rows = (start[e + 1] - start[e]) * a.B;
    used[e] = rows;
    if (a.by_used && rows > 0) {
      const int32_t* s = a.sid + p0 + rows - a.B;
      used[e] = rows - a.B + prefix_length(a.B, [&](int i) {
                  const int r = __ldg(s + i);
                  return r >= 0 && r < a.routes;
                });
    }
  }
  __syncthreads();
  auto tile_rows = [&](int e) {
    // (rows and a.rows, in 32 bits without a sign, stay below 2^32)
    const unsigned rows = used[e], most = a.rows, n = (rows + most - 1) >> a.log2R;
    if (!a.by_used || n <= 1) return n == 0 || !a.by_used ? most : min((rows + 31) & ~31u, most);
    return min(((rows + n - 1) / n + 31) & ~31u, most);
  };
  int count = 0;
  for (int e = e0; e < e1; ++e) {
    const unsigned rows = used[e], t = tile_rows(e);
    count += t == static_cast<unsigned>(a.rows) ? (rows + t - 1) >> a.log2R : (rows + t - 1) / t;
  }
  int sum = count;  // tiles up to this thread's experts
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) meet[warp] = sum;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) sum += meet[w];
    total += meet[w];
  }
  int at = sum - count;
  for (int e = e0; e < e1; ++e) {
    const int p0 = start[e] * a.B, rows = used[e], t = static_cast<int>(tile_rows(e));
    for (int64_t r = 0; r < rows; r += t, ++at)
      put(at, e, p0 + static_cast<int>(r), min(t, rows - static_cast<int>(r)));
  }
  return total;
}

// Of lists that are too long for every CTA of the product to cut them: one CTA, into the workspace.
constexpr int kTableThreads = 1024;

__global__ void __launch_bounds__(kTableThreads)
    mrs_product_table_kernel(const ListArgs a, const ProductTable t, int max_tiles) {
  __shared__ int start[kMaxExperts + 1], used[kMaxExperts], meet[32];
  pdl_trigger();
  pdl_wait();
  const int n = cut_list<kTableThreads>(a, start, used, meet, t.head,
                                        [&](int i, int e, int p0, int rows) {
                                          if (i < max_tiles) t.tiles[i] = make_int4(e, p0, rows, 0);
                                        });
  if (threadIdx.x == 0) t.head[1] = min(n, max_tiles);
}

// ------------------------------------------------------------------------- the products
struct ProductArgs {
  ListArgs list;
  ProductTable t;
  int here;  // every CTA cuts the list by itself
  const float *sw, *xs, *ws;  // or null
  const unsigned char* x;
  void* out;
  unsigned long long wait_limit_ns;
  int topk, per_route, max_tiles;
  int E, M, K, P;  // M: outputs of the product; K: the contraction; P: rows of the list at most
  int mtiles, chunk, nchunk, ksteps;
  int type;        // of the operands: 0 fp16 or e4m3, 1 bf16
  int out_type;
};

constexpr int kProductTmem = 512;
constexpr int kPairRows = 256;  // m of a tile
constexpr int kInfoSlots = 3;
constexpr int kTilesHere = 1024;    // of a list that every CTA cuts by itself
constexpr int kBlocksHere = 8192;
constexpr int kInfoUsers = 14;  // weights, announcer, eight that store, four with rows; the products
// A CTA's half of a tile's rows is copied by threads, 32 rows by a warp: those of wide tiles by four
// warps, the 32 of narrow ones by four that take steps in turn.
template <int R>
constexpr int kRowWarps = R > 64 ? 4 : 1;  // of a step
template <int R>
constexpr int kRowTurns = 4 / kRowWarps<R>;
constexpr int kProductThreads = 512;
// Accumulators.  With two, a narrow tile's products wait for the stores of the tile before the last:
// the ways from products to stores and back take longer than either.
template <int R>
constexpr int kAccs = kProductTmem / R;

template <int R>
struct ProductShape {
  static constexpr int kW = 128 * 128;
  static constexpr int kX = R / 2 * 128;
  static constexpr int kSlots = R == 256 ? 6 : 9;
  static constexpr size_t kSmem = static_cast<size_t>(kSlots) * (kW + kX) + 1024;
};

template <int R>
struct ProductInfo {
  int e, n, m0, tiles, half, pad[3];  // e < 0: no more units
  int src[R / 2];                     // rows of X that this CTA copies
  int route[R];                       // -1: none
  float factor[R];
};

// Two values to 16 bits, one rounding each.
__device__ __forceinline__ uint32_t rounded2(float lo, float hi, int type) {
  if (type == MOE_RS_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kFp8, bool kTranspose, int R, class Out>
__global__ void __launch_bounds__(kProductThreads, 1)
    mrs_product_kernel(const __grid_constant__ CUtensorMap wmap, const ProductArgs a) {
  using Sh = ProductShape<R>;
  constexpr int S = Sh::kSlots;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned long long full_s[S], free_s[S], rows_s[S], acc_full_s[kAccs<R>],
      acc_free_s[kAccs<R>], info_full_s[kInfoSlots], info_free_s[kInfoSlots], done_s;
  __shared__ __align__(16) ProductInfo<R> info_s[kInfoSlots];
  __shared__ __align__(16) uint16_t stage_s[sizeof(Out) == 2 ? 8 : 1][32 * 32];
  __shared__ int2 tiles_s[kTilesHere];  // first row of the list; expert, rows - 1
  __shared__ int meet_s[32];
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(pair_rank());
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t wbase = base, xbase = base + S * Sh::kW;
  const unsigned long long limit = a.wait_limit_ns;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_s[s], 3);  // the tensor copies, both CTAs' threads
      mbar_init(&free_s[s], 1);
      mbar_init(&rows_s[s], 32 * kRowWarps<R>);  // every copying thread
    }
    for (int b = 0; b < kAccs<R>; ++b) {
      mbar_init(&acc_full_s[b], 1);
      mbar_init(&acc_free_s[b], 16);  // the storing warps of both CTAs
    }
    for (int i = 0; i < kInfoSlots; ++i) {
      mbar_init(&info_full_s[i], 32);
      mbar_init(&info_free_s[i], kInfoUsers + (rank == 0 ? 1 : 0));
    }
    mbar_init(&done_s, 1);
    fence_mbar_init();
  }
  if (warp == 2) pair_tmem_alloc(&tmem_s, kProductTmem);
  tc_fence_before();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  pdl_wait();
  int tiles_here = 0;
  if (a.here) {  // (the rings are empty: their memory is used for the cut)
    int* start = reinterpret_cast<int*>(smem_raw);
    tiles_here = cut_list<kProductThreads>(
        a.list, start, start + kMaxExperts + 1, meet_s, a.t.head, [&](int i, int e, int p0, int rows) {
          if (i < kTilesHere) tiles_s[i] = make_int2(p0, (e << 16) | (rows - 1));
        });
    fence_proxy_async_smem();  // the rings' copies come behind these accesses
    __syncthreads();
  }

  bool ok = true;
  Ring<kInfoSlots> at_info;
  // The next unit for one of its users (a whole warp): false when there is none.
  auto next_unit = [&]() -> const ProductInfo<R>* {
    ok = ok && warp_wait(&info_full_s[at_info.slot], at_info.phase, limit);
    if (!ok) return nullptr;
    const ProductInfo<R>* q = &info_s[at_info.slot];
    return q->e < 0 ? nullptr : q;
  };
  auto leave_unit = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&info_free_s[at_info.slot]);
    at_info.advance();
  };

  // Boxes of weights that lie behind the last m are not copied: what is there meets no output.
  constexpr int kBoxM = kTranspose ? 64 : 128;
  auto weight_bytes = [&](int m) {  // of both CTAs, for the tile at m
    int boxes = 0;
#pragma unroll
    for (int i = 0; i < kPairRows / kBoxM; ++i) boxes += m + i * kBoxM < a.M ? 1 : 0;
    return boxes * kBoxM * 128;
  };

  if (warp == 0) {
    Ring<S> at;
    long long issued = 0;
    while (const ProductInfo<R>* q = next_unit()) {
      const int e = q->e, tiles = q->tiles;
      for (int c = 0; ok && c < tiles; ++c) {
        const int m = q->m0 + c * kPairRows;
        for (int ks = 0; ks < a.ksteps; ++ks) {
          ok = warp_wait(&free_s[at.slot], at.phase ^ 1u, limit);
          if (!ok) break;
          if (elect_one()) {
            if (rank == 0) mbar_expect(&full_s[at.slot], weight_bytes(m));
            const uint32_t bar = pair_first(&full_s[at.slot]);
#pragma unroll
            for (int i = 0; i < 128 / kBoxM; ++i) {
              const uint32_t to = wbase + at.slot * Sh::kW + i * (64 * 128);
              const int at_m = m + 128 * rank + i * kBoxM;
              if (at_m >= a.M) continue;
              if constexpr (kTranspose) pair_load_3d(to, &wmap, at_m, 64 * ks, e, bar);
              else pair_load_3d(to, &wmap, (kFp8 ? 128 : 64) * ks, at_m, e, bar);
            }
          }
          __syncwarp();
          ++issued;
          at.advance();
        }
      }
      leave_unit();
    }
    // Nothing may land in the shared memory of a CTA that has left: what was copied has been used,
    // or, where a wait gave up, had this long to land.
    for (long long i = issued > S ? issued - S : 0; i < issued; ++i)
      warp_wait(&free_s[i % S], static_cast<uint32_t>(i / S) & 1u, kWaitLimitNs);
  } else if (warp == 3) {
    // Rows written by threads are announced to the tensor cores.  (The thread that issues the
    // products would spend more clocks on these waits and the fence than the products take: 1340 us
    // for T = 8192, E = 64, 7168 -> 2048.)
    Ring<S> at;
    while (const ProductInfo<R>* q = next_unit()) {
      const int steps = q->tiles * a.ksteps;
      if (elect_one()) {
        Ring<S> s = at;
        for (int i = 0; ok && i < steps; ++i) {
          ok = thread_wait(&rows_s[s.slot], s.phase, limit);
          if (!ok) break;
          fence_proxy_async_smem();
          pair_arrive_first(&full_s[s.slot]);
          s.advance();
        }
      }
      ok = __all_sync(kFull, ok);
      at.skip(steps);
      leave_unit();
    }
  } else if (warp >= 12) {
    // a warp copies 32 rows of the CTA's half, four rows (8 lanes each) at a time, in every step or
    // in every kRowTurns-th
    constexpr int kTurns = kRowTurns<R>;
    Ring<S> at;
    const int w32 = kTurns == 1 ? 32 * (warp - 12) : 0, chunk = lane & 7, sub = lane >> 3;
    const int turn = (warp - 12) % kTurns;
    int now = 0;  // whose step it is
    const size_t row_bytes = static_cast<size_t>(a.K) * (kFp8 ? 1 : 2);
    // row 4 j + sub of the warp: two swizzles, for even and odd j
    const uint32_t place = xbase + (w32 + sub) * 128;
    const uint32_t even = place + 16 * (chunk ^ sub), odd = place + 16 * (chunk ^ (sub + 4));
    while (const ProductInfo<R>* q = next_unit()) {
      const int steps = q->tiles * a.ksteps, mine = q->half - w32;
      const unsigned char* from[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        from[j] = a.x + (4 * j < mine ? q->src[w32 + 4 * j + sub] * row_bytes : 0) + 16 * chunk;
      const int first = (turn - now + kTurns) % kTurns;
      at.skip(min(first, steps));
      int ks = first;
      for (int i = first; i < steps; i += kTurns) {
        while (ks >= a.ksteps) ks -= a.ksteps;
        ok = ok && thread_wait(&free_s[at.slot], at.phase ^ 1u, limit);
        if (ok) {  // (a lane whose wait gave up goes along until the unit ends)
          const uint32_t to = at.slot * Sh::kX;
          // columns past K are zeros
          const bool in = static_cast<size_t>(128 * ks + 16 * chunk) < row_bytes;
          const size_t off = in ? 128 * static_cast<size_t>(ks) : 0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (4 * j < mine) copy16(((j & 1) ? odd : even) + to + 512 * j, from[j] + off, in ? 16 : 0);
          copy_arrive(&rows_s[at.slot]);
        }
        at.skip(min(kTurns, steps - i));
        ks += kTurns;
      }
      now = (now + steps) % kTurns;
      ok = __all_sync(kFull, ok);
      leave_unit();
    }
    copy_wait_all();
  } else if (warp == 1) {
    // (of this call at most, whatever another one may have left there)
    const int tiles = a.here ? min(tiles_here, kTilesHere)
                             : min(max(__ldg(a.t.head + 1), 0), a.max_tiles);
    const int units = tiles * a.nchunk, step = gridDim.x >> 1;
    // What a unit takes is looked up over three rounds, so that no round waits for more than one
    // access: its tile, the tile's routes, their factors.
    struct Ahead {
      int e, p0, rows, m0, tiles;
      int r[R / 32], src[R / 32];
      float w[R / 32], x[R / 32];
    } now{}, next{}, later{};
    auto find = [&](int u, Ahead& q) {
      q.rows = 0;
      if (u >= units) return;
      const int t = a.nchunk == 1 ? u : u / a.nchunk, first = (u - t * a.nchunk) * a.chunk;
      int4 tile;
      if (a.here) {
        const int2 v = tiles_s[t];
        tile = make_int4(v.y >> 16, v.x, (v.y & 0xffff) + 1, 0);
      } else {
        tile = __ldg(a.t.tiles + t);
      }
      // (a table that another call overwrites must not lead out of this call's buffers)
      q.e = min(max(tile.x, 0), a.E - 1);
      q.p0 = min(max(tile.y, 0), a.P);
      q.rows = min(min(tile.z, R), a.P - q.p0);
      q.m0 = first * kPairRows;
      q.tiles = min(a.chunk, a.mtiles - first);
    };
    auto load_routes = [&](Ahead& q) {
#pragma unroll
      for (int j = 0; j < R / 32; ++j) {
        const int i = 32 * j + lane;
        q.r[j] = i < q.rows ? __ldg(a.list.sid + q.p0 + i) : -1;
      }
    };
    auto load_factors = [&](Ahead& q) {
#pragma unroll
      for (int j = 0; j < R / 32; ++j) {
        if (q.r[j] >= a.list.routes) q.r[j] = -1;
        const bool is = q.r[j] >= 0;
        if (!is) q.r[j] = -1;
        q.src[j] = is ? (a.per_route ? q.r[j] : q.r[j] / a.topk) : 0;
        q.w[j] = a.sw != nullptr && is ? __ldg(a.sw + q.p0 + 32 * j + lane) : 1.0f;
        q.x[j] = a.xs != nullptr && is ? __ldg(a.xs + q.src[j]) : 1.0f;
      }
    };
    const int u0 = blockIdx.x >> 1;
    find(u0, now);
    find(u0 + step, next);
    find(u0 + 2 * step, later);
    load_routes(now);
    load_routes(next);
    load_factors(now);
    for (int u = u0; ok && u < units; u += step) {
      load_routes(later);
      load_factors(next);
      Ahead last;
      find(u + 3 * step, last);
      int used = 0;
#pragma unroll
      for (int j = 0; j < R / 32; ++j) {
        const unsigned some = __ballot_sync(kFull, now.r[j] >= 0);
        if (some != 0u) used = 32 * j + 32 - __clz(some);
      }
      if (used > 0) {
        const int n = (used + 31) & ~31, half = n >> 1;
        ok = warp_wait(&info_free_s[at_info.slot], at_info.phase ^ 1u, limit);
        if (!ok) break;
        ProductInfo<R>* q = &info_s[at_info.slot];
        if (lane == 0) {
          q->e = now.e;
          q->n = n;
          q->m0 = now.m0;
          q->tiles = now.tiles;
          q->half = half;
        }
#pragma unroll
        for (int j = 0; j < R / 32; ++j) {
          const int i = 32 * j + lane, mine = i - rank * half;
          if (mine >= 0 && mine < half) q->src[mine] = now.src[j];
          q->route[i] = now.r[j];
          q->factor[i] = now.w[j] * now.x[j];
        }
        mbar_arrive(&info_full_s[at_info.slot]);
        at_info.advance();
      }
      now = next;
      next = later;
      later = last;
    }
    ok = ok && warp_wait(&info_free_s[at_info.slot], at_info.phase ^ 1u, limit);
    if (ok) {
      if (lane == 0) info_s[at_info.slot].e = -1;
      mbar_arrive(&info_full_s[at_info.slot]);
    }
  } else if (warp == 2 && rank == 0) {
    Ring<S> at;
    int buf = 0;
    uint32_t acc_phase = 0;
    bool any = false;
    while (const ProductInfo<R>* q = next_unit()) {
      const int n = q->n, tiles = q->tiles;
      any = true;
      if (elect_one()) {
        Ring<S> s = at;
        int to = buf;
        uint32_t to_phase = acc_phase;
        const uint32_t word = pair_word(a.type, kTranspose, false, n);
        for (int c = 0; ok && c < tiles; ++c) {
          ok = pair_wait(&acc_free_s[to], to_phase ^ 1u, limit);
          if (!ok) break;
          tc_fence_after();
          for (int ks = 0; ks < a.ksteps; ++ks) {
            ok = pair_wait(&full_s[s.slot], s.phase, limit);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dx = desc_rows128(xbase + s.slot * Sh::kX);
            const uint32_t wat = wbase + s.slot * Sh::kW;
            const uint64_t dw = kTranspose ? desc_lines128(wat, 64) : desc_rows128(wat);
#pragma unroll
            for (int g = 0; g < 4; ++g)
              // 32 bytes further along the rows; along the lines 16 of them
              pair_mma<kFp8>(tmem + to * R, dw + (kTranspose ? 16 * 128 / 16 : 2) * g, dx + 2 * g, word,
                             ks > 0 || g > 0);
            pair_commit(&free_s[s.slot]);
            s.advance();
          }
          if (ok) pair_commit(&acc_full_s[to]);
          if (++to == kAccs<R>) {
            to = 0;
            to_phase ^= 1u;
          }
        }
      }
      ok = __all_sync(kFull, ok);
      at.skip(tiles * a.ksteps);
      acc_phase ^= static_cast<uint32_t>((buf + tiles) / kAccs<R>) & 1u;
      buf = (buf + tiles) % kAccs<R>;
      leave_unit();
    }
    // nothing of the tensor core may be in flight when tensor memory is given back
    if (any) {
      if (elect_one()) pair_commit_first(&done_s);
      __syncwarp();
      warp_wait(&done_s, 0, kWaitLimitNs);
    }
  } else if (warp >= 4 && warp < 12) {
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t stage = smem_u32(stage_s[sizeof(Out) == 2 ? warp - 4 : 0]);
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    int buf = 0;
    uint32_t acc_phase = 0;
    while (const ProductInfo<R>* q = next_unit()) {
      const int n = q->n, e = q->e;
      const int count = q->tiles;
      // the outputs' scales, a tile ahead: of the lane's accumulator lanes among the warp's 32 m
      constexpr int kScales = sizeof(Out) == 4 ? 1 : 4;
      float ahead[kScales];
      auto load_scales = [&](int c) {
        const int m32 = q->m0 + c * kPairRows + 128 * rank + 32 * quarter;
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
          const int m = m32 + (sizeof(Out) == 4 ? lane : 8 * i + (lane >> 2));
          ahead[i] = a.ws != nullptr && c < count && m < a.M
                         ? __ldg(a.ws + static_cast<size_t>(e) * a.M + m) : 1.0f;
        }
      };
      load_scales(0);
      for (int c = 0; c < count; ++c) {
        const int m32 = q->m0 + c * kPairRows + 128 * rank + 32 * quarter;
        float scale[kScales];
#pragma unroll
        for (int i = 0; i < kScales; ++i) scale[i] = ahead[i];
        load_scales(c + 1);
        ok = warp_wait(&acc_full_s[buf], acc_phase, limit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + buf * R + lanes;
        auto load = [&](int j0, uint32_t(&to)[32]) {
          if constexpr (sizeof(Out) == 4) {
            tmem_load32(src + j0, to);
          } else {
            tmem_load_fragments(src + j0, to);
            tmem_load_fragments(src + j0 + (16u << 16), to + 16);
          }
        };
        // 32 rows of the list by 32 m, the next 32 rows on their way
        auto store = [&](int j0, uint32_t(&v)[32], uint32_t(&ahead)[32]) {
          tmem_wait(v);
          if (j0 + 64 < n) load(j0 + 64, ahead);
          if constexpr (sizeof(Out) == 4) {
            const int m = m32 + lane;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const int4 r = *reinterpret_cast<const int4*>(&q->route[j0 + j]);
              const float4 f = *reinterpret_cast<const float4*>(&q->factor[j0 + j]);
              const int to[4] = {r.x, r.y, r.z, r.w};
              const float by[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (to[i] >= 0 && m < a.M)
                  static_cast<float*>(a.out)[static_cast<size_t>(to[i]) * a.M + m] =
                      __uint_as_float(v[j + i]) * scale[0] * by[i];
            }
          } else {
            // through shared memory, so that four lanes store 64 bytes of a row side by side: 32
            // rows of 64 bytes, their 16-byte pieces spread over the banks
            __syncwarp();  // what was there has been read
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f =
                  *reinterpret_cast<const float2*>(&q->factor[j0 + 8 * k + 2 * (lane & 3)]);
              const F2 by = f2(f.x, f.y);
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t* p = v + 16 * (i >> 1) + 4 * k + 2 * (i & 1);
                // (one scale after the other: their product may leave fp32 where the result does not)
                const F2 y = f2(__uint_as_float(p[0]), __uint_as_float(p[1])) *
                             f2(scale[i], scale[i]) * by;
                const float2 r = f2_pair(y);
                w[i] = rounded2(r.x, r.y, a.out_type);
              }
              const int row = 8 * k + (lane & 7);
              store_transposed(stage + 64 * row + 16 * ((lane >> 3) ^ ((row >> 1) & 3)), w[0], w[1],
                               w[2], w[3]);
            }
            __syncwarp();
            const int m = m32 + 8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 8 * i + (lane >> 2), r = q->route[j0 + row];
              uint4 w;
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                           : "r"(stage + 64 * row + 16 * ((lane & 3) ^ ((row >> 1) & 3)))
                           : "memory");
              if (r >= 0 && m < a.M)  // M is a multiple of 8
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                          static_cast<size_t>(r) * a.M + m) = w;
            }
          }
        };
        // (of an odd number of 32 rows the two warps of a quarter have the one more in turn)
        const int begin = 32 * (half ^ (buf & 1));
        uint32_t one[32], two[32];
        if (begin < n && m32 < a.M) load(begin, one);
        if (m32 < a.M) {
          for (int j0 = begin; j0 < n; j0 += 128) {
            store(j0, one, two);
            if (j0 + 64 < n) store(j0 + 64, two, one);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair_arrive_first(&acc_free_s[buf]);
        if (++buf == kAccs<R>) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
      leave_unit();
    }
  }
  if (!ok && lane == 0) atomicOr(a.t.head, MOE_RS_DEVICE_WAIT_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  if (warp == 2) pair_tmem_free(tmem, kProductTmem);
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

CUtensorMapDataType map_type(int type) {
  return type == MOE_RS_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
         : type == MOE_RS_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
         : type == MOE_RS_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                               : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

}  // namespace

bool encode_few(CUtensorMap* map, const void* p, size_t row_bytes, size_t rows, size_t E) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  // words of 4 bytes: 1024 bytes are the most that a box has of a row
  const cuuint64_t dims[3] = {row_bytes / 4, rows, E};
  const cuuint64_t strides[2] = {row_bytes, row_bytes * rows};
  const cuuint32_t box[3] = {256, 32, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_weights3(CUtensorMap* map, const void* p, int type, int size, size_t cols, size_t rows,
                     size_t E, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cols, rows, E};
  const cuuint64_t strides[2] = {cols * size, cols * size * rows};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(box_rows),
                             1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, map_type(type), 3, const_cast<void*>(p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <bool kFp8, bool kTranspose, int R, class Out>
cudaError_t launch_product(const CUtensorMap& w, const ProductArgs& a, int pairs, cudaStream_t st) {
  auto* k = mrs_product_kernel<kFp8, kTranspose, R, Out>;
  constexpr size_t smem = ProductShape<R>::kSmem;
  static SmemGrant granted;
  const cudaError_t err = grant_smem(reinterpret_cast<const void*>(k), smem, granted);
  if (err != cudaSuccess) return err;
  return launch_pairs(k, pairs, kProductThreads, smem, st, w, a);
}

template <int R, class Out>
cudaError_t launch_product(bool fp8, bool transpose, const CUtensorMap& w, const ProductArgs& a,
                           int pairs, cudaStream_t st) {
  return transpose ? launch_product<false, true, R, Out>(w, a, pairs, st)
         : fp8     ? launch_product<true, false, R, Out>(w, a, pairs, st)
                   : launch_product<false, false, R, Out>(w, a, pairs, st);
}

size_t most_tiles(int T, int E, int topk, int block_m, int rows) {
  const size_t P = moe_sort_max_padded(T, E, topk, block_m), n = static_cast<size_t>(T) * topk;
  return P / rows + (n < static_cast<size_t>(E) ? n : E);
}

// Routes up to which a product goes by the blocks of the list.  us with it and in tiles, each call by
// itself, weights from HBM, 3584 -> 768:
//                       8 bits                                  bf16
//   routes   E = 1    4        8        64       896      1        4        8        64       896
//   16       14 18    12 18    15 18    21 23    21 23    14 25    14 25    18 26    27 31    27 33
//   64       14 21    16 18    20 18    37 39    45 49    16 27    18 25    23 27    52 57    74 80
//   128      22 23    23 18    23 18    45 47    74 75    25 27    27 25    27 27    70 79    122 125
//   256      29 24    29 20    31 18    49 49    127 117  34 31    35 29    35 27    76 80    197 201
//   512      49 24    49 23    49 23    68 49    213 185  57 31    59 29    59 29    81 80    332 350
// A unit has eight routes of a block at most, so that 128 routes of a few experts read the same weights
// again, from L2; at the limit that costs 5 us at most (8 bits, 4 or 8 experts).
constexpr int kFewRoutes = 128;

// The product (transpose: the rows' gradient, whose contraction runs over W's rows).
int product(const void* x, int type, const float* x_scales, int per_route, const void* w,
            const float* w_scales, int T, int E, int topk, int cols, int outs, int block_m,
            const int32_t* sid, const float* sw, const int32_t* eid, const int32_t* npp, void* out,
            int out_type, void* workspace, size_t workspace_bytes, bool transpose,
            cudaStream_t stream) {
  const bool fp8 = type == MOE_RS_FP8;
  if (T < 0) return MOE_RS_ERR_BAD_TOKENS;
  if (E < 1 || E > kMaxExperts) return MOE_RS_ERR_BAD_EXPERTS;
  if (topk < 1 || topk > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  if (block_m < 1 || block_m > 1024 || (block_m & (block_m - 1)) != 0)
    return MOE_RS_ERR_BAD_BLOCK_M;
  if (type != MOE_RS_BF16 && type != MOE_RS_FP16 && (!fp8 || transpose)) return MOE_RS_ERR_BAD_DTYPE;
  if (out_type != MOE_RS_BF16 && out_type != MOE_RS_FP16 && out_type != MOE_RS_FP32)
    return MOE_RS_ERR_BAD_DTYPE;
  if (cols < 8 || cols > MOE_RS_PRODUCT_MAX_COLS || cols % (fp8 ? 16 : 8) != 0 || outs < 8 ||
      outs > MOE_RS_PRODUCT_MAX_COLS || outs % 8 != 0)
    return MOE_RS_ERR_BAD_COLS;
  if (static_cast<int64_t>(T) * topk > INT32_MAX ||
      static_cast<int64_t>(moe_sort_max_padded(T, E, topk, block_m)) > INT32_MAX)
    return MOE_RS_ERR_OVERFLOW;
  const size_t need = moe_experts_product_workspace_bytes(T, E, topk, block_m);
  if (!workspace || workspace_bytes < need) return MOE_RS_ERR_WORKSPACE;
  if (T == 0) return MOE_RS_OK;
  if (!x || !w || !sid || !eid || !npp || !out || (fp8 && (!x_scales || !w_scales)))
    return MOE_RS_ERR_NULL_POINTER;
  if (!fp8 && (x_scales || w_scales)) return MOE_RS_ERR_BAD_DTYPE;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(sid, 4) || !aligned(sw, 4) || !aligned(eid, 4) || !aligned(npp, 4) ||
      !aligned(out, 16) || !aligned(workspace, 16))
    return MOE_RS_ERR_MISALIGNED;
  const size_t routes = static_cast<size_t>(T) * topk, size = fp8 ? 1 : 2;
  const size_t xrows = per_route ? routes : static_cast<size_t>(T);
  const size_t wrows = static_cast<size_t>(E) * outs;
  const size_t P = moe_sort_max_padded(T, E, topk, block_m);
  const int M = transpose ? cols : outs, K = transpose ? outs : cols;
  const Span outs_s[] = {span(out, routes * M * (out_type == MOE_RS_FP32 ? 4 : 2)),
                         span(workspace, workspace_bytes)};
  const Span ins[] = {span(x, xrows * K * size),
                      span(x_scales, x_scales ? 4 * xrows : 0),
                      span(w, wrows * cols * size),
                      span(w_scales, w_scales ? 4 * wrows : 0),
                      span(sid, 4 * P),
                      span(sw, sw ? 4 * P : 0),
                      span(eid, 4 * (P / block_m)),
                      span(npp, 4)};
  if (any_alias(outs_s, 2, ins, 8)) return MOE_RS_ERR_ALIAS;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  if (!transpose && routes <= kFewRoutes) {
    FewArgs f{};
    f.x = static_cast<const unsigned char*>(x);
    f.sid = sid;
    f.eid = eid;
    f.npp = npp;
    f.sw = sw;
    f.xs = x_scales;
    f.ws = w_scales;
    f.status = static_cast<int32_t*>(workspace);
    f.out = out;
    f.wait_limit_ns = product_wait_limit();
    f.routes = static_cast<int>(routes);
    f.topk = topk;
    f.per_route = per_route != 0;
    f.E = E;
    f.N = outs;
    f.K = cols;
    f.B = block_m;
    f.blocks = static_cast<int>(P / block_m);
    f.out_type = out_type;
    CUtensorMap map;
    if (!encode_few(&map, w, cols * size, outs, E))
      return MOE_RS_ERR_LAUNCH;
    return launch_status(launch_product_few(map, f, type, sms, stream));
  }
  const size_t hit = routes < static_cast<size_t>(E) ? routes : E;
  // us in tiles of 64 rows and of 256, of 32, 48, 64 and 96 rows an expert: E = 64, 3584 -> 768 in bf16 83
  // 85, 84 87, 87 89, 104 92; in 8 bits 50 53, 51 53, 53 55, 61 57; E = 16, 7168 -> 2048 in bf16 98 103,
  // 99 103, 115 105, 130 107; in 8 bits 61 64, 61 64, 68 66, 74 66
  const int R = routes <= 48 * hit ? 64 : 256;
  ListArgs list{};
  list.eid = eid;
  list.sid = sid;
  list.npp = npp;
  list.E = E;
  list.B = block_m;
  while ((1 << list.log2B) < block_m) ++list.log2B;
  list.max_rows = static_cast<int>(P);
  list.routes = static_cast<int>(routes);
  list.rows = R;
  list.log2R = R == 64 ? 6 : 8;
  list.by_used = R > 64;
  const size_t tiles = most_tiles(T, E, topk, block_m, R);
  ProductArgs a{};
  a.list = list;
  a.t = product_table(workspace);
  // (a cut takes a CTA 3 us, the table kernel 8)
  a.here = tiles <= kTilesHere && P / block_m <= kBlocksHere;
  a.sw = sw;
  a.xs = x_scales;
  a.ws = w_scales;
  a.x = static_cast<const unsigned char*>(x);
  a.out = out;
  a.wait_limit_ns = product_wait_limit();
  a.topk = topk;
  a.per_route = per_route != 0;
  a.max_tiles = static_cast<int>(tiles);
  a.E = E;
  a.M = M;
  a.K = K;
  a.P = static_cast<int>(P);
  a.ksteps = (K * static_cast<int>(size) + 127) / 128;
  // (512 m on the same rows take in a quarter less for the same products, but leave no second
  // accumulator for the next tile and half as many units.  Both in turn, us with 256 and with 512: T =
  // 16384, E = 64, topk = 8, 7168 -> 2048 2400 2450, its rows' gradient 2350 2750; T = 32768, 1024 -> 2048
  // 690 830; in 8 bits T = 8192, 7168 -> 2048 640 680; only T = 8192, 2048 -> 7168 and its like gain, 1240
  // 1210.)
  const int pairs = sms / 2;
  a.mtiles = (M + kPairRows - 1) / kPairRows;
  a.type = type == MOE_RS_BF16 ? 1 : 0;
  a.out_type = out_type;
  // A unit is as many output tiles of one row tile as leave 32 rounds of units (us with 4, 16, 32, 64
  // rounds and single tiles: 8192 skewed tokens, 384 -> 3584 in 8 bits 371 372 376 395 423; T = 8192, E =
  // 64, 7168 -> 2048 in bf16 1350 1250 1200 1205 1205), but no more than 32768 steps (some 20 ms): the list
  // waits for a unit as a whole, and 65536 x 65536 outputs and columns have 262144 of them, more than half
  // of the default limit.
  const size_t each = (routes / R + hit) * a.mtiles / (32 * static_cast<size_t>(pairs));
  const size_t most = std::min(static_cast<size_t>(a.mtiles), static_cast<size_t>(32768 / a.ksteps));
  a.chunk = static_cast<int>(each < 1 ? 1 : (each > most ? most : each));
  a.nchunk = (a.mtiles + a.chunk - 1) / a.chunk;
  a.chunk = (a.mtiles + a.nchunk - 1) / a.nchunk;
  a.nchunk = (a.mtiles + a.chunk - 1) / a.chunk;
  if (tiles * a.nchunk > INT32_MAX / 2) return MOE_RS_ERR_OVERFLOW;
  CUtensorMap wmap;
  if (!encode_weights3(&wmap, w, type, static_cast<int>(size), cols, outs, E, transpose ? 64 : 128))
    return MOE_RS_ERR_LAUNCH;
  if (!a.here) {
    const cudaError_t err = launch_pdl(mrs_product_table_kernel, dim3(1), dim3(kTableThreads), 0,
                                       stream, list, a.t, a.max_tiles);
    if (err != cudaSuccess) return launch_status(err);
  }
  const size_t units = tiles * a.nchunk;
  const int grid = units < static_cast<size_t>(pairs) ? static_cast<int>(units) : pairs;
  auto go = [&](auto o) {
    using Out = decltype(o);
    return R == 64 ? launch_product<64, Out>(fp8, transpose, wmap, a, grid, stream)
                   : launch_product<256, Out>(fp8, transpose, wmap, a, grid, stream);
  };
  return launch_status(out_type == MOE_RS_FP32 ? go(float{}) : go(uint16_t{}));
}

}  // namespace
}  // namespace mrs

using namespace mrs;

extern "C" {

size_t moe_experts_product_workspace_bytes(int T, int E, int topk, int block_m) {
  if (T < 0 || E < 1 || E > kMaxExperts || topk < 1 || topk > kMaxTopk || block_m < 1 ||
      block_m > 1024 || (block_m & (block_m - 1)) != 0)
    return 0;
  if (static_cast<int64_t>(T) * topk > INT32_MAX ||
      static_cast<int64_t>(moe_sort_max_padded(T, E, topk, block_m)) > INT32_MAX)
    return 0;
  return product_table_bytes(most_tiles(T, E, topk, block_m, kTileRowsLeast));
}

int moe_experts_product(const void* x, int x_dtype, const float* x_scales, int x_per_route,
                        const void* w, const float* w_scales, int T, int E, int topk, int cols,
                        int outs, int block_m, const int32_t* sorted_token_ids,
                        const float* sorted_weights, const int32_t* expert_ids,
                        const int32_t* num_tokens_post_pad, void* out, int out_dtype,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return product(x, x_dtype, x_scales, x_per_route, w, w_scales, T, E, topk, cols, outs, block_m,
                 sorted_token_ids, sorted_weights, expert_ids, num_tokens_post_pad, out, out_dtype,
                 workspace, workspace_bytes, false, stream);
}

int moe_experts_grad_rows(const void* grad, int dtype, int g_per_route, const void* w, int T, int E,
                          int topk, int cols, int outs, int block_m,
                          const int32_t* sorted_token_ids, const int32_t* expert_ids,
                          const int32_t* num_tokens_post_pad, void* grad_rows, int out_dtype,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return product(grad, dtype, nullptr, g_per_route, w, nullptr, T, E, topk, cols, outs, block_m,
                 sorted_token_ids, nullptr, expert_ids, num_tokens_post_pad, grad_rows, out_dtype,
                 workspace, workspace_bytes, true, stream);
}

}  // extern "C"
