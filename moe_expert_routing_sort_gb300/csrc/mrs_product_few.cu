// mrs_product_few.cu -- the experts' products of a few routes (single tokens): every expert's weights
// are read for a row or two, and nothing else takes time.
//
//   out[r, n] = w_r * sx_row * sw_en * sum over k of X[row, k] W[e, n, k]
// A CTA per SM takes units round robin, a unit being 32 outputs by up to eight routes of one block of
// the sorted list.  The list is read as it is, there is nothing to look up but a block's owner and its
// routes.  One warp keeps a ring of six steps (32 outputs by 1024 bytes, one tensor copy) full, over
// the ends of units; eight warps take 16 outputs by 256 bytes of a step each.  (A copy takes its warp
// 200 clocks to issue, a step each of the others 300 at least, whatever there is to do: steps of 128
// bytes took 29 us for one token in 8 bits, E = 896, topk = 16, 3584 -> 768, 512 bytes in four copies
// 23.)
// A lane reads 16 bytes of two rows of weights from shared memory and of one row of X, and these
// registers are the operands of a warp's matrix product as they are: the contraction's order does not
// matter as long as both operands have the same (lane t of four holds bytes 16 t .. 16 t + 15, which
// the product takes for other columns, the same ones of both).  (Fused multiply-adds have to convert
// every weight to fp32 first: 467 us for 512 routes in 8 bits, 3584 -> 768, E = 896, and 232 so.)
// The four warps' sums of an output meet in shared memory and are added in a fixed order.
//
// Bound by the weights' bytes and, before them, by an access to the list: one token in 8 bits, E = 896,
// topk = 16, 3584 -> 768, 44 MB in 13.9 us (in a graph 13.8, and 10.9 where the weights are in L2;
// 6.5 at the rate of a copy), in bf16 17.9 us in a graph, of 13.0.  In 16 bits sums are low by 1.4e-10 of
// themselves for every term (1.3e-7 over 1024, 9.6e-6 over 65536), in 8 bits by 1.3e-7 over 65536.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mrs_product.cuh"

namespace mrs {

constexpr int kFewThreads = 288;
constexpr int kFewWarps = 8;   // that compute
constexpr int kFewOuts = 32;
constexpr int kFewRows = 8;
constexpr int kFewSlots = 6;
constexpr int kFewWide = 1024;  // bytes of an output's row in a step
constexpr int kFewStep = kFewOuts * kFewWide;
constexpr int kFewPart = kFewWide / (kFewWarps / 2);  // bytes of a warp
constexpr int kFewInfo = 8;
constexpr size_t kFewSmem = static_cast<size_t>(kFewSlots) * kFewStep + 1024;

struct FewInfo {
  int e, n0, rows;      // e < 0: no more units
  int route[kFewRows];  // of the first `rows`
  int place[kFewRows];  // in the list
};

// 16 x 8 sums of 32 bytes of each row: a0, a2 of row g, a1, a3 of row g + 8, b of column g.
template <int kType>
__device__ __forceinline__ void few_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kType == MOE_RS_FP8)
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (kType == MOE_RS_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes, loaded here and not where they are used.
__device__ __forceinline__ uint4 load_now(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void store_rounded(void* out, size_t at, float v, int type) {
  if (type == MOE_RS_FP32) static_cast<float*>(out)[at] = v;
  else if (type == MOE_RS_BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[at] = __float2half_rn(v);
}

template <int kType>
__global__ void __launch_bounds__(kFewThreads, 1)
    mrs_product_few_kernel(const __grid_constant__ CUtensorMap wmap, const FewArgs a) {
  constexpr int S = kFewSlots;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned long long full_s[S], free_s[S], info_full_s[kFewInfo], info_free_s[kFewInfo],
      join_s;
  __shared__ FewInfo info_s[kFewInfo];
  __shared__ float sums[2][kFewWarps / 2][kFewRows][kFewOuts];  // of two units in turn
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const unsigned long long limit = a.wait_limit_ns;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_s[s], 1);
      mbar_init(&free_s[s], kFewWarps);
    }
    for (int i = 0; i < kFewInfo; ++i) {
      mbar_init(&info_full_s[i], 1);
      mbar_init(&info_free_s[i], kFewWarps);
    }
    mbar_init(&join_s, kFewWarps);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  bool ok = true;
  Ring<kFewInfo> at_info;
  Ring<S> at;
  if (warp == kFewWarps) {
    long long issued = 0;
    const int units = a.blocks * a.nchunk, step = gridDim.x;
    auto look = [&](int u, int& e, int& before, int& s) {
      e = -1;
      before = 0;
      s = -1;
      if (u >= units) return;
      const int b = u / a.nchunk;
      e = __ldg(a.eid + b);
      before = b > 0 ? __ldg(a.eid + b - 1) : 0;
      if (lane < a.B) s = __ldg(a.sid + b * a.B + lane);
    };
    int e, before, s;
    look(blockIdx.x, e, before, s);
    const int length = min(__ldg(a.npp), a.blocks * a.B);
    for (int u = blockIdx.x; ok && u < units; u += step) {
      int next_e, next_before, next_s;
      look(u + step, next_e, next_before, next_s);
      const int b = u / a.nchunk, p0 = b * a.B, n0 = (u - b * a.nchunk) * kFewOuts;
      const bool in = p0 < length, fine = e >= 0 && e < a.E;
      // (an owner out of order misleads the kernels of more routes)
      if (in && (!fine || before > e) && lane == 0) atomicOr(a.status, MOE_RS_DEVICE_BAD_EXPERT_ID);
      for (int w = 0; ok && in && fine && w < a.B; w += 32) {
        if (w > 0) s = w + lane < a.B ? __ldg(a.sid + p0 + w + lane) : -1;
        const bool is = s >= 0 && s < a.routes;
        const unsigned routes = __ballot_sync(kFull, is);
        if (routes == 0u) break;  // routes come first
        const int mine = __popc(routes & lanemask_lt(lane)), count = __popc(routes);
        for (int first = 0; ok && first < count; first += kFewRows) {
          ok = warp_wait(&info_free_s[at_info.slot], at_info.phase ^ 1u, limit);
          if (!ok) break;
          FewInfo* q = &info_s[at_info.slot];
          if (is && mine >= first && mine < first + kFewRows) {
            q->route[mine - first] = s;
            q->place[mine - first] = p0 + w + lane;
          }
          if (lane == 0) {
            q->e = e;
            q->n0 = n0;
            q->rows = min(count - first, kFewRows);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&info_full_s[at_info.slot]);
          at_info.advance();
          int part = 0;
          if (elect_one()) {
            Ring<S> to = at;
            for (; part < a.ksteps; ++part) {
              ok = thread_wait(&free_s[to.slot], to.phase ^ 1u, limit);
              if (!ok) break;
              fence_proxy_async_smem();  // the slot's reads are behind the wait, its copy ahead
              mbar_expect(&full_s[to.slot], kFewStep);
              tma_load_3d(base + to.slot * kFewStep, &wmap, kFewWide / 4 * part, n0, e,
                          &full_s[to.slot]);
              to.advance();
            }
          }
          issued += __reduce_max_sync(kFull, part);
          ok = __all_sync(kFull, ok);
          at.skip(a.ksteps);
        }
      }
      e = next_e;
      before = next_before;
      s = next_s;
    }
    ok = ok && warp_wait(&info_free_s[at_info.slot], at_info.phase ^ 1u, limit);
    if (ok && lane == 0) {
      info_s[at_info.slot].e = -1;
      mbar_arrive(&info_full_s[at_info.slot]);
    }
    // copies still on their way must land before the CTA leaves
    for (long long i = issued > S ? issued - S : 0; i < issued; ++i)
      thread_wait(&full_s[i % S], static_cast<uint32_t>(i / S) & 1u, kWaitLimitNs);
    __syncwarp();
  } else {
    const int o = warp & 1, part = warp >> 1;
    const int g = lane >> 2, t = lane & 3;
    const size_t row_bytes = static_cast<size_t>(a.K) * (kType == MOE_RS_FP8 ? 1 : 2);
    // rows 16 o + g (and 8 more), 16 bytes of every 64 of the warp's part
    const uint32_t from = base + (16 * o + g) * kFewWide + kFewPart * part + 16 * t;
    uint32_t unit = 0;  // units so far
    while (true) {
      ok = ok && warp_wait(&info_full_s[at_info.slot], at_info.phase, limit);
      if (!ok) break;
      const FewInfo* q = &info_s[at_info.slot];
      const int e = q->e, n = q->n0 + lane, rows = q->rows;
      if (e < 0) break;
      auto row_of = [&](int i) { return a.per_route ? i : i / a.topk; };
      // what this thread will store: output `lane` of the unit's route `warp`
      const bool stores = warp < rows && n < a.N;
      const int route = q->route[warp < rows ? warp : 0];
      float by = 1.0f, scale = 1.0f;
      if (stores) {
        if (a.sw != nullptr) by = __ldg(a.sw + q->place[warp]);
        if (a.xs != nullptr) {
          by *= __ldg(a.xs + row_of(route));
          scale = __ldg(a.ws + static_cast<size_t>(e) * a.N + n);
        }
      }
      const bool some = g < rows;  // a column of X that there is
      constexpr int kLoads = kFewPart / 64;  // of a lane and row in a step
      const size_t mine = kFewPart * part + 16 * t;  // of a step's bytes
      const unsigned char* x = a.x + (some ? row_of(q->route[g]) * row_bytes : 0) + mine;
      auto load_x = [&](int ks, uint4(&to)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const size_t k = kFewWide * static_cast<size_t>(ks) + 64 * i;
          to[i] = some && k + mine < row_bytes ? load_now(x + k) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      // X is loaded two steps ahead: another token's row comes from L2
      uint4 even[kLoads], odd[kLoads];
      load_x(0, even);
      load_x(1, odd);
      float c[2][4] = {};
      auto take = [&](int ks, uint4(&v)[kLoads]) {
        ok = ok && thread_wait(&full_s[at.slot], at.phase, limit);
        __syncwarp();
        const uint32_t w = from + at.slot * kFewStep;
        uint32_t p[kLoads][2][4];  // row g, row g + 8
#pragma unroll
        for (int i = 0; i < 2 * kLoads; ++i) {
          uint32_t(&d)[4] = p[i >> 1][i & 1];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                       : "r"(w + 64 * (i >> 1) + 8 * kFewWide * (i & 1))
                       : "memory");
        }
        // The slot is let go once its bytes are in registers: which lane arrives hangs on a word of each
        // load, and the copying thread has a proxy fence between its wait and the next copy.  (The
        // arrival by itself held up neither: tensor copies are of another proxy, and in e4m3 up to a
        // hundred of 200 thousand results had some of the next step's weights.  A proxy fence by every
        // lane mends it too, and takes one token from 13.8 to 15.1 us.)
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) word ^= p[i][0][0] ^ p[i][1][0];
        const int who = __any_sync(kFull, word == 0x9e3779b9u) ? 1 : 0;
        __syncwarp();
        if (lane == who) mbar_arrive(&free_s[at.slot]);
        at.advance();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          few_mma<kType>(c[0], p[i][0][0], p[i][1][0], p[i][0][1], p[i][1][1], v[i].x, v[i].y);
          few_mma<kType>(c[1], p[i][0][2], p[i][1][2], p[i][0][3], p[i][1][3], v[i].z, v[i].w);
        }
        load_x(ks + 2, v);
      };
      for (int ks = 0; ks < a.ksteps; ks += 2) {
        take(ks, even);
        if (ks + 1 < a.ksteps) take(ks + 1, odd);
      }
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      // outputs g and g + 8 of rows 2 t and 2 t + 1
      float(&to)[kFewRows][kFewOuts] = sums[unit & 1][warp >> 1];
      to[2 * t][16 * o + g] = c[0][0] + c[1][0];
      to[2 * t + 1][16 * o + g] = c[0][1] + c[1][1];
      to[2 * t][16 * o + g + 8] = c[0][2] + c[1][2];
      to[2 * t + 1][16 * o + g + 8] = c[0][3] + c[1][3];
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&info_free_s[at_info.slot]);
        mbar_arrive(&join_s);
      }
      at_info.advance();
      ok = warp_wait(&join_s, unit & 1u, limit);
      if (!ok) break;
      if (stores) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kFewWarps / 2; ++i) sum += sums[unit & 1][i][warp][lane];
        store_rounded(a.out, static_cast<size_t>(route) * a.N + n, sum * scale * by, a.out_type);
      }
      ++unit;
    }
  }
  if (!ok && lane == 0) atomicOr(a.status, MOE_RS_DEVICE_WAIT_TIMEOUT);
}

cudaError_t launch_product_few(const CUtensorMap& wmap, FewArgs a, int type, int sms,
                               cudaStream_t st) {
  a.nchunk = (a.N + kFewOuts - 1) / kFewOuts;
  const size_t row_bytes = static_cast<size_t>(a.K) * (type == MOE_RS_FP8 ? 1 : 2);
  a.ksteps = static_cast<int>((row_bytes + kFewWide - 1) / kFewWide);
  const int64_t units = static_cast<int64_t>(a.blocks) * a.nchunk;
  const dim3 grid(static_cast<unsigned>(units < sms ? units : sms)), block(kFewThreads);
  auto go = [&](auto* k, SmemGrant& granted) {
    const cudaError_t err = grant_smem(reinterpret_cast<const void*>(k), kFewSmem, granted);
    return err != cudaSuccess ? err : launch_pdl(k, grid, block, kFewSmem, st, wmap, a);
  };
  static SmemGrant granted[3];
  return type == MOE_RS_FP8    ? go(mrs_product_few_kernel<MOE_RS_FP8>, granted[0])
         : type == MOE_RS_BF16 ? go(mrs_product_few_kernel<MOE_RS_BF16>, granted[1])
                               : go(mrs_product_few_kernel<MOE_RS_FP16>, granted[2]);
}

}  // namespace mrs
