// Block-sparse decode (fdms_decode_attn_sparse): a cheap score selects the
// store blocks that a step attends to.
//
// Bounds: for every full 64-slot block the least and the largest stored K value
// of each channel, in bf16 (exact: bf16 rows as they are, E4M3 codes as the
// values they stand for, the block's scale being applied to the sum). A full
// block never changes, so its bounds are found once, by the first sparse decode
// that finds the block full and has to choose.
// Score: u = max over the query heads g of the kv head of
//   sum_c max(q_gc lo_c, q_gc hi_c) >= q_g . k for every key k of the block.
// A product of two bf16 values has 16 significant bits; the sums are kept to
// about 46, exact for all but extreme spreads of magnitude, so the order of the
// sum does not decide which of two near blocks is taken.
// The selection is a block table of its own, over which the decode kernels run
// (fdms_launch_decode_selected).
#include <cuda_bf16.h>

#include <algorithm>

#include "fdms_internal.cuh"

using namespace fdms;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtaBlocks = 4 * kWarps;   // blocks a CTA scores
constexpr int kStaged = 3600;            // scores of a head that shared memory takes (43 KB)

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A sum in two fp32 numbers: the sum and what its roundings lost, which an error-
// free addition gives (Knuth's). About 2^-46 of the magnitudes is lost in all, for
// seven operations a term; fp64 additions and conversions, a tenth as fast here,
// bounded the kernel (4.4k cycles of it for 252 blocks a head).
struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  __device__ __forceinline__ double value() const {   // (no error part beside inf, NaN)
    return fabsf(hi) < INFINITY ? (double)hi + (double)lo : (double)hi;
  }
};

// score in the selection's order: NaN as +infinity
__device__ __forceinline__ double ranked(double u) { return u != u ? (double)INFINITY : u; }

// a whole number in the order of the score (-0 and 0 equal)
__device__ __forceinline__ long long score_key(double u) {
  const long long b = __double_as_longlong(u + 0.0);
  return b ^ (long long)((unsigned long long)(b >> 63) >> 1);
}

// Bounds of one full block, by one warp: lane l holds the channels of its
// 2 * D / 32 16-bit values.
template <int D, bool FP8>
__device__ void block_bounds(const uint8_t* rows, uint16_t* out, int lane) {
  constexpr int C = D / 32;             // channels per lane, neighbours
  constexpr int RB = FP8 ? D : 2 * D;
  __nv_bfloat16 lo[C], hi[C];
  for (int r = 0; r < kBlockSlots; ++r) {
    __nv_bfloat16 x[C];
    if constexpr (FP8) {
      const uint8_t* p = rows + r * RB + swz_byte(RB, false, r, lane * C);
      for (int i = 0; i < C; i += 2) {
        const float2 f = e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(p + i));
        x[i] = __float2bfloat16_rn(f.x);      // exact
        x[i + 1] = __float2bfloat16_rn(f.y);
      }
    } else {
      const uint8_t* p = rows + r * RB + swz_byte(RB, false, r, lane * C * 2);
      for (int i = 0; i < C; ++i) x[i] = reinterpret_cast<const __nv_bfloat16*>(p)[i];
    }
    for (int i = 0; i < C; ++i) {
      lo[i] = r ? __hmin_nan(lo[i], x[i]) : x[i];
      hi[i] = r ? __hmax_nan(hi[i], x[i]) : x[i];
    }
  }
  for (int i = 0; i < C; ++i) {
    out[lane * C + i] = __bfloat16_as_ushort(lo[i]);
    out[D + lane * C + i] = __bfloat16_as_ushort(hi[i]);
  }
}

// CTAs (x, head): bounds and scores of the head's blocks 32 x .. 32 x + 31; the
// last CTA of a head to finish ranks them and writes the selection.
// Bound by its chain of dependent steps: lengths, block table, bounds, the count of
// CTAs that are done, scores, ranks. 13.5 us for 64 heads of 252 blocks of 128 channels
// (8.3 MB of bounds), 7 us for 8 heads of 35; the decode after it takes 16 and 7.
// The ranks compare each block with each. Whole calls that choose 32 blocks of 128
// channels (and dense decodes), bf16, one sequence of 8 heads: 252 blocks 15 us (19),
// 1024 61 (63), 2048 160 (120), 3500 430 (200); eight sequences: 25 (80), 1024 89 (300),
// 2048 268 (590). In a cache with room for more than kStaged blocks a head the scores
// are read from L2 in every comparison, however few there are: one sequence, 252 blocks
// 40 us, 1024 440, 3700 5.5 ms. CTAs without blocks only look: room for 114,688 tokens
// more costs 2.7 us.
// The first call on a prompt finds the bounds of all its full blocks, 64 dependent rows
// a warp: 96 to 153 us in all at 64 heads of 252 blocks, 640 to 790 at 2048.
// Eight lanes share a block, so that a sum over its D channels takes three
// shuffles for the four blocks of a warp at once.
template <int D, bool FP8, int G>
__global__ void __launch_bounds__(kThreads)
k_sparse_select(CacheView c, SparseWork sp, int layer, int num_select, int view_blocks,
                int staged, const uint16_t* __restrict__ q, int32_t* __restrict__ blocks) {
  constexpr int C = D / 8;                 // channels of a lane
  __shared__ __align__(16) uint16_t s_q[G * D];
  __shared__ int s_cnt[kWarps];
  __shared__ int s_last;
  // with `staged`: the head's scores as whole numbers in their order (fp64
  // comparisons are slow here), and rounded to fp32 (in their order, but for ties)
  extern __shared__ __align__(16) long long s_score[];
  float* s_near = reinterpret_cast<float*>(s_score + (c.max_blocks + 1) / 2 * 2);
  pdl_wait();
  pdl_launch_dependents();
  const int hs = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long hi = (long long)layer * c.Bmax * c.Hkv + hs;
  const int len = c.store_len[hi], full = len / kBlockSlots, part = len % kBlockSlots;
  const int32_t* bt = c.block_table + hi * c.max_blocks;
  const float* bs = c.bt_scale + hi * c.max_blocks * 2;
  int32_t* st = sp.sel_table + (long long)hs * view_blocks;
  float* ss = sp.sel_scale + (long long)hs * view_blocks * 2;
  double* score = sp.score + (long long)hs * c.max_blocks;
  const int nsel = min(full, num_select);
  const bool choose = full > num_select && num_select > 0;
  // CTAs that take part: those with blocks, or the first alone
  const int parts = choose ? (full + kCtaBlocks - 1) / kCtaBlocks : 1;
  if ((int)blockIdx.x >= parts) return;
  if (choose) {
    const int j0 = blockIdx.x * kCtaBlocks, j1 = min(full, j0 + kCtaBlocks);
    const int have = sp.bounds_done[hi];
    if (j1 > have) {
      for (int j = max(j0, have) + warp; j < j1; j += kWarps)
        block_bounds<D, FP8>(block_k(c, bt[j]), sp.bounds + (long long)bt[j] * 2 * D, lane);
    }
    const uint16_t* qh = q + ((long long)(hs / c.Hkv) * c.Hq + (long long)(hs % c.Hkv) * G) * D;
    for (int i = tid; i < G * D / 8; i += kThreads)
      reinterpret_cast<uint4*>(s_q)[i] = reinterpret_cast<const uint4*>(qh)[i];
    __syncthreads();
    const int j = j0 + warp * 4 + lane / 8, sub = lane % 8;
    uint32_t lo[C / 2], up[C / 2];
    if (j < j1) {
      const uint16_t* bd = sp.bounds + (long long)bt[j] * 2 * D + sub * C;
#pragma unroll
      for (int i = 0; i < C / 8; ++i) {
        *reinterpret_cast<uint4*>(lo + 4 * i) = *reinterpret_cast<const uint4*>(bd + 8 * i);
        *reinterpret_cast<uint4*>(up + 4 * i) = *reinterpret_cast<const uint4*>(bd + D + 8 * i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C / 2; ++i) lo[i] = up[i] = 0;
    }
    double best = -INFINITY;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      Sum u0, u1;
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(s_q + g * D + sub * C + 2 * i);
        // products of two bf16 values are exact; NaN stays
        const float x0 = bf16lo_to_f32(x), x1 = bf16hi_to_f32(x);
        u0.add(max_nan(x0 * bf16lo_to_f32(lo[i]), x0 * bf16lo_to_f32(up[i])));
        u1.add(max_nan(x1 * bf16hi_to_f32(lo[i]), x1 * bf16hi_to_f32(up[i])));
      }
      double u = u0.value() + u1.value();
      for (int off = 1; off < 8; off <<= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
      best = fmax(best, ranked(u));
    }
    if (sub == 0 && j < j1) score[j] = best * (FP8 ? (double)bs[2 * j] : 1.0);
    if (parts > 1) {
      __syncthreads();
      if (tid == 0) s_last = atom_add_acq_rel(sp.count + hs, 1) == parts - 1;
      __syncthreads();
      if (!s_last) return;
      if (tid == 0) sp.count[hs] = 0;
    }
    if (tid == 0) sp.bounds_done[hi] = max(full, have);
    __syncthreads();
    if (staged)
      for (int i = tid; i < (full + 3) / 4 * 4; i += kThreads) {
        const double u = i < full ? __ldcg(score + i) : -INFINITY;
        if (i < full) s_score[i] = score_key(u);
        s_near[i] = (float)u;
      }
    __syncthreads();
  }
  // Block j is chosen when fewer than num_select blocks come before it in the order
  // of (score, position). Counted in fp32 first, by the signs of differences (a
  // multiply-add pipe's and one other operation each): ties in fp32 only matter if
  // they bring in too many.
  unsigned fast = 0;                       // bit c: block c * kThreads + tid is chosen
  bool exact = choose;
  if (choose && staged) {
    int total = 0;
    for (int c0 = 0; c0 * kThreads < full; ++c0) {
      const int j = c0 * kThreads + tid;
      bool take = j < full;
      if (take) {
        const float x = s_near[j];
        int over = 0;
#pragma unroll 4
        for (int i = 0; i < full; i += 4) {   // (-inf behind the last one)
          const float4 y = *reinterpret_cast<const float4*>(s_near + i);
          over += (int)(__float_as_uint(x - y.x) >> 31) + (int)(__float_as_uint(x - y.y) >> 31) +
                  (int)(__float_as_uint(x - y.z) >> 31) + (int)(__float_as_uint(x - y.w) >> 31);
        }
        take = over < num_select;
      }
      fast |= (unsigned)take << c0;
      total += __syncthreads_count(take);
    }
    exact = total != nsel;
  }
  // the chosen blocks, ascending
  int base = 0;
  for (int j0 = 0; j0 < full; j0 += kThreads) {
    const int j = j0 + tid;
    bool take = j < full && nsel > 0;
    if (take && exact) {
      const long long x = staged ? s_score[j] : score_key(__ldcg(score + j));
      int rank = 0;
      for (int i = 0; i < full; ++i) {
        const long long y = staged ? s_score[i] : score_key(__ldcg(score + i));
        rank += y > x || (y == x && i < j);
      }
      take = rank < num_select;
    } else if (take && choose) {
      take = (fast >> (j0 / kThreads)) & 1;
    }
    const unsigned bal = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_cnt[warp] = __popc(bal);
    __syncthreads();
    int at = base;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += s_cnt[w];
      base += s_cnt[w];
    }
    at += __popc(bal & ((1u << lane) - 1));
    if (take) {
      st[at] = bt[j];
      ss[2 * at] = bs[2 * j];
      ss[2 * at + 1] = bs[2 * j + 1];
      if (blocks) blocks[(long long)hs * num_select + at] = j;
    }
    __syncthreads();
  }
  if (blocks)
    for (int i = nsel + tid; i < num_select; i += kThreads)
      blocks[(long long)hs * num_select + i] = -1;
  if (tid == 0) {
    sp.sel_len[hs] = nsel * kBlockSlots + part;
    if (part && !c.blk) {   // (per-block FP8: its rows are staged, not in a block)
      st[nsel] = bt[full];
      ss[2 * nsel] = bs[2 * full];
      ss[2 * nsel + 1] = bs[2 * full + 1];
    }
  }
}

template <int D, bool FP8, int G>
cudaError_t launch_select_g(fdms_cache* c, int layer, int batch, int num_select, int view_blocks,
                          const void* q, int32_t* blocks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int mb = c->view.max_blocks;
  cfg.gridDim = dim3((unsigned)(num_select > 0 ? (mb + kCtaBlocks - 1) / kCtaBlocks : 1),
                     (unsigned)(batch * c->view.Hkv));
  cfg.blockDim = dim3(kThreads);
  const int staged = mb <= kStaged;
  cfg.dynamicSmemBytes = staged ? (mb + 1) / 2 * 2 * sizeof(double) + (mb + 4) * sizeof(float) : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_sparse_select<D, FP8, G>, c->view, c->swork, layer, num_select,
                            view_blocks, staged, static_cast<const uint16_t*>(q), blocks);
}

template <int D, bool FP8>
cudaError_t launch_select(fdms_cache* c, int layer, int batch, int num_select, int view_blocks,
                          const void* q, int32_t* blocks, cudaStream_t s) {
  auto run = c->view.G == 1   ? launch_select_g<D, FP8, 1>
             : c->view.G == 2 ? launch_select_g<D, FP8, 2>
             : c->view.G == 4 ? launch_select_g<D, FP8, 4>
                              : launch_select_g<D, FP8, 8>;
  return run(c, layer, batch, num_select, view_blocks, q, blocks, s);
}

}  // namespace

extern "C" fdms_status fdms_bounds_create(fdms_cache* c, void* stream) {
  if (!c) return FDMS_ERR_INVALID_ARG;
  SparseWork& w = c->swork;
  if (w.bounds) return FDMS_OK;
  const CacheView& v = c->view;
  fdms_device_guard guard(c->device);
  const size_t heads = (size_t)v.L * v.Bmax * v.Hkv, call = (size_t)v.Bmax * v.Hkv;
  const size_t sizes[8] = {(size_t)v.num_blocks * 2 * v.D * sizeof(uint16_t),
                           heads * sizeof(int32_t),
                           call * v.max_blocks * sizeof(double),
                           call * v.max_blocks * sizeof(int32_t),
                           call * v.max_blocks * 2 * sizeof(float),
                           call * sizeof(int32_t),
                           call * sizeof(int4),
                           call * sizeof(int)};
  void* p[8] = {};
  int got = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool ok = true;
  for (; ok && got < 8; ++got) ok = cudaMalloc(&p[got], sizes[got]) == cudaSuccess;
  if (!ok) --got;
  ok = ok && cudaMemsetAsync(p[1], 0, sizes[1], s) == cudaSuccess &&
       cudaMemsetAsync(p[5], 0, sizes[5], s) == cudaSuccess &&
       cudaMemsetAsync(p[7], 0, sizes[7], s) == cudaSuccess &&
       cudaStreamSynchronize(s) == cudaSuccess &&
       c->nallocs + 8 <= (int)(sizeof(c->allocs) / sizeof(c->allocs[0]));
  if (!ok) {   // nothing is left allocated, the cache as it was
    for (int i = 0; i < got; ++i) cudaFree(p[i]);
    cudaGetLastError();
    return FDMS_ERR_CUDA;
  }
  for (int i = 0; i < 8; ++i) fdms_track(c, p[i], sizes[i]);
  w.bounds_done = static_cast<int32_t*>(p[1]);
  w.score = static_cast<double*>(p[2]);
  w.sel_table = static_cast<int32_t*>(p[3]);
  w.sel_scale = static_cast<float*>(p[4]);
  w.sel_len = static_cast<int32_t*>(p[5]);
  w.snap = static_cast<int4*>(p[6]);
  w.count = static_cast<int*>(p[7]);
  w.bounds = static_cast<uint16_t*>(p[0]);
  return FDMS_OK;
}

extern "C" fdms_status fdms_decode_attn_sparse(fdms_cache* c, int layer, int batch, int num_select,
                                               const void* q_dev, void* out_dev,
                                               int32_t* blocks_dev, void* stream) {
  if (!c) return FDMS_ERR_INVALID_ARG;
  const CacheView& v = c->view;
  if (layer < 0 || layer >= v.L || batch < 0 || batch > v.Bmax || num_select < 0)
    return FDMS_ERR_INVALID_ARG;
  if (!c->swork.bounds) return FDMS_ERR_INVALID_ARG;
  if (batch == 0) return FDMS_OK;
  if (!q_dev || !out_dev || (((uintptr_t)q_dev | (uintptr_t)out_dev) & 15))
    return FDMS_ERR_INVALID_ARG;
  fdms_device_guard guard(c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int view_blocks = num_select < v.max_blocks ? num_select + 1 : v.max_blocks;
  auto sel = v.D == 64 ? (v.fp8 ? launch_select<64, true> : launch_select<64, false>)
                       : (v.fp8 ? launch_select<128, true> : launch_select<128, false>);
  if (sel(c, layer, batch, num_select, view_blocks, q_dev, blocks_dev, s) != cudaSuccess)
    return FDMS_ERR_CUDA;
  fdms_log_launch(c, true);
  return fdms_launch_decode_selected(c, layer, batch, view_blocks, q_dev, out_dev, s);
}
