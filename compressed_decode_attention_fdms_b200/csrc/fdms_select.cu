// Keep bits from accumulated attention weights (fdms_select_keep): per
// (sequence, kv head) the `budget` largest scores of the tokens before the
// recent window, equal scores in order of position.
//
// One CTA per head finds the budget-th largest pair (score, earliest position)
// by radix select: a 32-bit key that orders like the score, in digits of 11, 11
// and 10 bits, then, where several scores equal the last one, their positions.
// Each digit is a histogram in shared memory. After the first digit few tokens
// are left in the running: they are gathered, and the scores themselves are
// passed over three times (histogram, gather, bits). A head's scores are copied
// to shared memory as a whole where they fit (up to kStage tokens): what bounds
// the kernel is the latency of one head's passes, and with four loads under way
// per thread reading them from L2 took 38.5 us for 256 heads of up to 32K tokens.
// Now 28.5 us (23.7 MB, 3.6 us at the memory's rate): a head of 32K tokens takes 20 us, of
// which the histogram is 4, the gather 4 and the bits 6 (bytes in every Hkv-th place,
// 1.2 M partial sectors in all), and 256 of them take two rounds of the SMs. Heads above
// kStage read their scores from L2 in each pass: 77 us for eight heads of 128K tokens,
// and for 64 of them too.
#include "fdms_tc.cuh"

using namespace fdms;

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;              // 11 bits, two bins a thread
constexpr int kList = 4096;              // gathered tokens
constexpr int kDigit = 11;
constexpr int kStage = 40960;            // scores of a head that shared memory takes
constexpr int kParts = 4;                // copies they come in

// 32-bit key in the order of the score: NaN 0 (the sum is the one NaN 0x7fffffff,
// whose key wraps), -0 and +0 equal
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u ^ ((uint32_t)((int)u >> 31) | 0x80000000u)) + 1u;
}

struct SelShared {
  unsigned hist[2][kBins];               // even and odd warps
  uint32_t key[kList];
  int pos[kList];
  unsigned warp[kSelWarps];
  unsigned bin, need, left, count;
  uint64_t part[kParts];                 // a part of the scores has landed
  int stop;
};

// f(key, position, there) for the tokens [from, to) of the CTA's head, whole warps
// at a time (`there`: position < to); four loads under way per thread. score(j)
// reads one.
template <class R, class F>
__device__ __forceinline__ void each_score(int from, int to, R score, F f) {
  const int tid = threadIdx.x;
  int j0 = from;
  for (; j0 + 4 * kSelThreads <= to; j0 += 4 * kSelThreads) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = score(j0 + u * kSelThreads + tid);
#pragma unroll
    for (int u = 0; u < 4; ++u) f(score_key(v[u]), j0 + u * kSelThreads + tid, true);
  }
  for (; j0 < to; j0 += kSelThreads) {
    const int j = j0 + tid;
    f(j < to ? score_key(score(j)) : 0u, j, j < to);
  }
}

// The bin, from the largest down, that holds the need-th element: s.bin, the
// elements of it still needed (s.need) and those it holds (s.left). Clears hist.
__device__ void find_bin(SelShared& s, unsigned need) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int b0 = kBins - 1 - 2 * tid;
  const unsigned c0 = s.hist[0][b0] + s.hist[1][b0], c1 = s.hist[0][b0 - 1] + s.hist[1][b0 - 1];
  s.hist[0][b0] = s.hist[1][b0] = s.hist[0][b0 - 1] = s.hist[1][b0 - 1] = 0;
  unsigned incl = c0 + c1;
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s.warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    unsigned w = s.warp[lane];
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    s.warp[lane] = w;
  }
  __syncthreads();
  unsigned before = (warp > 0 ? s.warp[warp - 1] : 0u) + incl - (c0 + c1);
  if (before < need && before + c0 >= need) {
    s.bin = b0;
    s.need = need - before;
    s.left = c0;
  }
  before += c0;
  if (before < need && before + c1 >= need) {
    s.bin = b0 - 1;
    s.need = need - before;
    s.left = c1;
  }
  __syncthreads();
}

constexpr int kStageAt = (sizeof(SelShared) + 15) / 16 * 16;

__global__ void __launch_bounds__(kSelThreads, 2)
k_select_keep(const int32_t* __restrict__ n_dev, int max_n, int Hkv, int W,
              const float* __restrict__ scores, const int32_t* __restrict__ budget,
              uint8_t* __restrict__ keep, int staged, DevCounters* ctr) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelShared& s = *reinterpret_cast<SelShared*>(smem);
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x / Hkv, h = blockIdx.x % Hkv, tid = threadIdx.x, lane = tid % 32;
  const int n = n_dev[b];
  if (n < 0 || n > max_n) {
    if (tid == 0 && h == 0) latch_error(ctr, FDMS_ERR_DEVICE);
    return;
  }
  const int m = max(0, n - W);                 // tokens that compete
  const int want = min(max(budget[blockIdx.x], 0), m);
  const float* x = scores + (size_t)blockIdx.x * max_n;
  uint8_t* out = keep + (size_t)b * max_n * Hkv + h;
  for (int j = m + tid; j < n; j += kSelThreads) out[(size_t)j * Hkv] = 1;
  if (want == 0 || want == m) {
    for (int j = tid; j < m; j += kSelThreads) out[(size_t)j * Hkv] = want ? 1 : 0;
    return;
  }
  // element j of the scores lies in shared memory as it does in global memory
  // to the 16 bytes: whole ones are copied, the ends read
  const int skew = (int)((uintptr_t)x / 4 % 4);
  float* sx = reinterpret_cast<float*>(smem + kStageAt) + skew;
  const int head = (4 - skew) % 4, body = m > head ? (m - head) / 4 * 4 : 0;
  const int step = (body / kParts + 4 * kSelThreads - 1) / (4 * kSelThreads) * (4 * kSelThreads);
  volatile int* stop = &s.stop;
  if (staged && tid == 0) {
    for (int i = 0; i < kParts; ++i) mbar_init(s.part + i, 1);
    *stop = 0;
    fence_mbar_init();
    for (int i = 0; i < kParts; ++i) {
      const int at = min(i * step, body), end = i == kParts - 1 ? body : min((i + 1) * step, body);
      mbar_arrive_expect_tx(s.part + i, (uint32_t)(end - at) * 4);
      if (end > at) bulk_g2s(sx + head + at, x + head + at, (uint32_t)(end - at) * 4, s.part + i);
    }
  }
  if (staged) {
    if (tid < min(head, m)) sx[tid] = x[tid];
    if (tid >= 32 && tid - 32 < m - head - body) sx[head + body + tid - 32] = x[head + body + tid - 32];
  }
  for (int i = tid; i < 2 * kBins; i += kSelThreads) s.hist[0][i] = 0;
  __syncthreads();
  unsigned* hist = s.hist[tid / 32 % 2];
  uint32_t thr = 0;                            // the digits found so far
  int cut = 0x7fffffff;                        // last position kept of those equal to thr
  unsigned need = (unsigned)want, left = (unsigned)m;
  bool listed = false;
  auto each_of_all = [&](auto f) {
    if (staged) each_score(0, m, [&](int j) { return sx[j]; }, f);
    else each_score(0, m, [&](int j) { return x[j]; }, f);
  };
  // f(key, position, there) for every gathered token
  auto each_listed = [&](auto f) {
    for (int i = tid; i < (int)s.count; i += kSelThreads) f(s.key[i], s.pos[i], true);
  };
  int shift = 32;
  while (shift > 0 && left != need) {
    const int width = shift < kDigit ? shift : kDigit, top = shift;
    const uint32_t mask = (1u << width) - 1;
    shift -= width;
    // (lanes that meet in a bin cost no turns worth avoiding)
    auto add = [&](uint32_t key, int, bool there) {
      if (there && (top == 32 || (key >> top) == (thr >> top)))
        atomicAdd(hist + ((key >> shift) & mask), 1u);
    };
    if (top == 32) {
      int from = 0;
      bool ok = true;
      for (int i = 0; i < kParts; ++i) {   // part after part, as they land
        const int to = i == kParts - 1 ? m : min(head + (i + 1) * step, m);
        if (staged) ok = ok && bar_wait(s.part + i, 0, stop);
        const auto count = [&](uint32_t key, int, bool there) {
          if (there) atomicAdd(hist + (key >> (32 - kDigit)), 1u);
        };
        if (!staged) each_score(from, to, [&](int j) { return x[j]; }, count);
        else if (ok) each_score(from, to, [&](int j) { return sx[j]; }, count);
        from = to;
      }
      if (!__syncthreads_and(ok)) {        // the scores did not land
        if (tid == 0) latch_error(ctr, FDMS_ERR_DEVICE);
        return;
      }
    } else if (listed)
      each_listed(add);
    else
      each_of_all(add);
    __syncthreads();
    find_bin(s, need);
    thr |= s.bin << shift;
    need = s.need;
    left = s.left;
    if (!listed && left <= (unsigned)kList && left != need) {
      if (tid == 0) s.count = 0;
      __syncthreads();
      const uint32_t lead = thr >> shift;
      // four tokens of each lane at a time: one reservation for a warp's 128
      for (int j0 = 0; j0 < m; j0 += 4 * kSelThreads) {
        uint32_t key[4];
        unsigned in[4], all = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = j0 + u * kSelThreads + tid;
          key[u] = j < m ? score_key(staged ? sx[j] : x[j]) : 0u;
          in[u] = __ballot_sync(0xffffffffu, j < m && (key[u] >> shift) == lead);
          all += __popc(in[u]);
        }
        if (all == 0) continue;
        unsigned at = 0;
        if (lane == 0) at = atomicAdd(&s.count, all);
        at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if ((in[u] >> lane) & 1) {
            const unsigned i = at + __popc(in[u] & ((1u << lane) - 1));
            s.key[i] = key[u];
            s.pos[i] = j0 + u * kSelThreads + tid;
          }
          at += __popc(in[u]);
        }
      }
      listed = true;
    }
    __syncthreads();
  }
  if (left != need) {
    // several equal the last score: the lowest positions of them, the same way
    int bits = 32 - __clz(m), at = 0;          // positions from the top: 2^bits - 1 - j
    const int last = (int)((1u << bits) - 1);
    while (bits > 0) {
      const int width = bits < kDigit ? bits : kDigit, top = bits, mask = (1 << width) - 1;
      bits -= width;
      auto add = [&](uint32_t key, int pos, bool there) {
        const int p = last - pos;
        if (there && key == thr && (p >> top) == (at >> top))
          atomicAdd(hist + ((p >> bits) & mask), 1u);
      };
      if (listed) each_listed(add);
      else each_of_all(add);
      __syncthreads();
      find_bin(s, need);
      at |= (int)s.bin << bits;
      need = s.need;
      __syncthreads();
    }
    cut = last - at;
  }
  each_of_all([&](uint32_t key, int pos, bool there) {
    if (there) out[(size_t)(unsigned)pos * Hkv] = key > thr || (key == thr && pos <= cut) ? 1 : 0;
  });
}

}  // namespace

fdms_status fdms_select_setup(fdms_cache*) {
  return cudaFuncSetAttribute(k_select_keep, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kStageAt + (kStage + 8) * 4) == cudaSuccess
             ? FDMS_OK
             : FDMS_ERR_CUDA;
}

extern "C" fdms_status fdms_select_keep(fdms_cache* c, int batch, const int32_t* n_dev, int max_n,
                                        const float* scores_dev, const int32_t* budget_dev,
                                        uint8_t* keep_dev, void* stream) {
  if (!c) return FDMS_ERR_INVALID_ARG;
  const CacheView& v = c->view;
  if (batch < 0 || batch > v.Bmax || max_n < 0 || max_n > v.max_seq_len)
    return FDMS_ERR_INVALID_ARG;
  if (batch == 0 || max_n == 0) return FDMS_OK;
  if (max_n > FDMS_MAX_PROMPT) return FDMS_ERR_UNSUPPORTED;
  if (!n_dev || !scores_dev || !budget_dev || !keep_dev) return FDMS_ERR_INVALID_ARG;
  fdms_device_guard guard(c->device);
  // (copies want scores_dev aligned to 16 bytes, as every tensor here)
  const int staged = max_n <= kStage && ((uintptr_t)scores_dev & 15) == 0;
  const size_t bytes = kStageAt + (staged ? ((size_t)max_n + 8) * 4 : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(batch * v.Hkv));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_select_keep, n_dev, max_n, v.Hkv, v.W, scores_dev, budget_dev,
                            keep_dev, staged, v.ctr) == cudaSuccess
             ? FDMS_OK
             : FDMS_ERR_CUDA;
}
