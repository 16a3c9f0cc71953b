// Attention of a prompt's queries under the cache's eviction rule
// (fdms_prefill_attn) and the weight every token collects over them
// (fdms_prefill_scores).
#include <cuda.h>

#include "fdms_tc.cuh"

using namespace fdms;

namespace {

struct PrefillArgs {
  const int32_t* n;
  const int32_t* nq;        // NULL: one query per token
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint8_t* keep;      // NULL: every token kept
  int batch, max_n, max_q, Hq, Hkv, G, W;
  float scale;
  DevCounters* ctr;
  // kept tokens, compacted (compact): bit words of the keep bytes, the kept
  // tokens before each word, their K and V rows
  int compact, words;
  uint32_t* bits;           // [batch * Hkv][words]
  uint32_t* before;         // [batch * Hkv][words]
  uint16_t* kc;             // [batch * Hkv][max_n][D]
  uint16_t* vc;             // (attention only)
  int32_t* pos;             // [batch * Hkv][max_n]: their positions (scores only)
  // work split over the keys: partial results, and their maxima and sums
  int splits;               // at most; a run of split_len key tiles or more each
  int split_len;
  float* part_o;            // [splits][batch * max_q * Hq][D]
  float* part_ml;           // [splits][batch * max_q * Hq][2]: reference (log2), sum
};

// Tokens and queries of sequence b; false when they are out of range.
__device__ __forceinline__ bool lengths(const PrefillArgs& a, int b, int& n, int& nq) {
  n = a.n[b];
  nq = a.nq ? a.nq[b] : n;
  return n >= 0 && n <= a.max_n && nq >= 0 && nq <= n && nq <= a.max_q;
}

template <int C>
__device__ __forceinline__ void load_row(const uint16_t* p, int lane, float (&x)[C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) x[i] = bf16lo_to_f32(p[lane * C + i]);
}
template <int C>
__device__ __forceinline__ float dot(const float (&x)[C], const float (&y)[C]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) s = fmaf(x[i], y[i], s);
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// One query row by one warp, token by token, touching only what it sees: the
// rows whose tiles held infinities or NaN (a matrix product carries them into
// rows that do not see them, as 0 * NaN), or whose sums passed what fp32 holds. Here
// they do not: weights are 1 at most, there are 2^30 of them, and a channel that meets a
// V value above 2^96 is summed in units of 2^32 from there on. (The mean so far, with a
// division per token, does not overflow either: 580 ms for 8K tokens of 32/8 heads of
// 128 with NaN in every V row; 363 ms like this.)
template <int D>
__device__ __noinline__ void attend_row(const PrefillArgs& a, int b, int n, int nq, int t, int h,
                                        uint16_t* out, float* lse) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x % 32;
  const int i = n - nq + t, kh = h / a.G;
  const long long row = ((long long)b * a.max_q + t) * a.Hq + h;
  float qx[C], o[C] = {}, unit[C], m = -INFINITY, l = 0.f;
  load_row<C>(a.q + row * D, lane, qx);
  for (int x = 0; x < C; ++x) unit[x] = 1.f;
  for (int j0 = 0; j0 <= i; j0 += 32) {
    const int jl = j0 + lane;
    const bool seen = jl <= i && (jl > i - a.W || !a.keep ||
                                  a.keep[((long long)b * a.max_n + jl) * a.Hkv + kh]);
    unsigned todo = __ballot_sync(0xffffffffu, seen);
    while (todo) {
      const int j = j0 + __ffs(todo) - 1;
      todo &= todo - 1;
      const long long at = (((long long)b * a.max_n + j) * a.Hkv + kh) * D;
      float kx[C], vx[C];
      load_row<C>(a.k + at, lane, kx);
      load_row<C>(a.v + at, lane, vx);
      const float s = dot<C>(qx, kx) * a.scale;
      const float m2 = fmaxf(m, s);
      // (a score of -inf beside nothing else so far: a weight of 0, not exp(-inf + inf))
      const float up = m2 == -INFINITY ? 1.f : __expf(m - m2);
      const float p = m2 == -INFINITY && s == m2 ? 0.f : __expf(s - m2);
      l = l * up + p;
      for (int x = 0; x < C; ++x) {
        if (fabsf(vx[x]) > 0x1p96f && unit[x] == 1.f) {
          unit[x] = 0x1p-32f;
          o[x] *= 0x1p-32f;
        }
        o[x] = o[x] * up + p * (vx[x] * unit[x]);
      }
      m = m2;
    }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  for (int x = 0; x < C; ++x)
    out[row * D + lane * C + x] = f32_to_bf16_rn(o[x] * inv / unit[x]);
  if (lse && lane == 0) lse[row] = m + logf(l);
}

// ------------------------------------------------------------ kept tokens
// Bit words of the keep bytes: a thread per token, a ballot per head (4 us for 8K
// tokens of 8 heads, nearly all of it launch).
__global__ void __launch_bounds__(256) k_keep_bits(PrefillArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  int n, nq;
  if (!lengths(a, b, n, nq)) n = 0;
  const int lane = threadIdx.x % 32;
  if (j - lane >= a.words * 32) return;
  for (int h = 0; h < a.Hkv; ++h) {
    const bool on = j < n && a.keep[((long long)b * a.max_n + j) * a.Hkv + h];
    const unsigned w = __ballot_sync(0xffffffffu, on);
    if (lane == 0) a.bits[((long long)b * a.Hkv + h) * a.words + j / 32] = w;
  }
}

// K and V rows of the kept tokens one after the other, so that TMA can bring them in
// tiles: a CTA per 128 tokens of a head, which counts the bits before its own (6.5 us
// for 8K tokens of 8 heads of 64; bound by the latency of that count and the copy).
template <int D>
__global__ void __launch_bounds__(256) k_keep_rows(PrefillArgs a) {
  __shared__ unsigned s_sum[8];
  __shared__ uint8_t s_tok[128];
  pdl_wait();
  pdl_launch_dependents();
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh % a.Hkv, tid = threadIdx.x, lane = tid % 32;
  const uint32_t* bits = a.bits + (long long)bh * a.words;
  const int w0 = blockIdx.x * 4;
  unsigned sum = 0;
  for (int w = tid; w < w0; w += 256) sum += __popc(bits[w]);
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_sum[tid / 32] = sum;
  __syncthreads();
  unsigned base = 0;
  for (int i = 0; i < 8; ++i) base += s_sum[i];
  int count = 0;   // of the CTA's 128 tokens
  for (int i = 0; i < 4 && w0 + i < a.words; ++i) {
    const unsigned w = bits[w0 + i];
    if (tid == 0) a.before[(long long)bh * a.words + w0 + i] = base + count;
    if (tid < 32 && ((w >> lane) & 1))
      s_tok[count + __popc(w & ((1u << lane) - 1))] = (uint8_t)(i * 32 + lane);
    count += __popc(w);
  }
  __syncthreads();
  constexpr int CH = D / 8;   // 16-byte chunks of a row
  const long long src0 = ((long long)b * a.max_n + (long long)w0 * 32) * a.Hkv + h;
  for (int x = tid; x < count * CH; x += 256) {
    const int r = x / CH, ch = x % CH;
    const long long src = (src0 + (long long)s_tok[r] * a.Hkv) * CH + ch;
    const long long dst = ((long long)bh * a.max_n + base + r) * CH + ch;
    reinterpret_cast<uint4*>(a.kc)[dst] = reinterpret_cast<const uint4*>(a.k)[src];
    if (a.vc) reinterpret_cast<uint4*>(a.vc)[dst] = reinterpret_cast<const uint4*>(a.v)[src];
  }
  if (a.pos)
    for (int r = tid; r < count; r += 256)
      a.pos[(long long)bh * a.max_n + base + r] = w0 * 32 + s_tok[r];
  // zeros behind the last one, to the end of its tile: a weight of 0 does not
  // hide what memory holds there
  if (blockIdx.x == gridDim.x - 1) {
    const int end = (int)base + count, fill = min((end + 127) / 128 * 128, a.max_n) - end;
    for (int x = tid; x < fill * CH; x += 256) {
      const long long dst = ((long long)bh * a.max_n + end) * CH + x;
      reinterpret_cast<uint4*>(a.kc)[dst] = make_uint4(0, 0, 0, 0);
      if (a.vc) reinterpret_cast<uint4*>(a.vc)[dst] = make_uint4(0, 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------ attention
struct PrefillMaps {
  CUtensorMap q, k, v, kc, vc;
};

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;       // query rows (token, head of the group) of a tile
constexpr int kKeys = 128;       // tokens of a key tile
constexpr int kMaskSlots = 8;

template <int D>
struct AttnL {
  static constexpr int TILE = 128 * D * 2;               // bytes of a Q, K or V tile
  static constexpr int NS = D == 128 ? 5 : 8;            // K / V stages
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_BAR = OFF_KV + NS * TILE;
  static constexpr int NBAR = 2 + 2 * NS + 6 + kMaskSlots;
  static constexpr int OFF_MASK = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;
  static constexpr int OFF_MISC = OFF_MASK + kMaskSlots * 16;
  static constexpr int OFF_BOARD = OFF_MISC + 16 + ItemQueue::BYTES;
  static constexpr int SMEM = OFF_BOARD + 256 + 1024;    // 1024: alignment
  static constexpr int THREADS = 384;
  // registers: 384 x 168 at launch = 64,512 = 256 x 208 + 128 x 88
  static constexpr int REGS_SOFTMAX = 208, REGS_REST = 88;
};

__device__ __forceinline__ float2 exp2_pair(float2 x, bool mad) {
  return mad ? exp2_mad(x) : make_float2(fast_exp2(x.x), fast_exp2(x.y));
}

__device__ __forceinline__ uint32_t low_bits(int k) {
  return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
}

// A row's sum of weights 2^(score - ref), once it passes 2^24, to between 1 and 4: the
// reference rises by the sum's exponent. What its results are to be scaled by. (An
// infinite sum stays, and so does NaN.)
__device__ __forceinline__ float raise_ref(float& l, float& ref) {
  if (!(l > 16777216.f)) return 1.f;
  const int k = min((int)(__float_as_uint(l) >> 23) - 127, 126);
  const float up = __uint_as_float((unsigned)(127 - k) << 23);   // 2^-k
  ref += (float)k;
  l *= up;
  return up;
}

template <bool M>
struct Masked {
  static constexpr bool value = M;
};

// Work item: up to 256 query rows (two tiles of 128 rows; row = token * G + head
// of the group) of one kv head over a run of key tiles. Blocks with the longest
// rows come first.
struct AttnItem {
  int b, kh, bh, n, nq, t0, i0, i_end, split;
  int tiles;                // row tiles, 0: nothing to do
  int raw0, cnt, nc;        // tokens before raw0: the cnt kept ones, compacted, nc tiles
  int kt0, N;               // its key tiles: N from tile kt0 on
  int splits;               // of its rows' keys: 1, the results are final
  int bad;                  // lengths out of range
  int end;                  // no more items
  __device__ __forceinline__ bool compacted(int x) const { return kt0 + x < nc; }
  // first token (or compacted row) of its key tile x
  __device__ __forceinline__ int first(int x) const {
    return compacted(x) ? (kt0 + x) * kKeys : raw0 + (kt0 + x - nc) * kKeys;
  }
};

__device__ __forceinline__ AttnItem attn_item(const PrefillArgs& a, int x) {
  AttnItem it;
  const int BH = a.batch * a.Hkv, TB = 2 * kRows / a.G;   // TB: tokens of a block
  it.split = x % a.splits;
  x /= a.splits;
  it.bh = x % BH;
  it.b = it.bh / a.Hkv;
  it.kh = it.bh % a.Hkv;
  it.t0 = ((a.max_q + TB - 1) / TB - 1 - x / BH) * TB;
  it.tiles = it.N = it.end = 0;
  it.splits = 1;
  it.bad = !lengths(a, it.b, it.n, it.nq);
  if (it.bad || it.t0 >= it.nq) return it;
  const int last = min(it.t0 + TB, it.nq);
  it.i0 = it.n - it.nq + it.t0;             // positions of its first and last query
  it.i_end = it.n - it.nq + last - 1;
  it.tiles = last - it.t0 > TB / 2 ? 2 : 1;
  // tokens before raw0 are outside every row's window: of them the kept ones;
  // from there on every token, masked
  it.raw0 = it.cnt = 0;
  if (a.compact) {
    it.raw0 = max(0, it.i0 - a.W + 1);
    if (it.raw0 > 0) {
      const long long w = (long long)it.bh * a.words + (it.raw0 - 1) / 32;
      it.cnt = a.before[w] + __popc(a.bits[w] & low_bits((it.raw0 - 1) % 32 + 1));
    }
  }
  it.nc = (it.cnt + kKeys - 1) / kKeys;
  const int all = it.nc + (it.i_end - it.raw0 + kKeys) / kKeys;
  it.splits = max(1, min(a.splits, (all + a.split_len - 1) / a.split_len));
  if (it.split >= it.splits) {
    it.tiles = 0;
    return it;
  }
  it.kt0 = (int)((long long)all * it.split / it.splits);
  it.N = (int)((long long)all * (it.split + 1) / it.splits) - it.kt0;
  return it;
}

// S = Q K^T, P = 2^(S c log2 e - ref), O = sum P V, l = sum P; out = O / l. Warps 0-3
// and 4-7: the softmax of row tile 0 and 1, a thread per row (no exchange between
// threads); warp 8 issues the matrix products, warp 9 the copies and the keep bits
// (10 and 11 only give their registers away). While one tile's weights are computed
// the tensor cores work for the other. Tensor memory holds S of both tiles (P takes
// its place, in bf16: half the columns, and the form the second product wants) and O.
// Rows of a kv head's group share K and V, so a tile of 128 rows spans 128 / G tokens.
//
// The weights enter the second product rounded to bf16 (one rounding, 2^-8 at most; 2.1e-3
// off 64 bits in the 2-norm where rounding the result alone gives 1.6e-3): with a head and a
// remainder, which decode carries, that product, half of the tensor work, would be done
// twice. Sums and denominators are fp32.
//
// What bounds it: of 3,500 cycles per key tile and row tile pair the products take
// 2,048 at heads of 128 (1,024 at 64) and the exponentials 2,048; neither is busy all
// the time, since a tile's products and softmax follow one another and two tiles only
// half cover the gaps. 8K tokens, 32/8 heads of 128, nothing evicted: 550 us, 470 in a
// burst of twenty passes: 1.00 and 1.17 PFLOP/s of measured 1.40 sustained, 1.66 in a
// burst. With 5 to 30 % kept, heads of 64: 142 to 160 us by the keep rates drawn, of
// which the compaction is 9; two key tiles of three cover the window there. The softmax
// branch spills 76 bytes a thread (its 128 scores fill 208 registers).
template <int D>
__global__ void __launch_bounds__(AttnL<D>::THREADS, 1)
k_prefill_mma(const __grid_constant__ PrefillArgs a, const __grid_constant__ PrefillMaps maps,
              uint16_t* __restrict__ out, float* __restrict__ lse) {
  using L = AttnL<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* kv_full = q_empty + 1;
  uint64_t* kv_empty = kv_full + L::NS;
  uint64_t* s_full = kv_empty + L::NS;    // [2] scores of a tile are there
  uint64_t* p_full = s_full + 2;          // [2] weights of a tile are there
  uint64_t* o_full = p_full + 2;          // [2] the product with V is done
  uint64_t* mask_full = o_full + 2;
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + L::OFF_MASK);   // [slots][4]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* stop = reinterpret_cast<int*>(s_tmem + 1);
  ItemQueue queue;
  queue.place(smem + L::OFF_MISC + 16);
  using Board = ItemBoard<AttnItem>;
  static_assert(Board::BYTES <= 256, "place of the items");
  Board board;
  board.place(smem + L::OFF_BOARD);

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int TH = kRows / a.G;             // tokens of a row tile
  if (warp == 8) {
    tmem_alloc(s_tmem, 512);
  } else if (tid == 9 * 32) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < L::NS; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_full + i, 1);
    }
    for (int i = 0; i < kMaskSlots; ++i) mbar_init(mask_full + i, 1);
    queue.init();
    board.init(9);
    *stop = 0;
    fence_mbar_init();
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();
  pdl_launch_dependents();
  bool ok = true;

  if (warp >= 8) regs_down<L::REGS_REST>();   // one instruction for the warpgroup
  if (warp == 9) {
    // ---------------------------------------------------- copies, keep bits
    int idx = 0, nq_tiles = 0;            // K / V stages and Q tiles used so far
    int puts = 0;
    for (int c = blockIdx.x, i = 0; ok; c = queue.next(i++, stop)) {
      AttnItem it;
      if (c < 0) {
        it.end = 1;
        board.put(puts, it, stop);
        break;
      }
      ok = queue.ask(i, stop);
      it = attn_item(a, c);
      if (it.bad && it.t0 == 0 && it.kh == 0 && it.split == 0 && lane == 0)
        latch_error(a.ctr, FDMS_ERR_DEVICE);
      if (it.tiles == 0) continue;
      ok = ok && board.put(puts++, it, stop);
      for (int x = 0; x < it.N && ok; ++x) {
        const int j0 = it.first(x);
        const bool cp = it.compacted(x);
        for (int kv = 0; kv < 2 && ok; ++kv, ++idx) {
          const int st = idx % L::NS, ph = idx / L::NS;
          if (ph > 0) ok = __all_sync(0xffffffffu, bar_wait(kv_empty + st, (ph - 1) & 1, stop));
          if (!ok) break;
          if (kv == 1 && !cp && j0 + kKeys > it.n && it.n < a.max_n) {
            // rows behind the sequence may hold anything, NaN included, which a
            // weight of 0 does not hide: zeros in their place
            uint8_t* dst = smem + L::OFF_KV + st * L::TILE;
            const uint4* src = reinterpret_cast<const uint4*>(a.v);
#pragma unroll 8
            for (int e = lane; e < kKeys * (D / 8); e += 32) {
              const int row = e / (D / 8), ch = e % (D / 8);
              uint4 y = make_uint4(0, 0, 0, 0);
              if (j0 + row < it.n)
                y = src[(((long long)it.b * a.max_n + j0 + row) * a.Hkv + it.kh) * (D / 8) + ch];
              *reinterpret_cast<uint4*>(dst + ch / 8 * 16384 + row * 128 +
                                        (((ch % 8) ^ (row & 7)) * 16)) = y;
            }
            fence_smem_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(kv_full + st);
          } else if (lane == 0) {
            mbar_arrive_expect_tx(kv_full + st, L::TILE);
            const CUtensorMap* map = cp ? (kv ? &maps.vc : &maps.kc) : (kv ? &maps.v : &maps.k);
            for (int y = 0; y < D / 64; ++y)
              tma_box4(smem + L::OFF_KV + st * L::TILE + y * 16384, map, y * 64,
                       cp ? 0 : it.kh, j0, cp ? it.bh : it.b, kv_full + st);
          }
          if (x == 0 && kv == 0) {
            // the queries, once the last item's products with K are done
            if (nq_tiles > 0)
              ok = __all_sync(0xffffffffu, bar_wait(q_empty, (nq_tiles - 1) & 1, stop));
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(q_full, it.tiles * L::TILE);
              for (int m = 0; m < it.tiles; ++m)
                for (int y = 0; y < D / 64; ++y)
                  tma_box4(smem + m * L::TILE + y * 16384, &maps.q, y * 64, it.kh * a.G,
                           it.t0 + m * TH, it.b, q_full);
            }
            ++nq_tiles;
          }
          if (kv == 0) {
            // keep bits of the tile's tokens. Key tile g takes slot g % 8: tile
            // g - 8 was read before the K stage of tile g - NS / 2 - 1 or later
            // was given back
            const int slot = idx / 2 % kMaskSlots;
            if (a.keep && !cp) {
              bool on[4];
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int j = j0 + w * 32 + lane;
                on[w] = j <= it.i_end &&
                        a.keep[((long long)it.b * a.max_n + min(j, it.i_end)) * a.Hkv + it.kh];
              }
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t bits = __ballot_sync(0xffffffffu, on[w]);
                if (lane == 0) mask[slot * 4 + w] = bits;
              }
            } else if (lane < 4) {
              mask[slot * 4 + lane] = 0xffffffffu;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(mask_full + slot);
          }
        }
      }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------- matrix products
    constexpr uint32_t kQK = mma_desc(128, 128, false), kPV = mma_desc(128, D, true);
    const uint32_t sq = smem_addr(smem), skv = smem_addr(smem + L::OFF_KV);
    int idx = 0, nq_tiles = 0, done[2] = {0, 0};   // done: key tiles of row tile m so far
    auto qk = [&](int m, int st) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint32_t at = (s / 4) * 16384 + (s % 4) * 32;
        mma_ss(tmem + m * 128, smem_desc(sq + m * L::TILE + at, 16),
               smem_desc(skv + st * L::TILE + at, 16), kQK, s > 0);
      }
      tc_commit(s_full + m);
    };
    for (int i = 0; ok; board.done(i), ++i) {
      const AttnItem* at = board.get(i, stop);
      if (!at || at->end) break;
      const AttnItem& it = *at;
      if (it.N == 0) continue;
      ok = __all_sync(0xffffffffu, bar_wait(q_full, nq_tiles & 1, stop) &&
                                       bar_wait(kv_full + idx % L::NS, (idx / L::NS) & 1, stop));
      if (ok) {
        tc_fence_after();
        if (elect_one()) {
          for (int m = 0; m < it.tiles; ++m) qk(m, idx % L::NS);
          tc_commit(kv_empty + idx % L::NS);
          if (it.N == 1) tc_commit(q_empty);
        }
        __syncwarp();
      }
      for (int x = 0; x < it.N && ok; ++x) {
        const int iv = idx + 2 * x + 1, ik = iv + 1;
        const int sv = iv % L::NS, sk = ik % L::NS;
        const bool more = x + 1 < it.N;
        ok = bar_wait(kv_full + sv, (iv / L::NS) & 1, stop) &&
             (!more || bar_wait(kv_full + sk, (ik / L::NS) & 1, stop));
        for (int m = 0; m < it.tiles; ++m) {
          const bool final = m == it.tiles - 1;
          // (a tile's first weights come after its last results were read)
          ok = __all_sync(0xffffffffu, ok && bar_wait(p_full + m, (done[m] + x) & 1, stop));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              mma_ts(tmem + 256 + m * D, tmem + m * 128 + s * 8,
                     smem_desc(skv + sv * L::TILE + s * 2048, 16384), kPV, x > 0 || s > 0);
            tc_commit(o_full + m);
            if (final) tc_commit(kv_empty + sv);
            if (more) {
              qk(m, sk);
              if (final) {
                tc_commit(kv_empty + sk);
                if (x + 2 == it.N) tc_commit(q_empty);
              }
            }
          }
          __syncwarp();
        }
      }
      idx += 2 * it.N;
      ++nq_tiles;
      for (int m = 0; m < it.tiles; ++m) done[m] += it.N;
    }
  } else if (warp < 8) {
    // ---------------------------------------------------- softmax
    regs_up<L::REGS_SOFTMAX>();
    const int m = warp / 4, r = tid % 128;
    const uint32_t ts = tmem + ((uint32_t)(warp % 4 * 32) << 16) + m * 128;
    const uint32_t to = tmem + ((uint32_t)(warp % 4 * 32) << 16) + 256 + m * D;
    const float sl2 = a.scale * 1.4426950408889634f;
    int done = 0, tiles_before = 0;       // key tiles of this row tile, and of all, so far
    for (int ci = 0; ok; board.done(ci), ++ci) {
      const AttnItem* item = board.get(ci, stop);
      if (!item || item->end) break;
      const AttnItem& it = *item;
      if (m >= it.tiles) {
        tiles_before += it.N;
        continue;
      }
      const int t = it.t0 + m * TH + r / a.G, h = it.kh * a.G + r % a.G;
      const int i = it.n - it.nq + t;                           // the row's position
      const int im0 = it.i0 + m * TH, im1 = im0 + TH - 1;       // the tile's
      // The weights are 2^(score - ref). Any reference gives the same quotient, and
      // none loses precision while nothing overflows: ref is the maximum of the first
      // tile that the row sees something of, and rises by the exponent of the row's sum
      // once that passes 2^24. (A tile that raises a weight past 2^127 at once makes
      // the row infinite, and it is computed again below. Maxima of every tile cost
      // 800 of 3,700 cycles per key tile.) What the last tile brought a split is left to the join.
      float ref = 0.f;
      bool has = false;       // a reference
      float l = 0.f;
      const int nc = it.nc - it.kt0, N = it.N, cnt = it.cnt;
      const int at_c = it.kt0 * kKeys, at_r = it.raw0 - nc * kKeys;
      for (int x = 0; x < N; ++x) {
        ok = __all_sync(0xffffffffu, bar_wait(s_full + m, (done + x) & 1, stop));
        if (!ok) break;
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          tmem_ld32(ts + w * 32, *reinterpret_cast<uint32_t(*)[32]>(s + w * 32));
        tmem_wait_ld();
        const bool cp = x < nc;
        const int j0 = (cp ? at_c : at_r) + x * kKeys;
        const bool masked = cp ? j0 + kKeys > cnt
                               : (j0 + kKeys - 1 > im0 || (a.keep && j0 <= im1 - a.W));
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};   // bit e of word w: column 32 w + e counts
        if (masked) {
          const int g = tiles_before + x;
          if (!cp) {
            ok = __all_sync(0xffffffffu, bar_wait(mask_full + g % kMaskSlots,
                                                  (g / kMaskSlots) & 1, stop));
            if (!ok) break;
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (cp) {
              see[w] = low_bits(cnt - j0 - w * 32);
            } else {
              see[w] = low_bits(i - j0 + 1 - w * 32) &
                       (mask[g % kMaskSlots * 4 + w] | ~low_bits(i - a.W - j0 + 1 - w * 32));
            }
          }
        }
        if (!__all_sync(0xffffffffu, has && l <= 16777216.f)) {
          float tm = -INFINITY;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            tm = fmaxf(tm, (see[e / 32] >> (e % 32)) & 1 ? s[e] : -INFINITY);
          if (!has && tm > -INFINITY) {
            ref = tm * sl2;
            has = true;
          }
          if (__any_sync(0xffffffffu, l > 16777216.f)) {
            // (x > 0) the sums so far are complete once the last product is
            const float up = raise_ref(l, ref);
            ok = __all_sync(0xffffffffu, bar_wait(o_full + m, (done + x - 1) & 1, stop));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < D; e += 16) {
              uint32_t o[16];
              tmem_ld16(to + e, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * up);
              tmem_st16(to + e, o);
            }
          }
        }
        float2 sum[4] = {};
        // (two copies: scores changed in place by a mask cost copies of all of them)
        auto weights = [&](auto mk) {
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            uint32_t p[8];
#pragma unroll
            for (int k0 = 0; k0 < 8; k0 += 4) {
              float2 e[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int c = w * 16 + 2 * (k0 + k);
                e[k] = ffma2(make_float2(s[c], s[c + 1]), make_float2(sl2, sl2),
                             make_float2(-ref, -ref));
                if (mk.value) {
                  if (!((see[c / 32] >> (c % 32)) & 1)) e[k].x = -INFINITY;
                  if (!((see[c / 32] >> (c % 32 + 1)) & 1)) e[k].y = -INFINITY;
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                e[k] = make_float2(fast_exp2(e[k].x), fast_exp2(e[k].y));
                sum[k] = add2(sum[k], e[k]);
                p[k0 + k] = pack_bf16(e[k].x, e[k].y);
              }
            }
            tmem_st8(ts + w * 8, p);
          }
        };
        if (masked) weights(Masked<true>{});
        else weights(Masked<false>{});
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(p_full + m);
        const float2 s2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += s2.x + s2.y;
      }
      // ---- the rows' results
      if (ok && it.N > 0)
        ok = __all_sync(0xffffffffu, bar_wait(o_full + m, (done + it.N - 1) & 1, stop));
      if (!ok) break;
      done += it.N;
      tiles_before += it.N;
      tc_fence_after();
      const bool live = t < it.nq;
      const long long row = ((long long)it.b * a.max_q + t) * a.Hq + h;
      if (it.splits == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bool bad = !(l < INFINITY);
#pragma unroll
        for (int e = 0; e < D; e += 32) {
          uint32_t o[32];
          if (it.N > 0) {
            tmem_ld32(to + e, o);
            tmem_wait_ld();
          }
          uint32_t y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float u = __uint_as_float(o[2 * k]) * inv, w = __uint_as_float(o[2 * k + 1]) * inv;
            if (l == 0.f) u = w = 0.f;
            bad |= !(fabsf(u) < INFINITY) | !(fabsf(w) < INFINITY);
            y[k] = pack_bf16(u, w);
          }
          if (live)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(out + row * D + e + k * 8) =
                  make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        }
        if (live && lse) lse[row] = l == 0.f ? -INFINITY : fmaf(ref, kLn2, logf(l));
        unsigned todo = __ballot_sync(0xffffffffu, bad && live);
        while (todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          attend_row<D>(a, it.b, it.n, it.nq, __shfl_sync(0xffffffffu, t, src),
                        __shfl_sync(0xffffffffu, h, src), out, lse);
        }
      } else {
        const long long at = (long long)it.split * a.batch * a.max_q * a.Hq + row;
        if (live) {
          a.part_ml[2 * at] = l == 0.f ? -INFINITY : ref;
          a.part_ml[2 * at + 1] = l;
        }
        if (it.N > 0) {
#pragma unroll
          for (int e = 0; e < D; e += 32) {
            uint32_t o[32];
            tmem_ld32(to + e, o);
            tmem_wait_ld();
            if (live)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(a.part_o + at * D + e + k * 4) =
                    make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*stop && tid == 0) latch_error(a.ctr, FDMS_ERR_DEVICE);
  if (*stop && tid == 9 * 32) {
    // a wait ran out: let the copies under way land before the CTA's memory goes
    const unsigned long long t1 = global_ns();
    while (global_ns() - t1 < 1000000ull) {
    }
  }
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ few rows
// Up to 64 query rows per kv head (draft tokens, a chunk's last queries): the time
// goes into reading K and V, so only the rows that some query sees are read, with
// no pass before. A warp takes every (4 * splits)-th word of 32 tokens, lists the
// tokens that count (this spreads the window, where all do, over the warps) and
// works through them 16 at a time: rows copied in the background two tiles ahead,
// products of 16 x 16 x 8, online softmax. The warps' results are joined in
// shared memory, the CTAs' by k_prefill_join.
// Bound by latencies: lengths, keep bits, the list and the first rows follow one
// another, then six or seven tiles. Five queries on each of eight sequences of up to
// 8197 tokens, 32/8 heads of 128, 6 to 20 % kept: 27 us in all, 36 MB read, where K and
// V whole are 201 MB and 31 us. (Tiles of k_prefill_mma, kept rows compacted first: 49.)
// 512 tokens of 4/2 heads of 64: 9 us against 16.5.
constexpr int kFewRows = 32;     // query rows of a CTA at most
constexpr int kFewWarps = 4;
constexpr int kFewTokens = 16;   // tokens of a tile
constexpr int kFewStages = 3;
constexpr int kFewWords = 16;    // words listed at a time

template <int D>
struct FewL {
  static constexpr int ROW = 2 * D;                                 // bytes
  static constexpr int STAGE = 2 * kFewTokens * ROW;                // K rows, then V rows
  static constexpr int LIST = (kFewWords * 32 + kFewTokens) * 4;
  static constexpr int OFF_STAGE = kFewRows * ROW;                  // after Q
  static constexpr int OFF_LIST = OFF_STAGE + kFewWarps * kFewStages * STAGE;
  static constexpr int OFF_ML = OFF_LIST;                           // [warps][rows][2], after
  static constexpr int SMEM = OFF_LIST + kFewWarps * LIST;          // the lists (two CTAs fit)
  static_assert(LIST >= kFewRows * 8, "maxima and sums reuse the lists");
  static_assert(kFewStages * STAGE >= kFewRows * D * 4, "results reuse the stages");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// R: row tiles of 16
template <int D, int R>
__global__ void __launch_bounds__(kFewWarps * 32, 2)
k_prefill_few(const __grid_constant__ PrefillArgs a, int row_chunks, uint16_t* __restrict__ out,
              float* __restrict__ lse) {
  using L = FewL<D>;
  constexpr int CH = D / 8;      // 16-byte chunks of a row
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_wait();
  pdl_launch_dependents();
  int x = blockIdx.x;
  const int split = x % a.splits;
  x /= a.splits;
  const int r0 = x % row_chunks * kFewRows;   // first row (token * G + head of the group)
  const int bh = x / row_chunks, b = bh / a.Hkv, kh = bh % a.Hkv;
  int n, nq;
  if (!lengths(a, b, n, nq)) {
    if (split == 0 && r0 == 0 && kh == 0 && tid == 0) latch_error(a.ctr, FDMS_ERR_DEVICE);
    return;
  }
  if (r0 >= nq * a.G) return;
  const int lg = __ffs(a.G) - 1;
  const int rows = min(kFewRows, nq * a.G - r0);
  const int off = n - nq, i0 = off + (r0 >> lg), i_end = off + ((r0 + rows - 1) >> lg);
  const uint32_t sq = smem_addr(smem);
  const uint32_t sst = sq + L::OFF_STAGE + warp * kFewStages * L::STAGE;
  int* list = reinterpret_cast<int*>(smem + L::OFF_LIST + warp * L::LIST);
  // Q rows, the chunks of row r permuted by r % 8 (as every row here)
  for (int e = tid; e < R * 16 * CH; e += kFewWarps * 32) {
    const int r = e / CH, ch = e % CH, t = (r0 + r) >> lg, g = (r0 + r) & (a.G - 1);
    const long long row = ((long long)b * a.max_q + min(t, nq - 1)) * a.Hq + kh * a.G + g;
    cp_async16(sq + r * L::ROW + ((ch ^ (r & 7)) * 16), a.q + row * D + ch * 8, r < rows);
  }
  const int words = i_end / 32 + 1, stride = a.splits * kFewWarps;
  const uint8_t* kb = a.keep ? a.keep + (long long)b * a.max_n * a.Hkv + kh : nullptr;
  auto keep_of = [&](int w0) {   // this lane's keep bits of the words w0, w0 + stride ..
    unsigned kept = 0;
#pragma unroll
    for (int u = 0; u < kFewWords; ++u) {
      const long long j = (long long)(w0 + u * stride) * 32 + lane;
      if (j <= i_end && kb[j * a.Hkv]) kept |= 1u << u;
    }
    return kept;
  };
  unsigned kept = kb ? keep_of(split * kFewWarps + warp) : ~0u;
  asm volatile("cp.async.commit_group;\n cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  float o[R][D / 8][4], mx[R][2], l[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) o[r][c][0] = o[r][c][1] = o[r][c][2] = o[r][c][3] = 0.f;
    mx[r][0] = mx[r][1] = -INFINITY;
    l[r][0] = l[r][1] = 0.f;
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  const uint16_t* kg = a.k + ((long long)b * a.max_n * a.Hkv + kh) * D;
  const uint16_t* vg = a.v + ((long long)b * a.max_n * a.Hkv + kh) * D;
  int count = 0;                 // listed tokens
  for (int w0 = split * kFewWarps + warp; w0 < words; w0 += stride * kFewWords) {
    // ---- list the tokens that some row sees (sign bit: kept)
    for (int u = 0; u < kFewWords && w0 + u * stride < words; ++u) {
      const int j = (w0 + u * stride) * 32 + lane;
      const bool k = (kept >> u) & 1, in = j <= i_end && (k || j > i0 - a.W);
      const unsigned all = __ballot_sync(0xffffffffu, in);
      if (in) list[count + __popc(all & ((1u << lane) - 1))] = j | (k ? 0x80000000 : 0);
      count += __popc(all);
    }
    __syncwarp();
    const bool last = w0 + (long long)stride * kFewWords >= words;
    const int tiles = last ? (count + kFewTokens - 1) / kFewTokens : count / kFewTokens;
    auto issue = [&](int t) {
      if (t < tiles) {
        const uint32_t st = sst + t % kFewStages * L::STAGE;
#pragma unroll
        for (int e = 0; e < kFewTokens * CH; e += 32) {
          const int r = (e + lane) / CH, ch = (e + lane) % CH, at = t * kFewTokens + r;
          const bool real = at < count;
          const long long src =
              (real ? (long long)(list[at] & 0x7fffffff) : 0) * a.Hkv * D + ch * 8;
          const uint32_t dst = st + r * L::ROW + ((ch ^ (r & 7)) * 16);
          cp_async16(dst, kg + src, real);
          cp_async16(dst + kFewTokens * L::ROW, vg + src, real);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    issue(0);
    issue(1);
    for (int t = 0; t < tiles; ++t) {
      __syncwarp();              // the stage of tile t - 1 is done with
      issue(t + 2);
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      __syncwarp();
      const uint32_t sk = sst + t % kFewStages * L::STAGE, sv = sk + kFewTokens * L::ROW;
      float s[R][2][4] = {};
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t bk[4];
        {
          const int key = lane % 8 + lane / 16 * 8, ch = ks * 2 + lane / 8 % 2;
          ldsm4(sk + key * L::ROW + ((ch ^ (key & 7)) * 16), bk);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          uint32_t aq[4];
          const int row = r * 16 + lane % 8 + lane / 8 % 2 * 8, ch = ks * 2 + lane / 16;
          ldsm4(sq + row * L::ROW + ((ch ^ (row & 7)) * 16), aq);
          mma16(s[r][0], aq, bk[0], bk[1]);
          mma16(s[r][1], aq, bk[2], bk[3]);
        }
      }
      // what each row sees of the tile (this lane's four columns)
      int pos[4];
      bool keptc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int at = t * kFewTokens + c / 2 * 8 + lane % 4 * 2 + c % 2;
        const int e = at < count ? list[at] : 0x7fffffff;   // behind every query
        pos[c] = e & 0x7fffffff;
        keptc[c] = e < 0;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint32_t p[4];
        float up[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int i = off + ((r0 + r * 16 + lane / 4 + y * 8) >> lg);
          float tm = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float& e = s[r][c / 2][y * 2 + c % 2];
            if (!(pos[c] <= i && (keptc[c] || pos[c] > i - a.W))) e = -INFINITY;
            tm = fmaxf(tm, e);
          }
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
          up[y] = 1.f;
          if (mx[r][y] == -INFINITY) {
            mx[r][y] = tm;
          } else if ((tm - mx[r][y]) * sl2 > 8.f) {   // weights stay under 2^8
            up[y] = fast_exp2((mx[r][y] - tm) * sl2);
            l[r][y] *= up[y];
            mx[r][y] = tm;
          }
          const float ref = mx[r][y] == -INFINITY ? 0.f : mx[r][y] * sl2;
          float e4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            e4[c] = fast_exp2(fmaf(s[r][c / 2][y * 2 + c % 2], sl2, -ref));
            l[r][y] += e4[c];
          }
          p[y] = pack_bf16(e4[0], e4[1]);
          p[y + 2] = pack_bf16(e4[2], e4[3]);
        }
        if (__any_sync(0xffffffffu, up[0] != 1.f || up[1] != 1.f)) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            o[r][c][0] *= up[0];
            o[r][c][1] *= up[0];
            o[r][c][2] *= up[1];
            o[r][c][3] *= up[1];
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][0][c] = __uint_as_float(p[c]);   // kept for the product
      }
#pragma unroll
      for (int dd = 0; dd < D / 16; ++dd) {
        uint32_t bv[4];
        const int key = lane % 8 + lane / 8 % 2 * 8, ch = dd * 2 + lane / 16;
        ldsm4_t(sv + key * L::ROW + ((ch ^ (key & 7)) * 16), bv);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t p[4] = {__float_as_uint(s[r][0][0]), __float_as_uint(s[r][0][1]),
                                 __float_as_uint(s[r][0][2]), __float_as_uint(s[r][0][3])};
          mma16(o[r][2 * dd], p, bv[0], bv[1]);
          mma16(o[r][2 * dd + 1], p, bv[2], bv[3]);
        }
      }
    }
    // the tokens of the last, incomplete tile wait for the next words
    const int rest = count - tiles * kFewTokens;
    __syncwarp();
    const int carry = lane < rest ? list[tiles * kFewTokens + lane] : 0;
    __syncwarp();
    if (lane < rest) list[lane] = carry;
    count = rest > 0 ? rest : 0;
    __syncwarp();
    if (kb && !last) kept = keep_of(w0 + stride * kFewWords);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // ---- join the warps
  __syncthreads();
  float* mine = reinterpret_cast<float*>(smem + L::OFF_STAGE + warp * kFewStages * L::STAGE);
  float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int row = r * 16 + lane / 4 + y * 8;
      float z = l[r][y];
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      if (lane % 4 == 0) {
        ml[(warp * kFewRows + row) * 2] = mx[r][y];
        ml[(warp * kFewRows + row) * 2 + 1] = z;
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2*>(mine + row * D + c * 8 + lane % 4 * 2) =
            make_float2(o[r][c][2 * y], o[r][c][2 * y + 1]);
    }
  __syncthreads();
  const long long all = (long long)a.batch * a.max_q * a.Hq;
  for (int row = warp; row < rows; row += kFewWarps) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, ml[(w * kFewRows + row) * 2]);
    float sum = 0.f, y[D / 32] = {};
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float lw = ml[(w * kFewRows + row) * 2 + 1];
      if (lw == 0.f) continue;
      const float f = fast_exp2((ml[(w * kFewRows + row) * 2] - m) * sl2);
      const float* part =
          reinterpret_cast<const float*>(smem + L::OFF_STAGE + w * kFewStages * L::STAGE) + row * D;
      sum = fmaf(f, lw, sum);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) y[c] = fmaf(f, part[c * 32 + lane], y[c]);
    }
    const int t = (r0 + row) >> lg, h = kh * a.G + ((r0 + row) & (a.G - 1));
    const long long at = ((long long)b * a.max_q + t) * a.Hq + h;
    if (a.splits == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      bool bad = !(sum < INFINITY);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        y[c] = sum == 0.f ? 0.f : y[c] * inv;
        bad |= !(fabsf(y[c]) < INFINITY);
      }
      if (__any_sync(0xffffffffu, bad)) {
        attend_row<D>(a, b, n, nq, t, h, out, lse);
        continue;
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) out[at * D + c * 32 + lane] = f32_to_bf16_rn(y[c]);
      if (lse && lane == 0) lse[at] = sum == 0.f ? -INFINITY : m * a.scale + logf(sum);
    } else {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) a.part_o[(split * all + at) * D + c * 32 + lane] = y[c];
      if (lane == 0) {
        a.part_ml[2 * (split * all + at)] = m * sl2;
        a.part_ml[2 * (split * all + at) + 1] = sum;
      }
    }
  }
}

// The partial results of a row's splits, joined: D / 4 lanes per row, eight CTAs per
// block of rows (as the items of k_prefill_mma; what it costs is the chain of loads of
// a warp's rows: one CTA per block took 29 us for 59k rows of two splits). A split's last
// tile may have left a sum of up to 2^127 beside a low reference, which is raised first:
// sums are small then (few rows', not TILES: 2^38) and that of the largest reference 1 or more, so
// that a split whose weight becomes 0, with a reference 126 lower, has no share. (Raised
// by the splits themselves: 2.5 us of 161 more for 8K tokens of heads of 64 with keep bits.)
template <int D, bool TILES>
__global__ void __launch_bounds__(256)
k_prefill_join(const __grid_constant__ PrefillArgs a, uint16_t* __restrict__ out,
               float* __restrict__ lse) {
  constexpr int LR = D / 4, RW = 32 / LR;   // lanes of a row, rows of a warp at a time
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % LR;
  const int BH = a.batch * a.Hkv, TB = 2 * kRows / a.G, lg = __ffs(a.G) - 1;
  const int part = blockIdx.x % 8, x = blockIdx.x / 8;
  const int bh = x % BH, t0 = x / BH * TB, b = bh / a.Hkv, kh = bh % a.Hkv;
  int n, nq;
  if (!lengths(a, b, n, nq) || t0 >= nq) return;
  int splits = a.splits;
  if (TILES) {                              // (few rows: all of them)
    const int blocks = (a.max_q + TB - 1) / TB;
    splits = attn_item(a, ((blocks - 1 - t0 / TB) * BH + bh) * a.splits).splits;
    if (splits == 1) return;                // its rows are final
  }
  const long long all = (long long)a.batch * a.max_q * a.Hq;
  const int rows = min(nq - t0, TB) << lg;
  for (int r0 = (part * 8 + warp) * RW; r0 < rows; r0 += 64 * RW) {
    const int r = r0 + lane / LR, t = t0 + (r >> lg), h = kh * a.G + (r & (a.G - 1));
    const bool live = r < rows;
    const long long row = live ? ((long long)b * a.max_q + t) * a.Hq + h : 0;
    float m = -INFINITY;
    for (int s = 0; live && s < splits; ++s) {
      float ref = a.part_ml[2 * (s * all + row)];
      if (TILES) {
        float sum = a.part_ml[2 * (s * all + row) + 1];
        raise_ref(sum, ref);
      }
      m = fmaxf(m, ref);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const long long at = s * all + row;
      float2 ml = live ? *reinterpret_cast<const float2*>(a.part_ml + 2 * at)
                       : make_float2(-INFINITY, 0.f);
      if (ml.y == 0.f) continue;            // nothing seen there (and no partial result)
      const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * D + sub * 4);
      const float up = TILES ? raise_ref(ml.y, ml.x) : 1.f, w = fast_exp2(ml.x - m);
      l = fmaf(w, ml.y, l);
      o.x = fmaf(w, x.x * up, o.x);
      o.y = fmaf(w, x.y * up, o.y);
      o.z = fmaf(w, x.z * up, o.z);
      o.w = fmaf(w, x.w * up, o.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    bool bad = !(l < INFINITY);
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    bad |= !(fabsf(o.x) < INFINITY) | !(fabsf(o.y) < INFINITY) | !(fabsf(o.z) < INFINITY) |
           !(fabsf(o.w) < INFINITY);
    if (live) {
      *reinterpret_cast<uint2*>(out + row * D + sub * 4) =
          make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      if (lse && sub == 0) lse[row] = l == 0.f ? -INFINITY : fmaf(m, kLn2, logf(l));
    }
    unsigned todo = __ballot_sync(0xffffffffu, bad && live);
    __syncwarp();
    while (todo) {                          // once per row
      const int src = (__ffs(todo) - 1) / LR * LR;
      todo &= ~((LR == 32 ? 0xffffffffu : (1u << LR) - 1u) << src);
      attend_row<D>(a, b, n, nq, __shfl_sync(0xffffffffu, t, src),
                    __shfl_sync(0xffffffffu, h, src), out, lse);
    }
  }
}

// ------------------------------------------------------------ scores
// S^T = K Q^T: a thread per token, whose sum over the queries stays in its
// registers; the queries' denominators are the columns'. What a token is seen
// by is a range of queries: from its own on, and (unless it is kept) for W of
// them. With `compact` the work is in two kinds of key tiles: every token over
// the queries in whose window it is, and the kept tokens, compacted, over the
// queries after that.
//
// What bounds it: the exponentials, one per query row and token. 8K tokens of 32/8 heads
// of 64: 314 us, 245 at the special-function unit's rate (of which a quarter is taken
// off it); the last 64 queries of eight prompts of up to 8K, heads of 128: 50 us, where
// what counts is the chain from key tile to product to sums at two steps an item.
// Two CTAs per SM take items: (kind, key tile, head) and a chunk of at most
// chunk_steps * 128 query rows. Warps 0-3 and 4-7 sum even and odd steps, warp
// 8 issues the matrix products, warp 9 the copies and the denominators.
struct ScoreArgs {
  int key_tiles;            // per head and kind
  int chunks, chunk_steps;
  const float* lse;
  float* scores;
  float* part;              // [chunks][kinds][batch * Hkv][max_n], or NULL: into `scores`
  int accumulate;
};

struct ScoreMaps {
  CUtensorMap q, k, kc;
};

// Of eight pairs of exponentials, those on the multiply-add pipe (8K prompt, 32/8
// heads of 64: 353 us with none, 339 with 2, 350 with 3, 372 with 4; in the
// attention kernels, which wait on the products more, none is best).
constexpr int kScoreMad = 2;

template <int D>
struct ScoreL {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NQ = D == 128 ? 2 : 4;            // Q stages
  static constexpr int SLOTS = 8;                        // denominator slots, >= NQ + 4
  static constexpr int OFF_Q = TILE;
  static constexpr int OFF_LSE = OFF_Q + NQ * TILE;
  static constexpr int OFF_SUM = OFF_LSE + SLOTS * 512;  // the odd steps' sums
  static constexpr int OFF_BAR = OFF_SUM + 512;
  static constexpr int NBAR = 2 + 2 * NQ + 4 + SLOTS + 2;
  static constexpr int OFF_MISC = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;
  static constexpr int OFF_BOARD = OFF_MISC + 16 + ItemQueue::BYTES;
  static constexpr int SMEM = OFF_BOARD + 256 + 1024;
  static constexpr int THREADS = 320;
};

// One item: its rows, and the queries [t_lo, t_hi) of its tokens.
struct ScoreItem {
  int b, kh, bh, n, nq, kind, j0, chunk, t_lo, t_hi;
  int count;                // tokens (or kept ones) of the sequence
  int mine;                 // the item is there (its sums are written, zeros included)
  int bad;                  // lengths out of range
  int end;                  // no more items
};

__device__ __forceinline__ int kept_total(const PrefillArgs& a, int bh, int n) {
  if (n == 0) return 0;
  const long long w = (long long)bh * a.words + (n - 1) / 32;
  return (int)(a.before[w] + __popc(a.bits[w]));
}

__device__ __forceinline__ ScoreItem score_item(const PrefillArgs& a, const ScoreArgs& sc, int x) {
  ScoreItem it;
  const int BH = a.batch * a.Hkv, kinds = a.compact ? 2 : 1;
  it.j0 = x % sc.key_tiles * kKeys;
  x /= sc.key_tiles;
  it.bh = x % BH;
  x /= BH;
  it.kind = x % kinds;
  it.chunk = x / kinds;
  it.b = it.bh / a.Hkv;
  it.kh = it.bh % a.Hkv;
  it.mine = it.bad = it.end = 0;
  it.t_lo = it.t_hi = it.count = 0;
  it.bad = !lengths(a, it.b, it.n, it.nq);
  if (it.bad) return it;
  const int off = it.n - it.nq, CT = sc.chunk_steps * (kRows / a.G);
  it.count = it.kind ? kept_total(a, it.bh, it.n) : it.n;
  if (it.j0 >= it.count) return it;
  it.mine = 1;
  int from, to = it.nq;
  if (it.kind) {
    from = a.pos[(long long)it.bh * a.max_n + it.j0] + a.W - off;
  } else {
    from = it.j0 - off;
    if (a.compact) to = min(to, min(it.j0 + kKeys, it.n) - 1 + a.W - off);
  }
  it.t_lo = max(max(from, 0), it.chunk * CT);
  it.t_hi = min(to, (it.chunk + 1) * CT);
  return it;
}

// Sum of one token's weights over a step's 128 columns (with MASKED the columns
// lo .. hi - 1); gives the scores' buffer back once they are read.
template <bool MASKED>
__device__ __forceinline__ float score_tile(uint32_t ts, const float* zs, float sl2,
                                            uint64_t* empty, int lo, int hi) {
  float2 sum[4] = {};
  uint32_t s[2][16];
  tmem_ld16(ts, s[0]);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    tmem_wait_ld();
    if (w < 7) {
      tmem_ld16(ts + w * 16 + 16, s[(w + 1) % 2]);
    } else {
      tc_fence_before();
      warp_arrive(empty);
    }
    const uint32_t* v = s[w % 2];
    const uint32_t see = low_bits(hi - w * 16) & ~low_bits(lo - w * 16);
    float2 e[8];
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const float4 y = *reinterpret_cast<const float4*>(zs + w * 16 + c);
      e[c / 2] = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                        make_float2(sl2, sl2), make_float2(y.x, y.y));
      e[c / 2 + 1] = ffma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                        make_float2(sl2, sl2), make_float2(y.z, y.w));
      if (MASKED) {
        if (!((see >> c) & 1)) e[c / 2].x = -INFINITY;
        if (!((see >> (c + 1)) & 1)) e[c / 2].y = -INFINITY;
        if (!((see >> (c + 2)) & 1)) e[c / 2 + 1].x = -INFINITY;
        if (!((see >> (c + 3)) & 1)) e[c / 2 + 1].y = -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = exp2_pair(e[k], !MASKED && k < kScoreMad);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k % 4] = add2(sum[k % 4], e[k]);
  }
  const float2 y = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
  return y.x + y.y;
}

__device__ __forceinline__ void score_out(const PrefillArgs& a, const ScoreArgs& sc,
                                          const ScoreItem& it, int e, float total) {
  if (sc.part) {
    const int plane = it.chunk * (a.compact ? 2 : 1) + it.kind;
    sc.part[((long long)plane * a.batch * a.Hkv + it.bh) * a.max_n + e] = total;
  } else {
    float* at = sc.scores + (long long)it.bh * a.max_n + e;
    *at = sc.accumulate ? *at + total : total;
  }
}

template <int D>
__global__ void __launch_bounds__(ScoreL<D>::THREADS, 2)
k_scores_mma(const __grid_constant__ PrefillArgs a, const __grid_constant__ ScoreArgs sc,
             const __grid_constant__ ScoreMaps maps) {
  using L = ScoreL<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_empty = k_full + 1;
  uint64_t* q_full = k_empty + 1;
  uint64_t* q_empty = q_full + L::NQ;
  uint64_t* s_full = q_empty + L::NQ;     // [2]
  uint64_t* s_empty = s_full + 2;         // [2]
  uint64_t* z_full = s_empty + 2;         // [SLOTS]
  uint64_t* sum_full = z_full + L::SLOTS; // the odd steps' sums are there / read
  uint64_t* sum_empty = sum_full + 1;
  float* odd = reinterpret_cast<float*>(smem + L::OFF_SUM);
  float* z = reinterpret_cast<float*>(smem + L::OFF_LSE);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* stop = reinterpret_cast<int*>(s_tmem + 1);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int TQ = kRows / a.G, lg = __ffs(a.G) - 1;   // queries of a step
  ItemQueue queue;
  queue.place(smem + L::OFF_MISC + 16);
  using Board = ItemBoard<ScoreItem>;
  static_assert(Board::BYTES <= 256, "place of the items");
  Board board;
  board.place(smem + L::OFF_BOARD);
  if (warp == 8) {
    tmem_alloc(s_tmem, 256);
  } else if (tid == 9 * 32) {
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    for (int i = 0; i < L::NQ; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, 4);
    }
    for (int i = 0; i < L::SLOTS; ++i) mbar_init(z_full + i, 1);
    mbar_init(sum_full, 4);
    mbar_init(sum_empty, 4);
    queue.init();
    board.init(9);
    *stop = 0;
    fence_mbar_init();
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // (every CTA has its tensor memory before the next kernel may start)
  pdl_wait();
  pdl_launch_dependents();
  bool ok = true;
  int step = 0, kt = 0;                   // steps and key tiles so far

  if (warp == 9) {
    // ---------------------------------------------------- copies, denominators
    int puts = 0;
    for (int x = blockIdx.x, i = 0; ok; x = queue.next(i++, stop)) {
      ScoreItem it;
      if (x < 0) {
        it.end = 1;
        board.put(puts, it, stop);
        break;
      }
      ok = queue.ask(i, stop);
      it = score_item(a, sc, x);
      if (it.bad && it.j0 == 0 && it.kh == 0 && it.chunk == 0 && it.kind == 0 && lane == 0)
        latch_error(a.ctr, FDMS_ERR_DEVICE);
      if (!it.mine) continue;
      ok = ok && board.put(puts++, it, stop);
      if (!ok || it.t_lo >= it.t_hi) continue;
      if (kt > 0) ok = __all_sync(0xffffffffu, bar_wait(k_empty, (kt - 1) & 1, stop));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(k_full, L::TILE);
        for (int c = 0; c < D / 64; ++c)
          tma_box4(smem + c * 16384, it.kind ? &maps.kc : &maps.k, c * 64, it.kind ? 0 : it.kh,
                   it.j0, it.kind ? it.bh : it.b, k_full);
      }
      ++kt;
      // minus the denominators of a step's columns (queries behind the last one:
      // any value, their columns are masked), loaded a step ahead
      const float* zg = sc.lse + (long long)it.b * a.max_q * a.Hq + it.kh * a.G;
      float ahead[4];
      auto fetch = [&](int t) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int c = w * 32 + lane;
          ahead[w] = zg[(long long)min(t + (c >> lg), it.nq - 1) * a.Hq + (c & (a.G - 1))];
        }
      };
      fetch(it.t_lo);
      for (int t = it.t_lo; t < it.t_hi; t += TQ, ++step) {
        float y[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) y[w] = ahead[w];
        if (t + TQ < it.t_hi) fetch(t + TQ);
        const int st = step % L::NQ, ph = step / L::NQ;
        if (ph > 0) ok = __all_sync(0xffffffffu, bar_wait(q_empty + st, (ph - 1) & 1, stop));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full + st, L::TILE);
          for (int c = 0; c < D / 64; ++c)
            tma_box4(smem + L::OFF_Q + st * L::TILE + c * 16384, &maps.q, c * 64, it.kh * a.G, t,
                     it.b, q_full + st);
        }
        // slot step % 8 was last read for step - 8. This Q stage was given back
        // by the product of step - NQ, which waited for the scores of step -
        // NQ - 2 to be read, so that the sums of step - NQ - 4 were done.
        const int slot = step % L::SLOTS;
#pragma unroll
        for (int w = 0; w < 4; ++w)   // a row that saw nothing: weights of 0
          z[slot * 128 + w * 32 + lane] = y[w] == -INFINITY ? y[w] : y[w] * -1.4426950408889634f;
        __syncwarp();
        if (lane == 0) mbar_arrive(z_full + slot);
      }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------- matrix products
    constexpr uint32_t kKQ = mma_desc(128, 128, false);
    const uint32_t sk = smem_addr(smem), sq = smem_addr(smem + L::OFF_Q);
    for (int i = 0; ok; board.done(i), ++i) {
      const ScoreItem* at = board.get(i, stop);
      if (!at || at->end) break;
      const ScoreItem it = *at;
      if (it.t_lo >= it.t_hi) continue;
      ok = __all_sync(0xffffffffu, bar_wait(k_full, kt & 1, stop));
      for (int t = it.t_lo; t < it.t_hi && ok; t += TQ, ++step) {
        const int st = step % L::NQ, buf = step % 2, use = step / 2;
        ok = __all_sync(0xffffffffu,
                        bar_wait(q_full + st, (step / L::NQ) & 1, stop) &&
                            (use == 0 || bar_wait(s_empty + buf, (use - 1) & 1, stop)));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t at = (s / 4) * 16384 + (s % 4) * 32;
            mma_ss(tmem + buf * 128, smem_desc(sk + at, 16),
                   smem_desc(sq + st * L::TILE + at, 16), kKQ, s > 0);
          }
          tc_commit(q_empty + st);
          tc_commit(s_full + buf);
          if (t + TQ >= it.t_hi) tc_commit(k_empty);
        }
        __syncwarp();
      }
      ++kt;
    }
  } else {
    // ---------------------------------------------------- sums
    const int buf = warp / 4, r = tid % 128;   // this warpgroup's steps, its token
    const uint32_t ts = tmem + ((uint32_t)(warp % 4 * 32) << 16) + buf * 128;
    const float sl2 = a.scale * 1.4426950408889634f;
    int done = 0;                              // items so far
    for (int i = 0; ok; board.done(i), ++i) {
      const ScoreItem* at = board.get(i, stop);
      if (!at || at->end) break;
      const ScoreItem it = *at;
      const int e = it.j0 + r, off = it.n - it.nq;
      const bool live = e < it.count;
      // this token's queries [from, to)
      int from = 0, to = 0;
      if (live && it.t_lo < it.t_hi) {
        if (it.kind) {
          from = a.pos[(long long)it.bh * a.max_n + e] + a.W - off;
          to = it.nq;
        } else {
          from = e - off;
          const bool bounded =
              a.compact ||
              (a.keep && !a.keep[((long long)it.b * a.max_n + e) * a.Hkv + it.kh]);
          to = bounded ? min(it.nq, e + a.W - off) : it.nq;
        }
        to = min(to, it.t_hi);
      }
      float total = 0.f;
      for (int t = it.t_lo; t < it.t_hi; t += TQ, ++step) {
        if (step % 2 != buf) continue;
        const int slot = step % L::SLOTS;
        ok = __all_sync(0xffffffffu, bar_wait(s_full + buf, (step / 2) & 1, stop) &&
                                         bar_wait(z_full + slot, (step / L::SLOTS) & 1, stop));
        if (!ok) break;
        tc_fence_after();
        const bool whole = __all_sync(0xffffffffu, from <= t && t + TQ <= to);
        const int lo = (from - t) * a.G, hi = (to - t) * a.G;   // columns that count
        const float* zs = z + slot * 128;
        total += whole ? score_tile<false>(ts, zs, sl2, s_empty + buf, lo, hi)
                       : score_tile<true>(ts, zs, sl2, s_empty + buf, lo, hi);
      }
      if (!ok) break;
      // the sums of even and odd steps, joined by the even steps' thread
      if (buf == 1) {
        if (done > 0) ok = __all_sync(0xffffffffu, bar_wait(sum_empty, (done - 1) & 1, stop));
        odd[r] = total;
        warp_arrive(sum_full);
      } else {
        ok = __all_sync(0xffffffffu, bar_wait(sum_full, done & 1, stop));
        if (ok && live) score_out(a, sc, it, e, total + odd[r]);
        warp_arrive(sum_empty);
      }
      ++done;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*stop && tid == 0) latch_error(a.ctr, FDMS_ERR_DEVICE);
  if (*stop && tid == 9 * 32) {
    // a wait ran out: let the copies under way land before the CTA's memory goes
    const unsigned long long t1 = global_ns();
    while (global_ns() - t1 < 1000000ull) {
    }
  }
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 256);
}

// The chunks' sums of each token, in order: first those over its window (or
// over every query), then those after it if it is kept.
__global__ void __launch_bounds__(256)
k_scores_join(const __grid_constant__ PrefillArgs a, const __grid_constant__ ScoreArgs sc) {
  pdl_wait();
  pdl_launch_dependents();
  const int bh = blockIdx.y, b = bh / a.Hkv, j = blockIdx.x * 256 + threadIdx.x;
  int n, nq;
  if (!lengths(a, b, n, nq) || j >= n) return;
  const long long plane = (long long)a.batch * a.Hkv * a.max_n, row = (long long)bh * a.max_n;
  const int kinds = a.compact ? 2 : 1;
  float sum = 0.f;
  for (int c = 0; c < sc.chunks; ++c) sum += sc.part[c * kinds * plane + row + j];
  if (a.compact) {
    const long long w = (long long)bh * a.words + j / 32;
    const uint32_t bits = a.bits[w];
    if ((bits >> (j % 32)) & 1) {
      const long long r = row + a.before[w] + __popc(bits & low_bits(j % 32));
      for (int c = 0; c < sc.chunks; ++c) sum += sc.part[(c * kinds + 1) * plane + r];
    }
  }
  float* at = sc.scores + row + j;
  *at = sc.accumulate ? *at + sum : sum;
}

// ------------------------------------------------------------ host
fdms_status check(fdms_cache* c, int batch, const int32_t* n_dev, int max_n, const int32_t* nq_dev,
                  int max_q, const void* q_dev, const void* k_dev) {
  const CacheView& v = c->view;
  if (batch < 0 || batch > v.Bmax || max_n < 0 || max_n > v.max_seq_len || max_q < 0 ||
      max_q > max_n || (!nq_dev && max_q != max_n))
    return FDMS_ERR_INVALID_ARG;
  if (batch == 0 || max_n == 0) return FDMS_OK;
  if (max_n > FDMS_MAX_PROMPT) return FDMS_ERR_UNSUPPORTED;
  if (!n_dev || !k_dev || (max_q > 0 && !q_dev)) return FDMS_ERR_INVALID_ARG;
  if (((uintptr_t)q_dev | (uintptr_t)k_dev) & 15) return FDMS_ERR_INVALID_ARG;
  return FDMS_OK;
}

PrefillArgs args_of(fdms_cache* c, int batch, const int32_t* n_dev, int max_n,
                    const int32_t* nq_dev, int max_q, const void* q, const void* k, const void* v,
                    const uint8_t* keep) {
  const CacheView& w = c->view;
  PrefillArgs a = {};
  a.n = n_dev;
  a.nq = nq_dev;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.keep = w.W >= max_n ? nullptr : keep;   // every token is in the window
  a.batch = batch;
  a.max_n = max_n;
  a.max_q = max_q;
  a.Hq = w.Hq;
  a.Hkv = w.Hkv;
  a.G = w.G;
  a.W = w.W;
  a.scale = w.softmax_scale;
  a.ctr = w.ctr;
  return a;
}

// How a call of these sizes runs: attention with its keys split over `splits`
// CTAs, scores with their queries in chunks, kept tokens compacted first; and
// where things lie in its workspace.
struct Plan {
  int splits, split_len;
  int row_chunks;                       // few rows: chunks of kFewRows, else 0
  bool compact;
  int words;
  int key_tiles, chunks, chunk_steps;   // scores
  size_t off_bits, off_before, off_kc, off_vc, off_pos, off_o, off_ml, off_few, off_part;
  // of workspace, enough for this call and for every smaller one
  size_t attn_bytes, score_bytes;
};
// Tokens from which the kept ones are compacted. Compacted / masked in place, attention
// of 32/8 heads of 64 with a fifth kept and a window of 256: 640 tokens 28 / 24 us, 1024
// 39 / 36 (window of 16: 30 / 37), 2048 37 / 56, 4096 70 / 144; heads of 128 at 1024
// 51 / 55. Fewer heads cross later (4/2 of 64: 2048 26 / 25, 4096 42 / 56), and so do the
// scores (32/8 of 64: 1024 30 / 21, 2048 44 / 42, 4096 80 / 112).
constexpr int kCompactMin = 1024;
// Tokens of a short prompt (most_few is 1), if its row chunks all run at once. By
// k_prefill_few / in tiles, 4/2 heads of 64: 128 tokens 6.6 / 9.2 us, 256 8.3 / 11.0,
// 512 11.7 / 14.1 (a quarter kept: 8.6 / 15.0), and beyond the rule still 768 15.3 / 19.7,
// 1024 18.5 / 21. 32/8 heads fill the device at 256 tokens (heads of 64 10.0 / 11.1 us, of
// 128 14.5 / 14.2) and go in tiles above.
constexpr int kFewShort = 512;

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
long long least_of(long long a, long long b) { return a < b ? a : b; }
long long most_of(long long a, long long b) { return a > b ? a : b; }

Plan plan_of(const fdms_cache* c, int batch, int max_n, int max_q, bool keep) {
  const CacheView& v = c->view;
  Plan p = {};
  const long long heads = (long long)batch * v.Hkv, rows = (long long)batch * max_q * v.Hq;
  const long long tiles = ceil_div(max_n, kKeys);
  auto up = [](long long bytes) { return (size_t)(bytes + 255) / 256 * 256; };
  // attention: an item (a block of rows) takes as many key tiles as its rows see,
  // half of all on average. Where the longest take over 3/2 of an SM's share of the
  // work, items are split to runs of 7/10 of it, four tiles or more (T = 5059, 8
  // heads of 64 without groups: the longest items alone took 76 us of 86).
  const long long items = heads * ceil_div(max_q, 2 * kRows / v.G), room = 2LL * c->num_sms;
  const long long len = most_of(4, ceil_div(7 * items * tiles, 20 * c->num_sms));
  const bool even = 4 * tiles * c->num_sms <= 3 * items * tiles;   // tiles <= 3/2 share
  p.split_len = (int)(even || len > tiles ? most_of(1, tiles) : len);
  p.splits = (int)most_of(1, ceil_div(tiles, p.split_len));
  // few rows: as many CTAs as there is room for, 128 tokens or more for a warp
  const long long head_rows = (long long)max_q * v.G, most_few = (max_n + 511) / 512;
  // (or a short prompt whose row chunks all run at once, without a split)
  const long long few_chunks = ceil_div(head_rows, kFewRows);
  if (head_rows > 0 && (head_rows <= 2 * kFewRows ||
                        (max_n <= kFewShort && heads * few_chunks <= room))) {
    p.row_chunks = (int)few_chunks;
    const long long want = room / most_of(1, heads * few_chunks);
    p.splits = (int)(want < 1 ? 1 : want < most_few ? want : most_few);
  }
  // scores: chunks of 8 to 32 steps of 128 query rows, six items or more (half of
  // the chunks are empty) for each of the two CTAs per SM. A chunk more is a plane of
  // partial sums more, and a join. At least 8 / 4 / 2 steps: 4/2 heads of 64, 512 tokens
  // 11.0 / 9.6 / 8.2 us, 1024 13.2 / 9.9 / 8.6; 32/8 heads, 512 13.7 / 10.3 / 10.3, 768
  // 14.4 / 14.0 / 14.6, 1024 18.7 / 19.7 / 17.8 (of 128: 20.0 / 21.4 / 19.2): 8 is not the
  // best for short prompts.
  const long long steps = ceil_div(max_q, kRows / v.G), base = heads * tiles;
  long long cs = ceil_div(base * steps, 12 * room);
  cs = cs < 8 ? 8 : cs > 32 ? 32 : cs;
  p.key_tiles = (int)tiles;
  p.chunk_steps = (int)cs;
  p.chunks = steps > 0 ? (int)ceil_div(steps, cs) : 1;
  // layout: the kept tokens, then either the attention's V rows and partial
  // results or the scores' positions and partial sums
  p.compact = keep && max_n >= kCompactMin && v.W < max_n;
  p.words = (int)ceil_div(max_n, 32);
  const int kinds = p.compact ? 2 : 1;
  size_t at = 0;
  if (p.compact) {
    p.off_bits = at;
    p.off_before = p.off_bits + up(heads * p.words * 4);
    p.off_kc = p.off_before + up(heads * p.words * 4);
    at = p.off_kc + up(heads * max_n * v.D * 2);
  }
  p.off_vc = p.off_pos = at;
  p.off_o = p.off_vc + (p.compact ? up(heads * max_n * v.D * 2) : 0);
  if (p.row_chunks) p.off_few = up((long long)p.splits * rows * v.D * 4);
  else p.off_ml = p.off_o + (p.splits > 1 ? up((long long)p.splits * rows * v.D * 4) : 0);
  p.off_part = p.off_pos + (p.compact ? up(heads * max_n * 4) : 0);
  // Bounds that grow with batch, max_n and max_q, of what this and smaller calls
  // lay there. Attention: splits - 1 < tiles / split_len <= 20/7 num_sms / items, none
  // from that many items on (and an item has 2 * kRows rows), and splits <= tiles / 4
  // + 1. Scores: chunks * base <= 12 * room + base, or the chunks are steps / 32, and
  // chunks <= steps / 8 in any case. Few rows: at most 2 * kFewRows of a head; splits
  // * heads * chunks <= room, or there is one split, and splits <= most_few.
  const long long many = 3LL * c->num_sms;
  const long long prow = tiles <= 4 ? 0 : least_of((many + least_of(items, many)) * 2 * kRows,
                                                   rows * (tiles / 4 + 1));
  const long long frow0 = least_of(rows, heads * 2 * kFewRows);
  const long long frow = most_of(frow0, least_of(room * kFewRows, frow0 * most_few));
  const long long sums =
      least_of(ceil_div(steps, 8) * base, most_of(12 * room + base, ceil_div(steps, 32) * base)) *
      kinds * kKeys;
  if (max_q == 0) return p;
  // (so few rows of a head that every smaller call has few too: nothing is compacted)
  const size_t few_end = up(frow * v.D * 4) + up(frow * 8);
  const size_t o_end = p.off_o + up(prow * v.D * 4) + up(prow * 8);
  p.attn_bytes = head_rows <= 2 * kFewRows || o_end < few_end ? few_end : o_end;
  p.score_bytes = p.off_part + (p.compact || steps > 8 ? up(sums * 4) : 0);
  return p;
}

// (every kernel of this file waits for the one before it before it touches
// memory and lets the next one start only then)
template <class... A>
cudaError_t launch(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
fdms_status attn(fdms_cache* c, PrefillArgs a, const Plan& p, uint8_t* ws, uint16_t* out,
                 float* lse, cudaStream_t s) {
  using L = AttnL<D>;
  const int TB = 2 * kRows / a.G;
  const long long blocks = (long long)a.batch * a.Hkv * ((a.max_q + TB - 1) / TB);
  a.splits = p.splits;
  a.split_len = p.split_len;
  if (p.row_chunks) {
    // partial results from the workspace's start on
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float*>(ws + p.off_few);
    const bool one = a.max_q * a.G <= 16;
    auto few = one ? k_prefill_few<D, 1> : k_prefill_few<D, 2>;
    if (launch(few, dim3((unsigned)(a.batch * a.Hkv * p.row_chunks * p.splits)), kFewWarps * 32,
               FewL<D>::SMEM, s, a, p.row_chunks, out, lse) != cudaSuccess ||
        (p.splits > 1 && launch(k_prefill_join<D, false>, dim3((unsigned)(blocks * 8)), 256, 0, s,
                                a, out, lse) != cudaSuccess))
      return FDMS_ERR_CUDA;
    return FDMS_OK;
  }
  PrefillMaps maps;
  const long long B = a.batch, T = a.max_n, Q = a.max_q;
  bool ok = fdms_tensor_map(&maps.q, a.q, {D, a.Hq, Q, B}, {D, (long long)a.Hq * D, Q * a.Hq * D},
                            a.G, kRows / a.G);
  for (int i = 0; i < 2 && ok; ++i)
    ok = fdms_tensor_map(i ? &maps.v : &maps.k, i ? a.v : a.k, {D, a.Hkv, T, B},
                         {D, (long long)a.Hkv * D, T * a.Hkv * D}, 1, kKeys);
  maps.kc = maps.k;
  maps.vc = maps.v;
  if (p.compact) {
    a.compact = 1;
    a.words = p.words;
    a.bits = reinterpret_cast<uint32_t*>(ws + p.off_bits);
    a.before = reinterpret_cast<uint32_t*>(ws + p.off_before);
    a.kc = reinterpret_cast<uint16_t*>(ws + p.off_kc);
    a.vc = reinterpret_cast<uint16_t*>(ws + p.off_vc);
    for (int i = 0; i < 2 && ok; ++i)
      ok = fdms_tensor_map(i ? &maps.vc : &maps.kc, i ? a.vc : a.kc, {D, 1, T, B * a.Hkv},
                           {D, D, T * D}, 1, kKeys);
    if (!ok) return FDMS_ERR_CUDA;
    if (launch(k_keep_bits, dim3((a.max_n + 255) / 256, a.batch), 256, 0, s, a) !=
            cudaSuccess ||
        launch(k_keep_rows<D>, dim3((a.max_n + 127) / 128, a.batch * a.Hkv), 256, 0, s, a) !=
            cudaSuccess)
      return FDMS_ERR_CUDA;
  }
  if (!ok) return FDMS_ERR_CUDA;
  if (p.splits > 1) {
    a.part_o = reinterpret_cast<float*>(ws + p.off_o);
    a.part_ml = reinterpret_cast<float*>(ws + p.off_ml);
  }
  const long long ctas = blocks * a.splits;
  if (ctas >= (1LL << 31)) return FDMS_ERR_UNSUPPORTED;
  if (launch(k_prefill_mma<D>, dim3((unsigned)ctas), L::THREADS, L::SMEM, s, a, maps, out,
             lse) != cudaSuccess)
    return FDMS_ERR_CUDA;
  if (a.splits > 1) {
    if (launch(k_prefill_join<D, true>, dim3((unsigned)(blocks * 8)), 256, 0, s, a, out,
               lse) != cudaSuccess)
      return FDMS_ERR_CUDA;
  }
  return FDMS_OK;
}

template <int D>
fdms_status scores(fdms_cache* c, PrefillArgs a, const Plan& p, uint8_t* ws, const float* lse,
                   float* out, int accumulate, cudaStream_t s) {
  using L = ScoreL<D>;
  ScoreMaps maps;
  const long long B = a.batch, T = a.max_n, Q = a.max_q;
  bool ok = fdms_tensor_map(&maps.q, a.q, {D, a.Hq, Q, B}, {D, (long long)a.Hq * D, Q * a.Hq * D},
                            a.G, kRows / a.G) &&
            fdms_tensor_map(&maps.k, a.k, {D, a.Hkv, T, B},
                            {D, (long long)a.Hkv * D, T * a.Hkv * D}, 1, kKeys);
  maps.kc = maps.k;
  if (p.compact) {
    a.compact = 1;
    a.words = p.words;
    a.bits = reinterpret_cast<uint32_t*>(ws + p.off_bits);
    a.before = reinterpret_cast<uint32_t*>(ws + p.off_before);
    a.kc = reinterpret_cast<uint16_t*>(ws + p.off_kc);
    a.pos = reinterpret_cast<int32_t*>(ws + p.off_pos);
    ok = ok && fdms_tensor_map(&maps.kc, a.kc, {D, 1, T, B * a.Hkv}, {D, D, T * D}, 1, kKeys);
    if (!ok) return FDMS_ERR_CUDA;
    if (launch(k_keep_bits, dim3((a.max_n + 255) / 256, a.batch), 256, 0, s, a) !=
            cudaSuccess ||
        launch(k_keep_rows<D>, dim3((a.max_n + 127) / 128, a.batch * a.Hkv), 256, 0, s, a) !=
            cudaSuccess)
      return FDMS_ERR_CUDA;
  }
  if (!ok) return FDMS_ERR_CUDA;
  ScoreArgs sc = {};
  sc.key_tiles = p.key_tiles;
  sc.chunks = p.chunks;
  sc.chunk_steps = p.chunk_steps;
  sc.lse = lse;
  sc.scores = out;
  sc.accumulate = accumulate;
  const bool join = a.compact || p.chunks > 1;
  if (join) sc.part = reinterpret_cast<float*>(ws + p.off_part);
  const long long items =
      (long long)p.key_tiles * a.batch * a.Hkv * (a.compact ? 2 : 1) * p.chunks;
  if (items >= (1LL << 30)) return FDMS_ERR_UNSUPPORTED;
  if (launch(k_scores_mma<D>, dim3((unsigned)items), L::THREADS, L::SMEM, s, a, sc, maps) !=
      cudaSuccess)
    return FDMS_ERR_CUDA;
  if (join && launch(k_scores_join, dim3((a.max_n + 255) / 256, a.batch * a.Hkv), 256, 0, s, a,
                     sc) != cudaSuccess)
    return FDMS_ERR_CUDA;
  return FDMS_OK;
}

template <int D>
bool setup() {
  auto room = [](auto kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
           cudaSuccess;
  };
  return room(k_prefill_mma<D>, AttnL<D>::SMEM) && room(k_prefill_few<D, 1>, FewL<D>::SMEM) &&
         room(k_prefill_few<D, 2>, FewL<D>::SMEM) && room(k_scores_mma<D>, ScoreL<D>::SMEM);
}

// no queries: zeros
__global__ void __launch_bounds__(256) k_scores_none(PrefillArgs a, float* scores) {
  pdl_wait();
  pdl_launch_dependents();
  const int bh = blockIdx.y, b = bh / a.Hkv, j = blockIdx.x * 256 + threadIdx.x;
  int n, nq;
  if (!lengths(a, b, n, nq)) {
    if (j == 0 && bh % a.Hkv == 0) latch_error(a.ctr, FDMS_ERR_DEVICE);
    return;
  }
  if (j < n) scores[(long long)bh * a.max_n + j] = 0.f;
}

}  // namespace

bool fdms_tensor_map(CUtensorMap* map, const void* base, const long long (&dim)[4],
                     const long long (&stride)[3], int b1, int b2) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)dim[0], (cuuint64_t)dim[1], (cuuint64_t)dim[2],
                              (cuuint64_t)dim[3]};
  const cuuint64_t strides[3] = {(cuuint64_t)stride[0] * 2, (cuuint64_t)stride[1] * 2,
                                 (cuuint64_t)stride[2] * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, unit[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

fdms_status fdms_prefill_setup(fdms_cache* c) {
  return (c->view.D == 64 ? setup<64>() : setup<128>()) ? FDMS_OK : FDMS_ERR_CUDA;
}

extern "C" fdms_status fdms_prefill_workspace_for(fdms_cache* c, int batch, int max_n, int max_q,
                                                  int uses, size_t* bytes_out) {
  if (!c || !bytes_out) return FDMS_ERR_INVALID_ARG;
  *bytes_out = 0;
  if (batch < 0 || batch > c->view.Bmax || max_n < 0 || max_n > c->view.max_seq_len ||
      max_q < 0 || max_q > max_n ||
      (uses & ~(FDMS_FOR_ATTN | FDMS_FOR_SCORES | FDMS_WITH_KEEP)))
    return FDMS_ERR_INVALID_ARG;
  const Plan p = plan_of(c, batch, max_n, max_q, uses & FDMS_WITH_KEEP);
  const size_t attn = uses & FDMS_FOR_ATTN ? p.attn_bytes : 0;
  const size_t scores = uses & FDMS_FOR_SCORES ? p.score_bytes : 0;
  *bytes_out = attn > scores ? attn : scores;
  return FDMS_OK;
}

extern "C" fdms_status fdms_prefill_workspace(fdms_cache* c, int batch, int max_n, int max_q,
                                              size_t* bytes_out) {
  return fdms_prefill_workspace_for(c, batch, max_n, max_q,
                                    FDMS_FOR_ATTN | FDMS_FOR_SCORES | FDMS_WITH_KEEP, bytes_out);
}

extern "C" fdms_status fdms_prefill_attn(fdms_cache* c, int batch, const int32_t* n_dev, int max_n,
                                         const int32_t* nq_dev, int max_q, const void* q_dev,
                                         const void* k_dev, const void* v_dev,
                                         const uint8_t* keep_dev, void* out_dev, float* lse_dev,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!c) return FDMS_ERR_INVALID_ARG;
  fdms_status st = check(c, batch, n_dev, max_n, nq_dev, max_q, q_dev, k_dev);
  if (st != FDMS_OK) return st;
  if (batch == 0 || max_q == 0) return FDMS_OK;
  if (!v_dev || !out_dev || (((uintptr_t)v_dev | (uintptr_t)out_dev) & 15))
    return FDMS_ERR_INVALID_ARG;
  const Plan p = plan_of(c, batch, max_n, max_q, keep_dev != nullptr);
  if (p.attn_bytes > 0 &&
      (!workspace || workspace_bytes < p.attn_bytes || ((uintptr_t)workspace & 255)))
    return FDMS_ERR_INVALID_ARG;
  fdms_device_guard guard(c->device);
  const PrefillArgs a =
      args_of(c, batch, n_dev, max_n, nq_dev, max_q, q_dev, k_dev, v_dev, keep_dev);
  auto run = c->view.D == 64 ? attn<64> : attn<128>;
  return run(c, a, p, static_cast<uint8_t*>(workspace), static_cast<uint16_t*>(out_dev), lse_dev,
             static_cast<cudaStream_t>(stream));
}

extern "C" fdms_status fdms_prefill_scores(fdms_cache* c, int batch, const int32_t* n_dev,
                                           int max_n, const int32_t* nq_dev, int max_q,
                                           const void* q_dev, const void* k_dev,
                                           const uint8_t* keep_dev, const float* lse_dev,
                                           float* scores_dev, int accumulate, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (!c) return FDMS_ERR_INVALID_ARG;
  fdms_status st = check(c, batch, n_dev, max_n, nq_dev, max_q, q_dev, k_dev);
  if (st != FDMS_OK) return st;
  if (batch == 0 || max_n == 0) return FDMS_OK;
  if (!scores_dev || (max_q > 0 && !lse_dev)) return FDMS_ERR_INVALID_ARG;
  const Plan p = plan_of(c, batch, max_n, max_q, keep_dev != nullptr);
  if (p.score_bytes > 0 &&
      (!workspace || workspace_bytes < p.score_bytes || ((uintptr_t)workspace & 255)))
    return FDMS_ERR_INVALID_ARG;
  fdms_device_guard guard(c->device);
  const PrefillArgs a =
      args_of(c, batch, n_dev, max_n, nq_dev, max_q, q_dev, k_dev, nullptr, keep_dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (max_q == 0) {
    if (accumulate) return FDMS_OK;
    return launch(k_scores_none, dim3((max_n + 255) / 256, batch * a.Hkv), 256, 0, s, a,
                  scores_dev) == cudaSuccess ? FDMS_OK : FDMS_ERR_CUDA;
  }
  auto run = c->view.D == 64 ? scores<64> : scores<128>;
  return run(c, a, p, static_cast<uint8_t*>(workspace), lse_dev, scores_dev, accumulate, s);
}
