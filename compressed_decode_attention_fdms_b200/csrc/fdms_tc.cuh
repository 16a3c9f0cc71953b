// Fifth-generation tensor cores (tcgen05, tensor memory) and tiled TMA copies:
// the instructions and descriptors the prompt kernels use. Not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fdms_internal.cuh"

namespace fdms {

// ------------------------------------------------------------ bounded waits
__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
constexpr unsigned long long kStopNs = 2000000000ull;

// Wait for a phase of `bar`. Gives up after kStopNs, or as soon as another
// thread of the CTA has (`stop`, in shared memory). (Reading the timer after the
// first miss also spaces the tries: polling at once cost the attention of an 8K
// prompt 18 %, 521 -> 613 us.)
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*stop) return false;
    if (global_ns() - t0 > kStopNs) {
      *stop = 1;
      return false;
    }
  }
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// this thread's accesses to shared memory, before what the
// tensor cores and copies do with it
__device__ __forceinline__ void fence_smem_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// one arrival for the warp, after what its lanes did before
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// ------------------------------------------------------------ next work item
// Asks for a CTA of this grid that has not started yet: its index is this CTA's
// next work item, and it is not launched any more. The answer (16 bytes) is
// counted on `bar`.
__device__ __forceinline__ void next_item_ask(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(smem_addr(answer)),
      "r"(smem_addr(bar))
      : "memory");
}
// The index from an answer, or -1: no CTA was left.
__device__ __forceinline__ int next_item_of(const void* answer) {
  int got, x;
  asm volatile(
      "{.reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.s32 %0, 1, 0, p;\n mov.s32 %1, -1;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;}"
      : "=r"(got), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  return got ? x : -1;
}
// The indexes of a persistent CTA's items, for the warp that asks for them: two
// answers in shared memory.
struct ItemQueue {
  uint8_t* answer;          // [2][16]
  uint64_t *full, *empty;   // [2]
  static constexpr int BYTES = 64;
  __device__ __forceinline__ void place(uint8_t* at) {
    answer = at;
    full = reinterpret_cast<uint64_t*>(at + 32);
    empty = full + 2;
  }
  __device__ __forceinline__ void init() {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
  }
  // the asking warp: ask for the item after item i (of this CTA)
  __device__ __forceinline__ bool ask(int i, volatile int* stop) {
    if (i >= 2 &&
        !__all_sync(0xffffffffu, bar_wait(empty + i % 2, (i / 2 - 1) & 1, stop)))
      return false;
    if (threadIdx.x % 32 == 0) {
      mbar_arrive_expect_tx(full + i % 2, 16);
      next_item_ask(answer + i % 2 * 16, full + i % 2);
    }
    return true;
  }
  // the asking warp: the item after item i, or -1
  __device__ __forceinline__ int next(int i, volatile int* stop) {
    if (!__all_sync(0xffffffffu, bar_wait(full + i % 2, (i / 2) & 1, stop))) return -1;
    const int x = next_item_of(answer + i % 2 * 16);
    fence_smem_async();
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(empty + i % 2);
    return x;
  }
};
// Items that one warp describes and the others read: two places in shared memory.
template <class Item>
struct ItemBoard {
  Item* item;               // [2]
  uint64_t *full, *empty;   // [2]
  static constexpr int BYTES = 2 * sizeof(Item) + 32;
  static_assert(sizeof(Item) % 8 == 0, "barriers follow the items");
  __device__ __forceinline__ void place(uint8_t* at) {
    item = reinterpret_cast<Item*>(at);
    full = reinterpret_cast<uint64_t*>(item + 2);
    empty = full + 2;
  }
  __device__ __forceinline__ void init(int readers) {   // warps that read
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, readers);
    }
  }
  // the describing warp: item i
  __device__ __forceinline__ bool put(int i, const Item& x, volatile int* stop) {
    if (i >= 2 &&
        !__all_sync(0xffffffffu, bar_wait(empty + i % 2, (i / 2 - 1) & 1, stop)))
      return false;
    if (threadIdx.x % 32 == 0) {
      item[i % 2] = x;
      mbar_arrive(full + i % 2);
    }
    return true;
  }
  // every reading warp, in turn: item i, to be read until done(i), or NULL
  __device__ __forceinline__ const Item* get(int i, volatile int* stop) {
    return __all_sync(0xffffffffu, bar_wait(full + i % 2, (i / 2) & 1, stop)) ? item + i % 2
                                                                              : nullptr;
  }
  __device__ __forceinline__ void done(int i) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(empty + i % 2);
  }
};

// ------------------------------------------------------------ tiled TMA
// One box of a 4-d tensor map into this CTA's shared memory.
__device__ __forceinline__ void tma_box4(void* dst, const CUtensorMap* map, int c0, int c1, int c2,
                                         int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ------------------------------------------------------------ tensor memory
__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst_smem)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// arrival on `bar` once every tensor-core operation this thread issued is done
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
// 32 columns of this warp's 32 lanes (lane i of the warp: tensor memory lane 32 (warp % 4) + i)
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// the same for 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Registers of the calling warpgroup's threads (every warp of it calls).
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------ matrix products
// Shared-memory operand in the 128-byte swizzle: rows of 128 bytes, groups of
// eight rows 1024 bytes apart. K-major operands (rows of 64 K values) leave
// `lead` unused; for an operand whose rows run along M or N, `lead` is the
// distance from one 64-value column block to the next.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// One lane of the warp, the same one each time (every lane calls). Products are
// issued under it: their descriptors then come from uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{.reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;}" : "=r"(on));
  return on != 0;
}
// bf16 x bf16 -> fp32, A K-major, B K-major or (b_rows_n) with rows along N
__host__ __device__ constexpr uint32_t mma_desc(int M, int N, bool b_rows_n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_rows_n ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// D (tensor memory) = A B, or += with `add`; A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{.reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// the same with A in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{.reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// two fp32 -> packed bf16 (x0 in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x1), "f"(x0));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
      " add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
      " mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// x clamped to [lo, hi], NaN kept
__device__ __forceinline__ float clamp_nan(float x, float lo, float hi) {
  float y;
  asm("{.reg .f32 t;\n max.NaN.f32 t, %1, %2;\n min.NaN.f32 %0, t, %3;}"
      : "=f"(y) : "f"(x), "f"(lo), "f"(hi));
  return y;
}
// 2^x of a pair on the multiply-add pipe, for kernels that the special-function
// unit (4 results a cycle and SM quarter) holds up: x = r + f with r whole and
// |f| <= 1/2, 2^f by a polynomial of degree 5 (least relative error over
// [-1/2, 1/2], found by weighted least squares; 2.1e-7 with fp32 steps, as good
// as the unit's), times 2^r put together in the exponent's bits: exact zeros where
// r is -127 (x below -126.5), infinity where it is 128 (from 127.5 up), NaN kept.
__device__ __forceinline__ float2 exp2_mad(float2 x) {
  const float big = 12582912.f;   // 1.5 * 2^23: adding it rounds to a whole number
  x.x = clamp_nan(x.x, -127.f, 128.f);
  x.y = clamp_nan(x.y, -127.f, 128.f);
  const float2 t = add2(x, make_float2(big, big));
  const float2 r = add2(t, make_float2(-big, -big));
  const float2 f = ffma2(r, make_float2(-1.f, -1.f), x);
  float2 p = ffma2(f, make_float2(1.3276472454890609e-3f, 1.3276472454890609e-3f),
                   make_float2(9.675540961325169e-3f, 9.675540961325169e-3f));
  p = ffma2(f, p, make_float2(5.550713092088699e-2f, 5.550713092088699e-2f));
  p = ffma2(f, p, make_float2(0.24022120237350464f, 0.24022120237350464f));
  p = ffma2(f, p, make_float2(0.6931469440460205f, 0.6931469440460205f));
  p = ffma2(f, p, make_float2(1.0000001192092896f, 1.0000001192092896f));
  return mul2(p, make_float2(
                     __uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                     __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u)));
}

}  // namespace fdms

// Host: a tensor map of bf16 rows [d3][d2][d1][d0], strides in elements of dims 1..3,
// boxes of b0 (64 values, the 128-byte swizzle), b1, b2, 1. False when the
// driver refuses it.
bool fdms_tensor_map(CUtensorMap* map, const void* base, const long long (&dim)[4],
                     const long long (&stride)[3], int b1, int b2);
