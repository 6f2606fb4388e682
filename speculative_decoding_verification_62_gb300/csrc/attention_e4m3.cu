// Attention of a verify step's rows over a paged cache of e4m3 codes with a scale for each
// block of tokens and key head.
//
//   s_j = c f q8.k8_j ks_j,  t_j = (s_j - m) + log2 vs_j,  w_j = 2^t_j
//   o = sum_j w_j v8_j / sum_j (w_j / vs_j)
// in one pass over the keys, with a maximum m of s + log2 vs that moves now and then; c is the scale
// times log2(e), f a power of two of the query row.  A key's scales are one thread's two
// registers: keys lie along the lanes, so both products are turned over,
//   S^T [128 keys][rows] = K Q^T,   O^T [D][rows] += V^T W^T,
// and the codes go from memory to the tensor cores as they are: no key or value is ever
// widened.  The other operands are sums of 8-bit floats:
// - queries: q / f = e4m3 + e5m2 (bf16: exact for values within 2^-13 of the row's largest, and
//   off by 2^-21 of it at most), fp16 a second e5m2;
// - weights: rounded to fp16, that to the nearest e5m2, what is left to the nearest again, and what is left
//   then, 2^-7 of the weight's power of two at most and a multiple of 2^-10 of it, is an e5m2: the sum is
//   the fp16, off by 2^-11 of the weight at most.  (With the first two cut off instead of rounded,
//   three terms hold nine of its eleven bits.)  The maximum of the weights lies in [2^13, 2^15] at all times
//   after its tile, so that e5m2's smallest step, 2^-16, is 2^-29 of it.  (Of scores near 2^27 it lies in
//   [2^-3, 2^15]: the maximum itself is a multiple of 16 there.)
// Each product is two or three products of kind::f8f6f4, into one 32-bit accumulator.
//
// Work: a unit is (request, up to kN rows of queries, key head) over the request's own keys, or
// (kN of all rows, key head) over the shared prefix; the rows of a key head are its
// query heads', token by token, and a block of them begins anywhere.  The units'
// tiles of 128 keys form one list (and a unit's start counts as kStart tiles); every CTA,
// two an SM, takes an equal contiguous share.  A unit that crosses a border leaves a part a share, and
// join_kernel adds them up with the prefix's, in list order: results repeat bit for bit.
//
// A CTA: a warpgroup for the softmax, a warp that issues the products, two that copy keys
// and values by TMA (a page's tokens of up to 128 a box, 128 bytes a token, 128-byte
// swizzle).  The next tile's scores are formed beside this one's softmax; a CTA's
// waits are filled by the other of its SM.
//
// Bound: the codes, read once (one request of 131000 tokens, 8 key heads of 128: 268 MB).
// Measured far from it: that request takes 137 us (39.5 at the copy rate), 256 requests of up to
// 5000 tokens 598 (197), at 36 % and (64 of them) 25 % of the issue slots and 15 % and 6 % of the
// tensor pipe: a tile's steps, scores, weights, moves of the maximum, wait for one another.
// The list counts a tile as one whatever its columns: behind a prefix (64 columns a tile beside
// 16) the busiest SM works 1.6 times as long as the average.
#include "../../include/spec_verify.h"
#include "internal.h"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

namespace {

constexpr int kTile = 128;     // keys a tile: the lanes of a product
constexpr int kThreads = 256;  // warps 0-3: softmax; 4: keys; 5: products; 6: values
constexpr int kMaxCtas = 320;  // CTAs at most (the slots of parts are sized for this)
constexpr int kSlots = 2 * kMaxCtas;
constexpr int kStages = 2;     // tiles of keys, and of values, on their way
// A unit's start and end, in tiles.  us with 1, 2, 3, 4: one request of 131000 tokens 150, 137, 153, 150; 37 of a
// key head a query head 74, 63, 60, 56; 32 behind a prefix 80, 80, 72, 80; 256 long ones 594, 600, 590, 586.
constexpr int kStart = 2;
constexpr int kTileBytes = kTile * 128;
constexpr int kMaxKeys = INT32_MAX - 4096;  // keys of a request: the last tile's places fit 32 bits
constexpr int kMaxList = 1 << 30;
constexpr float kNone = -3.0e38f;  // a maximum of nothing
constexpr float kTop = 13.f;       // log2 of the largest weight where the maximum just moved
constexpr float kLimit = 15.f;     // and where it moves (11 and 15: 577 us for 600 with 256 long
                                   // requests, and weights good to 2^-28 of the largest, not 2^-30)
constexpr float kFar = 0x1p20f;    // logarithms from here on are rounded by 2^-4 and more
constexpr unsigned long long kDrainNs = 2000000000ull;  // limit of the waits that end an aborted CTA

template <typename T>
struct Shape;
template <>
struct Shape<__nv_bfloat16> {
  static constexpr int terms = 2, chunks = 4;  // of a query; columns of a block, in sixteens
};
template <>
struct Shape<__half> {
  static constexpr int terms = 3, chunks = 3;
};
template <typename T>
struct Smem {
  static constexpr int n = 16 * Shape<T>::chunks;
  static constexpr int q_term = n * 128, q_bytes = Shape<T>::terms * q_term;
  static constexpr int w_term = n * 128, w_bytes = 3 * w_term;
  static constexpr int ring = 2 * kStages * kTileBytes;
  static constexpr int control = 3 * 1024;
  static constexpr int bytes = ring + q_bytes + w_bytes + control;
  static_assert(bytes <= 113 * 1024, "two CTAs an SM");
};

struct Params {
  int B, T, G, total, Hq, Hk, D, group, n;  // n: rows of a block
  int num_pages, page_size, page_shift, block_shift, per_page, max_pages, box_rows, max_keys;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  const int32_t* prefix_table;
  const float* k_scales;
  const float* v_scales;
  int prefix_len, prefix_tiles, prefix_blocks;
  const uint32_t* mask;
  float sl2;  // scale log2(e)
  const char* q;
  long long q_row, q_head;  // elements
  char* out;
  float* lse;
  unsigned int* status;
  int* starts;     // [B + 1]: where each request begins in the list, and the list's end
  float* own;      // [T][Hq][D]: whole units over own keys, where there is a prefix
  float* own_lse;
  float* pre;      // whole units over the prefix
  float* pre_lse;
  float* slot;     // [kSlots][n][D]: parts of units
  float* slot_lse;
  unsigned long long wait_ns;
};

// ---------------------------------------------------------------------------
// sm_103a instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for a phase, at most wait_ns; false (and *abort set) when that ran out or
// another warp of the CTA gave up.
__device__ __forceinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, unsigned long long wait_ns,
                                              volatile int* abort) {
  // ordinary waits end within the first tries (a try suspends the warp for a while
  // itself) and read no timer; a limit below 1 ms is looked at after every try
  const int tries = wait_ns >= 1000000ull ? 64 : 1;
  if (tries > 1) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (bar_try(bar, parity)) return true;
  }
  const unsigned long long t0 = now_ns();
#pragma unroll 1
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < tries; ++i)
      if (bar_try(bar, parity)) return true;
    if (*abort) return false;
    if (now_ns() - t0 > wait_ns) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned long long wait_ns,
                                         volatile int* abort) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, wait_ns, abort);
}
// Barrier of the softmax's 128 threads: whether any of them says so.
__device__ __forceinline__ bool any_of(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, 1, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(0), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// One thread of the warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// D = A B (+ D): 32 codes along the sum
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Four such steps in one block of text, so that operands move to uniform registers once.
template <int A, int B>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(A), "n"(B)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
#define SV_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), \
                    "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define SV_W8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), \
                    "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
#define SV_T8(v, o) "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), \
                    "+r"(v[o + 5]), "+r"(v[o + 6]), "+r"(v[o + 7])
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : SV_R8(v, 0), SV_R8(v, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      SV_W8(v, 0), SV_W8(v, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Keeps the uses of loaded values behind the wait for them.
__device__ __forceinline__ void tmem_loaded16(uint32_t* v) { asm volatile("" : SV_T8(v, 0), SV_T8(v, 8)); }
// pairs of floats in one instruction
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Shared-memory matrix descriptors (version 1): 128-byte swizzle, rows of 128 bytes, eight of
// them 1024 bytes apart; and no swizzle, eight rows of 16 bytes together, the next eight 128
// bytes on, the next 16 of a row's bytes `stride` bytes on.
__device__ __forceinline__ uint64_t swizzled(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
__device__ __forceinline__ uint64_t plain(uint32_t addr, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46);
}
// 32-bit accumulators, 128 rows, n columns; formats 0: e4m3, 1: e5m2; operands along the sum
// or across it (mn)
__device__ __forceinline__ uint32_t instr_desc(uint32_t b_format, uint32_t n, bool mn) {
  return (1u << 4) | (b_format << 10) | (mn ? 3u << 15 : 0u) | ((n / 8) << 17) | ((uint32_t)(kTile / 16) << 24);
}

// 8-bit floats, a in the low byte, and back
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_half(uint32_t h) {
  unsigned short r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ float2 of_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ float2 of_e5m2x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((unsigned short)c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// The nearest e5m2 of two halves (ties away from zero), in their upper bytes: half a step of those on
// top of the bits.  (A NaN turns into -0 here, and stays with what is left.)
__device__ __forceinline__ uint32_t nearest_e5m2(uint32_t h) { return h + 0x00800080u; }
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <typename T>
struct Type;
template <>
struct Type<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ __nv_bfloat16 down(float a) { return __float2bfloat16_rn(a); }
  static __device__ __forceinline__ uint32_t down2(float a, float b) {
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};
template <>
struct Type<__half> {
  static __device__ __forceinline__ float2 up(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ __half down(float a) { return __float2half_rn(a); }
  static __device__ __forceinline__ uint32_t down2(float a, float b) {
    __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};

// ---------------------------------------------------------------------------
// The tile list
// ---------------------------------------------------------------------------
struct Req {
  int row0, n, kv;  // first row; rows (0: skipped); own keys before the step
};
__device__ __forceinline__ Req request(const Params& P, int b, unsigned int& flags) {
  const int c0 = P.cu[b], c1 = P.cu[b + 1], kv = P.kv_len[b];
  if (c0 < 0 || c1 < c0 || c1 - c0 > P.G || c1 > P.total) {
    flags |= SV_STATUS_BAD_GAMMA;
    return Req{0, 0, 0};
  }
  if (kv < 0 || (long long)kv + (c1 - c0) + 1 > P.max_keys) {
    flags |= SV_STATUS_BAD_LENGTH;
    return Req{0, 0, 0};
  }
  return Req{c0 + b, c1 - c0 + 1, kv};
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
// blocks of a request's rows, and the keys that block i sees (by mask word: any row of the step)
__device__ __forceinline__ int blocks_of(const Params& P, const Req& r) {
  return (int)(((long long)r.n * P.group + P.n - 1) / P.n);
}
__device__ __forceinline__ int block_keys(const Params& P, const Req& r, int i) {
  const long long last = ((long long)(i + 1) * P.n + P.group - 1) / P.group;
  return r.kv + (!P.mask && last < r.n ? (int)last : r.n);
}
// The host refuses sizes whose lists could reach kMaxList where requests have rows of
// their own; inconsistent cu_draft entries (0, n, 0, n, ..) name the same rows again and
// again, so lengths are summed up to that and no further.
__device__ __forceinline__ int list_add(int a, int b) {
  return (int)min((unsigned int)a + (unsigned int)b, (unsigned int)kMaxList);
}
// Of a key head, the tiles of a request's first `blocks` row blocks, none of them its last:
// the sum over i of ceil((kv + ceil((i + 1) n / group)) / 128), which is
// floor((a i + b) / m) with a = n, m = 128 group and b = kv group + n + m - 1.  A sum of
// such terms is its whole parts and what counts the whole numbers below a line, which are
// the same counted by rows: Euclid's steps on (a, m).
__device__ __noinline__ long long blocks_sum(long long kv, int rows, int group, int blocks) {
  unsigned long long n = blocks, m = (unsigned long long)kTile * group, a = rows, b = kv * group + rows + m - 1, sum = 0;
#pragma unroll 1
  for (;;) {
    const unsigned long long qa = a / m, qb = b / m;
    sum += n * (n - 1) / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const unsigned long long top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top - n * m;
    const unsigned long long t = a;
    a = m;
    m = t;
  }
  return (long long)sum;
}
// ... and their starts
__device__ __forceinline__ int blocks_before(const Params& P, const Req& r, int blocks) {
  if (blocks == 0) return 0;
  const int tiles = P.mask ? blocks * tiles_of(r.kv + r.n) : (int)blocks_sum(r.kv, P.n, P.group, blocks);
  return tiles + blocks * kStart;
}
// A request's length in the list (below kMaxList).
__device__ __forceinline__ int request_tiles(const Params& P, const Req& r) {
  if (r.n <= 0) return 0;
  return (tiles_of(r.kv + r.n) + kStart + blocks_before(P, r, blocks_of(P, r) - 1)) * P.Hk;
}
__device__ __forceinline__ int prefix_list(const Params& P) {
  return P.prefix_blocks * P.Hk * (P.prefix_tiles + kStart);
}

// A run of tiles of one unit.
struct Piece {
  bool prefix;
  int b, h;
  int row0, rows;  // the rows' first token row, and rows x heads of the group behind it
  int r0, cols;    // the block's first of them, and how many
  int kv;          // own: keys before the step
  int keys, t0, t1, unit_t;
};

// Walks a share.  Every role walks it alone, from the same start.
struct Walk {
  int left, unit, b, i, h, off;  // unit: of the prefix, -1 behind it; i: block of rows
  Req r;
  __device__ __forceinline__ void load_request(const Params& P) {
    unsigned int ignored = 0;
    r = Req{0, 0, 0};
#pragma unroll 1
    for (; b < P.B; ++b) {
      r = request(P, b, ignored);
      if (r.n > 0) return;
    }
  }
  __device__ __forceinline__ bool next(const Params& P, Piece& p) {
    if (left <= 0) return false;
    if (unit >= P.prefix_blocks * P.Hk) {
      unit = -1;
      b = i = h = 0;
      load_request(P);
    }
    p.prefix = unit >= 0;
    if (p.prefix) {
      const int blk = unit / P.Hk;
      p.b = p.row0 = p.kv = 0;
      p.h = unit - blk * P.Hk;
      p.r0 = blk * P.n;
      p.rows = P.T * P.group;
      p.keys = P.prefix_len;
    } else {
      if (b >= P.B) return false;
      p.b = b;
      p.h = h;
      p.row0 = r.row0;
      p.r0 = i * P.n;
      p.rows = r.n * P.group;
      p.kv = r.kv;
      p.keys = block_keys(P, r, i);
    }
    p.cols = p.rows - p.r0 < P.n ? p.rows - p.r0 : P.n;
    p.unit_t = tiles_of(p.keys);
    const int all = p.unit_t + kStart;
    const int end = left < all - off ? off + left : all;
    p.t0 = off > kStart ? off - kStart : 0;
    p.t1 = end > kStart ? end - kStart : 0;
    left -= end - off;
    off = 0;
    if (p.t1 == p.t0) return false;  // the share ends in the unit's start
    if (p.prefix) {
      ++unit;
    } else if (++h == P.Hk) {
      h = 0;
      if ((long long)++i * P.n >= (long long)r.n * P.group) {
        i = 0;
        ++b;
        if (left > 0) load_request(P);
      }
    }
    return true;
  }
};

struct Control {
  uint64_t kv_full[2][kStages], kv_empty[2][kStages];  // keys, values
  uint64_t q_full, s_full[2], p_ready, pv_done, drain;
  uint32_t tmem;
  int abort, far;  // far: of the last moves of the maxima, one was by kFar or more
  unsigned int copied[2];
  int scan[kThreads / 32];
  Walk start;
  // of a block's columns
  alignas(16) float factor[64], neg[64];  // f c; less the maximum, 0 while there is none
  alignas(16) float top[64], scale[64];   // the maximum; what the sums shrink by, 1 / sum
  alignas(16) float most[4][64];                     // the warps' maxima, or sums
  int limit[64];                                     // own: keys below this are seen, or the mask word
  long long at[64];                                  // row and head of the output
};
static_assert(sizeof(Control) <= 3 * 1024, "control block");

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Params& P, Control* c) {
  const bool ok = bar_wait(smem_addr(bar), parity, P.wait_ns, &c->abort);
  return __all_sync(0xffffffffu, ok);
}

// Copies keys (v = 0) or values (1).
__device__ __forceinline__ void copy_role(const Params& P, Walk w, Control* c, int v, uint32_t ring,
                                          const CUtensorMap* map) {
  const int lane = threadIdx.x & 31;
  unsigned int flags = 0, n = 0;  // tiles so far
  Piece p;
  bool ok = true;
#pragma unroll 1
  while (ok && w.next(P, p)) {
    const int32_t* table = p.prefix ? P.prefix_table : P.table + (size_t)p.b * P.max_pages;
    // a lane's page of a tile (a box is at most a page), as the table has it
    auto look_up = [&](int t) {
      const int x = lane * P.box_rows;
      const long long key = (long long)t * kTile + x;
      return t < p.t1 && x < kTile && key < p.keys ? table[key >> P.page_shift] : 0;
    };
    int ahead = look_up(p.t0);
#pragma unroll 1
    for (int t = p.t0; t < p.t1; ++t, ++n) {
      int id = ahead;
      if (id < 0 || id >= P.num_pages) {
        flags |= SV_STATUS_BAD_PAGE;
        id = P.num_pages;  // past the pool: the copy fills zeros
      }
      ahead = look_up(t + 1);  // on its way while this tile's copies are issued
      const int key0 = t * kTile;
      const int keys = p.keys - key0 < kTile ? p.keys - key0 : kTile;
      const int stage = n % kStages;
      if (!(ok = warp_wait(&c->kv_empty[v][stage], (n / kStages & 1) ^ 1, P, c))) break;
      const uint32_t bar = smem_addr(&c->kv_full[v][stage]);
      uint32_t dst = ring + (2 * stage + v) * kTileBytes;
      if (elect_one()) bar_expect(bar, (uint32_t)((keys + P.box_rows - 1) & -P.box_rows) * 128);
      int lane_of = 0;
#pragma unroll 1
      for (int x = 0; x < keys; x += P.box_rows, dst += P.box_rows * 128, ++lane_of) {
        const int page = __shfl_sync(0xffffffffu, id, lane_of);
        if (elect_one()) tma_load(dst, map, bar, (key0 + x) & (P.page_size - 1), p.h, page);
      }
      __syncwarp();
    }
  }
  if (lane == 0) c->copied[v] = n;
  const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && any && v == 0) atomicOr(P.status, any);
}

// columns of a block that are worked on, in sixteens: the softmax is built for 1, 2 and all
template <typename T>
__device__ __forceinline__ int chunks_of(int cols) {
  return cols <= 16 ? 1 : cols <= 32 ? 2 : Shape<T>::chunks;
}

// The products, by one thread.
template <typename T>
__device__ __forceinline__ void matrix_role(const Params& P, Walk w, Control* c, uint32_t ring, uint32_t q, uint32_t ws) {
  if (!elect_one()) return;
  constexpr int kTerms = Shape<T>::terms;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return bar_wait(smem_addr(bar), parity, P.wait_ns, &c->abort); };
  const uint32_t s_col = c->tmem, o_col = c->tmem + 128;
  const int steps = (P.D + 31) / 32;
  unsigned int pieces = 0, nk = 0, nv = 0;  // tiles of keys and of values so far
  Piece p;
  bool ok = true;
#pragma unroll 1
  while (ok && w.next(P, p)) {
    const int n = p.t1 - p.t0, cols = 16 * chunks_of<T>(p.cols);
    const uint32_t qk0 = instr_desc(0, cols, false), qk1 = instr_desc(1, cols, false), pv = instr_desc(1, cols, true);
    auto scores = [&]() {
      const int stage = nk % kStages;
      if (!(ok = wait(&c->kv_full[0][stage], nk / kStages & 1))) return;
      const uint64_t a = swizzled(ring + 2 * stage * kTileBytes);
      const uint32_t d = s_col + (nk & 1) * 64;
#pragma unroll
      for (int x = 0; x < kTerms; ++x) {
        const uint64_t b = swizzled(q + x * Smem<T>::q_term);
        const uint32_t desc = x == 0 ? qk0 : qk1;
        if (steps == 4) {
          mma4<2, 2>(d, a, b, desc, x > 0);
        } else {
#pragma unroll 1
          for (int k = 0; k < steps; ++k) mma(d, a + 2 * k, b + 2 * k, desc, x > 0 || k > 0);
        }
      }
      mma_commit(smem_addr(&c->kv_empty[0][stage]));
      mma_commit(smem_addr(&c->s_full[nk & 1]));
      ++nk;
    };
    if (!(ok = wait(&c->q_full, pieces & 1))) break;
    scores();
    if (ok && n > 1) scores();
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      const int stage = nv % kStages;
      int keys = p.keys - (p.t0 + i) * kTile;
      keys = keys < kTile ? keys : kTile;
      if (!(ok = wait(&c->kv_full[1][stage], nv / kStages & 1))) break;
      if (!(ok = wait(&c->p_ready, nv & 1))) break;
      fence_after();
      const uint64_t a = swizzled(ring + (2 * stage + 1) * kTileBytes);
      const int groups = (keys + 31) / 32;
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        const uint64_t b = plain(ws + x * Smem<T>::w_term, kTile * 16);
        if (groups == 4) {
          mma4<256, 32>(o_col, a, b, pv, i > 0 || x > 0);
        } else {
#pragma unroll 1
          for (int k = 0; k < groups; ++k) mma(o_col, a + 256 * k, b + 32 * k, pv, i > 0 || x > 0 || k > 0);
        }
      }
      mma_commit(smem_addr(&c->kv_empty[1][stage]));
      mma_commit(smem_addr(&c->pv_done));
      ++nv;
      if (i + 2 < n) scores();
    }
    ++pieces;
  }
}

// A key's two scales
struct Scales {
  float k, v;
};

// What the softmax's threads keep between pieces.
struct SoftState {
  unsigned int tiles, flags;
  bool ok;
};

// The queries of a block into shared memory, as 8-bit floats: eight values a lane, half
// a warp a row.  Rows behind the last are zeros.
template <typename T>
__device__ __forceinline__ void queries(const Params& P, const Piece& p, Control* c, unsigned char* q_smem, int cols) {
  constexpr int kTerms = Shape<T>::terms;
  const int tid = threadIdx.x, in = tid & 15, first = tid >> 4;
  const int d = in * 8;
#pragma unroll 1
  for (int x0 = first; x0 < cols; x0 += 32) {  // four rows under way
    uint4 w[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int n = x0 + 8 * y;
      w[y] = make_uint4(0, 0, 0, 0);
      if (n < p.cols && d < P.D) {
        const int r = p.r0 + n, tok = r / P.group, g = r - tok * P.group;
        w[y] = *reinterpret_cast<const uint4*>(
            P.q + ((long long)(p.row0 + tok) * P.q_row + (long long)(p.h * P.group + g) * P.q_head + d) * 2);
      }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int n = x0 + 8 * y;
      if (n >= cols) break;
      const uint32_t u[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
      float v[8];
      uint32_t top = 0;  // the largest magnitude, as bits: NaN and infinities last
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = Type<T>::up(u[k]);
        v[2 * k] = a.x, v[2 * k + 1] = a.y;
        top = max(top, max(__float_as_uint(a.x) & 0x7fffffffu, __float_as_uint(a.y) & 0x7fffffffu));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // q 2^e has its largest in [2^7, 2^8) (from 2^-93 on)
      int e = 134 - (int)(top >> 23);
      e = top == 0 ? 0 : e > 100 ? 100 : e < -120 ? -120 : e;
      const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t code[kTerms][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a = v[2 * k] * up, b = v[2 * k + 1] * up;
        code[0][k] = e4m3x2(a, b);
        float2 back = of_e4m3x2(code[0][k]);
#pragma unroll
        for (int x = 1; x < kTerms; ++x) {
          a -= back.x, b -= back.y;
          code[x][k] = e5m2x2(a, b);
          back = of_e5m2x2(code[x][k]);
        }
      }
      const bool finite = top < 0x7f800000u;
      unsigned char* at = q_smem + (n >> 3) * 1024 + (n & 7) * 128 + (((in >> 1) ^ (n & 7)) * 16) + (in & 1) * 8;
#pragma unroll
      for (int x = 0; x < kTerms; ++x)
        *reinterpret_cast<uint2*>(at + x * Smem<T>::q_term) =
            finite ? make_uint2(code[x][0] | (code[x][1] << 16), code[x][2] | (code[x][3] << 16))
                   : make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      if (in == 0) c->factor[n] = fminf(P.sl2 * down, 0x1p127f);  // (finite: keys of zeros score 0)
    }
  }
}

// One piece, with CH times 16 columns.  A warp that gives up says so at the next barrier that
// all four pass, where all leave.
template <typename T, int CH>
__device__ __forceinline__ void soften(const Params& P, const Piece& p, Control* c, SoftState& st, unsigned char* ring,
                                       unsigned char* w_smem) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t s_col = c->tmem + lanes, o_col = c->tmem + 128 + lanes;
  const int n = p.t1 - p.t0;
  const int32_t* table = p.prefix ? P.prefix_table : P.table + (size_t)p.b * P.max_pages;
  // keys that every row of the block sees
  const int free = p.prefix ? P.prefix_len : P.mask ? p.kv : p.kv + p.r0 / P.group + 1;
  const bool by_word = !p.prefix && P.mask;
  auto look_up = [&](int t) {
    const long long key = (long long)t * kTile + tid;
    return t < p.t1 && key < p.keys ? table[key >> P.page_shift] : -1;
  };
  auto load_scales = [&](int t, int page) {
    Scales s{1.f, 1.f};
    if (page >= 0 && page < P.num_pages) {
      const int in = (t * kTile + tid) & (P.page_size - 1);
      const size_t at = ((size_t)page * P.per_page + (in >> P.block_shift)) * P.Hk + p.h;
      s.k = P.k_scales[at];
      s.v = P.v_scales[at];
    }
    return s;
  };
  Scales ahead = load_scales(p.t0, look_up(p.t0));
  int page_ahead = look_up(p.t0 + 1);
  uint64_t sum[8 * CH];  // of two columns each, this lane's keys
#pragma unroll
  for (int x = 0; x < 8 * CH; ++x) sum[x] = 0;
  bool forced = true;  // a column has no maximum yet
#pragma unroll 1
  for (int i = 0; i < n; ++i, ++st.tiles) {
    const uint32_t tile = st.tiles, buf = tile & 1;
    Scales sc = ahead;
    ahead = load_scales(p.t0 + i + 1, page_ahead);
    page_ahead = look_up(p.t0 + i + 2);
    if (!(sc.k >= 0x1p-32f && sc.k <= 0x1p64f)) sc.k = 1.f, st.flags |= SV_STATUS_BAD_SCALE;
    if (!(sc.v >= 0x1p-32f && sc.v <= 0x1p64f)) sc.v = 1.f, st.flags |= SV_STATUS_BAD_SCALE;
    const float lv = log2f(sc.v), inv_v = 1.f / sc.v;
    const int key = (p.t0 + i) * kTile + tid;
    const bool masked = (p.t0 + i) * kTile + kTile > free;
    st.ok = warp_wait(&c->s_full[buf], tile >> 1 & 1, P, c) && st.ok;
    fence_after();
    uint32_t v[16 * CH];  // log2 of the weights; -inf where a key is not seen
    const uint64_t ks2 = pair(sc.k, sc.k), lv2 = pair(lv, lv);
    // (the maximum comes off inside the multiply-add, so that what is rounded is small where a
    // weight is not)
    auto form = [&]() {
#pragma unroll
      for (int x = 0; x < CH; ++x) tmem_load16(s_col + buf * 64 + 16 * x, v + 16 * x);
      tmem_wait_load();
#pragma unroll
      for (int x = 0; x < CH; ++x) tmem_loaded16(v + 16 * x);
#pragma unroll
      for (int x = 0; x < 16 * CH; x += 4) {
        const float4 f = *reinterpret_cast<const float4*>(c->factor + x), m = *reinterpret_cast<const float4*>(c->neg + x);
        float t[4];
        unpair(pair_add(pair_fma(pair_mul(pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ks2), pair(f.x, f.y),
                                 pair(m.x, m.y)), lv2), t[0], t[1]);
        unpair(pair_add(pair_fma(pair_mul(pair(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), ks2),
                                 pair(f.z, f.w), pair(m.z, m.w)), lv2), t[2], t[3]);
#pragma unroll
        for (int y = 0; y < 4; ++y) v[x + y] = __float_as_uint(t[y]);
      }
      if (masked) {
#pragma unroll
        for (int x = 0; x < 16 * CH; x += 4) {
          const int4 l = *reinterpret_cast<const int4*>(c->limit + x);
          const int limit[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int d = key - p.kv;
            const bool sees = by_word ? d < 0 || (d < 32 && (limit[y] >> d & 1)) : key < limit[y];
            if (!sees) v[x + y] = __float_as_uint(-INFINITY);
          }
        }
      }
    };
    int moves = 0;       // of the maxima, in this tile
    bool moved = false;  // this thread's column
  formed:
    form();
    float over = -INFINITY;
#pragma unroll
    for (int x = 0; x < 16 * CH; x += 2) over = max3(over, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
    if (any_of((over > kLimit && moves < 4) || (moves == 0 ? forced : moves == 1 && c->far) || !st.ok)) {
      // The maxima move, and the logarithms are formed again.  Far from zero the first were rounded, by as
      // much as 16 each way, and so was what moved: it moves once more, by what is small and good now.
      if (any_of(!st.ok)) {
        st.ok = false;
        return;
      }
#pragma unroll
      for (int x = 0; x < 16 * CH; x += 16) {
        float mine = 0.f;
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const float top = warp_max(__uint_as_float(v[x + y]));
          if (lane == y) mine = top;
        }
        if (lane < 16) c->most[warp][x + lane] = mine;
      }
      if (tid == 0) c->far = 0;
      (void)any_of(false);
      if (tid < 16 * CH) {
        // over the old maximum (NaN left out)
        const float top = fmaxf(fmaxf(c->most[0][tid], c->most[1][tid]), fmaxf(c->most[2][tid], c->most[3][tid]));
        const float was = c->top[tid];
        float f = 1.f;
        if (was == kNone ? top > -INFINITY : top > kLimit || (moved && top > -INFINITY)) {
          // (rounded up: no weight passes 2^kTop, but for the rounding of a far `top`)
          const float now = was == kNone ? __fadd_ru(top, -kTop) : __fadd_ru(was, __fadd_ru(top, -kTop));
          f = exp2_fast(was - now);
          moved = true;
          if (fabsf(top) >= kFar) c->far = 1;
          c->top[tid] = now;
          c->neg[tid] = -now;
        }
        c->scale[tid] = f;
      }
      forced = any_of(tid < p.cols && c->top[tid] == kNone);
      if (i > 0) {
        st.ok = warp_wait(&c->pv_done, (tile - 1) & 1, P, c) && st.ok;
        fence_after();
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          uint32_t o[16];
          tmem_load16(o_col + 16 * x, o);
          tmem_wait_load();
          tmem_loaded16(o);
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const float2 f = *reinterpret_cast<const float2*>(c->scale + 16 * x + y);
            o[y] = __float_as_uint(__uint_as_float(o[y]) * f.x);
            o[y + 1] = __float_as_uint(__uint_as_float(o[y + 1]) * f.y);
            sum[8 * x + y / 2] = pair_mul(sum[8 * x + y / 2], pair(f.x, f.y));
          }
          tmem_store16(o_col + 16 * x, o);
        }
        tmem_wait_store();
        fence_before();
      }
      ++moves;
      goto formed;
    }
    if (i > 0) st.ok = warp_wait(&c->pv_done, (tile - 1) & 1, P, c) && st.ok;  // the weights' place is free
    // The value rows behind the last key of its 32 hold what memory held there, and weights of 0
    // times NaN would be NaN: their threads clear them.
    const int keys = p.keys - (p.t0 + i) * kTile;
    if (keys < kTile && (keys & 31)) {
      const int stage = tile % kStages;
      st.ok = warp_wait(&c->kv_full[1][stage], tile / kStages & 1, P, c) && st.ok;
      if (tid >= keys && tid < ((keys + 31) & ~31)) {
        uint4* at = reinterpret_cast<uint4*>(ring + (2 * stage + 1) * kTileBytes + tid * 128);
#pragma unroll
        for (int x = 0; x < 8; ++x) at[x] = make_uint4(0, 0, 0, 0);
      }
    }
    const uint64_t iv2 = pair(inv_v, inv_v);
#pragma unroll
    for (int x = 0; x < CH; ++x) {
      uint32_t h[8];
#pragma unroll
      for (int y = 0; y < 16; y += 4) {
        const uint32_t* t = v + 16 * x + y;
        const float a = exp2_fast(__uint_as_float(t[0])), b = exp2_fast(__uint_as_float(t[1])),
                    e = exp2_fast(__uint_as_float(t[2])), g = exp2_fast(__uint_as_float(t[3]));
        sum[8 * x + y / 2] = pair_fma(pair(a, b), iv2, sum[8 * x + y / 2]);
        sum[8 * x + y / 2 + 1] = pair_fma(pair(e, g), iv2, sum[8 * x + y / 2 + 1]);
        h[y / 2] = half2_of(a, b);
        h[y / 2 + 1] = half2_of(e, g);
      }
      uint4 code[3];
      uint32_t* first = reinterpret_cast<uint32_t*>(code);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t a = h[2 * y], b = h[2 * y + 1];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t an = nearest_e5m2(a), bn = nearest_e5m2(b);
          first[4 * k + y] = __byte_perm(an, bn, 0x7531);
          a = half2_sub(a, an & 0xff00ff00u), b = half2_sub(b, bn & 0xff00ff00u);
        }
        first[8 + y] = __byte_perm(e5m2x2_half(a), e5m2x2_half(b), 0x5410);
      }
#pragma unroll
      for (int y = 0; y < 3; ++y)
        *reinterpret_cast<uint4*>(w_smem + y * Smem<T>::w_term + x * (kTile * 16) + tid * 16) = code[y];
    }
    fence_smem();
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(smem_addr(&c->p_ready));
  }
  // the lanes' sums of a column: halves change hands until a lane has a column's (or two)
  st.ok = warp_wait(&c->pv_done, (st.tiles - 1) & 1, P, c) && st.ok;
  float l[16 * CH];
#pragma unroll
  for (int x = 0; x < 8 * CH; ++x) unpair(sum[x], l[2 * x], l[2 * x + 1]);
#pragma unroll
  for (int x = 0; x < CH; ++x) {
    float* s = l + 16 * x;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const bool upper = lane & o;
#pragma unroll
      for (int y = 0; y < o; ++y) {
        const float give = upper ? s[y] : s[y + o], keep = upper ? s[y + o] : s[y];
        s[y] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 16);
    if (lane < 16) c->most[warp][16 * x + lane] = s[0];
  }
  if (any_of(!st.ok)) {
    st.ok = false;
    return;
  }
  const bool whole = p.t0 == 0 && p.t1 == p.unit_t;
  const bool direct = whole && P.prefix_len == 0;
  const long long slot = 2 * blockIdx.x + (p.t0 == 0 ? 1 : 0);
  float* part = !whole ? P.slot + slot * P.n * P.D : p.prefix ? P.pre : P.own;
  float* part_lse = !whole ? P.slot_lse + slot * P.n : p.prefix ? P.pre_lse : P.own_lse;
  if (tid < p.cols) {
    const float s = c->most[0][tid] + c->most[1][tid] + c->most[2][tid] + c->most[3][tid];
    const float lse2 = c->top[tid] + log2f(s);
    c->scale[tid] = s > 0.f || s != s ? 1.f / s : 0.f;
    if (!direct)
      part_lse[whole ? c->at[tid] : tid] = lse2;
    else if (P.lse)
      P.lse[c->at[tid]] = lse2 * 0.693147180559945309f;
  }
  (void)any_of(false);
  fence_after();
#pragma unroll
  for (int x = 0; x < CH; ++x) {
    uint32_t o[16];
    tmem_load16(o_col + 16 * x, o);
    tmem_wait_load();
    tmem_loaded16(o);
    if (tid < P.D) {
#pragma unroll
      for (int y = 0; y < 16; ++y) {
        if (16 * x + y >= p.cols) break;
        const float inv = c->scale[16 * x + y];
        const float r = inv == 0.f ? 0.f : __uint_as_float(o[y]) * inv;
        if (direct)
          reinterpret_cast<T*>(P.out)[c->at[16 * x + y] * P.D + tid] = Type<T>::down(r);
        else
          part[(whole ? c->at[16 * x + y] : (long long)(16 * x + y)) * P.D + tid] = r;
      }
    }
  }
  fence_before();
}

template <typename T>
__device__ __forceinline__ void softmax_role(const Params& P, Walk w, Control* c, unsigned char* ring,
                                             unsigned char* q_smem, unsigned char* w_smem) {
  const int tid = threadIdx.x;
  SoftState st{0, 0, true};
  Piece p;
#pragma unroll 1
  while (st.ok && w.next(P, p)) {
    (void)any_of(false);  // the last piece's columns have been read
    const int chunks = chunks_of<T>(p.cols);
    if (tid < 16 * chunks) {
      const int r = p.r0 + tid, tok = r / P.group, g = r - tok * P.group;
      c->top[tid] = kNone;
      c->neg[tid] = 0.f;
      c->at[tid] = (long long)(p.row0 + tok) * P.Hq + p.h * P.group + g;
      if (tid >= p.cols)
        c->limit[tid] = 0;
      else
        c->limit[tid] = p.prefix ? P.prefix_len : P.mask ? (int)P.mask[p.row0 + tok] : p.kv + tok + 1;
      // (mask bits behind the step's rows name keys behind the request's)
      if (!p.prefix && P.mask && p.keys - p.kv < 32) c->limit[tid] &= (1 << (p.keys - p.kv)) - 1;
    }
    queries<T>(P, p, c, q_smem, 16 * chunks);
    fence_smem();
    (void)any_of(false);
    if (tid == 0) bar_arrive(smem_addr(&c->q_full));
    if (chunks == 1)
      soften<T, 1>(P, p, c, st, ring, w_smem);
    else if (chunks == 2)
      soften<T, 2>(P, p, c, st, ring, w_smem);
    else
      soften<T, Shape<T>::chunks>(P, p, c, st, ring, w_smem);
  }
  const unsigned int any = __reduce_or_sync(0xffffffffu, st.flags);
  if ((tid & 31) == 0 && any) atomicOr(P.status, any);
}

struct Maps {
  CUtensorMap k, v;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) attention8_kernel(const __grid_constant__ Maps maps,
                                                                 const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = Smem<T>;
  unsigned char* q_smem = smem + S::ring;
  unsigned char* w_smem = q_smem + S::q_bytes;
  Control* c = reinterpret_cast<Control*>(w_smem + S::w_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_addr(smem) & 1023) {  // the swizzle's period; never expected
    if (tid == 0) atomicOr(P.status, (unsigned int)SV_STATUS_INTERNAL);
    return;
  }
  // what needs no input is set up before the kernel ahead in the stream has ended
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_addr(&c->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else if (warp == 4 && lane < 2) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &maps.v : &maps.k) : "memory");
  } else if (tid == kThreads - 1) {
    c->abort = 0;
    c->copied[0] = c->copied[1] = 0;
    c->start.left = 0;
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < kStages; ++s) {
        bar_init(smem_addr(&c->kv_full[i][s]), 1);
        bar_init(smem_addr(&c->kv_empty[i][s]), 1);
      }
      bar_init(smem_addr(&c->s_full[i]), 1);
    }
    bar_init(smem_addr(&c->q_full), 1);
    bar_init(smem_addr(&c->p_ready), 4);
    bar_init(smem_addr(&c->pv_done), 1);
    bar_init(smem_addr(&c->drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the requests' tiles, scanned
  unsigned int flags = 0;
  const int chunk = (P.B + kThreads - 1) / kThreads;
  const int b0 = tid * chunk < P.B ? tid * chunk : P.B;
  const int b1 = b0 + chunk < P.B ? b0 + chunk : P.B;
  Req r{0, 0, 0};  // the thread's last request
  int mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    r = request(P, b, flags);
    mine = list_add(mine, request_tiles(P, r));
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = list_add(incl, v);
  }
  if (lane == 31) c->scan[warp] = incl;
  fence_before();
  __syncthreads();
  fence_after();
  const int before = prefix_list(P);
  int excl = list_add(before, incl - mine), total = before;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int v = c->scan[i];
    if (i < warp) excl = list_add(excl, v);
    total = list_add(total, v);
  }
  const bool over = total >= kMaxList;  // no request's rows are worked on
  if (over) {
    total = before;
    flags |= SV_STATUS_BAD_GAMMA;
  }
  const int per = (int)(((long long)total + gridDim.x - 1) / gridDim.x);
  // where the share begins, found by the thread whose requests hold it
  const long long g0 = (long long)per * blockIdx.x;
  const int left = total - g0 < per ? (int)(total - g0) : per;
  if (left > 0 && (g0 < before ? tid == 0 : !over && g0 >= excl && g0 < excl + mine)) {
    Walk w{left, -1, 0, 0, 0, 0, r};
    if (g0 < before) {
      const int t = P.prefix_tiles + kStart;
      w.unit = (int)g0 / t;
      w.off = (int)g0 - w.unit * t;
    } else {
      int rem = (int)g0 - excl;
      unsigned int ignored = 0;
#pragma unroll 1
      for (w.b = b0; w.b < b1 - 1; ++w.b) {
        const int t = request_tiles(P, request(P, w.b, ignored));
        if (rem < t) break;
        rem -= t;
      }
      w.r = request(P, w.b, ignored);
      // the last block that begins at or before `rem`
      int above = blocks_of(P, w.r);
#pragma unroll 1
      while (above - w.i > 1) {
        const int mid = (w.i + above) / 2;
        if ((long long)blocks_before(P, w.r, mid) * P.Hk <= rem)
          w.i = mid;
        else
          above = mid;
      }
      rem -= blocks_before(P, w.r, w.i) * P.Hk;
      const int t = tiles_of(block_keys(P, w.r, w.i)) + kStart;
      w.h = rem / t;
      w.off = rem - w.h * t;
    }
    c->start = w;
  }
  if (blockIdx.x == 0) {
    int at = excl;
#pragma unroll 1
    for (int b = b0; b < b1 && !over; ++b) {
      P.starts[b] = at;
      if (b + 1 < b1) {
        unsigned int ignored = 0;
        at += request_tiles(P, request(P, b, ignored));
      }
    }
    if (tid == 0) P.starts[P.B] = over ? -1 : total;
    if (flags) atomicOr(P.status, flags);
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t ring = smem_addr(smem);
  const Walk w = c->start;
  // the launch's registers (256 threads x 128) where they are needed: 128 x 184 + 128 x 72
  if (warp < 4)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp < 4)
    softmax_role<T>(P, w, c, smem, q_smem, w_smem);
  else if (warp == 4)
    copy_role(P, w, c, 0, ring, &maps.k);
  else if (warp == 5)
    matrix_role<T>(P, w, c, ring, smem_addr(q_smem), smem_addr(w_smem));
  else if (warp == 6)
    copy_role(P, w, c, 1, ring, &maps.v);
  fence_before();
  __syncthreads();
  if (c->abort) {
    // a wait ran out: copies and products in flight end (each wait bounded) before
    // shared and tensor memory are given back
    int ignored = 0;
    if (warp == 4 || warp == 6) {
      const int v = warp == 4 ? 0 : 1, end = (int)c->copied[v];
#pragma unroll 1
      for (int k = end > kStages ? end - kStages : 0; k < end; ++k)
        (void)bar_wait(smem_addr(&c->kv_full[v][k % kStages]), k / kStages & 1, kDrainNs, &ignored);
    } else if (warp == 5) {
      if (elect_one()) mma_commit(smem_addr(&c->drain));
      __syncwarp();
      (void)bar_wait(smem_addr(&c->drain), 0, kDrainNs, &ignored);
    }
    __syncthreads();
  }
  if (warp == 5) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(c->tmem));
  }
  if (tid == 0 && c->abort) atomicOr(P.status, (unsigned int)SV_STATUS_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Joining parts: o = sum 2^(lse_i - m) o_i / sum 2^(lse_i - m)
// ---------------------------------------------------------------------------
// A warp a row and head, four values a lane; or, where few rows have many parts (MANY), a CTA,
// whose warps share the parts and are joined at the end.
template <typename T, bool MANY>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Params P, int ctas) {
  __shared__ float s_o[4][128], s_m[4], s_l[4];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned int ignored = 0;
  const Req r = request(P, b, ignored);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's writes
  const int list = P.starts[P.B];
  if (r.n <= 0 || list < 0) return;
  const int per = (int)(((long long)list + ctas - 1) / ctas);
  if (per <= 0) return;
  const int first = P.starts[b];
  // without a prefix, requests whose units all lie within one share are done
  if (P.prefix_len == 0 && first / per == (first + request_tiles(P, r) - 1) / per) return;
  const long long rows = (long long)r.n * P.Hq;
  constexpr int kRowsCta = MANY ? 1 : 4;
#pragma unroll 1
  for (long long x = (long long)blockIdx.y * kRowsCta + (MANY ? 0 : warp); x < rows; x += (long long)gridDim.y * kRowsCta) {
    const int tok = (int)(x / P.Hq), head = (int)(x - (long long)tok * P.Hq);
    const int h = head / P.group, in = tok * P.group + head - h * P.group;
    const long long at = (long long)(r.row0 + tok) * P.Hq + head;
    const int i = in / P.n;
    const int tiles = tiles_of(block_keys(P, r, i));
    const int u0 = first + blocks_before(P, r, i) * P.Hk + h * (tiles + kStart) + kStart;  // its first tile
    const int own0 = u0 / per, own = (u0 + tiles - 1) / per - own0 + 1, own_col = in - i * P.n;
    int pre0 = 0, pre = 0, pre_col = 0;
    if (P.prefix_len > 0) {
      const long long all = (long long)(r.row0 + tok) * P.group + head - h * P.group;
      const int blk = (int)(all / P.n);
      pre_col = (int)(all - (long long)blk * P.n);
      const int v0 = (blk * P.Hk + h) * (P.prefix_tiles + kStart) + kStart;
      pre0 = v0 / per;
      pre = (v0 + P.prefix_tiles - 1) / per - pre0 + 1;
    }
    if (P.prefix_len == 0 && own == 1) continue;  // written already
    const int parts = pre + own;
    auto place = [&](int k, const float*& src, const float*& lse) {
      const bool prefix = k < pre;
      const int j = prefix ? k : k - pre, count = prefix ? pre : own;
      if (count == 1) {
        src = (prefix ? P.pre : P.own) + at * P.D;
        lse = (prefix ? P.pre_lse : P.own_lse) + at;
      } else {
        const long long slot = (2ll * ((prefix ? pre0 : own0) + j) + (j == 0)) * P.n + (prefix ? pre_col : own_col);
        src = P.slot + slot * P.D;
        lse = P.slot_lse + slot;
      }
    };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    constexpr int kAhead = 8, kStep = MANY ? 4 : 1;
#pragma unroll 1
    for (int k0 = MANY ? warp : 0; k0 < parts; k0 += kAhead * kStep) {
      float4 v[kAhead];
      float e[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int k = k0 + j * kStep;
        e[j] = -INFINITY;
        if (k < parts) {
          const float *src, *lse;
          place(k, src, lse);
          e[j] = *lse;
          if (lane * 4 < P.D) v[j] = *reinterpret_cast<const float4*>(src + lane * 4);
        }
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) top = fmaxf(top, e[j]);  // (a NaN is dropped here, and kept by its weight)
      const float scale = m == -INFINITY ? 0.f : exp2f(m - top);
      l *= scale;
      o.x *= scale, o.y *= scale, o.z *= scale, o.w *= scale;
      m = top;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (e[j] == -INFINITY) continue;  // no key seen there
        const float w = exp2f(e[j] - top);
        l += w;
        o.x += v[j].x * w, o.y += v[j].y * w, o.z += v[j].z * w, o.w += v[j].w * w;
      }
    }
    if (MANY) {
      __syncthreads();  // (the last row's sums have been read)
      *reinterpret_cast<float4*>(s_o[warp] + lane * 4) = o;
      if (lane == 0) s_m[warp] = m, s_l[warp] = l;
      __syncthreads();
      if (warp != 0) continue;
      m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
      l = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = s_m[k] == -INFINITY ? (s_l[k] != s_l[k] ? 1.f : 0.f) : exp2f(s_m[k] - m);
        if (f == 0.f) continue;
        const float4 v = *reinterpret_cast<const float4*>(s_o[k] + lane * 4);
        l += s_l[k] * f;
        o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
      }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    if (lane * 4 < P.D)
      *reinterpret_cast<uint2*>(P.out + (at * P.D + lane * 4) * 2) =
          make_uint2(Type<T>::down2(o.x * inv, o.y * inv), Type<T>::down2(o.z * inv, o.w * inv));
    if (P.lse && lane == 0) P.lse[at] = (m + log2f(l)) * 0.693147180559945309f;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (sv::code_of(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q)) ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// A pool's map: values, tokens of a page, heads, pages; a box is a head's 128 bytes of box_rows tokens
// (what lies behind head_dim is filled with zeros)
bool encode(CUtensorMap* map, const void* pool, const sv_kv_cache& c, const int64_t* strides, int box_rows) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                              (cuuint64_t)c.num_pages};
  const cuuint64_t by[3] = {(cuuint64_t)strides[1], (cuuint64_t)strides[2], (cuuint64_t)strides[0]};
  const cuuint32_t box[4] = {128, (cuuint32_t)box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(pool), dims, by, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
  size_t starts, own, own_lse, pre, pre_lse, slot, slot_lse, total;
};
Layout layout(long long T, int Hq, int D) {
  const size_t rows = (size_t)T * Hq;
  Layout L;
  size_t at = 256;  // the status word
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += sv::align256(bytes);
    return a;
  };
  L.starts = take((size_t)(T + 1) * sizeof(int));
  L.own = take(rows * D * 4);
  L.own_lse = take(rows * 4);
  L.pre = take(rows * D * 4);
  L.pre_lse = take(rows * 4);
  L.slot = take((size_t)kSlots * 64 * D * 4);
  L.slot_lse = take((size_t)kSlots * 64 * 4);
  L.total = at;
  return L;
}

template <typename T>
int grid_size() {
  static std::atomic<int> cached{0};
  int dev = 0, sms = 0;
  if (sv::code_of(cudaGetDevice(&dev))) return 0;
  const int c0 = cached.load(std::memory_order_relaxed);
  if ((c0 >> 16) == dev + 1) return c0 & 0xffff;
  if (sv::code_of(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) ||
      sv::code_of(cudaFuncSetAttribute(attention8_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<T>::bytes)))
    return 0;
  const int ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
  cached.store(((dev + 1) << 16) | ctas, std::memory_order_relaxed);
  return ctas;
}

template <typename T>
int launch(const Maps& m, const Params& P, cudaStream_t stream) {
  const int grid = grid_size<T>();
  if (grid <= 0) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned int)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<T>::bytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  sv::overlap_launch(at[0]);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int rc = sv::code_of(cudaLaunchKernelEx(&cfg, attention8_kernel<T>, m, P));
  if (rc) return rc;
  // The join overlaps the attention kernel, whose end it waits for; a CTA a row where the shares
  // are more than eight times the units (at their most) and the rows no more than 16 an SM.
  const long long longest = P.G < P.T ? P.G + 1 : P.T, rows = longest * P.Hq;
  const long long by_longest = (longest * P.group + P.n - 1) / P.n * P.B;
  const long long by_rows = (long long)P.T * P.group / P.n + P.B;
  const bool many = grid > 8 * P.Hk * (by_longest < by_rows ? by_longest : by_rows) &&
                    (long long)P.T * P.Hq <= 8ll * grid;
  const long long y = many ? rows : (rows + 3) / 4;
  cfg.gridDim = dim3((unsigned int)P.B, (unsigned int)(y < 1024 ? y : 1024));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return sv::code_of(cudaLaunchKernelEx(&cfg, many ? join_kernel<T, true> : join_kernel<T, false>, P, grid));
}

}  // namespace

extern "C" {

size_t spec_verify_attention_e4m3_workspace_size(int total_rows, int q_heads, int head_dim) {
  if (total_rows < 0 || q_heads < 1 || q_heads > 65535 || head_dim < 16 || head_dim > SV_MAX_HEAD_DIM ||
      head_dim % 16)
    return 0;
  return layout(total_rows, q_heads, head_dim).total;
}

int spec_verify_attention_e4m3(const void* q, const int64_t* q_strides, int q_heads, sv_dtype dtype,
                               const sv_kv_cache* cache, const sv_kv_scales* scales, const int32_t* prefix_table,
                               int prefix_len, const int32_t* cu_draft, int total_drafts, int max_drafts, float scale,
                               const uint32_t* draft_mask, void* out, float* lse, void* workspace, size_t ws_bytes,
                               sv_stream_t stream) {
  if (!cache || !scales || !q_strides) return SV_ERR_NULL;
  const sv_kv_cache& c = *cache;
  int rc = sv::check_cache_e4m3(c, *scales);
  if (rc) return rc;
  const long long rows = (long long)total_drafts + c.batch;
  if ((dtype != SV_BF16 && dtype != SV_F16) || total_drafts < 0 || max_drafts < 0 || rows > INT32_MAX ||
      prefix_len < 0 || prefix_len > kMaxKeys || q_heads < 1 || q_heads > 65535 || q_heads % c.kv_heads ||
      rows * (q_heads / c.kv_heads) > INT32_MAX - 64 || !(scale > 0.f) || !std::isfinite(scale * 1.44269504f) ||
      (draft_mask && max_drafts > SV_MAX_GAMMA))
    return SV_ERR_SCALAR;
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] <= 0 || q_strides[i] % 8 || q_strides[i] >= ((int64_t)1 << 38)) return SV_ERR_SCALAR;
  if (c.batch == 0) return SV_OK;
  if (!q || !cu_draft || !out || !workspace || (prefix_len > 0 && !prefix_table)) return SV_ERR_NULL;
  if (!sv::aligned(q, 16) || !sv::aligned(out, 16) || !sv::aligned(lse, 4) || !sv::aligned(cu_draft, 4) ||
      !sv::aligned(prefix_table, 4) || !sv::aligned(draft_mask, 4) || !sv::aligned(workspace, 256))
    return SV_ERR_ALIGN;
  const Layout L = layout(rows, q_heads, c.head_dim);
  if (ws_bytes < L.total) return SV_ERR_WORKSPACE;
  // every row's output is written while other rows' queries may still be read
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  const uintptr_t q_end = qa + 2 * ((uint64_t)(rows - 1) * (uint64_t)q_strides[0] +
                                    (uint64_t)(q_heads - 1) * (uint64_t)q_strides[1] + (uint64_t)c.head_dim);
  const uintptr_t o_end = oa + 2 * (uint64_t)rows * (uint64_t)q_heads * (uint64_t)c.head_dim;
  if (qa < o_end && oa < q_end) return SV_ERR_ALIGN;
  Params P = {};
  P.B = c.batch;
  P.T = (int)rows;
  P.G = max_drafts;
  P.total = total_drafts;
  P.Hq = q_heads;
  P.Hk = c.kv_heads;
  P.D = c.head_dim;
  P.group = q_heads / c.kv_heads;
  P.n = dtype == SV_BF16 ? Smem<__nv_bfloat16>::n : Smem<__half>::n;
  P.num_pages = c.num_pages;
  P.page_size = c.page_size;
  while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
  while ((1 << P.block_shift) < scales->block) ++P.block_shift;
  P.per_page = c.page_size / scales->block;
  P.max_pages = c.max_pages;
  P.box_rows = c.page_size < kTile ? c.page_size : kTile;
  const long long room = (long long)c.max_pages * c.page_size;
  P.max_keys = room < kMaxKeys ? (int)room : kMaxKeys;
  P.table = c.page_table;
  P.kv_len = c.kv_len;
  P.cu = cu_draft;
  P.prefix_table = prefix_table;
  P.k_scales = scales->k;
  P.v_scales = scales->v;
  P.prefix_len = prefix_len;
  P.prefix_tiles = (int)(((long long)prefix_len + kTile - 1) / kTile);
  P.prefix_blocks = prefix_len > 0 ? (int)((rows * P.group + P.n - 1) / P.n) : 0;
  // the longest list that the arguments allow
  const double reach = (double)room / kTile + 1.0 + kStart;
  const double blocks = (double)rows * P.group / P.n;
  if ((blocks + c.batch) * P.Hk * reach + (blocks + 1.0) * P.Hk * ((double)P.prefix_tiles + kStart) >= (double)kMaxList)
    return SV_ERR_SCALAR;
  P.mask = draft_mask;
  P.sl2 = scale * 1.44269504088896341f;
  P.q = static_cast<const char*>(q);
  P.q_row = q_strides[0], P.q_head = q_strides[1];
  P.out = static_cast<char*>(out);
  P.lse = lse;
  char* w = static_cast<char*>(workspace);
  P.status = reinterpret_cast<unsigned int*>(w);
  P.starts = reinterpret_cast<int*>(w + L.starts);
  P.own = reinterpret_cast<float*>(w + L.own);
  P.own_lse = reinterpret_cast<float*>(w + L.own_lse);
  P.pre = reinterpret_cast<float*>(w + L.pre);
  P.pre_lse = reinterpret_cast<float*>(w + L.pre_lse);
  P.slot = reinterpret_cast<float*>(w + L.slot);
  P.slot_lse = reinterpret_cast<float*>(w + L.slot_lse);
  P.wait_ns = sv::wait_limit_ns();
  Maps m;
  if (!encode(&m.k, c.k_pages, c, c.k_strides, P.box_rows) || !encode(&m.v, c.v_pages, c, c.v_strides, P.box_rows))
    return SV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SV_BF16 ? launch<__nv_bfloat16>(m, P, s) : launch<__half>(m, P, s);
}

}  // extern "C"
