// Attention of a verify step's rows over a paged cache.
//
// Row i of request b (its last token and its drafts, gamma_b + 1 rows, packed
// as in the other packed calls) reads the shared prefix's keys and the
// request's own keys 0 .. kv_len[b] + i (or, with draft_mask, the keys before
// the step and the rows of the step that its mask word names):
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q.k_j
// in one pass over the keys with a running maximum m and sum.  The query heads
// that share a key head are rows of the same product, so a key head's keys are
// read once a request, and the prefix's once for all requests.
//
// Work: a unit is (request, block of query rows, key head) over the request's
// own keys, or (block or pair of blocks of all requests' rows, key head) over
// the prefix.  Blocks are 128 rows: tokens x heads of the key head's group.  The
// units' tiles of keys form two lists, A (pairs of blocks over the prefix, 128
// keys a tile) and B (everything else, 64 keys).  The CTAs (one an SM) are dealt
// out to A and B by their weights, and each CTA of A, and each of a B CTA's two
// streams, takes an equal contiguous share of its list, so a batch of any
// raggedness, or one long request, loads every SM alike.  A unit that crosses a
// share's border leaves one part a share; combine_kernel joins them (and the
// prefix with the own keys) by their sums.  No part is waited for inside a
// kernel, and parts are joined in list order: results repeat bit for bit.
//
// A CTA holds two streams.  A stream is a softmax warpgroup, a matrix warp, a
// query tile in shared memory and 256 columns of tensor memory for S and O.
// S = Q K^T and O += P V are tcgen05 products; P overwrites its S.
// B reads keys from memory once and is bound by that: its streams are independent
// (each with a copy warp and a ring of 64-key slots), so that one stream's
// start and end of a unit hide behind the other's, and each has two score tiles,
// so that the product of the next keys runs beside the softmax.
// A is bound by the products: a product of 128 rows and 64 keys takes as long as
// one of 128 keys, so its tiles have 128.  Each stream has one block of rows and
// both read every key and value slot of one ring; one stream's softmax
// runs beside the other's products, and P goes over in halves.
// Keys and values arrive by TMA, a page (at most 64 tokens) and 64 values a box,
// with 128-byte swizzle; the layout of the page pool is only the tensor map's
// strides.
//
// S and the sums are 32 bits.  P is rounded to the cache's 16-bit type for the
// product: each weight is off by at most half a step of that type, so the output by
// at most what the rounding of an output of its magnitude takes (relative to the sum
// of the weighted magnitudes of the values); the sum of weights uses the unrounded
// ones.  m is the running maximum less a shift, and moves only when the maximum
// has grown by more than 8 since (a factor of 256 in P), which makes the rescaling of O
// rare.  The shift is 0 in bf16, whose weights have the range of 32 bits, and 7 in fp16:
// weights then reach 2^15 (fp16 ends at 65504), the largest of a part is 2^7 at
// least, and those below the normal numbers, 2^-14, are off by 2^-25: 2^-32 of the
// largest each.  (Without the shift, weights below 2^-25 of the largest were lost: 65536
// keys of 2^-25 each after one that is 1 are 0.16 % of an output.)
//
// Measured (GB300, with the join): one request's 131000 keys of 8 heads, 64 query heads
// of 128, 97.8 us (537 MB, 5.5 TB/s; 87.8 us and 6.1 TB/s without the join); 256 requests
// behind 8192 shared tokens 246 us (557 TFLOP/s); 37 requests in 16-token pages 45 us,
// bound by the issue of 2 KB boxes; one request of 600 tokens 11.8 us, 4.0 of them the
// join; a prompt of 2500 rows 96 us (533 TFLOP/s; 67 without the join), of 32768 rows 6.6 ms
// (1330 TFLOP/s).
#include "../../include/spec_verify.h"
#include "internal.h"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <mutex>

namespace {

constexpr int kRows = 128;      // rows a block
constexpr int kTile = 64;       // keys a tile of list B, and a box
constexpr int kPairTile = 128;  // keys a tile of list A
constexpr int kThreads = 384;   // warps 0-3, 4-7: softmax; 8, 10: copies; 9, 11: products
constexpr int kMaxKeys = INT32_MAX - 4096;  // keys of a request: the last tile's places fit 32 bits
constexpr int kMaxCtas = 160;   // CTAs at most (the slots of parts are sized for this)
constexpr int kSlots = 4 * kMaxCtas;  // parts: two a stream
constexpr unsigned long long kDrainNs = 2000000000ull;  // limit of the waits that end an aborted CTA
constexpr int kControl = 3 * 1024;  // barriers and small tables behind the tiles
// Cost of a pair's tile (A) and of a stream's tile (B), for dealing out the CTAs; and
// of a unit's start and end, in tiles, which the lists count in front of its tiles.
constexpr int kCostA = 36, kCostB = 9, kStartA = 3, kStartB = 2;

template <int DP, bool PAIR>
struct Shape {
  static constexpr int keys = PAIR ? kPairTile : kTile;
  static constexpr int halves = DP / 64;
  static constexpr int q_bytes = kRows * DP * 2;
  static constexpr int q_half = kRows * 128;       // 64 values of every row
  static constexpr int tile_bytes = keys * DP * 2;
  static constexpr int half_bytes = keys * 128;
  static constexpr int slots = DP == 64 ? 10 : 5;  // of a ring: A has one, B one a stream
  static constexpr int ring = slots * kPairTile * DP * 2;
  static constexpr int smem = 2 * q_bytes + ring + kControl;
  static_assert(smem <= 227 * 1024, "shared memory");
};

// n / d for 0 <= n < 2^31 by a multiplication: m = ceil(2^(31 + k) / d) with 2^k >= d
// is off by less than 2^k / 2^(31 + k) of 1 / d, so n m / 2^(31 + k) exceeds n / d by
// less than 1 / d.
struct Divisor {
  unsigned int d, k;
  unsigned long long m;
};
inline Divisor divisor(int d) {
  Divisor v{(unsigned int)d, 0u, 0ull};
  while ((1ull << v.k) < (unsigned long long)d) ++v.k;
  v.m = ((1ull << (31 + v.k)) + d - 1) / d;
  return v;
}
__device__ __forceinline__ int divide(int n, const Divisor& v) {
  return (int)(((unsigned long long)(unsigned int)n * v.m) >> (31 + v.k));
}
// n / d where the quotient is a small number (a share: at most 2 kMaxCtas; a key
// head: at most 65535): by a rounded reciprocal and one correction.
__device__ __forceinline__ int share_of(int n, int d, float inv) {
  int q = (int)((float)n * inv);
  const int r = n - q * d;
  q += r < 0 ? -1 : r >= d ? 1 : 0;
  return q;
}

struct AttnParams {
  int B, T, G, total, Hq, Hk, D, group, tpq, own_tok;
  int num_pages, page_size, page_shift, max_pages, box_rows;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  const int32_t* prefix_table;
  int max_keys;  // of a request
  Divisor by_heads, by_group, by_tpq;        // Hq, group, tpq
  int prefix_len, prefix_tiles, pair_tiles;  // tiles of the prefix in list B and in list A
  int pairs, odd;                            // pairs of row blocks, and a single one
  const uint32_t* mask;
  float sl2;  // scale log2(e)
  char* out;
  float* lse;
  unsigned int* status;
  int* starts;         // [B + 2]: where each request begins in list B, the list's end, the CTAs of list A
  // Parts: whole units over own keys as rows [T * Hq][DP]; whole prefix units by
  // block [Hk][blocks] and parts of units by slot [kSlots], both as [DP / 8][kRows][8]
  // (a warp's lanes have a row each: their stores are one run of memory)
  float* own;
  float* own_lse;
  float* whole;
  float* whole_lse;
  float* slot;
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
// Waits for a phase, at most wait_ns; false (and *abort set) when that ran out
// or another warp of the CTA gave up.  Loops here and below are kept rolled: with
// these waits unrolled the kernel had 304 KB of instructions and ran at half its
// speed.  (Not a function of its own: registers are moved between warps.)
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
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One thread of the warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// D = A B (+ D) over four steps of 16 values, A and B in shared memory, both
// K-major: a step is 32 bytes on.  The steps stand in one block of text so that
// the operands move to uniform registers once, not at every product.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D = A B (+ D) over one step, or four: A in tensor memory (a step is 8
// columns), B in shared memory with its 16 rows of 128 bytes a step.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
#define SV_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), \
                    "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define SV_W8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), \
                    "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
// 32 columns of this thread's lane
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SV_R8(v, 0), SV_R8(v, 8), SV_R8(v, 16), SV_R8(v, 24)
      : "r"(addr));
}
// The same, and the largest of them (NaN left out)
__device__ __forceinline__ float tmem_load32_max(uint32_t addr, uint32_t* v) {
  float m;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : SV_R8(v, 0), SV_R8(v, 8), SV_R8(v, 16), SV_R8(v, 24), "=f"(m)
      : "r"(addr));
  return m;
}
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
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      SV_W8(v, 0), SV_W8(v, 8), SV_W8(v, 16), SV_W8(v, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Keeps the uses of loaded values behind the wait for them.
#define SV_T8(v, o) "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), \
                    "+r"(v[o + 5]), "+r"(v[o + 6]), "+r"(v[o + 7])
__device__ __forceinline__ void tmem_loaded32(uint32_t* v) {
  asm volatile("" : SV_T8(v, 0), SV_T8(v, 8), SV_T8(v, 16), SV_T8(v, 24));
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_loaded(float& m) { asm volatile("" : "+f"(m)); }
__device__ __forceinline__ void tmem_loaded16(uint32_t* v) {
  asm volatile("" : SV_T8(v, 0), SV_T8(v, 8));
}
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

// 32 bytes: a lane has a row of its own, so that each store fills a sector
__device__ __forceinline__ void store8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), SV_W8(v, 0) : "memory");
}
// Shared-memory matrix descriptors, 128-byte swizzle: K-major (rows of 64
// values, eight rows 1024 bytes apart) and MN-major (tokens as rows; the next
// 64 values of a token `lead` bytes on, eight tokens 1024 bytes apart).
__device__ __forceinline__ uint64_t mat_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <typename T>
struct Type;
template <>
struct Type<__nv_bfloat16> {
  static constexpr uint32_t fmt = 1;
  static constexpr float shift = 0.f;  // log2 of the largest weight where the maximum just moved
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};
template <>
struct Type<__half> {
  static constexpr uint32_t fmt = 0;
  static constexpr float shift = 7.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};
// 32-bit accumulators, A and B of one 16-bit type
__host__ __device__ constexpr uint32_t instr_desc(uint32_t fmt, uint32_t n, bool b_mn) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((n / 8) << 17) |
         ((uint32_t)(kRows / 16) << 24);
}

// ---------------------------------------------------------------------------
// The tile list
// ---------------------------------------------------------------------------
struct Req {
  int row0;  // first row
  int n;     // rows (0: skipped)
  int kv;    // own keys before the step
};
__device__ __forceinline__ Req request(const AttnParams& P, int b, unsigned int& flags) {
  const int c0 = __ldg(P.cu + b), c1 = __ldg(P.cu + b + 1), kv = __ldg(P.kv_len + b);
  Req r{0, 0, 0};
  if (c0 < 0 || c1 < c0 || c1 - c0 > P.G || c1 > P.total) {
    flags |= SV_STATUS_BAD_GAMMA;
  } else if (kv < 0 || (long long)kv + (c1 - c0) + 1 > P.max_keys) {
    flags |= SV_STATUS_BAD_LENGTH;
  } else {
    r = Req{c0 + b, c1 - c0 + 1, kv};
  }
  return r;
}
// keys that row block rb of a request sees (by mask word: any row of the step), and their tiles
__device__ __forceinline__ int block_keys(const AttnParams& P, const Req& r, int rb) {
  const int last = !P.mask && (rb + 1) * P.tpq < r.n ? (rb + 1) * P.tpq : r.n;
  return r.kv + last;
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
// The host refuses sizes whose lists could reach kMaxList where requests have rows of
// their own; inconsistent cu_draft entries (0, n, 0, n, ..) name the same rows again and
// again, so lengths are summed up to that and no further.
constexpr int kMaxList = 1 << 30;
__device__ __forceinline__ int list_add(int a, int b) {
  return (int)min((unsigned int)a + (unsigned int)b, (unsigned int)kMaxList);
}
// Of a key head, the tiles of a request's first `blocks` row blocks, none of them its last:
// the sum over i of ceil((kv + (i + 1) tpq) / 64).  A sum of n terms floor((a i + b) / m) is
// its whole parts, n (n - 1) / 2 times a / m and n times b / m, and what is left counts
// the whole numbers below a line, which are the same counted by rows: (a n + b) / m terms
// with a and m exchanged, Euclid's steps on (tpq, 64).  One or two for groups of 1, 2, 4, 8
// heads, eight at most.  The sum is below kMaxList, so is every product.  (With a loop over
// the blocks the join of a prompt's rows was quadratic.  A function of its own: inlined at its
// six places it lengthened the code before the roles, which cost calls of single blocks 3
// to 7 %.)
__device__ __noinline__ int blocks_sum(int kv, int tpq, int blocks) {
  unsigned int n = blocks, a = tpq, b = (unsigned int)kv + tpq + kTile - 1, m = kTile, sum = 0;
  if (blocks <= 4) {  // sooner done one by one
#pragma unroll 1
    for (; n > 0; --n, b += a) sum += b / kTile;
    return (int)sum;
  }
#pragma unroll 1
  for (;;) {
    const unsigned int qa = a / m, qb = b / m;
    if (qa > 0) sum += (n & 1 ? n * ((n - 1) / 2) : (n / 2) * (n - 1)) * qa;
    sum += n * qb;
    a -= qa * m;
    b -= qb * m;
    const unsigned int top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top - n * m;
    const unsigned int t = a;
    a = m;
    m = t;
  }
  return (int)sum;
}
// ... and their starts
__device__ __forceinline__ int blocks_before(const AttnParams& P, const Req& r, int blocks) {
  if (blocks == 0) return 0;
  // (with mask words a row may see any row of its step)
  return P.mask ? blocks * (tiles_of(r.kv + r.n) + kStartB) : blocks_sum(r.kv, P.tpq, blocks) + blocks * kStartB;
}
// A request's length in list B: its units' tiles and starts (below kMaxList).
__device__ __forceinline__ int request_tiles(const AttnParams& P, const Req& r) {
  if (r.n <= 0) return 0;
  int t = tiles_of(r.kv + r.n) + kStartB;
  if (r.n > P.tpq) t += blocks_before(P, r, (r.n - 1) / P.tpq);
  return t * P.Hk;
}

// How the lists are dealt out.
struct Plan {
  int a, b;          // lengths of the lists: tiles and starts
  int per_a, per_b;  // of a CTA's share of A, of a stream's share of B
  int ctas_a, ctas_b;
};
// The CTAs of list A, by the lists' weights.  Only the attention kernel works this out,
// and the join reads it: the sum of floats may be contracted in two ways, which differ by a
// CTA for some lists past 2^24 tiles.
__device__ __forceinline__ int pair_ctas(int a, int b, int ctas) {
  if (a == 0) return 0;
  const float wa = (float)a * kCostA, wb = (float)b * kCostB;
  int na = (int)(ctas * (wa / (wa + wb)) + 0.5f);
  na = na < 1 ? 1 : na;
  return b > 0 && na > ctas - 1 ? ctas - 1 : na;
}
__device__ __forceinline__ int pair_list(const AttnParams& P) { return P.Hk * P.pairs * (P.pair_tiles + kStartA); }
__device__ __forceinline__ Plan make_plan(const AttnParams& P, int b_tiles, int ctas, int na) {
  Plan L;
  L.a = pair_list(P);
  L.b = b_tiles;
  L.ctas_a = na;
  L.ctas_b = ctas - na;
  L.per_a = na ? (L.a + na - 1) / na : 0;
  L.per_b = L.ctas_b ? (L.b + 2 * L.ctas_b - 1) / (2 * L.ctas_b) : 0;
  return L;
}
// list B before the requests' own units
__device__ __forceinline__ int single_tiles(const AttnParams& P) { return P.Hk * P.odd * (P.prefix_tiles + kStartB); }

// A run of tiles of one unit.
struct Piece {
  bool prefix;
  int b, h;
  int row0, ntok;    // first row and rows of the block (A: of stream 0's block)
  int kv, first;     // own: keys before the step, the block's first row within the request:
                     // row i of the block sees keys below kv + first + i + 1
  int keys;          // keys of the unit
  int t0, t1;        // tiles [t0, t1) of unit_t
  int unit_t;
};

// Walks a share.  Every role walks it alone, from the same start.
struct Walk {
  int left;
  bool pair, single;  // list A; the prefix's single block in list B
  int unit;           // prefix unit
  int b, rb, h;       // own unit
  int off;            // place within the unit: its start, then its tiles
  Req r;

  __device__ __forceinline__ void load_request(const AttnParams& P) {
    unsigned int ignored = 0;
    r = Req{0, 0, 0};
#pragma unroll 1
    while (b < P.B) {
      r = request(P, b, ignored);
      if (r.n > 0) return;
      ++b;
    }
  }
  __device__ __forceinline__ bool next(const AttnParams& P, Piece& p) {
    if (left <= 0) return false;
    if (single && unit >= P.Hk) {
      single = false;
      b = rb = h = 0;
      load_request(P);
    }
    p.prefix = pair || single;
    if (p.prefix) {
      p.b = 0;
      p.h = pair ? unit / P.pairs : unit;
      p.row0 = (pair ? (unit - p.h * P.pairs) * 2 : 2 * P.pairs) * P.tpq;
      p.ntok = P.T - p.row0;
      p.kv = p.first = 0;
      p.keys = P.prefix_len;
      p.unit_t = pair ? P.pair_tiles : P.prefix_tiles;
    } else {
      if (b >= P.B) return false;
      p.b = b;
      p.h = h;
      p.first = rb * P.tpq;
      p.row0 = r.row0 + p.first;
      p.ntok = r.n - p.first;
      p.kv = r.kv;
      p.keys = block_keys(P, r, rb);
      p.unit_t = tiles_of(p.keys);
    }
    const int start = pair ? kStartA : kStartB, all = p.unit_t + start;
    const int end = left < all - off ? off + left : all;
    p.t0 = off > start ? off - start : 0;
    p.t1 = end > start ? end - start : 0;
    left -= end - off;
    off = 0;
    if (p.t1 == p.t0) return false;  // the share ends in the unit's start
    if (p.prefix) {
      ++unit;
    } else if (++h == P.Hk) {
      h = 0;
      if (++rb * P.tpq >= r.n) {
        rb = 0;
        ++b;
        if (left > 0) load_request(P);
      }
    }
    return true;
  }
};

struct Control {
  uint64_t kv_full[20], kv_empty[20];
  // of each stream
  uint64_t q_full[2], q_empty[2], s_full[2][2], p_ready[2][2], o_full[2], o_free[2], drain[2];
  uint32_t tmem;
  int abort;
  unsigned int q_copied[2], kv_copied[2];
  int scan[kThreads / 32];
  Walk start[2];  // where the streams' shares begin
};
static_assert(sizeof(Control) <= kControl, "control block");

// A place in a ring of N slots.  A piece's tiles fill it as keys, values, keys, ..
template <int N>
struct Cursor {
  uint32_t slot, turn;  // turn: parity of the slot's use
  __device__ __forceinline__ void step(int k) {
    slot += k;
    if (slot >= (uint32_t)N) {
      slot -= N;
      turn ^= 1u;
    }
  }
  __device__ __forceinline__ Cursor next() const {
    Cursor c = *this;
    c.step(1);
    return c;
  }
  __device__ __forceinline__ Cursor previous() const {
    return slot == 0 ? Cursor{(uint32_t)N - 1, turn ^ 1u} : Cursor{slot - 1, turn};
  }
};

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const AttnParams& P, Control* c) {
  const bool ok = bar_wait(smem_addr(bar), parity, P.wait_ns, &c->abort);
  return __all_sync(0xffffffffu, ok);
}

// Copies: B: stream s's queries, keys and values; A: warp 0 both streams' queries
// and the keys, warp 1 the values.
template <int DP, bool PAIR>
__device__ __forceinline__ void copy_role(const AttnParams& P, Walk w, Control* c, int s, uint32_t q_smem,
                                          uint32_t ring, const CUtensorMap* qmap, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap) {
  using S = Shape<DP, PAIR>;
  const int lane = threadIdx.x & 31;
  const int first = PAIR ? 0 : s * S::slots;  // slot of the ring's start
  unsigned int flags = 0, qn = 0, copied = 0;  // query tiles of a stream, ring entries
  Cursor<S::slots> at{PAIR && s == 1 ? 1u : 0u, 0u};
  Piece p;
  bool ok = true;
#pragma unroll 1
  while (ok && w.next(P, p)) {
    const int n = p.t1 - p.t0;
    // a lane's page of tile i (a box is at most a page), as the table has it
    const int32_t* table = p.prefix ? P.prefix_table : P.table + (size_t)p.b * P.max_pages;
    auto look_up = [&](int i) {
      const int key = (p.t0 + i) * S::keys + lane * P.box_rows;
      return i < n && lane * P.box_rows < S::keys && key < p.keys ? __ldg(table + (key >> P.page_shift)) : 0;
    };
    int ahead = look_up(0);
    if (!PAIR || s == 0) {
      // the block's query rows: [token][head of the group] in 128-byte rows
#pragma unroll
      for (int x = 0; x < (PAIR ? 2 : 1); ++x) {
        const int qs = PAIR ? x : s;
        if (!(ok = warp_wait(&c->q_empty[qs], (qn & 1) ^ 1, P, c))) break;
        const uint32_t bar = smem_addr(&c->q_full[qs]);
        if (elect_one()) {
          bar_expect(bar, (uint32_t)(S::halves * 128 * P.group * (p.prefix ? P.tpq : P.own_tok)));
          for (int y = 0; y < S::halves; ++y)
            tma_load(q_smem + qs * S::q_bytes + y * S::q_half, qmap + (p.prefix ? 1 : 0), bar, y * 64, 0, p.h,
                     p.row0 + x * P.tpq);
        }
        __syncwarp();
        if (lane == 0) c->q_copied[qs] = qn + 1;
      }
      ++qn;
    }
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      int id = ahead;
      if (id < 0 || id >= P.num_pages) {
        flags |= SV_STATUS_BAD_PAGE;
        id = P.num_pages;  // past the pool: the copy fills zeros
      }
      ahead = look_up(i + 1);  // on its way while this tile's copies are issued
      const int key0 = (p.t0 + i) * S::keys;
      const int keys = p.keys - key0 < S::keys ? p.keys - key0 : S::keys;
#pragma unroll 1
      for (int v = PAIR ? s : 0; v < (PAIR ? s + 1 : 2); ++v) {  // keys, values
        const uint32_t slot = first + at.slot;
        if (!(ok = warp_wait(&c->kv_empty[slot], at.turn ^ 1, P, c))) break;
        const uint32_t bar = smem_addr(&c->kv_full[slot]);
        const CUtensorMap* map = v ? vmap : kmap;
        uint32_t dst = ring + slot * S::tile_bytes;
        if (elect_one()) bar_expect(bar, (uint32_t)(((keys + P.box_rows - 1) & -P.box_rows) * S::halves * 128));
        int lane_of = 0;
#pragma unroll 1
        for (int x = 0; x < keys; x += P.box_rows, dst += P.box_rows * 128, ++lane_of) {
          const int page = __shfl_sync(0xffffffffu, id, lane_of);
          if (elect_one()) {
            const int in = (key0 + x) & (P.page_size - 1);
            tma_load(dst, map, bar, 0, in, p.h, page);
            if (S::halves == 2) tma_load(dst + S::half_bytes, map, bar, 64, in, p.h, page);
          }
        }
        __syncwarp();
        at.step(PAIR ? 2 : 1);
        ++copied;
      }
    }
  }
  if (lane == 0) c->kv_copied[s] = copied;
  const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && any) atomicOr(P.status, any);
}

// Products of one stream, by one thread.  (All 512 columns are allocated, so they start at 0.)
template <typename T, int DP, bool PAIR>
__device__ __forceinline__ void matrix_role(const AttnParams& P, Walk w, Control* c, int s, uint32_t q_smem,
                                            uint32_t ring) {
  using S = Shape<DP, PAIR>;
  if (!elect_one()) return;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return bar_wait(smem_addr(bar), parity, P.wait_ns, &c->abort); };
  const uint32_t cols = s * 256;  // S (128 columns: B: two tiles), O of this stream
  constexpr uint32_t kQk = instr_desc(Type<T>::fmt, S::keys, false);
  constexpr uint32_t kPv = instr_desc(Type<T>::fmt, DP, true);
  constexpr int kAhead = PAIR ? 1 : 2;  // score tiles
  const uint32_t q = q_smem + s * S::q_bytes;
  const int first = PAIR ? 0 : s * S::slots;  // slot of the ring's start
  unsigned int pieces = 0, tk = 0, tv = 0;    // tiles of keys and of values so far
  Cursor<S::slots> ck{0u, 0u}, cv{1u, 0u};
  Piece p;
  bool ok = true;
#pragma unroll 1
  while (ok && w.next(P, p)) {
    const int n = p.t1 - p.t0;
    auto qk = [&](int i) {
      const uint32_t slot = first + ck.slot, buf = PAIR ? 0 : tk & 1;
      if (i == 0 && !(ok = wait(&c->q_full[s], pieces & 1))) return;
      if (!(ok = wait(&c->kv_full[slot], ck.turn))) return;
      const uint32_t b = ring + slot * S::tile_bytes;
#pragma unroll
      for (int x = 0; x < S::halves; ++x)
        mma_ss4(cols + buf * kTile, mat_desc(q + x * S::q_half, 16), mat_desc(b + x * S::half_bytes, 16), kQk, x > 0);
      mma_commit(smem_addr(&c->s_full[s][buf]));  // (the softmax warps hand the keys' slot back)
      if (i == n - 1) mma_commit(smem_addr(&c->q_empty[s]));
      ck.step(2);
      ++tk;
    };
    int ahead = 0;  // tiles whose scores are on their way
#pragma unroll 1
    for (; ok && ahead < kAhead && ahead < n; ++ahead) qk(ahead);
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      const uint32_t slot = first + cv.slot, t = tv;
      if (i == 0 && pieces > 0 && !(ok = wait(&c->o_free[s], (pieces - 1) & 1))) break;
      int keys = p.keys - (p.t0 + i) * S::keys;
      keys = keys < S::keys ? keys : S::keys;
      const int steps = (keys + 15) / 16;
      if (!(ok = wait(&c->kv_full[slot], cv.turn))) break;
      const uint32_t d = cols + 2 * kTile;
      const uint64_t v = mat_desc(ring + slot * S::tile_bytes, S::half_bytes);
#pragma unroll
      for (int x = 0; x < (PAIR ? 2 : 1); ++x) {
        const uint32_t buf = PAIR ? x : t & 1;
        if (!(ok = wait(&c->p_ready[s][buf], PAIR ? t & 1 : (t >> 1) & 1))) break;
        fence_after();
        const uint32_t a = PAIR ? cols + x * 32 : cols + buf * kTile;
        const int left = steps - 4 * x;
        {
          if (left >= 4) {
            mma_ts4(d, a, v + x * 512, kPv, i > 0 || x > 0);
          } else {
#pragma unroll 1
            for (int k = 0; k < left; ++k) mma_ts(d, a + k * 8, v + x * 512 + k * 128, kPv, i > 0 || x > 0 || k > 0);
          }
          if (!PAIR || x == 1) {
            mma_commit(smem_addr(&c->kv_empty[slot]));
            if (i == n - 1) mma_commit(smem_addr(&c->o_full[s]));
          }
        }
      }
      cv.step(2);
      ++tv;
      if (ok && i + kAhead < n) qk(i + kAhead);
    }
    ++pieces;
  }
}

// Which of the 32 keys from `at` a row sees: all below `limit`, or, with a mask
// word, those below kv and those of the step that it names.
__device__ __forceinline__ uint32_t seen(int at, int limit, bool by_word, uint32_t word, int kv) {
  if (by_word) {
    const int d = at - kv;  // the first key's place in the step's rows
    return d <= -32 ? ~0u : d < 0 ? (word << -d) | ((1u << -d) - 1u) : d < 32 ? word >> d : 0u;
  }
  const int k = limit - at;
  return k >= 32 ? ~0u : k > 0 ? (1u << k) - 1u : 0u;
}
__device__ __forceinline__ void hide(uint32_t* v, uint32_t see) {
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!((see >> x) & 1u)) v[x] = __float_as_uint(-INFINITY);
}
__device__ __forceinline__ float max32(const uint32_t* v) {
  float a = -INFINITY, b = -INFINITY;
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    a = max3(a, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
    b = max3(b, __uint_as_float(v[x + 2]), __uint_as_float(v[x + 3]));
  }
  return fmaxf(a, b);
}
// Weights of 32 scores: 2^(scale s - m), packed into v[0 .. 15], and their sums.
template <typename T>
__device__ __forceinline__ void weights32(const uint32_t* v, uint32_t* out, uint64_t sl2, uint64_t sub, uint64_t& sum0,
                                          uint64_t& sum1) {
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    float a, b, e, f;
    unpair(pair_fma(pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), sl2, sub), a, b);
    unpair(pair_fma(pair(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), sl2, sub), e, f);
    a = exp2_fast(a), b = exp2_fast(b), e = exp2_fast(e), f = exp2_fast(f);
    sum0 = pair_add(sum0, pair(a, b));
    sum1 = pair_add(sum1, pair(e, f));
    out[x / 2] = Type<T>::pack(a, b);
    out[x / 2 + 1] = Type<T>::pack(e, f);
  }
}

template <typename T, int DP, bool PAIR>
__device__ __forceinline__ void softmax_role(const AttnParams& P, Walk w, Control* c, int s, uint32_t part_base,
                                             unsigned char* ring) {
  const int row = threadIdx.x & 127, lane = row & 31;
  const uint32_t lanes = (uint32_t)(row & ~31) << 16;  // this warp's tensor-memory lanes
  const uint32_t s_cols = lanes + s * 256, o_col = s_cols + 2 * kTile;
  const float ninf = -INFINITY;
  const int tok = row / P.group, g = row - tok * P.group;
  using S = Shape<DP, PAIR>;
  const int first = PAIR ? 0 : s * S::slots;  // slot of the ring's start
  unsigned int tiles = 0, pieces = 0;
  Cursor<S::slots> at{0u, 0u};  // the tile's keys; its values come next
  Piece p;
  bool ok = true;
#pragma unroll 1
  while (ok && w.next(P, p)) {
    const int n = p.t1 - p.t0;
    const int skip = PAIR ? s * P.tpq : 0;  // rows of the other stream's block
    int btok = p.ntok - skip;
    btok = btok < P.tpq ? btok : P.tpq;
    const int rows = btok * P.group;
    const bool active = (row & ~31) < rows, mine = row < rows;
    // keys this row sees: all below `limit` or by its mask word; `free`: the keys
    // that every row of the block sees
    const bool by_word = !p.prefix && P.mask;
    const int limit = p.prefix ? P.prefix_len : p.kv + p.first + tok + 1;
    const int free = p.prefix ? P.prefix_len : (P.mask ? p.kv : p.kv + p.first + 1);
    uint32_t word = 0;
    if (by_word && mine) {
      word = P.mask[p.row0 + tok];
      if (p.keys - p.kv < 32) word &= (1u << (p.keys - p.kv)) - 1u;  // rows of the step
    }
    float m = ninf, l = 0.f;  // running maximum (times scale log2 e) less the shift, and sum
    // Moves the maximum to the new scores' (largest: `best`) where it has grown by more
    // than 8.  It is rounded up, and the growth is the exponent that `best` gets below, so
    // that no weight passes 2^(8 + shift), however large the scores are; the rounding lowers
    // a row's weights by one step of the maximum at most (16 below 2^28, which fp16 bears).
    auto settle = [&](int i, float best) {
      const float top = __fmaf_ru(best, P.sl2, -Type<T>::shift);
      if (i == 0) {
        m = top;
        return;
      }
      // (also from -inf; not where both are infinite or one is NaN)
      const bool grow = fmaf(best, P.sl2, -m) > 8.f + Type<T>::shift;
      if (!__any_sync(0xffffffffu, grow)) return;
      const float f = grow ? (m == ninf ? 0.f : exp2_fast(m - top)) : 1.f;
      // O is at rest once the last tile's product is done.  In A S of this tile
      // came after it; in B its values' slot has been handed back (the slot's
      // next use cannot end before this tile's own product).
      if (!PAIR) {
        const Cursor<S::slots> v = at.previous();
        if (!(ok = warp_wait(&c->kv_empty[first + v.slot], v.turn, P, c))) return;
        fence_after();
      }
#pragma unroll 1
      for (int x = 0; x < DP; x += 16) {
        uint32_t o[16];
        tmem_load16(o_col + x, o);
        tmem_wait_load();
        tmem_loaded16(o);
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
        tmem_store16(o_col + x, o);
      }
      l *= f;
      if (grow) m = top;
    };
    // The value rows behind the last key of its 16 hold what memory held there, and
    // weights of 0 times NaN would be NaN: this warpgroup clears them before it
    // hands P over.  (In A both streams' write the same zeros.)
    auto clear_tail = [&](int keys) {
      const Cursor<S::slots> v = at.next();
      const uint32_t slot = first + v.slot;
      if (!(ok = warp_wait(&c->kv_full[slot], v.turn, P, c))) return;
      constexpr int kRow = S::halves * 8;  // 16-byte words of a row
#pragma unroll 1
      for (int x = row; x < ((keys + 15) / 16 * 16 - keys) * kRow; x += 128) {
        const int r = keys + x / kRow, in = x % kRow;
        *reinterpret_cast<uint4*>(ring + slot * S::tile_bytes + (in / 8) * S::half_bytes + r * 128 + (in % 8) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    };
    const uint64_t sl2 = pair(P.sl2, P.sl2);
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++tiles, at.step(2)) {
      const uint32_t buf = PAIR ? 0 : tiles & 1, s_col = s_cols + buf * kTile;
      if (!(ok = warp_wait(&c->s_full[s][buf], PAIR ? tiles & 1 : (tiles >> 1) & 1, P, c))) break;
      if (threadIdx.x % 128 == 0) bar_arrive(smem_addr(&c->kv_empty[first + at.slot]));
      const int key0 = (p.t0 + i) * S::keys;
      const bool masked = key0 + S::keys > free;
      const int keys = p.keys - key0;
      const bool tail = keys < S::keys && (keys & 15);
      uint64_t sum0 = 0, sum1 = 0;  // two pairs of zeros
      if (PAIR) {
        uint32_t v[kPairTile];
        uint64_t sub = 0;
        if (active) {
          fence_after();
          float mx[4];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) mx[ch] = tmem_load32_max(s_col + 32 * ch, v + 32 * ch);
          tmem_wait_load();
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            tmem_loaded32(v + 32 * ch);
            tmem_loaded(mx[ch]);
          }
          if (masked) {
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              hide(v + 32 * ch, seen(key0 + 32 * ch, limit, by_word, word, p.kv));
              mx[ch] = max32(v + 32 * ch);
            }
          }
          settle(i, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
          const float neg = m == ninf ? 0.f : -m;
          sub = pair(neg, neg);
        }
        if (tail) clear_tail(keys);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (active) {
            weights32<T>(v + 64 * x, v + 32 * x, sl2, sub, sum0, sum1);
            weights32<T>(v + 64 * x + 32, v + 32 * x + 16, sl2, sub, sum0, sum1);
            tmem_store32(s_col + 32 * x, v + 32 * x);
            tmem_wait_store();
            fence_before();
          }
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(&c->p_ready[s][x]));
        }
      } else {
        if (active) {
          fence_after();
          uint32_t v[kTile];
          float mx0 = tmem_load32_max(s_col, v), mx1 = tmem_load32_max(s_col + 32, v + 32);
          tmem_wait_load();
          tmem_loaded32(v);
          tmem_loaded32(v + 32);
          tmem_loaded(mx0);
          tmem_loaded(mx1);
          if (masked) {
            hide(v, seen(key0, limit, by_word, word, p.kv));
            hide(v + 32, seen(key0 + 32, limit, by_word, word, p.kv));
            mx0 = max32(v), mx1 = max32(v + 32);
          }
          settle(i, fmaxf(mx0, mx1));
          if (!ok) break;
          const float neg = m == ninf ? 0.f : -m;
          const uint64_t sub = pair(neg, neg);
          weights32<T>(v, v, sl2, sub, sum0, sum1);
          weights32<T>(v + 32, v + 16, sl2, sub, sum0, sum1);
          tmem_store32(s_col, v);
          tmem_wait_store();
          fence_before();
        }
        if (tail) clear_tail(keys);
        if (!ok) break;
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&c->p_ready[s][buf]));
      }
      float a, b;
      unpair(pair_add(sum0, sum1), a, b);
      l += a + b;
    }
    if (!ok) break;
    // the piece's rows, after its last product (a barrier of its own: parity
    // would not tell that product from the one two before it)
    if (!(ok = warp_wait(&c->o_full[s], pieces & 1, P, c))) break;
    ++pieces;
    if (active) {
      fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse2 = m + log2f(l);
      const bool whole = p.t0 == 0 && p.t1 == p.unit_t;
      const bool direct = whole && !p.prefix && P.prefix_len == 0;
      const size_t at = (size_t)(p.row0 + skip + tok) * P.Hq + (size_t)p.h * P.group + g;
      float* part = nullptr;
      float* part_lse = nullptr;
      int jump = 8;  // from eight values of the row to the next
      if (!direct) {
        if (whole && !p.prefix) {
          part = P.own + at * DP;
          part_lse = P.own_lse + at;
        } else {
          const size_t tile = whole ? (size_t)p.h * (2 * P.pairs + P.odd) + p.row0 / P.tpq + (PAIR ? s : 0)
                                    : (size_t)(part_base + (p.t0 == 0 ? (PAIR ? 2 : 1) : 0));
          part = (whole ? P.whole : P.slot) + tile * kRows * DP + row * 8;
          part_lse = (whole ? P.whole_lse : P.slot_lse) + tile * kRows + row;
          jump = kRows * 8;
        }
      }
#pragma unroll 1
      for (int x = 0; x < DP; x += 32) {
        uint32_t o[32];
        tmem_load32(o_col + x, o);
        tmem_wait_load();
        tmem_loaded32(o);
#pragma unroll
        for (int y = 0; y < 32; ++y)
          o[y] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[y]) * inv);
        if (mine) {
          if (direct) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              if (x + y < P.D) {
                uint4 q;
                q.x = Type<T>::pack(__uint_as_float(o[y]), __uint_as_float(o[y + 1]));
                q.y = Type<T>::pack(__uint_as_float(o[y + 2]), __uint_as_float(o[y + 3]));
                q.z = Type<T>::pack(__uint_as_float(o[y + 4]), __uint_as_float(o[y + 5]));
                q.w = Type<T>::pack(__uint_as_float(o[y + 6]), __uint_as_float(o[y + 7]));
                *reinterpret_cast<uint4*>(P.out + (at * P.D + x + y) * 2) = q;
              }
            }
          } else {
#pragma unroll
            for (int y = 0; y < 32; y += 8) store8(part + (x + y) / 8 * jump, o + y);
          }
        }
      }
      fence_before();
      if (mine) {
        if (direct) {
          if (P.lse) P.lse[at] = lse2 * 0.693147180559945309f;
        } else {
          *part_lse = lse2;
        }
      }
    }
    __syncwarp();
    if (lane == 0) bar_arrive(smem_addr(&c->o_free[s]));
  }
}

template <typename T, int DP, bool PAIR>
__device__ __forceinline__ void run_roles(const AttnParams& P, Control* c, unsigned char* tiles, const CUtensorMap* qmap,
                                          const CUtensorMap* kmap,
                                          const CUtensorMap* vmap) {
  using S = Shape<DP, PAIR>;
  const int warp = threadIdx.x >> 5;
  const int s = warp < 8 ? warp >> 2 : (warp - 8) >> 1;
  const uint32_t q_smem = smem_addr(tiles), ring = q_smem + 2 * S::q_bytes;
  const Walk w = c->start[s];
  // the launch's registers (384 threads x 168) where they are needed: 256 x 200 +
  // 128 x 104 (a pair's 128 scores a thread: attn of 256 requests 257 -> 252 us; with
  // 208 and 88 the copy and matrix warps spill: 301 us)
  if (warp < 8)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp < 8)
    softmax_role<T, DP, PAIR>(P, w, c, s, 4 * blockIdx.x + (PAIR ? s : 2 * s), tiles + 2 * S::q_bytes);
  else if (!(warp & 1))
    copy_role<DP, PAIR>(P, w, c, s, q_smem, ring, qmap, kmap, vmap);
  else
    matrix_role<T, DP, PAIR>(P, w, c, s, q_smem, ring);
  fence_before();
  __syncthreads();
  if (c->abort) {
    // a wait ran out: copies and products in flight end (each wait bounded)
    // before shared and tensor memory are given back
    int ignored = 0;
    if (warp == 8 || warp == 10) {
      if (c->q_copied[s] > 0)
        (void)bar_wait(smem_addr(&c->q_full[s]), (c->q_copied[s] - 1) & 1, kDrainNs, &ignored);
      // the copies started last, one a slot of the ring (A: every other entry is
      // this warp's, in five slots of either ring size)
      constexpr int kKept = PAIR ? 5 : S::slots;
      const int first = PAIR ? 0 : s * S::slots, by = PAIR ? 2 : 1;
      const int end = (int)c->kv_copied[s], from = end > kKept ? end - kKept : 0;
#pragma unroll 1
      for (int k = from; k < end; ++k) {
        const int e = k * by + (PAIR ? s : 0);
        (void)bar_wait(smem_addr(&c->kv_full[first + e % S::slots]), (e / S::slots) & 1, kDrainNs, &ignored);
      }
    } else if (warp >= 8) {
      if (elect_one()) mma_commit(smem_addr(&c->drain[s]));
      __syncwarp();
      (void)bar_wait(smem_addr(&c->drain[s]), 0, kDrainNs, &ignored);
    }
    __syncthreads();
  }
}

struct Maps {
  CUtensorMap q[2], k, v;  // queries of a request's own block, and of a prefix block
};

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams P) {
  using S = Shape<DP, false>;
  extern __shared__ __align__(1024) unsigned char tiles[];
  Control* c = reinterpret_cast<Control*>(tiles + 2 * S::q_bytes + S::ring);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_addr(tiles) & 1023) {  // the swizzle's period; never expected
    if (tid == 0) atomicOr(P.status, (unsigned int)SV_STATUS_INTERNAL);
    return;
  }
  // what needs no input is set up before the kernel ahead in the stream has ended
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&c->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else if (warp == 8 && lane < 4) {
    const CUtensorMap* map = lane < 2 ? maps.q + lane : lane == 2 ? &maps.k : &maps.v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  } else if (tid == kThreads - 1) {
    c->abort = 0;
    c->q_copied[0] = c->q_copied[1] = c->kv_copied[0] = c->kv_copied[1] = 0;
    for (int s = 0; s < 2; ++s) {
      c->start[s].left = 0;
      bar_init(smem_addr(&c->q_full[s]), 1);
      bar_init(smem_addr(&c->q_empty[s]), 1);
      for (int i = 0; i < 2; ++i) {
        bar_init(smem_addr(&c->s_full[s][i]), 1);
        bar_init(smem_addr(&c->p_ready[s][i]), 4);
      }
      bar_init(smem_addr(&c->o_full[s]), 1);
      bar_init(smem_addr(&c->o_free[s]), 4);
      bar_init(smem_addr(&c->drain[s]), 1);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the requests' tiles, scanned
  unsigned int flags = 0;
  const int chunk = (P.B + kThreads - 1) / kThreads;
  const int b0 = tid * chunk < P.B ? tid * chunk : P.B;
  const int b1 = b0 + chunk < P.B ? b0 + chunk : P.B;
  Req r{0, 0, 0};  // the thread's last request: its only one up to 384 requests
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
  __syncthreads();
  const int singles = single_tiles(P);
  int excl = list_add(singles, incl - mine), total = singles;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int v = c->scan[i];
    if (i < warp) excl = list_add(excl, v);
    total = list_add(total, v);
  }
  const bool over = total >= kMaxList;  // no request's rows are worked on
  if (over) {
    total = singles;
    flags |= SV_STATUS_BAD_GAMMA;
  }
  const Plan L = make_plan(P, total, gridDim.x, pair_ctas(pair_list(P), total, gridDim.x));
  const bool pair_cta = (int)blockIdx.x < L.ctas_a;
  if (tid < 20) {
    bar_init(smem_addr(&c->kv_full[tid]), 1);
    bar_init(smem_addr(&c->kv_empty[tid]), pair_cta ? 2 : 1);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // where the streams' shares begin, found by the thread whose requests hold it
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int per = pair_cta ? L.per_a : L.per_b, end = pair_cta ? L.a : L.b;
    const int g0 = per * (pair_cta ? (int)blockIdx.x : 2 * ((int)blockIdx.x - L.ctas_a) + s);
    const int left = end - g0 < per ? end - g0 : per;
    if (left <= 0) continue;
    const bool unit = pair_cta || g0 < singles;
    if (unit ? tid == 0 : g0 >= excl && g0 < excl + mine) {
      Walk w;
      w.left = left;
      w.pair = pair_cta;
      w.single = unit && !pair_cta;
      w.unit = w.b = w.rb = w.h = w.off = 0;
      w.r = r;
      if (unit) {
        const int t = pair_cta ? P.pair_tiles + kStartA : P.prefix_tiles + kStartB;
        w.unit = g0 / t;
        w.off = g0 - w.unit * t;
      } else {
        int rem = g0 - excl;
        unsigned int ignored = 0;
#pragma unroll 1
        for (w.b = b0; w.b < b1 - 1; ++w.b) {
          const int t = request_tiles(P, request(P, w.b, ignored));
          if (rem < t) break;
          rem -= t;
        }
        if (b1 - b0 > 1) w.r = request(P, w.b, ignored);
        if (w.r.n > P.tpq) {
          // the last block that begins at or before `rem`
          int above = (w.r.n - 1) / P.tpq + 1;
#pragma unroll 1
          while (above - w.rb > 1) {
            const int mid = (w.rb + above) / 2;
            if (blocks_before(P, w.r, mid) * P.Hk <= rem)
              w.rb = mid;
            else
              above = mid;
          }
          rem -= blocks_before(P, w.r, w.rb) * P.Hk;
        }
        const int t = tiles_of(block_keys(P, w.r, w.rb)) + kStartB;
        w.h = share_of(rem, t, 1.f / (float)t);
        w.off = rem - w.h * t;
      }
      c->start[s] = w;
    }
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
    if (tid == 0) {
      P.starts[P.B] = over ? -1 : total;
      P.starts[P.B + 1] = L.ctas_a;
    }
    if (flags) atomicOr(P.status, flags);
  }
  fence_before();
  __syncthreads();
  fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (pair_cta)
    run_roles<T, DP, true>(P, c, tiles, maps.q, &maps.k, &maps.v);
  else
    run_roles<T, DP, false>(P, c, tiles, maps.q, &maps.k, &maps.v);
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(c->tmem));
  }
  if (tid == 0 && c->abort) atomicOr(P.status, (unsigned int)SV_STATUS_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Joining parts: o = sum 2^(lse_i - m) o_i / sum 2^(lse_i - m), one warp a row
// ---------------------------------------------------------------------------
// The parts of one row: the prefix's, then the own.
struct Unit {
  bool pair;
  int c0, count;   // first share, shares
  int slot_row, stream;
};

// A group of DP / 8 lanes a row, each with eight neighbouring values; or, where few
// rows have many parts (MANY; one request of 131000 tokens: 38), a CTA a row, whose
// groups share the row's parts and are joined at the end.
template <typename T, int DP, bool MANY>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ AttnParams P, int ctas) {
  constexpr int kLanes = DP / 8, kGroups = 32 / kLanes;  // lanes of a group, groups of a warp
  __shared__ float s_o[4][DP], s_m[4], s_l[4];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int in = lane % kLanes, group = lane / kLanes;
  unsigned int ignored = 0;
  const Req r = request(P, b, ignored);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's writes
  const int list = P.starts[P.B];
  if (r.n <= 0 || list < 0) return;
  const Plan L = make_plan(P, list, ctas, P.starts[P.B + 1]);
  const int first = P.starts[b];
  if (L.per_b <= 0) return;
  const float inv_a = 1.f / (float)(L.per_a > 0 ? L.per_a : 1), inv_b = 1.f / (float)L.per_b;
  // without a prefix, requests whose units all lie within one share are done
  if (P.prefix_len == 0 &&
      share_of(first, L.per_b, inv_b) == share_of(first + request_tiles(P, r) - 1, L.per_b, inv_b))
    return;
  const int rows = r.n * P.Hq;
  constexpr int kRowsCta = MANY ? 1 : 4 * kGroups;
  const int x0 = blockIdx.y * kRowsCta + (MANY ? 0 : warp * kGroups + group);
#pragma unroll 1
  for (int x = x0; x - (MANY ? 0 : group) < rows; x += gridDim.y * kRowsCta) {
    const bool live = x < rows;
    const int i = divide(live ? x : 0, P.by_heads), head = (live ? x : 0) - i * P.Hq;
    const int h = divide(head, P.by_group), g = head - h * P.group;
    const size_t at = (size_t)(r.row0 + i) * P.Hq + head;
    const int rb = divide(i, P.by_tpq);
    int u0 = first + blocks_before(P, r, rb) * P.Hk;
    const int tiles = tiles_of(block_keys(P, r, rb));
    u0 += h * (tiles + kStartB) + kStartB;  // its first tile
    Unit own, pre;
    own.pair = false;
    own.c0 = share_of(u0, L.per_b, inv_b);
    own.count = share_of(u0 + tiles - 1, L.per_b, inv_b) - own.c0 + 1;
    own.slot_row = (i - rb * P.tpq) * P.group + g;
    own.stream = 0;
    pre = own;
    pre.count = 0;
    int blk = 0;
    if (P.prefix_len > 0) {
      const int t = r.row0 + i;
      blk = divide(t, P.by_tpq);
      pre.pair = blk < 2 * P.pairs;
      pre.slot_row = (t - blk * P.tpq) * P.group + g;
      pre.stream = blk & 1;
      const int per = pre.pair ? L.per_a : L.per_b;
      const float inv = pre.pair ? inv_a : inv_b;
      const int t_unit = pre.pair ? P.pair_tiles : P.prefix_tiles;
      const int start = pre.pair ? kStartA : kStartB;
      const int v0 = (pre.pair ? h * P.pairs + blk / 2 : h) * (t_unit + start) + start;
      pre.c0 = share_of(v0, per, inv);
      pre.count = share_of(v0 + t_unit - 1, per, inv) - pre.c0 + 1;
    }
    const bool done = P.prefix_len == 0 && own.count == 1;  // written already
    const int parts = live && !done ? pre.count + own.count : 0;
    // where part k lies: its first eight values, the way to the next eight, its sum
    auto place = [&](int k, const float*& src, int& jump, const float*& lse) {
      const Unit& u = k < pre.count ? pre : own;
      const int j = k < pre.count ? k : k - pre.count;
      if (u.count == 1 && k >= pre.count) {
        src = P.own + at * DP;
        lse = P.own_lse + at;
        jump = 8;
        return;
      }
      const int c = u.c0 + j;
      const size_t tile =
          u.count == 1 ? (size_t)h * (2 * P.pairs + P.odd) + blk
                       : (size_t)(u.pair ? 4 * c + u.stream + 2 * (j == 0)
                                         : 4 * (L.ctas_a + c / 2) + 2 * (c & 1) + (j == 0));
      src = (u.count == 1 ? P.whole : P.slot) + tile * kRows * DP + u.slot_row * 8;
      lse = (u.count == 1 ? P.whole_lse : P.slot_lse) + tile * kRows + u.slot_row;
      jump = kRows * 8;
    };
    float o[8], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) o[y] = 0.f;
    constexpr int kAhead = MANY ? 8 : 5, kStep = MANY ? 4 * kGroups : 1;
#pragma unroll 1
    for (int k0 = MANY ? warp * kGroups + group : 0; k0 < parts; k0 += kAhead * kStep) {
      float v[kAhead][8], e[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int k = k0 + j * kStep;
        e[j] = -INFINITY;
        if (k < parts) {
          const float *src, *lse;
          int jump;
          place(k, src, jump, lse);
          e[j] = *lse;
          const float4 a = *reinterpret_cast<const float4*>(src + in * jump),
                       c = *reinterpret_cast<const float4*>(src + in * jump + 4);
          v[j][0] = a.x, v[j][1] = a.y, v[j][2] = a.z, v[j][3] = a.w;
          v[j][4] = c.x, v[j][5] = c.y, v[j][6] = c.z, v[j][7] = c.w;
        }
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) top = fmaxf(top, e[j]);  // (a NaN is dropped here, and kept by its weight)
      const float scale = m == -INFINITY ? 0.f : exp2f(m - top);
      l *= scale;
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] *= scale;
      m = top;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (e[j] == -INFINITY) continue;  // no key seen there
        const float w = exp2f(e[j] - top);
        l += w;
#pragma unroll
        for (int y = 0; y < 8; ++y) o[y] += v[j][y] * w;
      }
    }
    if (MANY && done) continue;  // (one row a CTA: all of it)
    if (MANY) {
      // the groups' joins, in a fixed order
#pragma unroll
      for (int d = kLanes; d < 32; d <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, d), l2 = __shfl_xor_sync(0xffffffffu, l, d);
        const float top = fmaxf(m, m2);
        const float f = m == -INFINITY ? (l != l ? 1.f : 0.f) : exp2f(m - top);
        const float f2 = m2 == -INFINITY ? (l2 != l2 ? 1.f : 0.f) : exp2f(m2 - top);
        l = l * f + l2 * f2;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float o2 = __shfl_xor_sync(0xffffffffu, o[y], d);
          o[y] = (f == 0.f ? 0.f : o[y] * f) + (f2 == 0.f ? 0.f : o2 * f2);
        }
        m = top;
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int y = 0; y < 8; ++y) s_o[warp][in * 8 + y] = o[y];
        if (in == 0) s_m[warp] = m, s_l[warp] = l;
      }
      __syncthreads();
      if (warp == 0 && group == 0) {
        m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        l = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) o[y] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = s_m[k] == -INFINITY ? (s_l[k] != s_l[k] ? 1.f : 0.f) : exp2f(s_m[k] - m);
          l += s_l[k] * f;
#pragma unroll
          for (int y = 0; y < 8; ++y) o[y] += f == 0.f ? 0.f : s_o[k][in * 8 + y] * f;
        }
      }
    }
    if (!live || done || (MANY && (warp != 0 || group != 0))) continue;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    if (in * 8 < P.D) {
      uint4 q;
      q.x = Type<T>::pack(o[0] * inv, o[1] * inv);
      q.y = Type<T>::pack(o[2] * inv, o[3] * inv);
      q.z = Type<T>::pack(o[4] * inv, o[5] * inv);
      q.w = Type<T>::pack(o[6] * inv, o[7] * inv);
      *reinterpret_cast<uint4*>(P.out + (at * P.D + in * 8) * 2) = q;
    }
    if (P.lse && in == 0) P.lse[at] = (m + log2f(l)) * 0.693147180559945309f;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

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

// A map of four dimensions, values innermost; strides in elements.
bool encode(CUtensorMap* map, sv_dtype dtype, const void* base, const uint64_t (&dims)[4],
            const int64_t (&strides)[3], const uint32_t (&box)[4]) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t x[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < 4; ++i) d[i] = dims[i], x[i] = box[i];
  for (int i = 0; i < 3; ++i) s[i] = (cuuint64_t)strides[i] * 2;
  return fn(map, dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), d, s, x, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttnLayout {
  size_t starts, own, own_lse, whole, whole_lse, slot, slot_lse, total;
};
AttnLayout attn_layout(long long T, int Hq, int D) {
  const size_t dp = D <= 64 ? 64 : 128, rows = (size_t)T * Hq;
  // blocks of the prefix in every grouping of the heads: a block holds at least
  // kRows / 2 + 1 rows (kRows - group + 1 of a larger group) but the last of a key head
  const size_t tiles = rows / (kRows / 2) + Hq;
  AttnLayout L;
  size_t at = 256;  // the status word
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += sv::align256(bytes);
    return a;
  };
  L.starts = take((size_t)(T + 2) * sizeof(int));
  L.own = take(rows * dp * 4);
  L.own_lse = take(rows * 4);
  L.whole = take(tiles * kRows * dp * 4);
  L.whole_lse = take(tiles * kRows * 4);
  L.slot = take((size_t)kSlots * kRows * dp * 4);
  L.slot_lse = take((size_t)kSlots * kRows * 4);
  L.total = at;
  return L;
}

template <typename T, int DP>
int grid_size() {
  static std::atomic<int> cached{0};
  int dev = 0, sms = 0;
  if (sv::code_of(cudaGetDevice(&dev))) return 0;
  const int c0 = cached.load(std::memory_order_relaxed);
  if ((c0 >> 16) == dev + 1) return c0 & 0xffff;
  if (sv::code_of(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) ||
      sv::code_of(cudaFuncSetAttribute(attention_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Shape<DP, false>::smem)))
    return 0;
  sms = sms < kMaxCtas ? sms : kMaxCtas;
  cached.store(((dev + 1) << 16) | sms, std::memory_order_relaxed);
  return sms;
}

template <typename T, int DP>
int launch(const Maps& m, const AttnParams& P, cudaStream_t stream) {
  const int grid = grid_size<T, DP>();
  if (grid <= 0) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned int)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<DP, false>::smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  sv::overlap_launch(at[0]);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int rc = sv::code_of(cudaLaunchKernelEx(&cfg, attention_kernel<T, DP>, m, P));
  if (rc) return rc;
  // The launch itself overlaps the attention kernel, whose end the CTAs wait for.
  // A CTA a row where the shares are more than eight times the units (counted at their most:
  // a row block has a unit a key head) and the rows no more than 16 an SM.
  // By a CTA a row and by lane groups, 304 shares: one request of 131000 tokens and 8 rows of
  // 64 heads (8 units, 512 rows and heads) 98 and 117 us; four of 30000 tokens (32, 1024)
  // 91 and 93; 64 rows of 32 heads behind 30000 tokens (16, 2048) 55 both, 128 rows
  // (32, 4096) 91 and 79; a prompt of 128 rows (32, 4096) 25 and 17, of 2500 (632, 80000)
  // 254 and 95.
  const long long longest = P.G < P.T ? P.G + 1 : P.T;
  const long long by_longest = (longest + P.tpq - 1) / P.tpq * P.B, by_rows = P.T / P.tpq + (long long)P.B;
  const bool many = 2ll * grid > 8 * P.Hk * (by_longest < by_rows ? by_longest : by_rows) &&
                    (long long)P.T * P.Hq <= 16ll * grid;
  const long long rows = longest * P.Hq;
  const int per_cta = many ? 1 : 4 * (32 / (DP / 8));
  const long long y = (rows + per_cta - 1) / per_cta;
  cfg.gridDim = dim3((unsigned int)P.B, (unsigned int)(y < 1024 ? y : 1024));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return sv::code_of(
      cudaLaunchKernelEx(&cfg, many ? combine_kernel<T, DP, true> : combine_kernel<T, DP, false>, P, grid));
}

}  // namespace

extern "C" {

size_t spec_verify_attention_workspace_size(int total_rows, int q_heads, int head_dim) {
  if (total_rows < 0 || q_heads < 1 || q_heads > 65535 || head_dim < 8 || head_dim > SV_MAX_HEAD_DIM ||
      head_dim % 8)
    return 0;
  return attn_layout(total_rows, q_heads, head_dim).total;
}

int spec_verify_attention(const void* q, const int64_t* q_strides, int q_heads,
                          const sv_kv_cache* cache, const int32_t* prefix_table, int prefix_len,
                          const int32_t* cu_draft, int total_drafts, int max_drafts, float scale,
                          const uint32_t* draft_mask, void* out, float* lse, void* workspace,
                          size_t ws_bytes, sv_stream_t stream) {
  if (!cache || !q_strides) return SV_ERR_NULL;
  const sv_kv_cache& c = *cache;
  int rc = sv::check_cache(c);
  if (rc) return rc;
  const long long rows = (long long)total_drafts + c.batch;
  if (total_drafts < 0 || max_drafts < 0 || rows > INT32_MAX || prefix_len < 0 ||
      prefix_len > kMaxKeys || q_heads < 1 ||
      q_heads > 65535 || q_heads % c.kv_heads || q_heads / c.kv_heads > kRows || !(scale > 0.f) ||
      !std::isfinite(scale * 1.44269504f) || (draft_mask && max_drafts > SV_MAX_GAMMA))
    return SV_ERR_SCALAR;
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] <= 0 || q_strides[i] % 8 || q_strides[i] >= ((int64_t)1 << 38)) return SV_ERR_SCALAR;
  if (c.batch == 0) return SV_OK;
  if (!q || !cu_draft || !out || !workspace || (prefix_len > 0 && !prefix_table)) return SV_ERR_NULL;
  if (!sv::aligned(q, 16) || !sv::aligned(out, 16) || !sv::aligned(lse, 4) ||
      !sv::aligned(cu_draft, 4) || !sv::aligned(prefix_table, 4) || !sv::aligned(draft_mask, 4) ||
      !sv::aligned(workspace, 256))
    return SV_ERR_ALIGN;
  const AttnLayout L = attn_layout(rows, q_heads, c.head_dim);
  if (ws_bytes < L.total) return SV_ERR_WORKSPACE;
  // every row's output is written while other rows' queries may still be read
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  const uintptr_t q_end = qa + 2 * ((uint64_t)(rows - 1) * (uint64_t)q_strides[0] +
                                    (uint64_t)(q_heads - 1) * (uint64_t)q_strides[1] + (uint64_t)c.head_dim);
  const uintptr_t o_end = oa + 2 * (uint64_t)rows * (uint64_t)q_heads * (uint64_t)c.head_dim;
  if (qa < o_end && oa < q_end) return SV_ERR_ALIGN;
  AttnParams P = {};
  P.B = c.batch;
  P.T = (int)rows;
  P.G = max_drafts;
  P.total = total_drafts;
  P.Hq = q_heads;
  P.Hk = c.kv_heads;
  P.D = c.head_dim;
  P.group = q_heads / c.kv_heads;
  P.tpq = kRows / P.group;
  P.by_heads = divisor(P.Hq);
  P.by_group = divisor(P.group);
  P.by_tpq = divisor(P.tpq);
  P.own_tok = max_drafts < P.tpq ? max_drafts + 1 : P.tpq;
  P.num_pages = c.num_pages;
  P.page_size = c.page_size;
  while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
  P.max_pages = c.max_pages;
  P.box_rows = c.page_size < kTile ? c.page_size : kTile;
  P.table = c.page_table;
  P.kv_len = c.kv_len;
  P.cu = cu_draft;
  P.prefix_table = prefix_table;
  const long long room = (long long)c.max_pages * c.page_size;
  P.max_keys = room < kMaxKeys ? (int)room : kMaxKeys;
  P.prefix_len = prefix_len;
  P.prefix_tiles = (prefix_len + kTile - 1) / kTile;
  P.pair_tiles = (prefix_len + kPairTile - 1) / kPairTile;
  if (prefix_len > 0) {
    const int blocks = (P.T + P.tpq - 1) / P.tpq;
    P.pairs = blocks / 2;
    P.odd = blocks & 1;
  }
  // the longest lists that the arguments allow (the prefix's single block stands in B)
  const double reach = (double)c.max_pages * c.page_size / kTile + 1.0 + kStartB;
  const double prefix = P.Hk * ((double)P.prefix_tiles + kStartA);
  if (((double)rows / P.tpq + c.batch) * P.Hk * reach + prefix >= (double)kMaxList ||
      ((double)rows / P.tpq + 1.0) * prefix >= (double)kMaxList)
    return SV_ERR_SCALAR;
  P.mask = draft_mask;
  P.sl2 = scale * 1.44269504088896341f;
  P.out = static_cast<char*>(out);
  P.lse = lse;
  char* w = static_cast<char*>(workspace);
  P.status = reinterpret_cast<unsigned int*>(w);
  P.starts = reinterpret_cast<int*>(w + L.starts);
  P.own = reinterpret_cast<float*>(w + L.own);
  P.own_lse = reinterpret_cast<float*>(w + L.own_lse);
  P.whole = reinterpret_cast<float*>(w + L.whole);
  P.whole_lse = reinterpret_cast<float*>(w + L.whole_lse);
  P.slot = reinterpret_cast<float*>(w + L.slot);
  P.slot_lse = reinterpret_cast<float*>(w + L.slot_lse);
  P.wait_ns = sv::wait_limit_ns();
  Maps m;
  const uint64_t D = (uint64_t)c.head_dim;
  const uint64_t qd[4] = {D, (uint64_t)P.group, (uint64_t)P.Hk, (uint64_t)P.T};
  const int64_t qs[3] = {q_strides[1], q_strides[1] * P.group, q_strides[0]};
  const uint32_t q_own[4] = {64, (uint32_t)P.group, 1, (uint32_t)P.own_tok};
  const uint32_t q_pre[4] = {64, (uint32_t)P.group, 1, (uint32_t)P.tpq};
  const uint64_t cd[4] = {D, (uint64_t)c.page_size, (uint64_t)c.kv_heads, (uint64_t)c.num_pages};
  const int64_t ks[3] = {c.k_strides[1], c.k_strides[2], c.k_strides[0]};
  const int64_t vs[3] = {c.v_strides[1], c.v_strides[2], c.v_strides[0]};
  const uint32_t cb[4] = {64, (uint32_t)P.box_rows, 1, 1};
  if (!encode(&m.q[0], c.dtype, q, qd, qs, q_own) || !encode(&m.q[1], c.dtype, q, qd, qs, q_pre) ||
      !encode(&m.k, c.dtype, c.k_pages, cd, ks, cb) || !encode(&m.v, c.dtype, c.v_pages, cd, vs, cb))
    return SV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c.dtype == SV_BF16)
    return c.head_dim <= 64 ? launch<__nv_bfloat16, 64>(m, P, s) : launch<__nv_bfloat16, 128>(m, P, s);
  return c.head_dim <= 64 ? launch<__half, 64>(m, P, s) : launch<__half, 128>(m, P, s);
}

}  // extern "C"
