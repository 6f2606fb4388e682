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
// own keys, or (pair of blocks of all requests' rows, key head) over the
// prefix.  The units' tiles of 128 keys, prefix first, form one list, and each
// of the CTAs (one an SM) takes an equal contiguous share of it, so a batch of
// any raggedness, or one long request, loads every SM alike.  A unit that
// crosses a share's border leaves one part a CTA; combine_kernel joins them
// (and the prefix with the own keys) by their sums.  No part is waited for
// inside a kernel, and parts are joined in list order: results repeat bit for
// bit.
//
// A CTA: two softmax warpgroups, a copy warp and a matrix warp.  Query blocks
// are 128 rows (tokens x heads of the key head's group).  S = Q K^T and
// O += P V are tcgen05 products with S, P and O in tensor memory: two streams
// of (S, O), 512 columns.  With two row blocks (prefix) each stream has one
// and both read every tile; with one, the streams take the tiles in turn and
// are joined at the end, so that one stream's softmax runs beside the other's
// products.  Keys and values arrive by TMA, a page (at most 128 tokens) and 64
// values a box, in a ring of slots with 128-byte swizzle; the layout in the
// page pool is only the tensor map's strides.
//
// S and the sums are 32 bits.  P is rounded to the cache's 16-bit type for the
// product (at most half a step of a weight, below the rounding of the output's
// own type where weights are spread); the sum of weights uses the unrounded
// ones.  The running maximum moves only when it grows by more than 8 (a factor
// of 256 in P, harmless in 32 bits and in the range of fp16), which makes the
// rescaling of O rare.
#include "../../include/spec_verify.h"
#include "internal.h"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <mutex>

namespace {

constexpr int kTile = 128;      // keys a tile, rows a block
constexpr int kThreads = 320;   // warps 0-3 and 4-7: softmax; 8: copies; 9: products
constexpr int kMaxCtas = 160;   // shares of the tile list (partial slots are sized for this)
constexpr int kSlotRows = 256;
constexpr unsigned long long kDrainNs = 2000000000ull;  // limit of the waits that end an aborted CTA
constexpr int kControl = 3072;  // barriers and small tables behind the tiles

template <int DP>
struct Shape {
  static constexpr int halves = DP / 64;
  static constexpr int tile_bytes = kTile * DP * 2;
  static constexpr int half_bytes = kTile * 128;  // 64 values of every token
  static constexpr int slots = DP == 128 ? 5 : 8;
  static constexpr int smem = (slots + 2) * tile_bytes + kControl;
  static_assert(smem <= 227 * 1024, "shared memory");
};

struct AttnParams {
  int B, T, G, total, Hq, Hk, D, group, tpq, own_tok;
  int num_pages, page_size, page_shift, max_pages, box_rows;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  const int32_t* prefix_table;
  int prefix_len, prefix_tiles, prefix_blocks, prefix_units;
  const uint32_t* mask;
  float sl2;  // scale log2(e)
  char* out;
  float* lse;
  unsigned int* status;
  long long* starts;   // [B + 1]: first tile of each request, and the total
  float* dense[2];     // own, prefix: rows of whole units [T * Hq][DP]
  float* dense_lse[2];
  float* slot;         // [2 * kMaxCtas][kSlotRows][DP]
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
// or another warp of the CTA gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned long long wait_ns,
                                         volatile int* abort) {
  // ordinary waits end within these tries (a try suspends the warp for a while
  // itself) and read no timer
  for (int i = 0; i < 256; ++i)
    if (bar_try(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (bar_try(bar, parity)) return true;
    if (*abort) return false;
    if (now_ns() - t0 > wait_ns) {
      *abort = 1;
      return false;
    }
  }
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
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
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
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};
template <>
struct Type<__half> {
  static constexpr uint32_t fmt = 0;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};
// 32-bit accumulators, A and B of one 16-bit type
__host__ __device__ constexpr uint32_t instr_desc(uint32_t fmt, uint32_t n, bool b_mn) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((n / 8) << 17) |
         ((uint32_t)(kTile / 16) << 24);
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
  const int c0 = P.cu[b], c1 = P.cu[b + 1], kv = P.kv_len[b];
  Req r{0, 0, 0};
  if (c0 < 0 || c1 < c0 || c1 - c0 > P.G || c1 > P.total) {
    flags |= SV_STATUS_BAD_GAMMA;
  } else if (kv < 0 || (long long)kv + (c1 - c0) + 1 > (long long)P.max_pages * P.page_size) {
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
__device__ __forceinline__ long long request_tiles(const AttnParams& P, const Req& r) {
  if (r.n <= 0) return 0;
  long long t = 0;
  for (int rb = 0; rb * P.tpq < r.n; ++rb) t += tiles_of(block_keys(P, r, rb));
  return t * P.Hk;
}

// One CTA's run of tiles of one unit.
struct Piece {
  bool prefix, two;  // two row blocks, one a stream; else the streams share one
  int b, h;
  int row0, ntok;    // first row and rows of the block(s)
  int kv;            // own: keys before the step; row i of the block sees kv + first + i + 1
  int first;         // own: the block's first row within the request
  int keys;          // keys of the unit
  int t0, t1;        // tiles [t0, t1) of unit_t
  int unit_t;
};

// Walks a CTA's share.  Every role walks it alone, from the same start.
struct Walk {
  long long left;
  bool prefix;
  int unit;         // prefix unit
  int b, rb, h;     // own unit
  int off;          // first tile within the unit
  Req r;

  __device__ __forceinline__ void load_request(const AttnParams& P) {
    unsigned int ignored = 0;
    r = Req{0, 0, 0};
    while (b < P.B) {
      r = request(P, b, ignored);
      if (r.n > 0) return;
      ++b;
    }
  }
  __device__ __forceinline__ bool next(const AttnParams& P, Piece& p) {
    if (left <= 0) return false;
    if (prefix && unit >= P.prefix_units) {
      prefix = false;
      b = rb = h = off = 0;
      load_request(P);
    }
    if (prefix) {
      p.prefix = true;
      p.b = 0;
      p.h = unit / P.prefix_blocks;
      p.row0 = (unit - p.h * P.prefix_blocks) * 2 * P.tpq;
      p.ntok = P.T - p.row0 < 2 * P.tpq ? P.T - p.row0 : 2 * P.tpq;
      p.two = p.ntok > P.tpq;
      p.kv = p.first = 0;
      p.keys = P.prefix_len;
      p.unit_t = P.prefix_tiles;
    } else {
      if (b >= P.B) return false;
      p.prefix = p.two = false;
      p.b = b;
      p.h = h;
      p.first = rb * P.tpq;
      p.row0 = r.row0 + p.first;
      p.ntok = r.n - p.first < P.tpq ? r.n - p.first : P.tpq;
      p.kv = r.kv;
      p.keys = block_keys(P, r, rb);
      p.unit_t = tiles_of(p.keys);
    }
    p.t0 = off;
    p.t1 = left < p.unit_t - off ? off + (int)left : p.unit_t;
    left -= p.t1 - p.t0;
    off = 0;
    if (prefix) {
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
  uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], s_full[2], p_ready[2], o_full, o_free,
      ml_ready, drain;
  uint32_t tmem;
  int abort;
  int start_b, start_prefix, start_unit, start_off, per_b;
  long long start_rem, left;
  long long scan[kThreads / 32];
  float2 ml[2][kTile];
};
static_assert(sizeof(Control) <= kControl, "control block");

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------
// The order of a piece's tiles in the ring: keys one tile ahead of values.
__device__ __forceinline__ int k_entry(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_entry(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

template <int DP>
__device__ __forceinline__ void copy_role(const AttnParams& P, Walk w, Control* c, uint32_t q_smem,
                                          uint32_t ring, const CUtensorMap* qmap,
                                          const CUtensorMap* qmap_prefix, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap, unsigned int& entry,
                                          unsigned int& qn) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  unsigned int flags = 0;
  Piece p;
  bool ok = true;
  while (ok && w.next(P, p)) {
    // the block's query rows: [token][head of the group] in 128-byte rows
    for (int s = 0; ok && s < (p.two ? 2 : 1); ++s, ++qn) {
      const uint32_t slot = qn & 1;
      ok = bar_wait(smem_addr(&c->q_empty[slot]), ((qn >> 1) & 1) ^ 1, P.wait_ns, &c->abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t bar = smem_addr(&c->q_full[slot]);
      const int box = p.prefix ? P.tpq : P.own_tok;
      if (lane == 0) {
        bar_expect(bar, (uint32_t)(S::halves * 128 * P.group * box));
        for (int x = 0; x < S::halves; ++x)
          tma_load(q_smem + slot * S::tile_bytes + x * S::half_bytes, p.prefix ? qmap_prefix : qmap, bar,
                   x * 64, 0, p.h, p.row0 + s * P.tpq);
      }
    }
    const int n = p.t1 - p.t0;
    for (int e = 0; ok && e < 2 * n; ++e, ++entry) {
      const bool is_v = e == 2 * n - 1 || (e > 0 && !(e & 1));
      const int i = is_v ? (e == 2 * n - 1 ? n - 1 : e / 2 - 1) : (e + 1) / 2;
      const int key0 = (p.t0 + i) * kTile;
      const int keys = p.keys - key0 < kTile ? p.keys - key0 : kTile;
      const int pages = (keys + P.box_rows - 1) / P.box_rows;  // boxes of at most a page
      const int boxes = pages * S::halves;
      // this lane's page, looked up before the wait for the slot
      const int pg = lane / S::halves;
      int id = 0;
      if (lane < boxes) {
        const int key = key0 + pg * P.box_rows;
        id = p.prefix ? P.prefix_table[key >> P.page_shift]
                      : P.table[(size_t)p.b * P.max_pages + (key >> P.page_shift)];
        if (id < 0 || id >= P.num_pages) {
          flags |= SV_STATUS_BAD_PAGE;
          id = P.num_pages;  // past the pool: the copy fills zeros
        }
      }
      const uint32_t slot = entry % S::slots;
      ok = bar_wait(smem_addr(&c->kv_empty[slot]), ((entry / S::slots) & 1) ^ 1, P.wait_ns, &c->abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t bar = smem_addr(&c->kv_full[slot]);
      if (lane == 0) bar_expect(bar, (uint32_t)(boxes * 128 * P.box_rows));
      __syncwarp();
      if (lane < boxes) {
        const int half = lane - pg * S::halves;
        const int key = key0 + pg * P.box_rows;
        tma_load(ring + slot * S::tile_bytes + half * S::half_bytes + pg * P.box_rows * 128,
                 is_v ? vmap : kmap, bar, half * 64, key & (P.page_size - 1), p.h, id);
      }
    }
  }
  const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && any) atomicOr(P.status, any);
}

template <typename T, int DP>
__device__ __forceinline__ void matrix_role(const AttnParams& P, Walk w, Control* c, uint32_t q_smem,
                                            uint32_t ring, unsigned char* ring_ptr) {
  using S = Shape<DP>;
  const int lane = threadIdx.x & 31;
  const uint32_t tmem = c->tmem;
  constexpr uint32_t kQk = instr_desc(Type<T>::fmt, kTile, false);
  constexpr uint32_t kPv = instr_desc(Type<T>::fmt, DP, true);
  unsigned int base = 0, qn = 0, pieces = 0, np[2] = {0, 0};
  Piece p;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = bar_wait(smem_addr(bar), parity, P.wait_ns, &c->abort);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  while (ok && w.next(P, p)) {
    const int n = p.t1 - p.t0, nv = p.two ? 2 * n : n;
    // S of virtual tile j: stream j & 1
    auto qk = [&](int j) {
      const int s = j & 1, i = p.two ? j >> 1 : j;
      const unsigned int e = base + k_entry(i), slot = e % S::slots;
      const unsigned int qs = (p.two ? qn + s : qn) & 1, qp = ((p.two ? qn + s : qn) >> 1) & 1;
      if ((p.two ? j < 2 : j == 0) && !wait(&c->q_full[qs], qp)) return;
      if ((!p.two || s == 0) && !wait(&c->kv_full[slot], (e / S::slots) & 1)) return;
      if (lane == 0) {
        const uint32_t a = q_smem + qs * S::tile_bytes, b = ring + slot * S::tile_bytes;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t at = (k / 4) * S::half_bytes + (k % 4) * 32;
          mma_ss(tmem + s * kTile, mat_desc(a + at, 16), mat_desc(b + at, 16), kQk, k > 0);
        }
        mma_commit(smem_addr(&c->s_full[s]));
        if (!p.two || s == 1) mma_commit(smem_addr(&c->kv_empty[slot]));
        if (j + (p.two ? 2 : 1) >= nv) mma_commit(smem_addr(&c->q_empty[qs]));
      }
      __syncwarp();
    };
    for (int j = 0; ok && j < 2 && j < nv; ++j) qk(j);
    for (int j = 0; ok && j < nv; ++j) {
      const int s = j & 1, i = p.two ? j >> 1 : j;
      const unsigned int e = base + v_entry(i, n), slot = e % S::slots;
      if (j == 0 && pieces > 0 && !wait(&c->o_free, (pieces - 1) & 1)) break;
      int keys = p.keys - (p.t0 + i) * kTile;
      keys = keys < kTile ? keys : kTile;
      const int steps = (keys + 15) / 16;
      if (!p.two || s == 0) {
        if (!wait(&c->kv_full[slot], (e / S::slots) & 1)) break;
        if (keys & 15) {
          // rows behind the last key of the last 16: what memory held there
          // (weights of 0 times NaN would be NaN)
          for (int x = lane; x < (steps * 16 - keys) * S::halves * 8; x += 32) {
            const int row = keys + x / (S::halves * 8), in = x % (S::halves * 8);
            *reinterpret_cast<uint4*>(ring_ptr + slot * S::tile_bytes + (in / 8) * S::half_bytes +
                                      row * 128 + (in % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
      }
      if (!wait(&c->p_ready[s], np[s] & 1)) break;
      ++np[s];
      fence_after();
      if (lane == 0) {
        const uint32_t b = ring + slot * S::tile_bytes;
        const uint32_t a = tmem + s * kTile, d = tmem + 2 * kTile + s * kTile;
        for (int k = 0; k < steps; ++k)
          mma_ts(d, a + k * 8, mat_desc(b + k * 2048, S::half_bytes), kPv, j > 1 || k > 0);
        if (!p.two || s == 1) mma_commit(smem_addr(&c->kv_empty[slot]));
        if (j == nv - 1) mma_commit(smem_addr(&c->o_full));
      }
      __syncwarp();
      if (j + 2 < nv) qk(j + 2);
    }
    base += 2 * n;
    qn += p.two ? 2 : 1;
    ++pieces;
  }
}

template <typename T, int DP>
__device__ __forceinline__ void softmax_role(const AttnParams& P, Walk w, Control* c) {
  const int wg = threadIdx.x >> 7;                       // stream
  const int row = threadIdx.x & 127, lane = row & 31;
  const uint32_t lanes = (uint32_t)(row & ~31) << 16;    // this warp's tensor-memory lanes
  const uint32_t s_col = c->tmem + lanes + wg * kTile;
  const uint32_t o_col = c->tmem + lanes + 2 * kTile;
  const float ninf = -INFINITY;
  unsigned int ns = 0, pieces = 0, joins = 0;
  Piece p;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = bar_wait(smem_addr(bar), parity, P.wait_ns, &c->abort);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  const int tok = row / P.group, g = row - tok * P.group;
  while (ok && w.next(P, p)) {
    const int n = p.t1 - p.t0;
    const int blk = p.two ? wg : 0;  // row block of this stream
    const int btok = p.ntok - blk * P.tpq < P.tpq ? p.ntok - blk * P.tpq : P.tpq;
    const int rows = btok * P.group;
    const bool active = (row & ~31) < rows, mine = row < rows;
    // keys this row sees: all below `limit`, or below `free` and by its mask word
    int limit = p.prefix ? P.prefix_len : p.kv + p.first + tok + 1;
    int free = p.prefix ? P.prefix_len : (P.mask ? p.kv : p.kv + p.first + 1);
    uint32_t word = 0;
    if (!p.prefix && P.mask && mine) {
      word = P.mask[p.row0 + tok];
      if (p.keys - p.kv < 32) word &= (1u << (p.keys - p.kv)) - 1u;  // rows of the step
    }
    float m = ninf, l = 0.f;  // running maximum (times scale log2 e) and sum
    const int step = p.two ? 1 : 2;
    for (int i = p.two ? 0 : wg; i < n; i += step) {
      if (!wait(&c->s_full[wg], ns & 1)) break;
      ++ns;
      if (active) {
        fence_after();
        const int key0 = (p.t0 + i) * kTile;
        const bool masked = key0 + kTile > free;
        // keys [key0 + 32 ch, + 32) that this row does not see
        auto hide = [&](uint32_t* v, int ch) {
          const int at = key0 + 32 * ch;
          uint32_t see;  // bit x: key at + x is seen
          if (!p.prefix && P.mask) {
            const int d = at - p.kv;  // the chunk's first key in the step's rows
            see = d <= -32 ? ~0u : d < 0 ? (word << -d) | ((1u << -d) - 1u) : d < 32 ? word >> d : 0u;
          } else {
            const int n = limit - at;
            see = n >= 32 ? ~0u : n > 0 ? (1u << n) - 1u : 0u;
          }
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!((see >> x) & 1u)) v[x] = __float_as_uint(ninf);
        };
        // S is read twice, 32 columns at a time, the next ones on their way:
        // for the maximum, then for the weights (128 values held at once spill)
        uint32_t v[2][32];
        float mx0 = ninf, mx1 = ninf;
        tmem_load32(s_col, v[0]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t* u = v[ch & 1];
          tmem_wait_load();
          tmem_loaded32(u);
          tmem_load32(s_col + ((ch + 1) & 3) * 32, v[(ch + 1) & 1]);
          if (masked) hide(u, ch);
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            mx0 = max3(mx0, __uint_as_float(u[x]), __uint_as_float(u[x + 1]));
            mx1 = max3(mx1, __uint_as_float(u[x + 2]), __uint_as_float(u[x + 3]));
          }
        }
        const float top = fmaxf(mx0, mx1) * P.sl2;
        if (i < step) {
          m = top;
        } else {
          const bool grow = top > m + 8.f || (m == ninf && top > ninf);
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? (m == ninf ? 0.f : exp2_fast(m - top)) : 1.f;
            // the products so far are complete: S of this tile came after them
            for (int x = 0; x < DP; x += 16) {
              uint32_t o[16];
              tmem_load16(o_col + wg * kTile + x, o);
              tmem_wait_load();
              tmem_loaded16(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_store16(o_col + wg * kTile + x, o);
            }
            l *= f;
            if (grow) m = top;
          }
        }
        const uint64_t sub = pair(m == ninf ? 0.f : -m, m == ninf ? 0.f : -m);
        const uint64_t sl2 = pair(P.sl2, P.sl2);
        uint64_t sum0 = 0, sum1 = 0;  // two pairs of zeros
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t* u = v[ch & 1];
          tmem_wait_load();
          tmem_loaded32(u);
          if (ch < 3) tmem_load32(s_col + (ch + 1) * 32, v[(ch + 1) & 1]);
          if (masked) hide(u, ch);
          uint32_t w16[16];
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            float a, b, e, f;
            unpair(pair_fma(pair(__uint_as_float(u[x]), __uint_as_float(u[x + 1])), sl2, sub), a, b);
            unpair(pair_fma(pair(__uint_as_float(u[x + 2]), __uint_as_float(u[x + 3])), sl2, sub), e, f);
            a = exp2_fast(a), b = exp2_fast(b), e = exp2_fast(e), f = exp2_fast(f);
            sum0 = pair_add(sum0, pair(a, b));
            sum1 = pair_add(sum1, pair(e, f));
            w16[x / 2] = Type<T>::pack(a, b);
            w16[x / 2 + 1] = Type<T>::pack(e, f);
          }
          // over columns of S that are read already
          tmem_store16(s_col + ch * 16, w16);
        }
        float a, b;
        unpair(pair_add(sum0, sum1), a, b);
        l += a + b;
        tmem_wait_store();
        fence_before();
      }
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&c->p_ready[wg]));
    }
    if (!ok) break;
    // the piece's rows: this stream's columns, or half the columns of both
    const int row_t = p.row0 + blk * P.tpq + tok;
    float f0 = 0.f, f1 = 0.f, lse2;
    if (p.two) {
      f0 = l > 0.f || l != l ? 1.f / l : 0.f;
      lse2 = m + log2f(l);
    } else {
      c->ml[wg][row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&c->ml_ready));
      if (!wait(&c->ml_ready, joins & 1)) break;
      ++joins;
      const float2 a = c->ml[0][row], b = n > 1 ? c->ml[1][row] : make_float2(ninf, 0.f);
      const float mm = fmaxf(a.x, b.x);
      const float sub = mm == ninf ? 0.f : mm;
      const float wa = a.x == ninf && a.y == 0.f ? 0.f : exp2_fast(a.x - sub);
      const float wb = b.x == ninf && b.y == 0.f ? 0.f : exp2_fast(b.x - sub);
      const float ll = a.y * wa + b.y * wb;
      const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
      f0 = wa * inv;
      f1 = wb * inv;
      lse2 = mm + log2f(ll);
    }
    if (!wait(&c->o_full, pieces & 1)) break;
    ++pieces;
    if (active) {
      fence_after();
      const bool whole = p.t0 == 0 && p.t1 == p.unit_t;
      const bool direct = whole && !p.prefix && P.prefix_len == 0;
      const size_t at = (size_t)row_t * P.Hq + (size_t)p.h * P.group + g;
      float* part = nullptr;
      float* part_lse = nullptr;
      if (!direct) {
        if (whole) {
          part = P.dense[p.prefix] + at * DP;
          part_lse = P.dense_lse[p.prefix] + at;
        } else {
          const size_t r = ((size_t)blockIdx.x * 2 + (p.t0 == 0)) * kSlotRows + blk * kTile + row;
          part = P.slot + r * DP;
          part_lse = P.slot_lse + r;
        }
      }
      const int x0 = p.two ? 0 : wg * (DP / 2), x1 = p.two ? DP : x0 + DP / 2;
      const uint32_t first = o_col + (p.two ? wg * kTile : 0);
      for (int x = x0; x < x1; x += 32) {
        uint32_t o[32], o2[32];
        tmem_load32(first + x, o);
        if (!p.two && n > 1) tmem_load32(o_col + kTile + x, o2);
        tmem_wait_load();
        tmem_loaded32(o);
        if (!p.two && n > 1) {
          tmem_loaded32(o2);
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            const float a = f0 == 0.f ? 0.f : __uint_as_float(o[y]) * f0;
            const float b = f1 == 0.f ? 0.f : __uint_as_float(o2[y]) * f1;
            o[y] = __float_as_uint(a + b);
          }
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y)
            o[y] = f0 == 0.f ? 0u : __float_as_uint(__uint_as_float(o[y]) * f0);
        }
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
            for (int y = 0; y < 32; y += 4)
              *reinterpret_cast<uint4*>(part + x + y) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
        }
      }
      if (mine && (p.two || wg == 0)) {
        if (direct) {
          if (P.lse) P.lse[at] = lse2 * 0.693147180559945309f;
        } else {
          *part_lse = lse2;
        }
      }
      fence_before();
    }
    __syncwarp();
    if (lane == 0) bar_arrive(smem_addr(&c->o_free));
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap qmap_prefix,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ AttnParams P) {
  using S = Shape<DP>;
  extern __shared__ __align__(1024) unsigned char tiles[];
  Control* c = reinterpret_cast<Control*>(tiles + (S::slots + 2) * S::tile_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_addr(tiles) & 1023) {  // the swizzle's period; never expected
    if (tid == 0) atomicOr(P.status, (unsigned int)SV_STATUS_INTERNAL);
    return;
  }
  // the share of the tile list: a scan over the requests' tiles
  unsigned int flags = 0;
  const int chunk = (P.B + kThreads - 1) / kThreads;
  const int b0 = tid * chunk < P.B ? tid * chunk : P.B;
  const int b1 = b0 + chunk < P.B ? b0 + chunk : P.B;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += request_tiles(P, request(P, b, flags));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) c->scan[warp] = incl;
  if (tid == 0) {
    c->abort = 0;
    c->start_b = P.B;
    for (int i = 0; i < 8; ++i) {
      bar_init(smem_addr(&c->kv_full[i]), 1);
      bar_init(smem_addr(&c->kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&c->q_full[i]), 1);
      bar_init(smem_addr(&c->q_empty[i]), 1);
      bar_init(smem_addr(&c->s_full[i]), 1);
      bar_init(smem_addr(&c->p_ready[i]), 4);
    }
    bar_init(smem_addr(&c->o_full), 1);
    bar_init(smem_addr(&c->o_free), 8);
    bar_init(smem_addr(&c->ml_ready), 8);
    bar_init(smem_addr(&c->drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  const long long prefix_all = (long long)P.prefix_units * P.prefix_tiles;
  long long excl = prefix_all + incl - mine, total = prefix_all;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) excl += c->scan[i];
    total += c->scan[i];
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long g0 = per * blockIdx.x;
  const long long left = total - g0 < per ? total - g0 : per;
  if (blockIdx.x == 0) {
    long long at = excl;
    for (int b = b0; b < b1; ++b) {
      P.starts[b] = at;
      unsigned int ignored = 0;
      at += request_tiles(P, request(P, b, ignored));
    }
    if (tid == 0) P.starts[P.B] = total;
    if (flags) atomicOr(P.status, flags);
  }
  if (left <= 0) return;  // the whole CTA
  if (g0 >= prefix_all && g0 >= excl && g0 < excl + mine) {
    long long at = excl;
    int b = b0;
    unsigned int ignored = 0;
    for (; b < b1 - 1; ++b) {
      const long long t = request_tiles(P, request(P, b, ignored));
      if (g0 < at + t) break;
      at += t;
    }
    c->start_b = b;
    c->start_rem = g0 - at;
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&c->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  Walk w;
  w.left = left;
  w.prefix = g0 < prefix_all;
  w.unit = w.b = w.rb = w.h = w.off = 0;
  w.r = Req{0, 0, 0};
  if (w.prefix) {
    w.unit = (int)(g0 / P.prefix_tiles);
    w.off = (int)(g0 - (long long)w.unit * P.prefix_tiles);
  } else {
    w.b = c->start_b;
    w.load_request(P);
    long long rem = c->start_rem;
    for (; w.rb * P.tpq < w.r.n; ++w.rb) {
      const int t = tiles_of(block_keys(P, w.r, w.rb));
      if (rem < (long long)t * P.Hk) {
        w.h = (int)(rem / t);
        w.off = (int)(rem - (long long)w.h * t);
        break;
      }
      rem -= (long long)t * P.Hk;
    }
  }
  const uint32_t q_smem = smem_addr(tiles), ring = q_smem + 2 * S::tile_bytes;
  unsigned int entry = 0, qn = 0;  // ring entries and query tiles copied (warp 8)
  if (warp < 8)
    softmax_role<T, DP>(P, w, c);
  else if (warp == 8)
    copy_role<DP>(P, w, c, q_smem, ring, &qmap, &qmap_prefix, &kmap, &vmap, entry, qn);
  else
    matrix_role<T, DP>(P, w, c, q_smem, ring, tiles + 2 * S::tile_bytes);
  fence_before();
  __syncthreads();
  if (c->abort) {
    // a wait ran out: copies and products in flight end (each wait bounded)
    // before shared and tensor memory are given back
    int ignored = 0;
    if (warp == 8) {
      for (unsigned int i = qn > 2 ? qn - 2 : 0; i < qn; ++i)
        (void)bar_wait(smem_addr(&c->q_full[i & 1]), (i >> 1) & 1, kDrainNs, &ignored);
      for (unsigned int e = entry > (unsigned int)S::slots ? entry - S::slots : 0; e < entry; ++e)
        (void)bar_wait(smem_addr(&c->kv_full[e % S::slots]), (e / S::slots) & 1, kDrainNs, &ignored);
    } else if (warp == 9) {
      if (lane == 0) mma_commit(smem_addr(&c->drain));
      __syncwarp();
      (void)bar_wait(smem_addr(&c->drain), 0, kDrainNs, &ignored);
    }
    __syncthreads();
  }
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(c->tmem));
  }
  if (tid == 0 && c->abort) atomicOr(P.status, (unsigned int)SV_STATUS_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Joining parts: o = sum 2^(lse_i - m) o_i / sum 2^(lse_i - m), one warp a row
// ---------------------------------------------------------------------------
template <int DP>
struct Joined {
  float o[DP / 32];
  float m, l;
  __device__ __forceinline__ void add(const float* part, float lse2) {
    if (lse2 == -INFINITY) return;  // no key seen there
    const float top = fmaxf(m, lse2);
    const float a = m == -INFINITY ? 0.f : exp2f(m - top), b = exp2f(lse2 - top);
    const int lane = threadIdx.x & 31;
    if (DP == 128) {
      const float4 v = *reinterpret_cast<const float4*>(part + lane * 4);
      o[0] = o[0] * a + v.x * b;
      o[1] = o[1] * a + v.y * b;
      o[2 % (DP / 32)] = o[2 % (DP / 32)] * a + v.z * b;
      o[3 % (DP / 32)] = o[3 % (DP / 32)] * a + v.w * b;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(part + lane * 2);
      o[0] = o[0] * a + v.x * b;
      o[1] = o[1] * a + v.y * b;
    }
    l = l * a + b;
    m = lse2 != lse2 ? lse2 : top;  // fmaxf drops a NaN
  }
};

template <typename T, int DP>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ AttnParams P, int ctas) {
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  unsigned int ignored = 0;
  const Req r = request(P, b, ignored);
  if (r.n <= 0) return;
  const long long total = P.starts[P.B], per = (total + ctas - 1) / ctas;
  const long long first = P.starts[b];
  if (per <= 0) return;
  // without a prefix, requests whose units all lie within one share are done
  const long long tiles_all = request_tiles(P, r);
  if (P.prefix_len == 0 && first / per == (first + tiles_all - 1) / per) return;
  const int rows = r.n * P.Hq;
  for (int x = (blockIdx.y * 4 + (threadIdx.x >> 5)); x < rows; x += gridDim.y * 4) {
    const int i = x / P.Hq, head = x - i * P.Hq;
    const int h = head / P.group, g = head - h * P.group;
    const size_t at = (size_t)(r.row0 + i) * P.Hq + head;
    Joined<DP> acc;
#pragma unroll
    for (int y = 0; y < DP / 32; ++y) acc.o[y] = 0.f;
    acc.m = -INFINITY;
    acc.l = 0.f;
    auto unit = [&](long long u0, int tiles, int which, int slot_row) {
      const long long c0 = u0 / per, c1 = (u0 + tiles - 1) / per;
      if (c0 == c1) {
        acc.add(P.dense[which] + at * DP, P.dense_lse[which][at]);
        return;
      }
      for (long long c = c0; c <= c1; ++c) {
        const size_t s = ((size_t)c * 2 + (c == c0)) * kSlotRows + slot_row;
        acc.add(P.slot + s * DP, P.slot_lse[s]);
      }
    };
    const int rb = i / P.tpq;
    long long u0 = first;
    for (int y = 0; y < rb; ++y) u0 += (long long)tiles_of(block_keys(P, r, y)) * P.Hk;
    const int tiles = tiles_of(block_keys(P, r, rb));
    u0 += (long long)h * tiles;
    if (P.prefix_len == 0 && u0 / per == (u0 + tiles - 1) / per) continue;  // written already
    if (P.prefix_len > 0) {
      const int t = r.row0 + i, pair = t / (2 * P.tpq), in = t - pair * 2 * P.tpq;
      const int blk = in / P.tpq;
      unit((long long)(h * P.prefix_blocks + pair) * P.prefix_tiles, P.prefix_tiles, 1,
           blk * kTile + (in - blk * P.tpq) * P.group + g);
    }
    unit(u0, tiles, 0, (i - rb * P.tpq) * P.group + g);
    const float inv = acc.l > 0.f || acc.l != acc.l ? 1.f / acc.l : 0.f;
    if (DP == 128) {
      if (lane * 4 < P.D)
        *reinterpret_cast<uint2*>(P.out + (at * P.D + lane * 4) * 2) =
            make_uint2(Type<T>::pack(acc.o[0] * inv, acc.o[1] * inv),
                       Type<T>::pack(acc.o[2 % (DP / 32)] * inv, acc.o[3 % (DP / 32)] * inv));
    } else if (lane * 2 < P.D) {
      *reinterpret_cast<uint32_t*>(P.out + (at * P.D + lane * 2) * 2) =
          Type<T>::pack(acc.o[0] * inv, acc.o[1] * inv);
    }
    if (P.lse && lane == 0) P.lse[at] = (acc.m + log2f(acc.l)) * 0.693147180559945309f;
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
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
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
  size_t starts, dense[2], dense_lse[2], slot, slot_lse, total;
};
AttnLayout attn_layout(long long T, int Hq, int D) {
  const size_t dp = D <= 64 ? 64 : 128, rows = (size_t)T * Hq;
  AttnLayout L;
  size_t at = 256;  // the status word
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += sv::align256(bytes);
    return a;
  };
  L.starts = take((size_t)(T + 1) * sizeof(long long));
  for (int i = 0; i < 2; ++i) L.dense[i] = take(rows * dp * 4);
  for (int i = 0; i < 2; ++i) L.dense_lse[i] = take(rows * 4);
  L.slot = take((size_t)2 * kMaxCtas * kSlotRows * dp * 4);
  L.slot_lse = take((size_t)2 * kMaxCtas * kSlotRows * 4);
  L.total = at;
  return L;
}

template <typename T, int DP>
int grid_size() {
  static std::atomic<int> cached{0};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int c0 = cached.load(std::memory_order_relaxed);
  if ((c0 >> 16) == dev + 1) return c0 & 0xffff;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaFuncSetAttribute(attention_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<DP>::smem) != cudaSuccess)
    return 0;
  sms = sms < kMaxCtas ? sms : kMaxCtas;
  cached.store(((dev + 1) << 16) | sms, std::memory_order_relaxed);
  return sms;
}

struct Maps {
  CUtensorMap q, q_prefix, k, v;
};

template <typename T, int DP>
int launch(const Maps& m, const AttnParams& P, cudaStream_t stream) {
  const int grid = grid_size<T, DP>();
  if (grid <= 0) return SV_ERR_CUDA;
  attention_kernel<T, DP><<<grid, kThreads, Shape<DP>::smem, stream>>>(m.q, m.q_prefix, m.k, m.v, P);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  // CTAs a request: four rows each, at most 64 of them
  const long long rows = ((long long)(P.G < P.T ? P.G + 1 : P.T) * P.Hq + 3) / 4;
  const dim3 g((unsigned int)P.B, (unsigned int)(rows < 64 ? rows : 64));
  combine_kernel<T, DP><<<g, 128, 0, stream>>>(P, grid);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
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
  if (total_drafts < 0 || max_drafts < 0 || rows > INT32_MAX || prefix_len < 0 || q_heads < 1 ||
      q_heads > 65535 || q_heads % c.kv_heads || q_heads / c.kv_heads > kTile || !(scale > 0.f) ||
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
  AttnParams P = {};
  P.B = c.batch;
  P.T = (int)rows;
  P.G = max_drafts;
  P.total = total_drafts;
  P.Hq = q_heads;
  P.Hk = c.kv_heads;
  P.D = c.head_dim;
  P.group = q_heads / c.kv_heads;
  P.tpq = kTile / P.group;
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
  P.prefix_len = prefix_len;
  P.prefix_tiles = (prefix_len + kTile - 1) / kTile;
  P.prefix_blocks = (P.T + 2 * P.tpq - 1) / (2 * P.tpq);
  if (prefix_len > 0) {
    const long long units = (long long)P.prefix_blocks * P.Hk;
    if (units > INT32_MAX) return SV_ERR_SCALAR;
    P.prefix_units = (int)units;
  }
  P.mask = draft_mask;
  P.sl2 = scale * 1.44269504088896341f;
  P.out = static_cast<char*>(out);
  P.lse = lse;
  char* w = static_cast<char*>(workspace);
  P.status = reinterpret_cast<unsigned int*>(w);
  P.starts = reinterpret_cast<long long*>(w + L.starts);
  for (int i = 0; i < 2; ++i) {
    P.dense[i] = reinterpret_cast<float*>(w + L.dense[i]);
    P.dense_lse[i] = reinterpret_cast<float*>(w + L.dense_lse[i]);
  }
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
  if (!encode(&m.q, c.dtype, q, qd, qs, q_own) || !encode(&m.q_prefix, c.dtype, q, qd, qs, q_pre) ||
      !encode(&m.k, c.dtype, c.k_pages, cd, ks, cb) || !encode(&m.v, c.dtype, c.v_pages, cd, vs, cb))
    return SV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c.dtype == SV_BF16)
    return c.head_dim <= 64 ? launch<__nv_bfloat16, 64>(m, P, s) : launch<__nv_bfloat16, 128>(m, P, s);
  return c.head_dim <= 64 ? launch<__half, 64>(m, P, s) : launch<__half, 128>(m, P, s);
}

}  // extern "C"
