// The pages of a cache: who holds them, the page table of the next step, and the pool
// moved together.
//
// Both calls are a kernel of one cluster that works out whole numbers, and one over the whole
// GPU that moves pages.  The cluster's CTAs share the rows (a warp a row) or the pool's
// pages; what one phase leaves in memory the next reads behind a cluster barrier, so nothing
// is waited for in a loop.  Counts are kept with atomics, whose order does not show: a
// page's count after all of them, the first place that dropped it (a maximum), the lowest row
// that writes to it (a maximum).  Places in the list of free pages come from sums over
// the rows in order.
//
// Bound: the table's entries of the rows that change, two dependent reads each; then the copied tokens
// (read and written once).  Measured: 256 rows, forks of four, contexts of up to 20000 tokens in
// pages of 64, 48 us, nearly all of it the cluster's (its CTAs read every entry of a changed
// row up to five times; 8 SMs work); without forks 16.
// A compaction that moves 1440 pages of 256 KB takes 125 us, 89 % of the copy rate.
#include "../../include/spec_verify.h"
#include "internal.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kCopyThreads = 256;
constexpr int kPart = 32 * 1024;  // bytes that a CTA moves at once

// One pool's layout in bytes: a page is page_size tokens of heads of row_bytes.
struct Pool {
  char* at;
  long long page, token, head;
};

struct PagesParams {
  int B, W, num_pages, page_size, Hk, row_bytes;
  int dense;            // a page is one run of memory in both pools
  int parts;            // CTAs that share a page's keys or values
  int32_t* table;
  int32_t* kv_len;
  int32_t* held;
  int32_t* ref;
  int32_t* free_pages;
  int32_t* free_count;
  const int32_t* parents;
  const int32_t* tokens;
  int32_t* remap;
  Pool k, v;
  float* k_scales;      // NULL: 16 bits
  float* v_scales;
  int block;
  unsigned int* status;
  // scratch, cleared for the pages that a call looks at (a workspace may have served another
  // number of pages, whose arrays began elsewhere)
  int32_t* first;       // [num_pages]: INT_MAX less the first place that dropped a page
  int32_t* lowest;      // [num_pages]: INT_MAX less the lowest row that writes to a page
  int32_t* writers;     // [num_pages]: rows that do
  // scratch that needs no value
  int4* rows;           // [B]: tokens, pages with tokens, pages needed, entries held before
  int4* more;           // [B]: freed, taken, copies or not, the page to copy
  int2* before;         // [B]: freed and taken by the rows before
  int4* copies;         // [B]: source, destination, tokens
  int32_t* entries;     // [B][W]: the parents' entries
  int32_t* counts;      // sums of the cluster's CTAs, pages moved
  int32_t* src;         // [num_pages]: compact: where live pages from n on lie, by rank
  int32_t* dst;         // [num_pages]: the free places below n
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// Exclusive sums over the CTA of a thread's two values, and their totals.
struct Sums {
  int a, b, all_a, all_b;
};
__device__ __forceinline__ Sums scan(int a, int b, int2* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += p, y += q;
  }
  if (lane == 31) s_warp[warp] = make_int2(x, y);
  __syncthreads();
  Sums r{x - a, y - b, 0, 0};
#pragma unroll 8
  for (int i = 0; i < kWarps; ++i) {
    const int2 w = s_warp[i];
    if (i < warp) r.a += w.x, r.b += w.y;
    r.all_a += w.x, r.all_b += w.y;
  }
  __syncthreads();
  return r;
}

// What a row is after the call: its parent, tokens, pages.
struct Row {
  int a;      // row it continues; -1: it ends
  bool stays;
  int kv, live, need, held;  // tokens, pages of them, pages after the takes, entries before
  int n;
};
__device__ __forceinline__ Row row_of(const PagesParams& P, int b, unsigned int& flags) {
  Row r;
  r.a = P.parents ? P.parents[b] : b;
  if (r.a < -1 || r.a >= P.B) {
    flags |= SV_STATUS_BAD_ROW;
    r.a = b;
  }
  r.stays = r.a == b;
  r.held = clamp(P.held[b], 0, P.W);
  r.n = P.tokens[b];
  r.kv = r.live = 0;
  if (r.a >= 0) {
    const int h = clamp(P.held[r.a], 0, P.W);
    r.kv = P.kv_len[r.a];
    const long long room = (long long)h * P.page_size;
    if (r.kv < 0 || r.kv > room) {
      flags |= SV_STATUS_BAD_LENGTH;
      r.kv = r.kv < 0 ? 0 : (int)room;
    }
    r.live = (int)(((long long)r.kv + P.page_size - 1) / P.page_size);
  } else {
    r.n = 0;
  }
  const long long need = ((long long)r.kv + r.n + P.page_size - 1) / P.page_size;
  r.need = (int)need;
  if (r.n < 0 || need > P.W) {
    flags |= SV_STATUS_BAD_LENGTH;
    r.n = 0;
    r.need = r.live;
  }
  return r;
}

__global__ void __launch_bounds__(kThreads, 1) step_kernel(const __grid_constant__ PagesParams P) {
  __shared__ int2 s_warp[kWarps];
  const int lane = threadIdx.x & 31;
  const int rank = blockIdx.x, ctas = gridDim.x;  // (the grid is one cluster)
  const int warp0 = rank * kWarps + (threadIdx.x >> 5), warps = ctas * kWarps;
  unsigned int flags = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const auto fits = [&](int page) { return page >= 0 && page < P.num_pages; };
  const int count = clamp(*P.free_count, 0, P.num_pages);
  // 1: what each row is; references dropped and added
#pragma unroll 1
  for (int b = warp0; b < P.B; b += warps) {
    const Row r = row_of(P, b, flags);
    const int32_t* mine = P.table + (size_t)b * P.W;
    const int32_t* from = P.table + (size_t)(r.a < 0 ? 0 : r.a) * P.W;
#pragma unroll 4
    for (int j = (r.stays ? r.live : 0) + lane; j < r.held; j += 32) {
      const int p = mine[j];
      if (fits(p)) {
        atomicSub(P.ref + p, 1);
        P.first[p] = 0;
      } else {
        flags |= SV_STATUS_BAD_PAGE;
      }
    }
    if (!r.stays) {
#pragma unroll 4
      for (int j = lane; j < r.live; j += 32) {
        const int p = from[j];
        P.entries[(size_t)b * P.W + j] = p;
        if (fits(p))
          atomicAdd(P.ref + p, 1);
        else
          flags |= SV_STATUS_BAD_PAGE;
      }
    }
    if (lane == 0) {
      P.rows[b] = make_int4(r.kv, r.live, r.need, r.held);
      int page = -1;  // the page of older tokens that it writes behind
      if (r.n > 0 && r.kv % P.page_size) {
        page = (r.stays ? mine : from)[r.kv / P.page_size];
        if (fits(page)) {
          P.writers[page] = P.lowest[page] = 0;
        } else {
          flags |= SV_STATUS_BAD_PAGE;
          page = -1;
        }
      }
      P.more[b].w = page;
    }
  }
  cluster_sync();
  // 2: pages that nobody holds: the first place that dropped them; shared pages that rows
  // write to: how many do, and the lowest
#pragma unroll 1
  for (int b = warp0; b < P.B; b += warps) {
    const int4 r = __ldcg(P.rows + b);
    const bool stays = !P.parents || P.parents[b] == b || P.parents[b] < -1 || P.parents[b] >= P.B;
    const int32_t* mine = P.table + (size_t)b * P.W;
#pragma unroll 4
    for (int j = (stays ? r.y : 0) + lane; j < r.w; j += 32) {
      const int p = mine[j];
      if (fits(p) && __ldcg(P.ref + p) == 0) atomicMax(P.first + p, INT32_MAX - (b * P.W + j));
    }
    if (lane == 0) {
      const int page = __ldcg(&P.more[b].w);
      if (page >= 0 && __ldcg(P.ref + page) <= 1) {
        P.more[b].w = -1;
      } else if (page >= 0) {
        atomicAdd(P.writers + page, 1);
        atomicMax(P.lowest + page, INT32_MAX - b);
      }
    }
  }
  cluster_sync();
  // 3: what each row frees and takes
#pragma unroll 1
  for (int b = warp0; b < P.B; b += warps) {
    const int4 r = __ldcg(P.rows + b);
    const bool stays = !P.parents || P.parents[b] == b || P.parents[b] < -1 || P.parents[b] >= P.B;
    const int32_t* mine = P.table + (size_t)b * P.W;
    int frees = 0;
#pragma unroll 4
    for (int j = (stays ? r.y : 0) + lane; j < r.w; j += 32) {
      const int p = mine[j];
      if (fits(p) && __ldcg(P.first + p) == INT32_MAX - (b * P.W + j)) ++frees;
    }
    frees = __reduce_add_sync(0xffffffffu, frees);
    if (lane == 0) {
      const int page = __ldcg(&P.more[b].w);
      const bool copies = page >= 0 && !(__ldcg(P.writers + page) == __ldcg(P.ref + page) &&
                                         __ldcg(P.lowest + page) == INT32_MAX - b);
      P.more[b] = make_int4(frees, (copies ? 1 : 0) + r.z - r.y, copies ? 1 : 0, page);
    }
  }
  cluster_sync();
  // 4: sums over the rows in order, by the first CTA
  if (rank == 0) {
    int base_f = 0, base_t = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int4 m = b < P.B ? __ldcg(P.more + b) : make_int4(0, 0, 0, 0);
      const Sums s = scan(m.x, m.y, s_warp);
      if (b < P.B) P.before[b] = make_int2(base_f + s.a, base_t + s.b);
      base_f += s.all_a, base_t += s.all_b;
    }
    if (threadIdx.x == 0) P.counts[0] = base_f, P.counts[1] = base_t;
  }
  cluster_sync();
  // 5: freed pages go behind the free ones, in the order of rows and places
  int freed = __ldcg(P.counts), taken = __ldcg(P.counts + 1);
  if (freed > P.num_pages - count) {  // (counts that do not agree with the table)
    flags |= SV_STATUS_BAD_PAGE;
    freed = P.num_pages - count;
  }
  const bool enough = taken <= count + freed;
  if (!enough) flags |= SV_STATUS_NO_PAGES;
#pragma unroll 1
  for (int b = warp0; b < P.B; b += warps) {
    const int4 r = __ldcg(P.rows + b), m = __ldcg(P.more + b);
    const bool stays = !P.parents || P.parents[b] == b || P.parents[b] < -1 || P.parents[b] >= P.B;
    const int32_t* mine = P.table + (size_t)b * P.W;
    int at = __ldcg(P.before + b).x;
#pragma unroll 1
    for (int j0 = stays ? r.y : 0; m.x > 0 && j0 < r.w; j0 += 32) {
      const int j = j0 + lane;
      const int p = j < r.w ? mine[j] : -1;
      const bool frees = fits(p) && __ldcg(P.first + p) == INT32_MAX - (b * P.W + j);
      const unsigned int who = __ballot_sync(0xffffffffu, frees);
      const int place = at + __popc(who & ((1u << lane) - 1u));
      if (frees) {
        if (place < freed) P.free_pages[count + place] = p;
        P.first[p] = 0;
      }
      at += __popc(who);
    }
    if (lane == 0 && m.w >= 0) {
      if (m.z && enough) atomicSub(P.ref + m.w, 1);
      P.writers[m.w] = 0;
      P.lowest[m.w] = 0;
    }
  }
  cluster_sync();
  // 6: pages are taken from the list's end; the table
  const int top = count + freed - 1;
#pragma unroll 1
  for (int b = warp0; b < P.B; b += warps) {
    const int4 r = __ldcg(P.rows + b), m = __ldcg(P.more + b);
    const bool stays = !P.parents || P.parents[b] == b || P.parents[b] < -1 || P.parents[b] >= P.B;
    int32_t* mine = P.table + (size_t)b * P.W;
    const int at = top - __ldcg(P.before + b).y;
    const int own = r.x / P.page_size;  // the page that is copied
    const bool copies = m.z && enough;
    const int need = enough ? r.z : r.y;
    const auto take = [&](int i) {
      const int p = __ldcg(P.free_pages + at - i);
      if (!fits(p)) {
        flags |= SV_STATUS_BAD_PAGE;
        return -1;
      }
      P.ref[p] = 1;
      return p;
    };
    if (!stays) {
#pragma unroll 4
      for (int j = lane; j < r.y; j += 32)
        if (!copies || j != own) mine[j] = __ldcg(P.entries + (size_t)b * P.W + j);
    }
    for (int j = r.y + lane; j < need; j += 32) mine[j] = take((copies ? 1 : 0) + j - r.y);
    for (int j = need + lane; j < r.w; j += 32) mine[j] = -1;
    if (lane == 0) {
      int p = -1;
      if (copies) {
        p = take(0);
        mine[own] = p;
      }
      P.copies[b] = make_int4(m.w, p, p >= 0 ? r.x % P.page_size : 0, 0);
      P.held[b] = need;
      P.kv_len[b] = r.x;
    }
  }
  if (rank == 0 && threadIdx.x == 0) *P.free_count = count + freed - (enough ? taken : 0);
  const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && any) atomicOr(P.status, any);
}

// Tokens [0, n) of a page to another, 16 bytes a thread and step: `part` of `parts` threads.
__device__ __forceinline__ void move(const PagesParams& P, const Pool& pool, int src, int dst, int n, int part,
                                     int parts) {
  const char* from = pool.at + (long long)src * pool.page;
  char* to = pool.at + (long long)dst * pool.page;
  const int vecs = P.row_bytes / 16, all = n * P.Hk * vecs;
  const bool run = P.dense && (pool.head == P.row_bytes || n == P.page_size);
  constexpr int kAhead = 8;
#pragma unroll 1
  for (int x0 = part; x0 < all; x0 += kAhead * parts) {
    uint4 w[kAhead];
    long long at[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int x = x0 + k * parts;
      if (run) {
        at[k] = (long long)x * 16;
      } else {
        const int row = x / vecs, t = row / P.Hk;
        at[k] = t * pool.token + (long long)(row - t * P.Hk) * pool.head + (x - row * vecs) * 16;
      }
      if (x < all) w[k] = __ldcs(reinterpret_cast<const uint4*>(from + at[k]));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (x0 + k * parts < all) __stcs(reinterpret_cast<uint4*>(to + at[k]), w[k]);
  }
}
__device__ __forceinline__ void move_scales(const PagesParams& P, float* s, int src, int dst, int n) {
  const int per = P.page_size / P.block * P.Hk, all = (n + P.block - 1) / P.block * P.Hk;
  for (int x = threadIdx.x; x < all; x += blockDim.x)
    s[(long long)dst * per + x] = s[(long long)src * per + x];
}

// A row's copy: grid (rows, parts of the keys' and values' pages)
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PagesParams P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int parts = gridDim.y / 2, part = blockIdx.y / 2;
  const bool keys = (blockIdx.y & 1) == 0;
#pragma unroll 1
  for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
    const int4 c = P.copies[b];
    if (c.z <= 0) continue;
    move(P, keys ? P.k : P.v, c.x, c.y, c.z, part * kCopyThreads + threadIdx.x, parts * kCopyThreads);
    if (part == 0 && P.k_scales) move_scales(P, keys ? P.k_scales : P.v_scales, c.x, c.y, c.z);
  }
}

// Compact: n pages are in use; the ones from n on (rank r among the live: n - m .. n - 1)
// move to the m free places below n.  (Both lists are in order.)
__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const __grid_constant__ PagesParams P) {
  __shared__ int2 s_warp[kWarps];
  const int rank = blockIdx.x, ctas = gridDim.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = (P.num_pages + ctas - 1) / ctas;
  const int p0 = rank * per < P.num_pages ? rank * per : P.num_pages;
  const int p1 = p0 + per < P.num_pages ? p0 + per : P.num_pages;
  int live = 0;
  for (int p = p0 + threadIdx.x; p < p1; p += kThreads) live += P.ref[p] > 0;
  const Sums s = scan(live, 0, s_warp);
  if (threadIdx.x == 0) P.counts[rank] = s.all_a;
  cluster_sync();
  int n = 0, below = 0;  // live pages, those of the CTAs before
  for (int i = 0; i < ctas; ++i) {
    const int c = __ldcg(P.counts + i);
    if (i < rank) below += c;
    n += c;
  }
  int holes = 0;
#pragma unroll 1
  for (int x0 = p0; x0 < p1; x0 += kThreads) {
    const int p = x0 + threadIdx.x;
    const bool is = p < p1 && P.ref[p] > 0;
    const Sums t = scan(is, p < p1 && !is && p < n, s_warp);
    const int before = below + t.a;  // live pages before p
    if (p < p1) {
      if (is && p >= n) P.src[before] = p;
      if (!is && p < n) P.dst[p - before] = p;
      if (!is || p < n) P.remap[p] = is ? p : -1;
    }
    below += t.all_a;
    holes += t.all_b;
  }
  cluster_sync();  // (counts have been read)
  if (threadIdx.x == 0) P.counts[rank] = holes;
  cluster_sync();
  int m = 0;
  for (int i = 0; i < ctas; ++i) m += __ldcg(P.counts + i);
  const int at = rank * kThreads + threadIdx.x, by = ctas * kThreads;
  for (int i = at; i < m; i += by) {
    const int src = __ldcg(P.src + n - m + i), dst = __ldcg(P.dst + i);
    P.remap[src] = dst;
    P.ref[dst] = P.ref[src];
    P.ref[src] = 0;
  }
  for (int i = at; i < P.num_pages - n; i += by) P.free_pages[i] = P.num_pages - 1 - i;
  if (at == 0) {
    *P.free_count = P.num_pages - n;
    P.counts[kCluster] = m;
    P.counts[kCluster + 1] = n;
  }
}

// Moves the pages, keys and values apart, and turns the table's entries over.
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const __grid_constant__ PagesParams P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int m = P.counts[kCluster], n = P.counts[kCluster + 1];
#pragma unroll 1
  for (long long x = blockIdx.x; x < 2ll * m * P.parts; x += gridDim.x) {
    const int item = (int)(x / P.parts), part = (int)(x - (long long)item * P.parts);
    const int i = item >> 1, src = P.src[n - m + i], dst = P.dst[i];
    const bool keys = (item & 1) == 0;
    move(P, keys ? P.k : P.v, src, dst, P.page_size, part * kCopyThreads + threadIdx.x, P.parts * kCopyThreads);
    if (part == 0 && P.k_scales) move_scales(P, keys ? P.k_scales : P.v_scales, src, dst, P.page_size);
  }
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kCopyThreads / 32);
#pragma unroll 1
  for (int b = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); b < P.B; b += warps) {
    const int held = clamp(P.held[b], 0, P.W);
    for (int j = lane; j < held; j += 32) {
      int32_t* e = P.table + (size_t)b * P.W + j;
      const int p = *e;
      if (p >= 0 && p < P.num_pages)
        *e = P.remap[p];
      else
        atomicOr(P.status, (unsigned int)SV_STATUS_BAD_PAGE);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct PagesLayout {
  size_t first, lowest, writers, rows, more, before, copies, entries, counts, src, dst, total;
};
PagesLayout pages_layout(size_t pages, size_t B, size_t W) {
  PagesLayout L;
  size_t at = 256;  // the status word
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += sv::align256(bytes);
    return a;
  };
  L.first = take(pages * 4);
  L.lowest = take(pages * 4);
  L.writers = take(pages * 4);
  L.rows = take(B * 16);
  L.more = take(B * 16);
  L.before = take(B * 8);
  L.copies = take(B * 16);
  L.entries = take(B * W * 4);
  L.counts = take(64 * 4);
  L.src = take(pages * 4);
  L.dst = take(pages * 4);
  L.total = at;
  return L;
}

// (A call about rows alone has nothing to do for none of them.)
int make_params(PagesParams& P, const sv_kv_cache* cache, const sv_kv_scales* scales, const sv_page_pool* pool,
                void* workspace, size_t ws_bytes, bool rows_alone) {
  if (!cache || !pool) return SV_ERR_NULL;
  const sv_kv_cache& c = *cache;
  if (c.dtype == SV_E4M3 && !scales) return SV_ERR_NULL;
  const int rc = c.dtype == SV_E4M3 ? sv::check_cache_e4m3(c, *scales) : sv::check_cache(c);
  if (rc) return rc;
  if (c.max_pages < 1 || (long long)c.batch * c.max_pages > INT32_MAX - 1 ||
      (long long)c.max_pages * c.page_size > INT32_MAX ||
      (long long)c.page_size * c.kv_heads * c.head_dim > INT32_MAX / 2)
    return SV_ERR_SCALAR;
  if (c.batch == 0) {
    if (rows_alone) return SV_OK;
    // (the pools' addresses are checked with the rows')
    if (!c.k_pages || !c.v_pages || (c.dtype == SV_E4M3 && (!scales->k || !scales->v))) return SV_ERR_NULL;
    if (!sv::aligned(c.k_pages, 16) || !sv::aligned(c.v_pages, 16) ||
        (c.dtype == SV_E4M3 && (!sv::aligned(scales->k, 4) || !sv::aligned(scales->v, 4))))
      return SV_ERR_ALIGN;
  }
  if ((c.batch > 0 && !pool->held) || !pool->ref || !pool->free_pages || !pool->free_count || !workspace) return SV_ERR_NULL;
  for (const void* p : {pool->held, pool->ref, pool->free_pages, pool->free_count})
    if (!sv::aligned(p, 4)) return SV_ERR_ALIGN;
  if (!sv::aligned(workspace, 256)) return SV_ERR_ALIGN;
  const PagesLayout L = pages_layout(c.num_pages, c.batch, c.max_pages);
  if (ws_bytes < L.total) return SV_ERR_WORKSPACE;
  const int es = c.dtype == SV_E4M3 ? 1 : 2;
  P.B = c.batch;
  P.W = c.max_pages;
  P.num_pages = c.num_pages;
  P.page_size = c.page_size;
  P.Hk = c.kv_heads;
  P.row_bytes = c.head_dim * es;
  P.table = const_cast<int32_t*>(c.page_table);
  P.kv_len = const_cast<int32_t*>(c.kv_len);
  P.held = pool->held;
  P.ref = pool->ref;
  P.free_pages = pool->free_pages;
  P.free_count = pool->free_count;
  P.k = Pool{static_cast<char*>(c.k_pages), c.k_strides[0] * es, c.k_strides[1] * es, c.k_strides[2] * es};
  P.v = Pool{static_cast<char*>(c.v_pages), c.v_strides[0] * es, c.v_strides[1] * es, c.v_strides[2] * es};
  P.dense = 1;
  for (const Pool* p : {&P.k, &P.v}) {
    const bool by_token = p->head == P.row_bytes && p->token == (long long)P.row_bytes * P.Hk;
    const bool by_head = p->token == P.row_bytes && p->head == (long long)P.row_bytes * P.page_size;
    P.dense &= by_token || by_head;
  }
  if (c.dtype == SV_E4M3) {
    P.k_scales = scales->k;
    P.v_scales = scales->v;
    P.block = scales->block;
  }
  char* w = static_cast<char*>(workspace);
  P.status = reinterpret_cast<unsigned int*>(w);
  P.first = reinterpret_cast<int32_t*>(w + L.first);
  P.lowest = reinterpret_cast<int32_t*>(w + L.lowest);
  P.writers = reinterpret_cast<int32_t*>(w + L.writers);
  P.rows = reinterpret_cast<int4*>(w + L.rows);
  P.more = reinterpret_cast<int4*>(w + L.more);
  P.before = reinterpret_cast<int2*>(w + L.before);
  P.copies = reinterpret_cast<int4*>(w + L.copies);
  P.entries = reinterpret_cast<int32_t*>(w + L.entries);
  P.counts = reinterpret_cast<int32_t*>(w + L.counts);
  P.src = reinterpret_cast<int32_t*>(w + L.src);
  P.dst = reinterpret_cast<int32_t*>(w + L.dst);
  return SV_OK;
}

int launch(void (*kernel)(PagesParams), const PagesParams& P, dim3 grid, int threads, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  sv::overlap_launch(at[0]);
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return sv::code_of(cudaLaunchKernelEx(&cfg, kernel, P));
}

}  // namespace

extern "C" {

size_t spec_verify_pages_workspace_size(int num_pages, int batch, int max_pages) {
  if (num_pages < 1 || batch < 0 || max_pages < 1 || (long long)batch * max_pages > INT32_MAX - 1) return 0;
  return pages_layout(num_pages, batch, max_pages).total;
}

int spec_verify_pages_step(const sv_kv_cache* cache, const sv_kv_scales* scales, const sv_page_pool* pool,
                           const int32_t* parents, const int32_t* tokens, void* workspace, size_t ws_bytes,
                           sv_stream_t stream) {
  PagesParams P = {};
  int rc = make_params(P, cache, scales, pool, workspace, ws_bytes, true);
  if (rc || P.B == 0) return rc;
  if (!tokens) return SV_ERR_NULL;
  if (!sv::aligned(tokens, 4) || !sv::aligned(parents, 4)) return SV_ERR_ALIGN;
  P.parents = parents;
  P.tokens = tokens;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Rows for more warps than a CTA has: us a call with one CTA and with eight, no forks and forks of four: 36
  // rows of 16 pages 11.6 / 10.5, 17.4 / 15.1; 64 of 64 13.5 / 12.4, 23.2 / 19.0; 256 of 64 35 / 14, 71 / 22.  Up to
  // 32 rows a CTA has a warp for each: 8 of 64 8.3 / 10.8, 12.7 / 16.0; 32 of 1000 9.2 / 10.9, 72 / 79.
  const int cluster = P.B > kWarps ? kCluster : 1;
  rc = launch(step_kernel, P, dim3(cluster), kThreads, cluster, s);
  if (rc) return rc;
  return launch(copy_kernel, P, dim3(P.B < 4096 ? P.B : 4096, 8), kCopyThreads, 1, s);
}

int spec_verify_pages_compact(const sv_kv_cache* cache, const sv_kv_scales* scales, const sv_page_pool* pool,
                              int32_t* remap, void* workspace, size_t ws_bytes, sv_stream_t stream) {
  PagesParams P = {};
  int rc = make_params(P, cache, scales, pool, workspace, ws_bytes, false);
  if (rc) return rc;
  if (!remap) return SV_ERR_NULL;
  if (!sv::aligned(remap, 4)) return SV_ERR_ALIGN;
  P.remap = remap;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // us with one CTA and with eight: 6.0 / 8.0 (388 pages), 9.2 / 10.3 (1988), 11.4 / 10.9 (2521), 13.9 / 11.6
  // (3992), 23 / 14.5 (8000), 96 / 46 (40000)
  const int cluster = P.num_pages > 2 * kThreads ? kCluster : 1;
  rc = launch(plan_kernel, P, dim3(cluster), kThreads, cluster, s);
  if (rc) return rc;
  // (eight CTAs an SM fill it; moves of 700 pages of 256 KB take 73 us with one, 60 with two, 60 with eight)
  P.parts = (int)(((long long)P.page_size * P.Hk * P.row_bytes + kPart - 1) / kPart);
  const long long tasks = 2ll * P.num_pages * P.parts > P.B / 8 ? 2ll * P.num_pages * P.parts : P.B / 8 + 1;
  return launch(compact_kernel, P, dim3((unsigned int)(tasks < 152 * 8 ? tasks : 152 * 8)), kCopyThreads, 1, s);
}

}  // extern "C"
