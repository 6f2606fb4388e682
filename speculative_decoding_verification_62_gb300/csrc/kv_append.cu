// A step's keys and values into a paged cache, with the rotary position
// rotation applied on the way.
//
// Row i of request b sits at position p = position_offset + kv_len[b] + i (or
// positions[row]) and goes to slot kv_len[b] + i of the request's pages.  Pair
// j of a head (values j and j + rot/2, or 2j and 2j + 1) turns by the angle
// p f_j: (a, c) -> s (a cos - c sin, c cos + a sin).  f_j is given in turns a
// position, as a whole multiple of 2^-64, so p f_j modulo one turn is a 64-bit
// product that wraps: far positions lose nothing (the rounding of f_j, 2^-65
// turns, grows to 2^-34 turns at position 2^31).  The turn goes to 32-bit
// floats as a fraction in [-1/2, 1/2), and cos and sin are taken of that.
//
// Bound: q, k and v are read once and written once; a CTA's chain of look-ups
// (request, length, page), angles and stores is hidden by its first values, which are
// under way before the look-ups, and by the other CTAs of its SM.  The angles of a row
// are formed once, in shared memory, and serve every head.  Hence many small CTAs:
// - up to 608 rows (four CTAs an SM, one wave) a CTA of 256 threads a row;
// - up to 2047 rows 128 threads a row, eight CTAs an SM, three reads a thread under
//   way: 618 rows 6.3 us (two rows a CTA: 7.4), 1174 rows 7.4 (10.0), 1920 rows 13.0 (14.0).
//   This is the best form up to one wave, eight CTAs an SM (1216 rows on 152).  Past it forms
//   that are not built in were faster: 1260 rows 10.8 us, with two reads under way 8.8;
//   1330 rows 10.5 and 8.4; 1646 rows 11.5, with one read and twelve CTAs 9.6; 1920 rows
//   13.0, with one read and sixteen CTAs 11.6 (and 2377 rows, two a CTA, 15.2 and 13.2);
// - from there two rows a CTA of 128 threads, twelve CTAs an SM: 23018 rows 59 us, one
//   row a CTA of 128 threads 68, four rows 69, two rows of 256 threads 64.
// Measured (GB300): one row 3.5 us; 256 requests' steps 7.4 us (29 MB, 3.9 TB/s);
// prompts of 12 requests, 24 + 6 + 6 heads of 96 in fp16, 59.4 us (318 MB, 5.4 TB/s: 79 %
// of a copy).
#include "../../include/spec_verify.h"
#include "append.h"
#include "internal.h"

namespace {

using namespace sv::append;

constexpr int kFewRows = 608;    // up to here 256 threads a row
constexpr int kManyRows = 2048;  // from here on two rows a CTA

struct AppendParams {
  const char* q;
  const char* k;
  const char* v;
  char* q_out;
  char* k_pages;
  char* v_pages;
  long long q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;  // elements
  long long kp, kt, kh, vp, vt, vh;  // cache strides: page, token, head
  int Hq, Hk, D, rot, B, T, G, num_pages, page_size, max_pages;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  const long long* freq;
  const int32_t* positions;
  int offset;
  float scale;
  unsigned int* status;
};

struct RowInfo {
  long long k_at, v_at;  // element offsets of the row's slot in the pools; -1: skipped
};

// A task: two vectors of a head (VW 1: a pair of values), one task a thread and
// row.  Turning heads pair values j and j + rot / 2 (INTER: neighbours).
template <int VW>
struct Words {
  Vec<VW> x, y;
};
template <>
struct Words<1> {
  unsigned short x, y;
};

template <typename T, int VW, bool INTER, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : ROWS == 1 ? 8 : 12) append_kernel(AppendParams P) {
  constexpr int kThreads = THREADS;
  extern __shared__ float2 s_turn[];  // [ROWS][rot / 2] cos, sin
  __shared__ RowInfo s_row[ROWS];
  __shared__ long long s_pos[ROWS];
  __shared__ int s_ok[ROWS];
  const int tid = threadIdx.x, lane = tid & 31;
  const int half = P.rot / 2;
  const int r0 = blockIdx.x * ROWS;
  const int nrows = P.T - r0 < ROWS ? P.T - r0 : ROWS;
  const int per_head = VW == 1 ? (P.D + 1) / 2 : P.D / (2 * VW);
  const int Hs = P.Hq + P.Hk;  // heads that turn
  const int n = (Hs + P.Hk) * per_head;
  constexpr int kTasks = ROWS > 1 ? 1 : THREADS == 256 ? 2 : 3;  // under way together

  // of a task: its head, the values that it moves (elements of the head)
  struct Task {
    int h, s, j, j2;
    bool turns;
  };
  auto task_of = [&](int e) {
    Task t;
    t.h = e / per_head;
    t.s = e - t.h * per_head;
    t.turns = t.h < Hs && t.s < (VW == 1 ? half : P.rot / (2 * VW));
    const bool apart = t.turns && !INTER;
    t.j = t.s * (apart ? VW : 2 * VW);
    t.j2 = apart ? t.j + half : t.j + VW;
    return t;
  };
  auto source = [&](const Task& t, int row) {
    if (t.h < P.Hq) return P.q + ((long long)row * P.q_row + (long long)t.h * P.q_head) * 2;
    if (t.h < Hs) return P.k + ((long long)row * P.k_row + (long long)(t.h - P.Hq) * P.k_head) * 2;
    return P.v + ((long long)row * P.v_row + (long long)(t.h - Hs) * P.v_head) * 2;
  };
  Words<VW> w[kTasks][ROWS];
  auto fetch = [&](int e0) {
#pragma unroll
    for (int k = 0; k < kTasks; ++k) {
      if (e0 + k * kThreads >= n) continue;
      const Task t = task_of(e0 + k * kThreads);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (r >= nrows) continue;
        const char* src = source(t, r0 + r);
        if constexpr (VW == 1) {
          const unsigned short* a = reinterpret_cast<const unsigned short*>(src);
          w[k][r].x = a[t.j];
          w[k][r].y = t.j2 < P.D ? a[t.j2] : (unsigned short)0;
        } else {
          w[k][r].x = load_vec<VW>(src + t.j * 2);
          w[k][r].y = load_vec<VW>(src + t.j2 * 2);
        }
      }
    }
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  fetch(tid);

  if (tid < 32) {
    const int b0 = request_of(P.cu, P.B, r0);
    unsigned int flags = 0;
    if (lane < nrows) {
      const int t = r0 + lane;
      int b = b0;
      while (b + 1 < P.B && (long long)P.cu[b + 1] + b + 1 <= t) ++b;
      const int c0 = P.cu[b], c1 = P.cu[b + 1], len = P.kv_len[b];
      const int i = t - b - c0;
      RowInfo info{-1, -1};
      long long pos = 0;
      const bool fits = c0 >= 0 && c1 >= c0 && c1 - c0 <= P.G && c1 <= P.T - P.B;
      const bool row = fits && i >= 0 && i <= c1 - c0;
      if (!row) {
        // (rows behind a consistent last request: a step of fewer rows than the call's)
        if (!fits || i < 0 || b + 1 < P.B) flags = SV_STATUS_BAD_GAMMA;
      } else {
        const long long slot = (long long)len + i;
        if (len < 0 || slot >= (long long)P.max_pages * P.page_size) {
          flags = SV_STATUS_BAD_LENGTH;
        } else {
          const int page = P.table[(size_t)b * P.max_pages + slot / P.page_size];
          if (page < 0 || page >= P.num_pages) {
            flags = SV_STATUS_BAD_PAGE;
          } else {
            const long long in = slot % P.page_size;
            info.k_at = page * P.kp + in * P.kt;
            info.v_at = page * P.vp + in * P.vt;
          }
        }
        pos = P.positions ? (long long)P.positions[t] : (long long)P.offset + slot;
      }
      s_row[lane] = info;
      s_pos[lane] = pos;
      s_ok[lane] = row;
    }
    const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && any) atomicOr(P.status, any);
  }
  __syncthreads();
  for (int e = tid; e < nrows * half; e += kThreads) {
    const int r = e / half;
    const long long turn = (long long)((unsigned long long)s_pos[r] * (unsigned long long)P.freq[e - r * half]);
    float sn, cs;
    sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn, &cs);
    s_turn[e] = make_float2(cs * P.scale, sn * P.scale);
  }
  __syncthreads();

#pragma unroll 1
  for (int e0 = tid; e0 < n; e0 += kTasks * kThreads) {
    if (e0 != tid) fetch(e0);
#pragma unroll
    for (int k = 0; k < kTasks; ++k) {
      if (e0 + k * kThreads >= n) continue;
      const Task t = task_of(e0 + k * kThreads);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (r >= nrows || !s_ok[r]) continue;
        char* dst;
        if (t.h < P.Hq) {
          dst = P.q_out + ((long long)(r0 + r) * P.o_row + (long long)t.h * P.o_head) * 2;
        } else {
          const RowInfo info = s_row[r];
          if (info.k_at < 0) continue;
          dst = t.h < Hs ? P.k_pages + (info.k_at + (long long)(t.h - P.Hq) * P.kh) * 2
                         : P.v_pages + (info.v_at + (long long)(t.h - Hs) * P.vh) * 2;
        }
        const float2* turn = s_turn + r * half;
        Words<VW> u = w[k][r];
        if constexpr (VW == 1) {
          unsigned short* d = reinterpret_cast<unsigned short*>(dst);
          if (t.turns) {
            const float2 a = Conv<T>::up((unsigned int)u.x | ((unsigned int)u.y << 16)), c = turn[t.s];
            const unsigned int y = Conv<T>::down(a.x * c.x - a.y * c.y, a.y * c.x + a.x * c.y);
            u.x = (unsigned short)y;
            u.y = (unsigned short)(y >> 16);
          }
          d[t.j] = u.x;
          if (t.j2 < P.D) d[t.j2] = u.y;
        } else {
          if (t.turns && INTER) {
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) {
              const float2 a = Conv<T>::up(u.x.w[i]), b = Conv<T>::up(u.y.w[i]);
              const float2 c0 = turn[t.s * VW + i], c1 = turn[t.s * VW + VW / 2 + i];
              u.x.w[i] = Conv<T>::down(a.x * c0.x - a.y * c0.y, a.y * c0.x + a.x * c0.y);
              u.y.w[i] = Conv<T>::down(b.x * c1.x - b.y * c1.y, b.y * c1.x + b.x * c1.y);
            }
          } else if (t.turns) {
#pragma unroll
            for (int i = 0; i < VW / 2; ++i) {
              const float2 a = Conv<T>::up(u.x.w[i]), b = Conv<T>::up(u.y.w[i]);
              const float2 c0 = turn[t.s * VW + 2 * i], c1 = turn[t.s * VW + 2 * i + 1];
              u.x.w[i] = Conv<T>::down(a.x * c0.x - b.x * c0.y, a.y * c1.x - b.y * c1.y);
              u.y.w[i] = Conv<T>::down(b.x * c0.x + a.x * c0.y, b.y * c1.x + a.y * c1.y);
            }
          }
          store_vec<VW>(dst + t.j * 2, u.x);
          store_vec<VW>(dst + t.j2 * 2, u.y);
        }
      }
    }
  }
}

template <typename T, int VW, bool INTER, int ROWS, int THREADS>
int launch_rows(const AppendParams& P, cudaStream_t stream) {
  const unsigned int grid = (unsigned int)((P.T + ROWS - 1) / ROWS);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)ROWS * (P.rot / 2) * sizeof(float2);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  sv::overlap_launch(at[0]);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return sv::code_of(cudaLaunchKernelEx(&cfg, append_kernel<T, VW, INTER, ROWS, THREADS>, P));
}

template <typename T, int VW, bool INTER>
int launch_order(const AppendParams& P, cudaStream_t stream) {
  if (P.T <= kFewRows) return launch_rows<T, VW, INTER, 1, 256>(P, stream);
  if (P.T < kManyRows) return launch_rows<T, VW, INTER, 1, 128>(P, stream);
  return launch_rows<T, VW, INTER, 2, 128>(P, stream);
}

template <typename T, int VW>
int launch(const AppendParams& P, bool inter, cudaStream_t stream) {
  return inter ? launch_order<T, VW, true>(P, stream) : launch_order<T, VW, false>(P, stream);
}

template <typename T>
int launch_width(const AppendParams& P, int vw, bool inter, cudaStream_t stream) {
  if (vw == 8) return launch<T, 8>(P, inter, stream);
  if (vw == 4) return launch<T, 4>(P, inter, stream);
  return launch<T, 1>(P, inter, stream);
}

}  // namespace

extern "C" int spec_verify_kv_append(const void* q, const int64_t* q_strides, int q_heads,
                                     const void* k, const int64_t* k_strides, const void* v,
                                     const int64_t* v_strides, void* q_out,
                                     const int64_t* q_out_strides, const sv_kv_cache* cache,
                                     const int32_t* cu_draft, int total_drafts, int max_drafts,
                                     const int64_t* freq, int rot_dim, int interleaved,
                                     float rope_scale, const int32_t* positions,
                                     int position_offset, void* workspace, size_t ws_bytes,
                                     sv_stream_t stream) {
  if (!cache || !k_strides || !v_strides) return SV_ERR_NULL;
  const sv_kv_cache& c = *cache;
  int rc = sv::check_cache(c);
  if (rc) return rc;
  if (total_drafts < 0 || max_drafts < 0 || q_heads < 0 || rot_dim < 0 || rot_dim % 2 ||
      rot_dim > c.head_dim || (interleaved != 0 && interleaved != 1) || !(rope_scale > 0.f) ||
      rope_scale > 3.0e38f || (long long)total_drafts + c.batch > INT32_MAX)
    return SV_ERR_SCALAR;
  if (!k || !v || !cu_draft || !workspace || (rot_dim > 0 && !freq)) return SV_ERR_NULL;
  if (q_heads > 0 && (!q || !q_out || !q_strides || !q_out_strides)) return SV_ERR_NULL;
  if (ws_bytes < sizeof(uint32_t)) return SV_ERR_WORKSPACE;
  if (!sv::aligned(q, 2) || !sv::aligned(k, 2) || !sv::aligned(v, 2) || !sv::aligned(q_out, 2) ||
      !sv::aligned(cu_draft, 4) || !sv::aligned(freq, 8) || !sv::aligned(positions, 4) ||
      !sv::aligned(workspace, 256))
    return SV_ERR_ALIGN;
  if (c.batch == 0) return SV_OK;
  if (q_heads > 0) {
    const long long rows = (long long)total_drafts + c.batch;
    const View o = view(q_out, q_out_strides, rows, q_heads, c.head_dim);
    const View in = view(q, q_strides, rows, q_heads, c.head_dim);
    if (overlaps_itself(o)) return SV_ERR_SCALAR;
    if ((!same(o, in) && !apart(o, in)) ||
        !apart(o, view(k, k_strides, rows, c.kv_heads, c.head_dim)) ||
        !apart(o, view(v, v_strides, rows, c.kv_heads, c.head_dim)))
      return SV_ERR_ALIGN;
  }
  AppendParams P = {};
  P.q = static_cast<const char*>(q);
  P.k = static_cast<const char*>(k);
  P.v = static_cast<const char*>(v);
  P.q_out = static_cast<char*>(q_out);
  P.k_pages = static_cast<char*>(c.k_pages);
  P.v_pages = static_cast<char*>(c.v_pages);
  if (q_heads > 0) {
    P.q_row = q_strides[0], P.q_head = q_strides[1];
    P.o_row = q_out_strides[0], P.o_head = q_out_strides[1];
  }
  P.k_row = k_strides[0], P.k_head = k_strides[1];
  P.v_row = v_strides[0], P.v_head = v_strides[1];
  P.kp = c.k_strides[0], P.kt = c.k_strides[1], P.kh = c.k_strides[2];
  P.vp = c.v_strides[0], P.vt = c.v_strides[1], P.vh = c.v_strides[2];
  P.Hq = q_heads;
  P.Hk = c.kv_heads;
  P.D = c.head_dim;
  P.rot = rot_dim;
  P.B = c.batch;
  P.T = total_drafts + c.batch;
  P.G = max_drafts;
  P.num_pages = c.num_pages;
  P.page_size = c.page_size;
  P.max_pages = c.max_pages;
  P.table = c.page_table;
  P.kv_len = c.kv_len;
  P.cu = cu_draft;
  P.freq = reinterpret_cast<const long long*>(freq);
  P.positions = positions;
  P.offset = position_offset;
  P.scale = rope_scale;
  P.status = static_cast<unsigned int*>(workspace);
  // The widest vector that every head's start and both halves of a rotation
  // allow: 8 values (16 bytes), 4, or single pairs.
  int vw = 8;
  for (; vw > 1; vw >>= 1) {
    if (vw == 2) { vw = 1; break; }
    const long long strides[] = {P.q_row, P.q_head, P.o_row, P.o_head, P.k_row, P.k_head, P.v_row,
                                 P.v_head, P.kp, P.kt, P.kh, P.vp, P.vt, P.vh};
    bool ok = P.D % (2 * vw) == 0 && P.rot % (2 * vw) == 0;
    for (long long s : strides) ok = ok && s % vw == 0;
    for (const void* p : {q, k, v, (const void*)q_out, (const void*)c.k_pages, (const void*)c.v_pages})
      ok = ok && sv::aligned(p, 2 * vw);
    if (ok) break;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return c.dtype == SV_BF16 ? launch_width<__nv_bfloat16>(P, vw, interleaved, s)
                            : launch_width<__half>(P, vw, interleaved, s);
}
