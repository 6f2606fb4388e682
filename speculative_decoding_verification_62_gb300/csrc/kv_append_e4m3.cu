// A step's keys and values into a paged cache of e4m3 codes, with a scale for each block
// of tokens and head, and the rotary position rotation on the way (kv_append.cu).
//
// A run is what a call appends to one block of tokens: rows of one request that follow one
// another.  For each run and head, keys and values apart:
//   m2 = max of x^2, and of a^2 + c^2 for pairs that turn
//   s  = smallest 2^e, -32 <= e <= 56, with m2 <= (448 2^e)^2; at least the old scale
//        where the block holds older tokens
//   code = rn_e4m3(x / s);  older codes: rn_e4m3(code s_old / s)
// (The rotation's factor counts: its power of two before the squares, which so overflow or vanish only
// where s ends, what is left of it behind them.)
// A turn leaves a^2 + c^2, so that the scale is known before any angle, and no rounding of
// an angle can move it: products of 16-bit values are exact in 32 bits and their sum is
// rounded once.  (Of a power of two too much a code of 3 mantissa bits loses nothing
// but below 2^-6 s.)
//
// Bound: q, k and v are read once and written once, k and v in half the bytes.  A warp
// takes one head's keys or values of a run: its first 16 rows stay in registers between
// the maximum and the codes (a longer run's others are read twice).  Rows of q are turned by CTAs
// of their own beside them.  Measured (24 / 6 heads of 96, 23000 prompt rows in fp16, 43 us at
// the copy rate): 73 us in blocks of 16 tokens, 147 in blocks of 128.  A verify step of 1150 rows
// (32 / 8 heads of 128) takes 13.8 us (3.9), its look-ups one after another.  A rotation of a
// width that is no multiple of 16, or rows that are not 16-byte aligned, go value by value: 40 of 80
// values 21 us for such a step.
#include "../../include/spec_verify.h"
#include "append.h"
#include "internal.h"

#include <cmath>

namespace {

using namespace sv::append;

constexpr int kHold = 4;      // tasks of a lane that stay in registers: 16 rows of 128 values
constexpr int kMaxRuns = 16;  // rows a CTA looks for runs among
constexpr int kSlots = 1216;  // CTAs of a wave: eight an SM
constexpr int kMaxRows = INT32_MAX - 4096;  // so that sums of a row and a CTA's or a wave's fit 32 bits

struct Append8Params {
  const char* q;
  const char* k;
  const char* v;
  char* q_out;
  unsigned char* k_pages;
  unsigned char* v_pages;
  long long q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;  // elements
  long long kp, kt, kh, vp, vt, vh;  // cache strides in bytes: page, token, head
  int Hq, Hk, D, rot, B, T, G, num_pages, page_size, max_pages, block;
  int run_rows, kv_ctas, q_rows;  // rows a CTA looks for runs among, and CTAs; rows of q a CTA
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  float* k_scales;
  float* v_scales;
  const long long* freq;
  const int32_t* positions;
  int offset;
  float scale, power, rest2;  // the rotation's factor; its square is power^2 rest2, power a power of two
  unsigned int* status;
};

// What a call appends to one block.
struct Run {
  int t, rows, old;           // first row, rows; older tokens of the block
  long long k_at, v_at;       // bytes from the pools to the first row's slot
  long long scale_at;         // the block's first head's scale
  long long slot;             // the first row's place in the request
};

// Where row t stands: its request, its place in the step; false: nowhere
struct RowAt {
  int b, i, n;
  long long slot;
};
__device__ __forceinline__ bool row_at(const Append8Params& P, int b0, int t, RowAt& r, unsigned int& flags) {
  int b = b0;
  while (b + 1 < P.B && (long long)P.cu[b + 1] + b + 1 <= t) ++b;
  const int c0 = P.cu[b], c1 = P.cu[b + 1];
  const int i = t - b - c0;
  const bool fits = c0 >= 0 && c1 >= c0 && c1 - c0 <= P.G && c1 <= P.T - P.B;
  if (!fits || i < 0 || i > c1 - c0) {
    // (rows behind a consistent last request: a step of fewer rows than the call's)
    if (!fits || i < 0 || b + 1 < P.B) flags |= SV_STATUS_BAD_GAMMA;
    return false;
  }
  r.b = b, r.i = i, r.n = c1 - c0 + 1;
  r.slot = (long long)P.kv_len[b] + i;
  return true;
}

__device__ __forceinline__ long long position(const Append8Params& P, int t, long long slot) {
  return P.positions ? (long long)P.positions[t] : (long long)P.offset + slot;
}
__device__ __forceinline__ float2 turn_of(const Append8Params& P, long long pos, int j) {
  const long long turn = (long long)((unsigned long long)pos * (unsigned long long)P.freq[j]);
  float sn, cs;
  sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn, &cs);
  return make_float2(cs * P.scale, sn * P.scale);
}

// The exponent of a block's scale: m2 = m 2^x with m in [1/2, 1), 448^2 = 0.765625 2^18.
__device__ __forceinline__ int exponent_of(float m2) {
  const unsigned int bits = __float_as_uint(m2);
  const int d = (int)(bits >> 23) - 126 - 18;
  const bool above = (bits & 0x7fffffu) > 0x440000u;  // m > 0.765625
  const int e = d & 1 ? (d + 1) >> 1 : (d >> 1) + (above ? 1 : 0);
  return e < -32 ? -32 : e > 56 ? 56 : e;
}

// two e4m3 codes, a in the low byte
__device__ __forceinline__ unsigned int codes2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 values2(unsigned short c) {
  unsigned int h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// A task: two vectors of a head (VW 1: a pair of values) of one row.
template <int VW>
struct Words {
  Vec<VW> x, y;
};
template <>
struct Words<1> {
  unsigned short x, y;
};
struct Place {
  int s, j, j2;  // the task's number, and where its two vectors begin
  bool turns;
};
template <int VW, bool INTER>
__device__ __forceinline__ Place place_of(int s, bool may_turn, int rot) {
  Place p;
  p.s = s;
  p.turns = may_turn && s < (VW == 1 ? rot / 2 : rot / (2 * VW));
  const bool apart = p.turns && !INTER;
  p.j = s * (apart ? VW : 2 * VW);
  p.j2 = apart ? p.j + rot / 2 : p.j + VW;
  return p;
}
template <int VW>
__device__ __forceinline__ Words<VW> fetch(const char* src, const Place& p) {
  Words<VW> w;
  if constexpr (VW == 1) {
    const unsigned short* a = reinterpret_cast<const unsigned short*>(src);
    w.x = a[p.j];
    w.y = a[p.j2];
  } else {
    w.x = load_vec<VW>(src + p.j * 2);
    w.y = load_vec<VW>(src + p.j2 * 2);
  }
  return w;
}
// The task's values in 32 bits, turned: 2 VW of them, x's before y's.
template <typename T, int VW, bool INTER>
__device__ __forceinline__ void turned(const Words<VW>& w, const Place& p, const float2* turn, float* o) {
  if constexpr (VW == 1) {
    const float2 a = Conv<T>::up((unsigned int)w.x | ((unsigned int)w.y << 16));
    o[0] = a.x, o[1] = a.y;
    if (p.turns) {
      const float2 c = turn[p.s];
      o[0] = a.x * c.x - a.y * c.y, o[1] = a.y * c.x + a.x * c.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) {
      const float2 a = Conv<T>::up(w.x.w[i]), b = Conv<T>::up(w.y.w[i]);
      o[2 * i] = a.x, o[2 * i + 1] = a.y, o[VW + 2 * i] = b.x, o[VW + 2 * i + 1] = b.y;
    }
    if (p.turns && INTER) {
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float2 c = turn[p.s * VW + i];
        const float a = o[2 * i], b = o[2 * i + 1];
        o[2 * i] = a * c.x - b * c.y, o[2 * i + 1] = b * c.x + a * c.y;
      }
    } else if (p.turns) {
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float2 c = turn[p.s * VW + i];
        const float a = o[i], b = o[VW + i];
        o[i] = a * c.x - b * c.y, o[VW + i] = b * c.x + a * c.y;
      }
    }
  }
}
// The largest square of a value or of a turning pair's length (NaN left out)
template <typename T, int VW, bool INTER>
__device__ __forceinline__ float squares(const Words<VW>& w, const Place& p, float power, float rest2) {
  float pairs = 0.f, single = 0.f;
  const float by = p.turns ? power : 1.f;
  if constexpr (VW == 1) {
    float2 a = Conv<T>::up((unsigned int)w.x | ((unsigned int)w.y << 16));
    a.x *= by, a.y *= by;
    if (p.turns)
      pairs = fmaf(a.x, a.x, a.y * a.y);
    else
      single = fmaxf(a.x * a.x, a.y * a.y);
  } else {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) {
      float2 a = Conv<T>::up(w.x.w[i]), b = Conv<T>::up(w.y.w[i]);
      a.x *= by, a.y *= by, b.x *= by, b.y *= by;
      const float ax = a.x * a.x, bx = b.x * b.x;
      if (p.turns)
        pairs = fmaxf(pairs, INTER ? fmaxf(fmaf(a.y, a.y, ax), fmaf(b.y, b.y, bx))
                                   : fmaxf(fmaf(b.x, b.x, ax), fmaf(b.y, b.y, a.y * a.y)));
      else
        single = fmaxf(single, fmaxf(fmaxf(ax, a.y * a.y), fmaxf(bx, b.y * b.y)));
    }
  }
  return fmaxf(pairs * rest2, single);
}

template <typename T, int VW, bool INTER, int THREADS>
__device__ __forceinline__ void kv_part(const Append8Params& P, float2* s_turn) {
  __shared__ Run s_run[kMaxRuns];
  __shared__ int s_runs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = P.rot / 2, per = P.D / (2 * VW);
  if (warp == 0) {
    const int r0 = blockIdx.x * P.run_rows, t = r0 + lane;
    const int b0 = request_of(P.cu, P.B, r0);
    unsigned int flags = 0;
    Run run{};
    bool starts = false;
    RowAt r;
    if (lane < P.run_rows && t < P.T && row_at(P, b0, t, r, flags)) {
      const int in_block = (int)(r.slot & (P.block - 1));
      if (r.slot < r.i || r.slot >= (long long)P.max_pages * P.page_size) {  // (kv_len below 0)
        flags |= SV_STATUS_BAD_LENGTH;
      } else if (r.i == 0 || in_block == 0) {
        const int page = P.table[(size_t)r.b * P.max_pages + r.slot / P.page_size];
        if (page < 0 || page >= P.num_pages) {
          flags |= SV_STATUS_BAD_PAGE;
        } else {
          const int in = (int)(r.slot & (P.page_size - 1));
          starts = true;
          run.t = t;
          run.rows = P.block - in_block < r.n - r.i ? P.block - in_block : r.n - r.i;
          run.old = in_block;
          run.k_at = page * P.kp + in * P.kt;
          run.v_at = page * P.vp + in * P.vt;
          run.scale_at = ((long long)page * (P.page_size / P.block) + in / P.block) * P.Hk;
          run.slot = r.slot;
        }
      }
    }
    const unsigned int who = __ballot_sync(0xffffffffu, starts);
    if (starts) s_run[__popc(who & ((1u << lane) - 1u))] = run;
    if (lane == 0) s_runs = __popc(who);
    const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && any) atomicOr(P.status, any);
  }
  __syncthreads();
#pragma unroll 1
  for (int x = 0; x < s_runs; ++x) {
    const Run run = s_run[x];
    const int tasks = run.rows * per;
    bool angles = false;  // this run's are formed
#pragma unroll 1
    for (int item = warp; item < 2 * P.Hk || !angles; item += THREADS / 32) {
      const bool live = item < 2 * P.Hk, keys = item < P.Hk;
      const int h = keys ? item : item - P.Hk;
      const char* src = keys ? P.k + ((long long)run.t * P.k_row + (long long)h * P.k_head) * 2
                             : P.v + ((long long)run.t * P.v_row + (long long)h * P.v_head) * 2;
      const long long row_bytes = (keys ? P.k_row : P.v_row) * 2;
      Words<VW> held[kHold];
      if (live) {
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
          const int e = lane + 32 * k;
          if (e < tasks) {
            const int r = e / per;
            held[k] = fetch<VW>(src + r * row_bytes, place_of<VW, INTER>(e - r * per, keys, P.rot));
          }
        }
      }
      if (!angles) {  // with the first values under way
        for (int e = tid; e < run.rows * half; e += THREADS) {
          const int r = e / half;
          s_turn[e] = turn_of(P, position(P, run.t + r, run.slot + r), e - r * half);
        }
        __syncthreads();
        angles = true;
      }
      if (!live) continue;
      float m2 = 0.f;
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const int e = lane + 32 * k;
        if (e < tasks) m2 = fmaxf(m2, squares<T, VW, INTER>(held[k], place_of<VW, INTER>(e % per, keys, P.rot), P.power, P.rest2));
      }
#pragma unroll 1
      for (int e = lane + 32 * kHold; e < tasks; e += 32) {
        const int r = e / per;
        const Place p = place_of<VW, INTER>(e - r * per, keys, P.rot);
        m2 = fmaxf(m2, squares<T, VW, INTER>(fetch<VW>(src + r * row_bytes, p), p, P.power, P.rest2));
      }
      m2 = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m2)));
      float s = __uint_as_float((unsigned int)(exponent_of(m2) + 127) << 23);
      float* scale_at = (keys ? P.k_scales : P.v_scales) + run.scale_at + h;
      unsigned char* dst = keys ? P.k_pages + run.k_at + (long long)h * P.kh : P.v_pages + run.v_at + (long long)h * P.vh;
      const long long slot_bytes = keys ? P.kt : P.vt;
      if (run.old > 0) {
        const float was = *scale_at;
        if (!(was >= 0x1p-32f && was <= 0x1p64f)) {
          if (lane == 0) atomicOr(P.status, (unsigned int)SV_STATUS_BAD_SCALE);
        } else if (was >= s) {
          s = was;
        } else {
          const float f = was / s;
          const int vecs = P.D / 16;
          for (int e = lane; e < run.old * vecs; e += 32) {
            const int r = e / vecs;
            uint4* at = reinterpret_cast<uint4*>(dst - (run.old - r) * slot_bytes + (e - r * vecs) * 16);
            uint4 w = *at;
            unsigned int* u = reinterpret_cast<unsigned int*>(&w);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 a = values2((unsigned short)u[y]), b = values2((unsigned short)(u[y] >> 16));
              u[y] = codes2(a.x * f, a.y * f) | (codes2(b.x * f, b.y * f) << 16);
            }
            *at = w;
          }
        }
        __syncwarp();  // (every lane has read the old scale)
      }
      if (lane == 0) *scale_at = s;
      const float inv = 1.f / s;
      auto put = [&](const Words<VW>& w, int r, const Place& p) {
        float o[2 * VW];
        turned<T, VW, INTER>(w, p, s_turn + r * half, o);
        unsigned char* d = dst + r * slot_bytes;
        if constexpr (VW == 1) {
          const unsigned int c = codes2(o[0] * inv, o[1] * inv);
          d[p.j] = (unsigned char)c;
          d[p.j2] = (unsigned char)(c >> 8);
        } else {
          unsigned int c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c[i] = codes2(o[4 * i] * inv, o[4 * i + 1] * inv) | (codes2(o[4 * i + 2] * inv, o[4 * i + 3] * inv) << 16);
          if (p.turns && !INTER) {
            *reinterpret_cast<uint2*>(d + p.j) = make_uint2(c[0], c[1]);
            *reinterpret_cast<uint2*>(d + p.j2) = make_uint2(c[2], c[3]);
          } else {
            *reinterpret_cast<uint4*>(d + p.j) = make_uint4(c[0], c[1], c[2], c[3]);
          }
        }
      };
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const int e = lane + 32 * k;
        if (e < tasks) {
          const int r = e / per;
          put(held[k], r, place_of<VW, INTER>(e - r * per, keys, P.rot));
        }
      }
#pragma unroll 1
      for (int e = lane + 32 * kHold; e < tasks; e += 32) {
        const int r = e / per;
        const Place p = place_of<VW, INTER>(e - r * per, keys, P.rot);
        put(fetch<VW>(src + r * row_bytes, p), r, p);
      }
    }
    __syncthreads();  // before the next run's angles
  }
}

template <typename T, int VW, bool INTER, int THREADS>
__device__ __forceinline__ void q_part(const Append8Params& P, float2* s_turn) {
  constexpr int kAhead = 2;  // tasks under way together
  __shared__ long long s_pos[4];
  __shared__ int s_ok[4];
  const int tid = threadIdx.x, lane = tid & 31;
  const int half = P.rot / 2, per = P.D / (2 * VW), n = P.Hq * per;
  const int r0 = (blockIdx.x - P.kv_ctas) * P.q_rows;
  const int rows = P.T - r0 < P.q_rows ? P.T - r0 : P.q_rows;
  Words<VW> w[kAhead];
  auto load = [&](int e0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int e = e0 + k * THREADS;
      if (e >= rows * n) continue;
      const int r = e / n, y = e - r * n, h = y / per;
      w[k] = fetch<VW>(P.q + ((long long)(r0 + r) * P.q_row + (long long)h * P.q_head) * 2,
                       place_of<VW, INTER>(y - h * per, true, P.rot));
    }
  };
  load(tid);
  if (tid < 32) {
    const int b0 = request_of(P.cu, P.B, r0);
    if (lane < rows) {
      unsigned int ignored = 0;  // (the keys' part sets the status)
      RowAt r;
      const bool ok = row_at(P, b0, r0 + lane, r, ignored);
      s_ok[lane] = ok;
      s_pos[lane] = ok ? position(P, r0 + lane, r.slot) : 0;
    }
  }
  __syncthreads();
  for (int e = tid; e < rows * half; e += THREADS) {
    const int r = e / half;
    s_turn[e] = turn_of(P, s_pos[r], e - r * half);
  }
  __syncthreads();
#pragma unroll 1
  for (int e0 = tid; e0 < rows * n; e0 += kAhead * THREADS) {
    if (e0 != tid) load(e0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int e = e0 + k * THREADS;
      if (e >= rows * n) continue;
      const int r = e / n, y = e - r * n, h = y / per;
      if (!s_ok[r]) continue;
      const Place p = place_of<VW, INTER>(y - h * per, true, P.rot);
      float o[2 * VW];
      turned<T, VW, INTER>(w[k], p, s_turn + r * half, o);
      char* d = P.q_out + ((long long)(r0 + r) * P.o_row + (long long)h * P.o_head) * 2;
      // (values that do not turn go through 32 bits and back unchanged)
      if constexpr (VW == 1) {
        const unsigned int c = Conv<T>::down(o[0], o[1]);
        unsigned short* u = reinterpret_cast<unsigned short*>(d);
        u[p.j] = (unsigned short)c;
        u[p.j2] = (unsigned short)(c >> 16);
      } else {
        Words<VW> c;
#pragma unroll
        for (int i = 0; i < VW / 2; ++i) {
          c.x.w[i] = Conv<T>::down(o[2 * i], o[2 * i + 1]);
          c.y.w[i] = Conv<T>::down(o[VW + 2 * i], o[VW + 2 * i + 1]);
        }
        store_vec<VW>(d + p.j * 2, c.x);
        store_vec<VW>(d + p.j2 * 2, c.y);
      }
    }
  }
}

template <typename T, int VW, bool INTER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) append8_kernel(const __grid_constant__ Append8Params P) {
  extern __shared__ float2 s_turn[];  // cos, sin of a run's or of the CTA's rows
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x < P.kv_ctas)
    kv_part<T, VW, INTER, THREADS>(P, s_turn);
  else
    q_part<T, VW, INTER, THREADS>(P, s_turn);
}

template <typename T, int VW, bool INTER, int THREADS>
int launch_threads(Append8Params P, cudaStream_t stream) {
  constexpr int kMaxSmem = SV_MAX_BLOCK * (SV_MAX_HEAD_DIM / 2) * (int)sizeof(float2);
  const int run = P.G < P.block ? P.G + 1 : P.block;  // rows of a run at most
  const int rows = run > P.q_rows ? run : P.q_rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned int)(P.kv_ctas + (P.Hq > 0 ? (P.T + P.q_rows - 1) / P.q_rows : 0)));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)rows * (P.rot / 2) * sizeof(float2);
  if (cfg.dynamicSmemBytes > 40 * 1024) {
    const int rc = sv::code_of(cudaFuncSetAttribute(append8_kernel<T, VW, INTER, THREADS>,
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem));
    if (rc) return rc;
  }
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  sv::overlap_launch(at[0]);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return sv::code_of(cudaLaunchKernelEx(&cfg, append8_kernel<T, VW, INTER, THREADS>, P));
}

// us a call (32 / 8 heads of 128, bf16; the calls of a graph):
// - a CTA looks for runs among one row while CTAs are few, and up to 16: 17.9 with one, 26.2 with 4 (1200
//   rows); 115 with one, 106 with 4 and with 16 (20000); 4 / 1 heads of 64: 34.8, 23.2, 20.6 (20000)
// - 256 threads while CTAs are few, and longer where a run has heads for 8 warps: 5.5 against 8.3 with 128
//   (1 row), 12.9 / 16.6 (800), 19.6 / 27.2 (2048), 30.9 / 40.4 (5000), 111 / 106 (20000); 16 / 4 heads 18.8 / 20.8
//   (5000), 28.7 / 25.8 (8000); 4 / 1 heads of 64: 4.9 / 5.0 (256), 6.3 / 5.4 (800)
// - two rows of q a CTA from 2048 on: 20.5 against 32.1 with one (4 / 1 heads of 64, 20000), 22.2 / 25.7 (24 / 6
//   of 96, 5000), no difference with 32 / 8 heads; below, 6.9 / 6.8 (64 rows), 6.4 / 7.1 for one (8 / 1 heads, 800)
template <typename T, int VW, bool INTER>
int launch(Append8Params& P, cudaStream_t stream) {
  const int rows = (P.T + kSlots - 1) / kSlots;
  P.run_rows = rows < kMaxRuns ? rows : kMaxRuns;
  P.kv_ctas = (P.T + P.run_rows - 1) / P.run_rows;
  P.q_rows = P.T < 2048 ? 1 : 2;
  if (P.T < 608 || (P.Hk >= 4 && P.T < 6144)) return launch_threads<T, VW, INTER, 256>(P, stream);
  return launch_threads<T, VW, INTER, 128>(P, stream);
}

}  // namespace

extern "C" int spec_verify_kv_append_e4m3(
    const void* q, const int64_t* q_strides, int q_heads, const void* k, const int64_t* k_strides, const void* v,
    const int64_t* v_strides, sv_dtype dtype, void* q_out, const int64_t* q_out_strides, const sv_kv_cache* cache,
    const sv_kv_scales* scales, const int32_t* cu_draft, int total_drafts, int max_drafts, const int64_t* freq,
    int rot_dim, int interleaved, float rope_scale, const int32_t* positions, int position_offset, void* workspace,
    size_t ws_bytes, sv_stream_t stream) {
  if (!cache || !scales || !k_strides || !v_strides) return SV_ERR_NULL;
  const sv_kv_cache& c = *cache;
  int rc = sv::check_cache_e4m3(c, *scales);
  if (rc) return rc;
  if ((dtype != SV_BF16 && dtype != SV_F16) || total_drafts < 0 || max_drafts < 0 || q_heads < 0 || rot_dim < 0 ||
      rot_dim % 2 || rot_dim > c.head_dim || (interleaved != 0 && interleaved != 1) || !(rope_scale > 0.f) ||
      rope_scale > 3.0e38f || (long long)total_drafts + c.batch > kMaxRows)
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
    if ((!same(o, in) && !apart(o, in)) || !apart(o, view(k, k_strides, rows, c.kv_heads, c.head_dim)) ||
        !apart(o, view(v, v_strides, rows, c.kv_heads, c.head_dim)))
      return SV_ERR_ALIGN;
  }
  Append8Params P = {};
  P.q = static_cast<const char*>(q);
  P.k = static_cast<const char*>(k);
  P.v = static_cast<const char*>(v);
  P.q_out = static_cast<char*>(q_out);
  P.k_pages = static_cast<unsigned char*>(c.k_pages);
  P.v_pages = static_cast<unsigned char*>(c.v_pages);
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
  P.block = scales->block;
  P.table = c.page_table;
  P.kv_len = c.kv_len;
  P.cu = cu_draft;
  P.k_scales = scales->k;
  P.v_scales = scales->v;
  P.freq = reinterpret_cast<const long long*>(freq);
  P.positions = positions;
  P.offset = position_offset;
  P.scale = rope_scale;
  int e = std::ilogb(rope_scale);
  P.power = std::ldexp(1.f, e < -126 ? -126 : e);
  P.rest2 = (rope_scale / P.power) * (rope_scale / P.power);
  P.status = static_cast<unsigned int*>(workspace);
  // vectors of 8 values where every head's start and both halves of a rotation allow it
  bool wide = rot_dim % 16 == 0;
  for (long long x : {P.q_row, P.q_head, P.o_row, P.o_head, P.k_row, P.k_head, P.v_row, P.v_head}) wide = wide && x % 8 == 0;
  for (const void* p : {q, k, v, (const void*)q_out}) wide = wide && sv::aligned(p, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const auto go = [&](auto t) {
    using T = decltype(t);
    if (wide) return interleaved ? launch<T, 8, true>(P, s) : launch<T, 8, false>(P, s);
    return interleaved ? launch<T, 1, true>(P, s) : launch<T, 1, false>(P, s);
  };
  return dtype == SV_BF16 ? go(__nv_bfloat16()) : go(__half());
}
