// Verification of drafted tokens against given probabilities.
//
// Per request: draft i is accepted iff q_i(x_i) = 0 or u_i q_i(x_i) < p_i(x_i);
// k is the first draft refused, or gamma_b.  The last token is drawn from
//   w = max(0, p_k - q_k)   (k < gamma_b; from p_k where every w is 0)
//   w = p_{gamma_b}         (every draft accepted)
// by the inverse CDF: the smallest j with w_0 + .. + w_j > u w_total.
//
// The test is exact: u q is a product of two 24-bit numbers, formed in double.
// The draw is exact up to the weights' grain: each weight is a whole multiple of
// 2^-47 (of 2^-46 without q), found by additions alone (weight() below), and weights are
// summed as integers, so that no sum depends on an order; u w_total is compared after a
// 128-bit product.  Weights below 2^-22 are rounded (by at most 2^-47, and by
// 2^-48 more where p - q itself is rounded), and the roundings of n entries move a
// boundary by about 2^-48 sqrt(n): a uniform lands on the other side of one of V boundaries
// with a chance of about V sqrt(V) 2^-48 (2^-23 at V = 128256, if all entries
// were that small).  Sums saturate at 2^63 = 65536 (a row sums to about 1).
//
// Bound: the one or two rows that the draw needs are read once from HBM; all
// other reads are gathers.  A cluster of C CTAs shares a request, each warp a
// contiguous range of the row.  The owner of the target re-reads only the
// range of the warp that holds it, from L2.  Measured (GB300): 512 requests over
// 128256 entries of bf16, 350 of them with a refused draft, 59.5 us (222 MB, 3.7 TB/s;
// instruction issue 54 %, integer pipe 46 %), 64 requests over 152064 of fp32, 50
// refused, 19.0 us (70 MB), one request 5.7 us: latency, a chain of gathers, sums,
// exchange and walk.  Staging by asynchronous copies (66 us), a second set of registers
// (64 us) and three CTAs an SM (87 us) were slower at 512 requests.
#include "../../include/spec_verify.h"
#include "internal.h"

#include <atomic>

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr unsigned long long kCap = 1ull << 63;

struct ProbsParams {
  const char* target;
  const char* draft;  // null: the draft is certain of its token
  int B, G, V, total, C;
  const int32_t* tokens;
  const int32_t* gamma;  // padded layout
  const int32_t* cu;     // packed layout
  const float* uniforms;
  int32_t* out;
  int32_t* accepted;
  unsigned int* status;
};

__device__ __forceinline__ unsigned long long sat_add(unsigned long long a, unsigned long long b) {
  const unsigned long long s = a + b;  // both at most 2^63
  return s < kCap ? s : kCap;
}

template <int EB>
__device__ __forceinline__ float load_one(const char* row, size_t i) {
  if (EB == 4) return __ldg(reinterpret_cast<const float*>(row) + i);
  return __uint_as_float((unsigned int)__ldg(reinterpret_cast<const unsigned short*>(row) + i) << 16);
}

// A probability's bits; what is none counts as 0, what is above 1 as 1, and both
// are flagged (-0 is 0).
__device__ __forceinline__ unsigned int clean(unsigned int bits, unsigned int& flags) {
  if (bits <= 0x3f800000u) return bits;
  if (bits == 0x80000000u) return 0u;
  flags |= SV_STATUS_BAD_PROB;
  return bits <= 0x7f800000u ? 0x3f800000u : 0u;
}

// A weight in units of 2^-47 is hi 2^24 + 2 lo + le.  With d = p - q rounded and e
// its exact error (q <= p, so that (p - d) - q is exact), adding 1 rounds d to a
// multiple of 2^-23, which stands in the sum's low bits; what is left of d, at most
// 2^-24, is rounded to a multiple of 2^-46 by adding 1.5 2^-23 in the same way, and
// e, at most 2^-25, to one of 2^-47 by adding 1.5 2^-24.  Additions run at twice the
// rate of integer instructions, and a conversion to 64-bit integers at an eighth.
constexpr unsigned int kOne = 0x3f800000u;     // 1
constexpr unsigned int kRest = 0x34400000u;    // 1.5 2^-23
constexpr unsigned int kError = 0x33c00000u;   // 1.5 2^-24
struct Parts {
  unsigned int hi, lo, le;  // sums of the parts, with kOne, kRest and kError in each
};

// Two weights at a time.
template <bool TWO>
__device__ __forceinline__ void add_weights(unsigned int p0, unsigned int p1, unsigned int q0, unsigned int q1,
                                            Parts& sum) {
  auto pack = [](unsigned int a, unsigned int b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
  };
  auto add = [](unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
  };
  // a - b
  auto sub = [&](unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(0xbf800000bf800000ull), "l"(a));
    return r;
  };
  const unsigned long long one = 0x3f8000003f800000ull, minus_one = 0xbf800000bf800000ull,
                           rest = 0x3440000034400000ull, error = 0x33c0000033c00000ull;
  const unsigned long long p = pack(p0, p1);
  unsigned long long d = p, e = 0;
  if (TWO) {
    const unsigned long long q = pack(min(p0, q0), min(p1, q1));  // as floats: none is negative
    d = sub(p, q);
    e = sub(sub(p, d), q);
  }
  const unsigned long long t = add(d, one);
  const unsigned long long t2 = add(sub(d, add(t, minus_one)), rest);
  unsigned int a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(t));
  sum.hi += a + b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(t2));
  sum.lo += a + b;
  if (TWO) {
    const unsigned long long t3 = add(e, error);
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(t3));
    sum.le += a + b;
  }
}
// The sum of n weights from their parts' sums (n at most 256: hi stays below 2^32)
template <bool TWO>
__device__ __forceinline__ unsigned long long joined(const Parts& s, unsigned int n) {
  return ((unsigned long long)(s.hi - n * kOne) << 24) + 2 * (long long)(int)(s.lo - n * kRest) +
         (TWO ? (long long)(int)(s.le - n * kError) : 0ll);
}
__device__ __forceinline__ unsigned long long weight(unsigned int p, unsigned int q) {
  Parts s{0u, 0u, 0u};
  add_weights<true>(p, 0u, q, 0u, s);
  return joined<true>(s, 2);
}

// floor(u S) for a float u in [0, 1): u = m 2^-s with a 24-bit m.
__device__ __forceinline__ unsigned long long scaled(float u, unsigned long long S) {
  if (u == 0.f) return 0;
  const unsigned int bits = __float_as_uint(u);
  const unsigned int e = bits >> 23;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int s = 150 - (int)(e ? e : 1u);  // 24 .. 149
  const unsigned long long hi = __umul64hi(m, S), lo = m * S;
  if (s >= 128) return 0;
  if (s >= 64) return hi >> (s - 64);
  return (hi << (64 - s)) | (lo >> s);
}

__device__ __forceinline__ unsigned int cluster_rank() {
  unsigned int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_to_rank(unsigned long long* p, unsigned int rank, unsigned long long v) {
  unsigned int a = (unsigned int)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(r), "l"(v) : "memory");
}

// The weights that a draw sums: of rows p and q (q may be null), or of p with
// token `skip` left out.
struct Draw {
  const char* p;
  const char* q;
  int skip;
};

template <int EB>
__device__ __forceinline__ unsigned long long weight_at(const Draw& d, int i) {
  unsigned int ignored = 0;
  if (i == d.skip) return 0;
  const unsigned int p = clean(__float_as_uint(load_one<EB>(d.p, i)), ignored);
  return weight(p, d.q ? clean(__float_as_uint(load_one<EB>(d.q, i)), ignored) : 0u);
}

template <int EB>
__device__ __forceinline__ unsigned int word_bits(const uint4& v, int j) {
  const unsigned int w = j * EB / 4 == 0 ? v.x : j * EB / 4 == 1 ? v.y : j * EB / 4 == 2 ? v.z : v.w;
  if (EB == 4) return w;
  return j & 1 ? w & 0xffff0000u : w << 16;
}

// Adds the weights of N entries.
template <int N, bool TWO>
__device__ __forceinline__ void add_batch(unsigned int (&p)[N], unsigned int (&q)[N], Parts& sum,
                                          unsigned int& flags) {
  unsigned int top = 0;
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    top = __vimax3_u32(top, p[j], p[j + 1]);
    if (TWO) top = __vimax3_u32(top, q[j], q[j + 1]);
  }
  if (top > kOne) {  // something that is no probability, or -0
#pragma unroll
    for (int j = 0; j < N; ++j) {
      p[j] = clean(p[j], flags);
      if (TWO) q[j] = clean(q[j], flags);
    }
  }
#pragma unroll
  for (int j = 0; j < N; j += 2) add_weights<TWO>(p[j], p[j + 1], q[j], q[j + 1], sum);
}

// The sum of one warp's units [u0, u1): a unit is 32 x 16 bytes of the row.
// VEC: rows are 16-byte aligned and V is a whole number of 16-byte words.
template <int EB, bool VEC, bool TWO>
__device__ __forceinline__ unsigned long long range_sum(const Draw& d, int V, int u0, int u1,
                                                        unsigned int& flags) {
  constexpr int E = 16 / EB;
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 31;
  unsigned long long acc = 0;
  if (VEC) {
    const uint4* p = reinterpret_cast<const uint4*>(d.p);
    const uint4* q = reinterpret_cast<const uint4*>(d.q);
    const int words = V / E;
#pragma unroll 1
    for (int u = u0; u < u1; u += kUnroll) {
      uint4 a[kUnroll], b[kUnroll];
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        const int w = (u + r) * 32 + lane;
        const bool in = u + r < u1 && w < words;
        a[r] = in ? __ldcs(p + w) : make_uint4(0, 0, 0, 0);
        if (TWO) b[r] = in ? __ldcs(q + w) : make_uint4(0, 0, 0, 0);
      }
      Parts sum{0u, 0u, 0u};
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        unsigned int x[E], y[E];
        const int skip = d.skip - ((u + r) * 32 + lane) * E;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          x[j] = word_bits<EB>(a[r], j);
          y[j] = TWO ? word_bits<EB>(b[r], j) : 0u;
          if (!TWO && j == skip) x[j] = 0u;
        }
        add_batch<E, TWO>(x, y, sum, flags);
      }
      acc = sat_add(acc, joined<TWO>(sum, kUnroll * E));
    }
  } else {
    constexpr int N = 2 * E;
#pragma unroll 1
    for (int u = u0; u < u1; u += 2) {
      unsigned int x[N], y[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = (u * E + j) * 32 + lane;
        const bool in = u + j / E < u1 && i < V && i != d.skip;
        x[j] = in ? __float_as_uint(load_one<EB>(d.p, i)) : 0u;
        y[j] = TWO && in ? __float_as_uint(load_one<EB>(d.q, i)) : 0u;
      }
      Parts sum{0u, 0u, 0u};
      add_batch<N, TWO>(x, y, sum, flags);
      acc = sat_add(acc, joined<TWO>(sum, N));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc = sat_add(acc, __shfl_xor_sync(0xffffffffu, acc, o));
  return acc;
}

template <int EB, bool PK, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) probs_kernel(ProbsParams P) {
  __shared__ int s_k, s_gb, s_skip;
  __shared__ unsigned long long s_warp[kWarps];
  __shared__ unsigned long long s_rank[2][kMaxCluster];
  __shared__ unsigned long long s_scan[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = P.C, b = blockIdx.x / C, V = P.V, G = P.G;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  unsigned int flags = 0;
  if (C > 1) cluster_arrive();  // waited for before the first store to a peer
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // rows of this request
  int gb;
  size_t trow, drow;
  if (PK) {
    const int c0 = P.cu[b], c1 = P.cu[b + 1];
    const bool ok = c0 >= 0 && c1 >= c0 && c1 - c0 <= G && c1 <= P.total;
    gb = ok ? c1 - c0 : 0;
    drow = (size_t)(c0 < 0 ? 0 : (c0 > P.total ? P.total : c0));
    trow = drow + b;
    if (!ok) flags |= SV_STATUS_BAD_GAMMA;
  } else {
    gb = P.gamma[b];
    if (gb < 0 || gb > G) flags |= SV_STATUS_BAD_GAMMA;
    gb = gb < 0 ? 0 : (gb > G ? G : gb);
    drow = (size_t)b * G;
    trow = (size_t)b * (G + 1);
  }
  const size_t last_u = PK ? trow + gb : trow + G;
  float u_last = P.uniforms[last_u];
  // the tests: one lane a draft, in every CTA of the cluster
  if (warp == 0) {
    bool ok = true;
    int x = 0;
    if (lane < gb) {
      x = P.tokens[drow + lane];
      if (x < 0 || x >= V) {
        flags |= SV_STATUS_BAD_TOKEN;
        x = x < 0 ? 0 : V - 1;
      }
      float p = load_one<EB>(P.target, (trow + lane) * V + x);
      float q = P.draft ? load_one<EB>(P.draft, (drow + lane) * V + x) : 1.f;
      float u = P.uniforms[trow + lane];
      p = __uint_as_float(clean(__float_as_uint(p), flags));
      q = __uint_as_float(clean(__float_as_uint(q), flags));
      if (!(u >= 0.f && u < 1.f)) {
        flags |= SV_STATUS_BAD_UNIFORM;
        u = 0.f;
      }
      ok = q == 0.f || (double)u * (double)q < (double)p;
    }
    const unsigned int refused = __ballot_sync(0xffffffffu, lane < gb && !ok);
    const int k = refused ? __ffs(refused) - 1 : gb;
    const int xk = __shfl_sync(0xffffffffu, x, k < 32 ? k : 0);
    if (lane == 0) {
      s_k = k;
      s_gb = gb;
      s_skip = k < gb && !P.draft ? xk : -1;
    }
    if (rank == 0) {
      if (lane <= G && lane != k) P.out[(size_t)b * (G + 1) + lane] = lane < k ? x : -1;
      if (lane == 0) P.accepted[b] = k;
    }
  }
  if (!(u_last >= 0.f && u_last < 1.f)) {
    flags |= SV_STATUS_BAD_UNIFORM;
    u_last = 0.f;
  }
  __syncthreads();
  const int k = s_k;
  const bool refused = k < s_gb;
  Draw d;
  d.p = P.target + (trow + k) * V * EB;
  d.q = refused && P.draft ? P.draft + (drow + k) * V * EB : nullptr;
  d.skip = s_skip;
  // this warp's units of the row
  constexpr int kUnit = 32 * (16 / EB);
  const int units = (V + kUnit - 1) / kUnit, NW = C * kWarps;
  const int w0 = rank * kWarps;
  unsigned long long S = 0, before = 0;
  int pass = 0;
  for (;; ++pass) {
    const int gw = w0 + warp;
    const int u0 = (int)((long long)units * gw / NW), u1 = (int)((long long)units * (gw + 1) / NW);
    const unsigned long long ws = d.q ? range_sum<EB, VEC, true>(d, V, u0, u1, flags)
                                      : range_sum<EB, VEC, false>(d, V, u0, u1, flags);
    if (lane == 0) s_warp[warp] = ws;
    __syncthreads();
    if (C > 1) {
      if (pass == 0) cluster_wait();  // every peer runs
      if (tid < C) {
        unsigned long long mine = 0;
        for (int w = 0; w < kWarps; ++w) mine = sat_add(mine, s_warp[w]);
        store_to_rank(&s_rank[pass][rank], tid, mine);
      }
      cluster_arrive();
      cluster_wait();
    } else {
      if (tid == 0) {
        unsigned long long mine = 0;
        for (int w = 0; w < kWarps; ++w) mine = sat_add(mine, s_warp[w]);
        s_rank[pass][0] = mine;
      }
      __syncthreads();
    }
    S = 0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) before = S;
      S = sat_add(S, s_rank[pass][r]);
    }
    // every residual weight 0: the draw is from p_k
    if (S != 0 || !refused || pass == 1) break;
    d.q = nullptr;
    d.skip = -1;
    __syncthreads();
  }
  if (S == 0 || S >= kCap) flags |= SV_STATUS_BAD_PROB;
  const unsigned long long goal = scaled(u_last, S);
  int32_t* drawn = P.out + (size_t)b * (G + 1) + k;
  if (S == 0) {
    if (rank == 0 && tid == 0) *drawn = V - 1;
  } else if (goal >= before && goal < sat_add(before, s_rank[pass][rank])) {
    // the warp whose range holds the target, then a thread of this CTA
    unsigned long long c = before;
    int w = 0;
    for (; w < kWarps - 1; ++w) {
      const unsigned long long n = sat_add(c, s_warp[w]);
      if (goal < n) break;
      c = n;
    }
    const int gw = w0 + w;
    const int e0 = (int)((long long)units * gw / NW) * kUnit;
    int e1 = (int)((long long)units * (gw + 1) / NW) * kUnit;
    if (e1 > V) e1 = V;
    const int per = (e1 - e0 + kThreads - 1) / kThreads;
    const int i0 = e0 + tid * per, i1 = i0 + per < e1 ? i0 + per : e1;
    unsigned long long mine = 0;
    for (int i = i0; i < i1; ++i) mine = sat_add(mine, weight_at<EB>(d, i));
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = sat_add(incl, v);
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    for (int v = 0; v < warp; ++v) c = sat_add(c, s_scan[v]);
    const unsigned long long prev = __shfl_up_sync(0xffffffffu, incl, 1);
    const unsigned long long from = lane ? sat_add(c, prev) : c;
    if (goal >= from && goal < sat_add(from, mine)) {
      unsigned long long at = from;
      for (int i = i0; i < i1; ++i) {
        at = sat_add(at, weight_at<EB>(d, i));
        if (goal < at) {
          *drawn = i;
          break;
        }
      }
    }
  }
  const unsigned int any = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0 && any) atomicOr(P.status, any);
}

// CTAs a request: the largest cluster of at most 8 that keeps the grid within
// two CTAs an SM, so that a small batch still reads with the whole GPU.
int cluster_for(int B) {
  static std::atomic<int> cached{0};
  int dev = 0, sms = 0;
  if (sv::code_of(cudaGetDevice(&dev))) return 0;
  const int c0 = cached.load(std::memory_order_relaxed);
  if ((c0 >> 16) == dev + 1) {
    sms = c0 & 0xffff;
  } else {
    if (sv::code_of(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev))) return 0;
    cached.store(((dev + 1) << 16) | sms, std::memory_order_relaxed);
  }
  int C = kMaxCluster;
  while (C > 1 && (long long)B * C > 2ll * sms) C >>= 1;
  return C;
}

template <int EB, bool PK, bool VEC>
int launch(ProbsParams P, cudaStream_t stream) {
  P.C = cluster_for(P.B);
  if (P.C <= 0) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned int)P.B * (unsigned int)P.C);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  sv::overlap_launch(at[1]);
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned int)P.C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return sv::code_of(cudaLaunchKernelEx(&cfg, probs_kernel<EB, PK, VEC>, P));
}

int verify_probs(const void* target, const void* draft, sv_dtype dtype, int B, int G, int V,
                 const int32_t* cu, int total, const int32_t* tokens, const int32_t* gamma,
                 const float* uniforms, int32_t* out, int32_t* accepted, void* ws, size_t ws_bytes,
                 sv_stream_t stream, bool packed) {
  if (B < 0 || G < 0 || G > SV_MAX_GAMMA || V < 1 || V > SV_MAX_VOCAB || total < 0)
    return SV_ERR_SCALAR;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_SCALAR;
  if (B == 0) return SV_OK;
  if (!target || !uniforms || !out || !accepted || !ws || (packed ? !cu : !gamma)) return SV_ERR_NULL;
  if ((packed ? total > 0 : G > 0) && !tokens) return SV_ERR_NULL;
  const size_t eb = dtype == SV_BF16 ? 2 : 4;
  if (ws_bytes < spec_verify_workspace_size(B, G, V)) return SV_ERR_WORKSPACE;
  if (!sv::aligned(target, eb) || !sv::aligned(draft, eb) || !sv::aligned(tokens, 4) ||
      !sv::aligned(gamma, 4) || !sv::aligned(cu, 4) || !sv::aligned(uniforms, 4) ||
      !sv::aligned(out, 4) || !sv::aligned(accepted, 4) || !sv::aligned(ws, 256))
    return SV_ERR_ALIGN;
  ProbsParams P;
  P.target = static_cast<const char*>(target);
  P.draft = static_cast<const char*>(draft);
  P.B = B;
  P.G = G;
  P.V = V;
  P.total = total;
  P.C = 1;
  P.tokens = tokens;
  P.gamma = gamma;
  P.cu = cu;
  P.uniforms = uniforms;
  P.out = out;
  P.accepted = accepted;
  P.status = static_cast<unsigned int*>(ws);
  // 16-byte loads where every row starts on a 16-byte boundary
  const bool vec = (size_t)V * eb % 16 == 0 && sv::aligned(target, 16) && sv::aligned(draft, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SV_BF16) {
    if (packed) return vec ? launch<2, true, true>(P, s) : launch<2, true, false>(P, s);
    return vec ? launch<2, false, true>(P, s) : launch<2, false, false>(P, s);
  }
  if (packed) return vec ? launch<4, true, true>(P, s) : launch<4, true, false>(P, s);
  return vec ? launch<4, false, true>(P, s) : launch<4, false, false>(P, s);
}

}  // namespace

extern "C" {

int spec_verify_sample_probs(const void* target_probs, const void* draft_probs, sv_dtype dtype,
                             int B, int G, int V, const int32_t* draft_tokens,
                             const int32_t* gamma, const float* uniforms, int32_t* out_tokens,
                             int32_t* num_accepted, void* workspace, size_t ws_bytes,
                             sv_stream_t stream) {
  return verify_probs(target_probs, draft_probs, dtype, B, G, V, nullptr, 0, draft_tokens, gamma,
                      uniforms, out_tokens, num_accepted, workspace, ws_bytes, stream, false);
}

int spec_verify_sample_probs_packed(const void* target_probs, const void* draft_probs,
                                    sv_dtype dtype, int B, int G, int V, const int32_t* cu_draft,
                                    int total_drafts, const int32_t* draft_tokens,
                                    const float* uniforms, int32_t* out_tokens,
                                    int32_t* num_accepted, void* workspace, size_t ws_bytes,
                                    sv_stream_t stream) {
  return verify_probs(target_probs, draft_probs, dtype, B, G, V, cu_draft, total_drafts,
                      draft_tokens, nullptr, uniforms, out_tokens, num_accepted, workspace,
                      ws_bytes, stream, true);
}

}  // extern "C"
