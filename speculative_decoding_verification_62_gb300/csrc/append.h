// What the appends to a paged cache share: 16-bit values as pairs of floats, a row's
// request, and which outputs may not reach which inputs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace sv {
namespace append {

template <typename T>
struct Conv;
template <>
struct Conv<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(unsigned int w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ unsigned int down(float a, float b) {
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<unsigned int*>(&r);
  }
};
template <>
struct Conv<__half> {
  static __device__ __forceinline__ float2 up(unsigned int w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
  static __device__ __forceinline__ unsigned int down(float a, float b) {
    __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<unsigned int*>(&r);
  }
};

// VW 16-bit values as 32-bit words
template <int VW>
struct Vec {
  unsigned int w[VW / 2];
};
template <int VW>
__device__ __forceinline__ Vec<VW> load_vec(const char* p) {
  Vec<VW> r;
  if (VW == 8) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    r.w[0] = v.x, r.w[1] = v.y, r.w[2 % (VW / 2)] = v.z, r.w[3 % (VW / 2)] = v.w;
  } else {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x, r.w[1] = v.y;
  }
  return r;
}
template <int VW>
__device__ __forceinline__ void store_vec(char* p, const Vec<VW>& r) {
  if (VW == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2 % (VW / 2)], r.w[3 % (VW / 2)]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
}

// The request of row t: the largest b with cu[b] + b <= t, by one warp, 32
// probes a round.
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool le = at < hi && (long long)cu[at] + at <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    if (n == 0) return lo;
    lo += (n - 1) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Host side: CTAs read and write their rows in no order, so q_out may not reach what
// another row still reads, nor itself.
// ---------------------------------------------------------------------------
using Wide = __int128;  // offsets in bytes, at any stride
inline Wide size_of(long long s) { return s < 0 ? -(Wide)s : (Wide)s; }

// [n[0]][n[1]][dim] values of 2 bytes, strides in elements (dimension 0: rows, 1: heads)
struct View {
  Wide at;
  long long n[2], stride[2];
  int dim;
  Wide inner(int d) const {  // bytes from the first to behind the last value along dimension d
    return (Wide)(n[d] - 1) * size_of(stride[d]) * 2 + dim * 2;
  }
  Wide first(int d) const {  // the lowest address along dimension d
    return at + (stride[d] < 0 ? (Wide)(n[d] - 1) * stride[d] * 2 : (Wide)0);
  }
};
inline View view(const void* p, const int64_t* strides, long long rows, long long heads, int dim) {
  return View{(Wide)reinterpret_cast<uintptr_t>(p), {rows, heads}, {strides[0], strides[1]}, dim};
}
inline bool overlaps_itself(const View& v) {
  const int in = v.n[0] == 1 || (v.n[1] > 1 && size_of(v.stride[1]) <= size_of(v.stride[0])) ? 1 : 0;
  const int out = 1 - in;
  return (v.n[in] > 1 && size_of(v.stride[in]) < v.dim) ||
         (v.n[out] > 1 && size_of(v.stride[out]) * 2 < v.inner(in));
}
// Whether two views are known to share no value: their reaches are apart, or they are
// slices of one tensor (the q, k and v parts of a projection's rows): one stride along
// rows or along heads, and windows within it that are apart.
inline bool apart(const View& a, const View& b) {
  auto low = [](const View& v) { return v.first(0) + v.first(1) - v.at; };
  auto high = [&](const View& v) { return low(v) + v.inner(0) + v.inner(1) - v.dim * 2; };
  if (high(a) <= low(b) || high(b) <= low(a)) return true;
  for (int d = 0; d < 2; ++d) {
    const Wide step = size_of(a.stride[d]) * 2;
    if (a.stride[d] != b.stride[d] || a.inner(1 - d) > step || b.inner(1 - d) > step) continue;
    const Wide by = ((b.first(1 - d) - a.first(1 - d)) % step + step) % step;
    if (by >= a.inner(1 - d) && by + b.inner(1 - d) <= step) return true;
  }
  return false;
}
inline bool same(const View& a, const View& b) {
  return a.at == b.at && (a.n[0] == 1 || a.stride[0] == b.stride[0]) &&
         (a.n[1] == 1 || a.stride[1] == b.stride[1]);
}

}  // namespace append
}  // namespace sv
