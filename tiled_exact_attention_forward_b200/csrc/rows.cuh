// One row of a head (d elements) spread over d / 8 lanes: loads, stores, the row
// sum, and the position rotation, shared by the norm-and-rotate kernels and the
// paged append.
//
// Lane layout: lane s of a row holds two runs of four elements, `lo` and `hi`,
// chosen so that both elements of every rotated pair sit in the same lane and no
// element crosses lanes:
//   half-split pairs (i, i + rot/2):  lo = [4s, 4s+4), hi = lo + rot/2   for s < rot/8,
//                                     the unrotated rest split in two halves alike;
//   adjacent pairs (2i, 2i+1):        lo = [8s, 8s+4), hi = [8s+4, 8s+8).
// Either way lane s < rot/8 needs cos and sin of the pairs 4s .. 4s+3 only.  A run
// is one 8-byte (16-bit types) or 16-byte (float32) access; the 16 lanes of a
// d = 128 row read 128 contiguous bytes per access.  (The alternative, 16-byte
// accesses with the partner fetched by shuffles, needs eight shuffles a row.)
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace fa {
namespace rows {

// Element types: 16-bit (Bf16, F16, from common.cuh) and float32.
struct F32 {};

template <class E> struct Raw { using type = uint2; };          // four 16-bit elements
template <> struct Raw<F32> { using type = float4; };
template <class E> __host__ __device__ constexpr int elem_bytes() { return 2; }
template <> __host__ __device__ constexpr int elem_bytes<F32>() { return 4; }

template <class E> __device__ __forceinline__ void unpack4(const typename Raw<E>::type& r, float (&f)[4]);
template <> __device__ __forceinline__ void unpack4<Bf16>(const uint2& r, float (&f)[4]) {
  f[0] = __uint_as_float(r.x << 16);
  f[1] = __uint_as_float(r.x & 0xffff0000u);
  f[2] = __uint_as_float(r.y << 16);
  f[3] = __uint_as_float(r.y & 0xffff0000u);
}
template <> __device__ __forceinline__ void unpack4<F16>(const uint2& r, float (&f)[4]) {
  f[0] = __half2float(__ushort_as_half(static_cast<unsigned short>(r.x & 0xffffu)));
  f[1] = __half2float(__ushort_as_half(static_cast<unsigned short>(r.x >> 16)));
  f[2] = __half2float(__ushort_as_half(static_cast<unsigned short>(r.y & 0xffffu)));
  f[3] = __half2float(__ushort_as_half(static_cast<unsigned short>(r.y >> 16)));
}
template <> __device__ __forceinline__ void unpack4<F32>(const float4& r, float (&f)[4]) {
  f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
}
// float32 results rounded once, to nearest even, to the element type.
template <class E> __device__ __forceinline__ typename Raw<E>::type pack4(const float (&f)[4]) {
  return make_uint2(pack2<E>(f[0], f[1]), pack2<E>(f[2], f[3]));
}
template <> __device__ __forceinline__ float4 pack4<F32>(const float (&f)[4]) {
  return make_float4(f[0], f[1], f[2], f[3]);
}

// Four elements at element offset `i` of `base`.
template <class E> __device__ __forceinline__ typename Raw<E>::type load4(const void* base, long long i) {
  return *reinterpret_cast<const typename Raw<E>::type*>(static_cast<const char*>(base) + i * elem_bytes<E>());
}
template <class E>
__device__ __forceinline__ void store4(void* base, long long i, const typename Raw<E>::type& v) {
  *reinterpret_cast<typename Raw<E>::type*>(static_cast<char*>(base) + i * elem_bytes<E>()) = v;
}

// Element offsets of lane s's two runs.
struct Lane {
  int lo, hi;
  bool turn;  // the lane's elements are rotated
};
template <int D, bool INTER>
__device__ __forceinline__ Lane lane_of(int s, int rot) {
  Lane l;
  l.turn = s < rot / 8;
  if (INTER) {
    l.lo = 8 * s;
    l.hi = 8 * s + 4;
  } else if (l.turn) {
    l.lo = 4 * s;
    l.hi = 4 * s + rot / 2;
  } else {
    l.lo = rot + 4 * (s - rot / 8);
    l.hi = l.lo + (D - rot) / 2;
  }
  return l;
}

// Sum over the lanes of a row (L = 8 or 16 consecutive lanes of a warp; every lane
// of the warp calls it).
template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float dot8(const float (&a)[4], const float (&b)[4], const float (&c)[4], const float (&d)[4]) {
  float s = a[0] * c[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fmaf(a[i], c[i], s);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(b[i], d[i], s);
  return s;
}

// The rotation by the angles whose cosines and sines are c, s: (a, b) becomes
// (a c - b s, b c + a s).  Call with -s for the transpose.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&lo)[4], float (&hi)[4], const float (&c)[4], const float (&s)[4]) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = lo[2 * i], b = lo[2 * i + 1];
      lo[2 * i] = a * c[i] - b * s[i];
      lo[2 * i + 1] = b * c[i] + a * s[i];
      const float a2 = hi[2 * i], b2 = hi[2 * i + 1];
      hi[2 * i] = a2 * c[i + 2] - b2 * s[i + 2];
      hi[2 * i + 1] = b2 * c[i + 2] + a2 * s[i + 2];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = lo[i], b = hi[i];
      lo[i] = a * c[i] - b * s[i];
      hi[i] = b * c[i] + a * s[i];
    }
  }
}

// cos and sin of lane s's four pairs at `pos`: row `pos` of the table holds rot/2
// cosines, then rot/2 sines.  Lanes that do not turn get (1, 0); a position outside
// the table reads nothing and gets NaN.
__device__ __forceinline__ void load_angles(const float* table, long long pos, bool inside, int rot, int s, bool turn,
                                            float (&c)[4], float (&sn)[4]) {
  float4 vc = make_float4(1.f, 1.f, 1.f, 1.f), vs = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turn) {
    if (inside) {
      const float* row = table + pos * rot;
      vc = *reinterpret_cast<const float4*>(row + 4 * s);
      vs = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * s);
    } else {
      const float nan = __uint_as_float(0x7fc00000u);
      vc = vs = make_float4(nan, nan, nan, nan);
    }
  }
  c[0] = vc.x; c[1] = vc.y; c[2] = vc.z; c[3] = vc.w;
  sn[0] = vs.x; sn[1] = vs.y; sn[2] = vs.z; sn[3] = vs.w;
}

// A lane's share of a weight vector (ones when there is none), in E or in float32.
template <class E>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, const Lane& l, float (&lo)[4], float (&hi)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) lo[i] = hi[i] = 1.f;
  if (w == nullptr) return;
  if (w_f32) {
    unpack4<F32>(load4<F32>(w, l.lo), lo);
    unpack4<F32>(load4<F32>(w, l.hi), hi);
  } else {
    unpack4<E>(load4<E>(w, l.lo), lo);
    unpack4<E>(load4<E>(w, l.hi), hi);
  }
}

}  // namespace rows
}  // namespace fa
