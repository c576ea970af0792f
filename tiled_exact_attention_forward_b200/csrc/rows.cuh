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
//
// Arithmetic is on pairs of floats (packed f32x2): with one value an instruction the
// kernels were bound by instruction issue (23 an element, 0.77 of the issue slots,
// 4.5 TB/s), not by memory.
#pragma once

#include "common.cuh"

namespace fa {
namespace rows {

// Element types: 16-bit (Bf16, F16, from common.cuh) and float32.
struct F32 {};

template <class E> struct Raw { using type = uint2; };          // four 16-bit elements
template <> struct Raw<F32> { using type = float4; };
template <class E> __host__ __device__ constexpr int elem_bytes() { return 2; }
template <> __host__ __device__ constexpr int elem_bytes<F32>() { return 4; }

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ uint64_t f2_swap(uint64_t a) { return a << 32 | a >> 32; }

// A lane's eight elements (or coefficients): pairs 0, 1 are the lo run, 2, 3 the hi run.
struct Oct {
  uint64_t p[4];
};

template <class E> __device__ __forceinline__ void unpack(const typename Raw<E>::type& r, uint64_t& a, uint64_t& b);
template <> __device__ __forceinline__ void unpack<Bf16>(const uint2& r, uint64_t& a, uint64_t& b) {
  a = f2_pack(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
  b = f2_pack(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
template <> __device__ __forceinline__ void unpack<F16>(const uint2& r, uint64_t& a, uint64_t& b) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
  a = f2_pack(x.x, x.y);
  b = f2_pack(y.x, y.y);
}
template <> __device__ __forceinline__ void unpack<F32>(const float4& r, uint64_t& a, uint64_t& b) {
  a = f2_pack(r.x, r.y);
  b = f2_pack(r.z, r.w);
}
template <class E>
__device__ __forceinline__ Oct unpack(const typename Raw<E>::type& lo, const typename Raw<E>::type& hi) {
  Oct o;
  unpack<E>(lo, o.p[0], o.p[1]);
  unpack<E>(hi, o.p[2], o.p[3]);
  return o;
}
// float32 results rounded once, to nearest even, to the element type.
template <class E> __device__ __forceinline__ typename Raw<E>::type pack(uint64_t a, uint64_t b) {
  float x, y, z, w;
  f2_unpack(a, x, y);
  f2_unpack(b, z, w);
  return make_uint2(pack2<E>(x, y), pack2<E>(z, w));
}
template <> __device__ __forceinline__ float4 pack<F32>(uint64_t a, uint64_t b) {
  float4 r;
  f2_unpack(a, r.x, r.y);
  f2_unpack(b, r.z, r.w);
  return r;
}

// Four elements at byte offset `at` of `base`.
template <class E> __device__ __forceinline__ typename Raw<E>::type load4(const char* at) {
  return *reinterpret_cast<const typename Raw<E>::type*>(at);
}
template <class E> __device__ __forceinline__ void store4(char* at, const typename Raw<E>::type& v) {
  *reinterpret_cast<typename Raw<E>::type*>(at) = v;
}

// Byte offsets of lane s's two runs in a row of E.
struct Lane {
  int lo, hi;
  bool turn;  // the lane's elements are rotated
};
template <class E, int D, bool INTER>
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
  l.lo *= elem_bytes<E>();
  l.hi *= elem_bytes<E>();
  return l;
}

// Sum over the lanes of a row (L = 8 or 16 consecutive lanes of a warp; every lane
// of the warp calls it).
template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// A lane's share of the dot product of two rows.
__device__ __forceinline__ float dot(const Oct& a, const Oct& b) {
  uint64_t s = f2_mul(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = f2_fma(a.p[i], b.p[i], s);
  float x, y;
  f2_unpack(s, x, y);
  return x + y;
}
// 1 / sqrt(v): the approximate instruction (within 2 units in the last place) and one
// Newton step, r + r (1 - v r^2) / 2.  The step is left out where it has nothing to add:
// r infinite (v = 0) or zero (v infinite), where it would make NaN.
__device__ __forceinline__ float rsqrt_row(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return v > 0.f && v < 1e38f ? fmaf(0.5f * r, e, r) : r;
}

// A linear map on a lane's pairs: z_i = x_i keep_i + partner_i cross_i, where the partner
// of a half-split pair is the other run's pair, of adjacent pairs the same one swapped.
struct Turn {
  Oct keep, cross;
};
template <bool INTER> __device__ __forceinline__ uint64_t partner(const Oct& x, int i) {
  return INTER ? f2_swap(x.p[i]) : x.p[i ^ 2];
}
// z = turned x (t.cross unused, and no partner read, in a lane that does not turn: its
// partner's infinity must not meet a zero).
template <bool INTER> __device__ __forceinline__ Oct apply(const Turn& t, bool turn, const Oct& x) {
  Oct z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.p[i] = f2_mul(x.p[i], t.keep.p[i]);
  if (turn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) z.p[i] = f2_fma(partner<INTER>(x, i), t.cross.p[i], z.p[i]);
  }
  return z;
}

// The rotation at `pos` for lane s: row `pos` of the table holds rot/2 cosines, then rot/2
// sines; (a, b) becomes (a c - b s, b c + a s).  A lane that does not turn keeps its
// elements; a position outside the table reads nothing and gives NaN.
template <bool INTER>
__device__ __forceinline__ Turn rotation(const float* table, long long pos, bool inside, int rot, int s, bool turn) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turn) {
    if (inside) {
      const float* row = table + pos * rot + 4 * s;
      c = *reinterpret_cast<const float4*>(row);
      sn = *reinterpret_cast<const float4*>(row + rot / 2);
    } else {
      const float nan = __uint_as_float(0x7fc00000u);
      c = sn = make_float4(nan, nan, nan, nan);
    }
  }
  Turn t;
  if (INTER) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.keep.p[i] = f2_both(cc[i]);
      t.cross.p[i] = f2_pack(-ss[i], ss[i]);
    }
  } else {
    t.keep.p[0] = t.keep.p[2] = f2_pack(c.x, c.y);
    t.keep.p[1] = t.keep.p[3] = f2_pack(c.z, c.w);
    t.cross.p[2] = f2_pack(sn.x, sn.y);
    t.cross.p[3] = f2_pack(sn.z, sn.w);
    t.cross.p[0] = f2_neg(t.cross.p[2]);
    t.cross.p[1] = f2_neg(t.cross.p[3]);
  }
  return t;
}
// The transpose: the same angles backwards.
__device__ __forceinline__ Turn transposed(Turn t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) t.cross.p[i] = f2_neg(t.cross.p[i]);
  return t;
}
// The rotation of w x as one map of x: each coefficient times the weight of the element
// that it multiplies.
template <bool INTER> __device__ __forceinline__ Turn weighted(Turn t, const Oct& w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.keep.p[i] = f2_mul(t.keep.p[i], w.p[i]);
    t.cross.p[i] = f2_mul(t.cross.p[i], partner<INTER>(w, i));
  }
  return t;
}

// A lane's share of a weight vector (ones when there is none), in E or in float32.
template <class E, int D, bool INTER>
__device__ __forceinline__ Oct load_weight(const void* w, int w_f32, int s, int rot) {
  Oct o;
  o.p[0] = o.p[1] = o.p[2] = o.p[3] = f2_both(1.f);
  if (w == nullptr) return o;
  const char* at = static_cast<const char*>(w);
  if (w_f32) {
    const Lane l = lane_of<F32, D, INTER>(s, rot);
    return unpack<F32>(load4<F32>(at + l.lo), load4<F32>(at + l.hi));
  }
  const Lane l = lane_of<E, D, INTER>(s, rot);
  return unpack<E>(load4<E>(at + l.lo), load4<E>(at + l.hi));
}

}  // namespace rows
}  // namespace fa
