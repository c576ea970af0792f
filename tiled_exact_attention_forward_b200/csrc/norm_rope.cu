// Per-head RMS norm and position rotation of queries and keys in one pass, and its
// backward pass.
//
// With x one head's row of d elements, at position p of its sequence:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  z = R(p) y,
// where R(p) turns the first `rot` elements pairwise by the table's angles.
// Backward, with dz given:
//   g = R(p)^T dz,  dw = sum over rows of g x r,  u = g w,
//   dx = r (u - x r^2 mean(u x)).
// r is recomputed from x (which the backward reads anyway) instead of being saved.
// All arithmetic is float32; each output is rounded once.
//
// Both passes are bound by memory: the forward reads x and writes z, the backward
// reads x and dz and writes dx, each byte once; the table's rows are shared by the
// heads of a position and come from L2.  Input and output strides are free, so a
// projection's [B, N, H, d] output is read where it lies and written in the
// [B, H, N, d] order that the attention kernels take.
//
// Work split: a group of d / 8 lanes takes HG heads of one position, all its loads
// issued before the first is used; a block's groups take consecutive positions of
// the same heads, so its writes to [B, H, N, d] are runs of consecutive rows.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace fa {
namespace nrope {

using namespace rows;

constexpr int THREADS = 256;
constexpr int HG = 4;  // heads per group of lanes

template <int D> __host__ __device__ constexpr int positions_per_block() { return THREADS / (D / 8); }

// A block's work: HG heads of tensor t (0 = q, 1 = k) from head h0 on, for the
// positions [p0, p0 + positions_per_block).
struct Tile {
  int t, h0, heads;
  long long p0;
};
template <int D> __device__ __forceinline__ Tile tile_of(long long i, const NormRopeArgs& a) {
  const int gq = (a.H[0] + HG - 1) / HG, gk = (a.H[1] + HG - 1) / HG;
  const int hg = static_cast<int>(i % (gq + gk));
  Tile w;
  w.p0 = (i / (gq + gk)) * positions_per_block<D>();
  w.t = hg < gq ? 0 : 1;
  w.h0 = (hg < gq ? hg : hg - gq) * HG;
  w.heads = min(HG, a.H[w.t] - w.h0);
  return w;
}

// The angles of row n of batch b.
__device__ __forceinline__ void angles(const NormRopeArgs& a, long long b, long long n, bool live, int s, const Lane& l,
                                       float (&c)[4], float (&sn)[4]) {
  const long long pos = a.positions && live ? a.positions[b * a.pos_stride + n] : n;
  const bool inside = pos >= 0 && pos < a.max_pos;
  if (l.turn && live && !inside) atomicOr(&g_status, kStatusBadBlock);
  load_angles(a.rope, pos, inside, a.rot, s, l.turn && live, c, sn);
}

template <class E, int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int L = D / 8;
  const int s = threadIdx.x % L;
  const Tile w = tile_of<D>(blockIdx.x, a);
  const long long p = w.p0 + threadIdx.x / L;
  const bool live = p < static_cast<long long>(a.B) * a.N;
  const Lane l = lane_of<D, INTER>(s, a.rot);
  const long long b = live ? p / a.N : 0, n = live ? p - b * a.N : 0;

  const long long* xs = a.x_stride[w.t];
  const long long x0 = b * xs[0] + w.h0 * xs[1] + n * xs[2];
  typename Raw<E>::type rlo[HG], rhi[HG];
#pragma unroll
  for (int h = 0; h < HG; ++h)
    if (live && h < w.heads) {
      rlo[h] = load4<E>(a.x[w.t], x0 + h * xs[1] + l.lo);
      rhi[h] = load4<E>(a.x[w.t], x0 + h * xs[1] + l.hi);
    } else {
      rlo[h] = rhi[h] = typename Raw<E>::type{};
    }
  float c[4], sn[4], wlo[4], whi[4];
  angles(a, b, n, live, s, l, c, sn);
  if (NORM) load_weight<E>(a.w[w.t], a.w_f32, l, wlo, whi);

  const long long* ys = a.y_stride[w.t];
  const long long y0 = b * ys[0] + w.h0 * ys[1] + n * ys[2];
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    float lo[4], hi[4];
    unpack4<E>(rlo[h], lo);
    unpack4<E>(rhi[h], hi);
    if (NORM) {
      const float r = 1.f / sqrtf(row_sum<L>(dot8(lo, hi, lo, hi)) * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] *= r * wlo[i];
        hi[i] *= r * whi[i];
      }
    }
    if (l.turn) rotate<INTER>(lo, hi, c, sn);
    if (live && h < w.heads) {
      store4<E>(a.y[w.t], y0 + h * ys[1] + l.lo, pack4<E>(lo));
      store4<E>(a.y[w.t], y0 + h * ys[1] + l.hi, pack4<E>(hi));
    }
  }
}

// Backward.  A persistent grid: each block walks tiles gridDim.x apart and keeps its
// share of dw in registers, so the weight gradients cost one partial row per block;
// sum_partials_kernel adds the blocks' rows in a fixed order (no atomics: the result
// does not depend on timing).
template <class E, int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(THREADS) norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, long long tiles) {
  constexpr int L = D / 8, P = positions_per_block<D>();
  const int s = threadIdx.x % L;
  const Lane l = lane_of<D, INTER>(s, a.rot);
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;

  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const Tile w = tile_of<D>(i, a);
    const long long p = w.p0 + threadIdx.x / L;
    const bool live = p < static_cast<long long>(a.B) * a.N;
    const long long b = live ? p / a.N : 0, n = live ? p - b * a.N : 0;
    const long long* xs = a.x_stride[w.t];
    const long long* gs = a.g_stride[w.t];
    const long long x0 = b * xs[0] + w.h0 * xs[1] + n * xs[2];
    const long long g0 = b * gs[0] + w.h0 * gs[1] + n * gs[2];
    typename Raw<E>::type xlo[HG], xhi[HG], glo[HG], ghi[HG];
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      xlo[h] = xhi[h] = glo[h] = ghi[h] = typename Raw<E>::type{};
      if (live && h < w.heads) {
        glo[h] = load4<E>(a.g[w.t], g0 + h * gs[1] + l.lo);
        ghi[h] = load4<E>(a.g[w.t], g0 + h * gs[1] + l.hi);
        if (NORM) {
          xlo[h] = load4<E>(a.x[w.t], x0 + h * xs[1] + l.lo);
          xhi[h] = load4<E>(a.x[w.t], x0 + h * xs[1] + l.hi);
        }
      }
    }
      float c[4], sn[4], wlo[4], whi[4];
    angles(a, b, n, live, s, l, c, sn);
#pragma unroll
    for (int e = 0; e < 4; ++e) sn[e] = -sn[e];
    if (NORM) load_weight<E>(a.w[w.t], a.w_f32, l, wlo, whi);

    const long long* ys = a.y_stride[w.t];
    const long long y0 = b * ys[0] + w.h0 * ys[1] + n * ys[2];
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      float lo[4], hi[4];
      unpack4<E>(glo[h], lo);
      unpack4<E>(ghi[h], hi);
      if (l.turn) rotate<INTER>(lo, hi, c, sn);
      if (NORM) {
        float x1[4], x2[4], u1[4], u2[4];
        unpack4<E>(xlo[h], x1);
        unpack4<E>(xhi[h], x2);
        const float r = 1.f / sqrtf(row_sum<L>(dot8(x1, x2, x1, x2)) * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x1[e] *= r;  // the normalised row
          x2[e] *= r;
          u1[e] = lo[e] * wlo[e];
          u2[e] = hi[e] * whi[e];
        }
        // A dead row or head adds nothing: its g is zero, its r finite or multiplied by zero.
        const bool count = live && h < w.heads;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d1 = count ? lo[e] * x1[e] : 0.f, d2 = count ? hi[e] * x2[e] : 0.f;
          if (w.t == 0) {
            dw[0][e] += d1;
            dw[0][4 + e] += d2;
          } else {
            dw[1][e] += d1;
            dw[1][4 + e] += d2;
          }
        }
        const float m = row_sum<L>(dot8(u1, u2, x1, x2)) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = r * (u1[e] - x1[e] * m);
          hi[e] = r * (u2[e] - x2[e] * m);
        }
      }
      if (live && h < w.heads) {
        store4<E>(a.y[w.t], y0 + h * ys[1] + l.lo, pack4<E>(lo));
        store4<E>(a.y[w.t], y0 + h * ys[1] + l.hi, pack4<E>(hi));
      }
    }
  }

  if (NORM && a.partials != nullptr) {
    __shared__ float sm[P][D];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t) __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sm[threadIdx.x / L][l.lo + e] = dw[t][e];
        sm[threadIdx.x / L][l.hi + e] = dw[t][4 + e];
      }
      __syncthreads();
      if (threadIdx.x < D) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) v += sm[i][threadIdx.x];
        a.partials[(static_cast<long long>(blockIdx.x) * 2 + t) * D + threadIdx.x] = v;
      }
    }
  }
}

// dw[t][e] = sum over the blocks of their partial rows: a block adds 32 columns, 32
// threads to a column, each over every 32nd block.
template <class E>
__global__ void __launch_bounds__(1024) sum_partials_kernel(const __grid_constant__ NormRopeArgs a, int blocks) {
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);  // over [2][d]
  const int part = threadIdx.x >> 5;
  float v = 0.f;
  for (int i = part; i < blocks; i += 32) v += a.partials[static_cast<long long>(i) * 2 * a.d + col];
  __shared__ float sm[32][33];
  sm[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sm[i][threadIdx.x];
    const int which = col / a.d, e = col % a.d;
    if (a.dw[which] != nullptr) {
      if (a.w_f32) {
        static_cast<float*>(a.dw[which])[e] = t;
      } else if constexpr (elem_bytes<E>() == 2) {
        static_cast<unsigned short*>(a.dw[which])[e] = to16<E>(t);
      }
    }
  }
}

template <class E, int D, bool INTER>
cudaError_t launch(const NormRopeArgs& a, bool backward, cudaStream_t stream) {
  const long long positions = static_cast<long long>(a.B) * a.N;
  const long long groups = (a.H[0] + HG - 1) / HG + (a.H[1] + HG - 1) / HG;
  const long long tiles = (positions + positions_per_block<D>() - 1) / positions_per_block<D>() * groups;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (!backward) {
    (a.norm ? norm_rope_kernel<E, D, INTER, true> : norm_rope_kernel<E, D, INTER, false>)
        <<<static_cast<unsigned>(tiles), THREADS, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const unsigned grid = static_cast<unsigned>(tiles < kNormRopeBlocks ? tiles : kNormRopeBlocks);
  (a.norm ? norm_rope_bwd_kernel<E, D, INTER, true> : norm_rope_bwd_kernel<E, D, INTER, false>)
      <<<grid, THREADS, 0, stream>>>(a, tiles);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.norm || a.partials == nullptr) return e;
  sum_partials_kernel<E><<<2 * D / 32, 1024, 0, stream>>>(a, static_cast<int>(grid));
  return cudaGetLastError();
}

template <class E>
cudaError_t launch_typed(const NormRopeArgs& a, bool backward, cudaStream_t stream) {
  if (a.d == 128) return a.interleaved ? launch<E, 128, true>(a, backward, stream) : launch<E, 128, false>(a, backward, stream);
  return a.interleaved ? launch<E, 64, true>(a, backward, stream) : launch<E, 64, false>(a, backward, stream);
}

}  // namespace nrope

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool backward, cudaStream_t stream) {
  if (a.f32) return nrope::launch_typed<rows::F32>(a, backward, stream);
  return a.f16 ? nrope::launch_typed<F16>(a, backward, stream) : nrope::launch_typed<Bf16>(a, backward, stream);
}

cudaError_t take_status_norm_rope(unsigned int* out) { return take_local_status(out); }

}  // namespace fa
