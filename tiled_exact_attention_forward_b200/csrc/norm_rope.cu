// Per-head RMS norm and position rotation of queries and keys in one pass, and its
// backward pass.
//
// With x one head's row of d elements, at position p of its sequence:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  z = R(p) y,
// where R(p) turns the first `rot` elements pairwise by the table's angles.
// Backward, with dz given:
//   g = R(p)^T dz,  dw = sum over rows of g x r,  u = g w,
//   dx = r u - x r^3 mean(u x).
// r is recomputed from x (which the backward reads anyway) instead of being saved.
// All arithmetic is float32; each output is rounded once.
//
// Both passes are bound by memory: the forward reads x and writes z, the backward
// reads x and dz and writes dx, each byte once; the table's rows are shared by the
// heads of a position and come from L2.  Measured (bf16, B 2, 16 + 16 heads, 4096
// positions, d = 128): forward 23.9 us, 5.7 TB/s; backward 40.8 us, 4.9 TB/s, the sum of
// the weight gradients included; 32 + 8 heads, 16384 positions, float16: 54.2 us, 6.3 TB/s
// and 90 us, 5.7 TB/s.  What keeps the smaller shape from the copy rate (6.55) is the
// start and the end of a short kernel; the backward also has half the warps (94 registers
// a thread).  Input and output strides are free, so a
// projection's [B, N, H, d] output is read where it lies and written in the
// [B, H, N, d] order that the attention kernels take.
//
// Work split: a group of d / 8 lanes takes HG heads of one position, all its loads
// issued before the first is used; a block's groups take consecutive positions of
// the same heads, so its writes to [B, H, N, d] are runs of consecutive rows.
#include "cache_ops.h"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace fa {
namespace nrope {

using namespace rows;

// Measured on 8192 packed tokens of 32 + 32 heads (forward, bf16) and on both passes of
// the 4096-position shape above: 128 threads 48.5 and 64.4 us, 256 threads 53.9 and 68.5.
constexpr int THREADS = 128;
// Heads per group of lanes: 64 bytes a lane in flight per tensor read.  Fewer pay for the
// position's angles too often, more cost the backward its warps and short batches their
// blocks (16-bit types, as above: 2 heads 60.9 and 80.4 us, 4 heads 48.5 and 64.4, 8 heads
// 48.0 and 78.9; 300 tokens of 32 + 8 heads, forward: 4 heads 3.1, 8 heads 3.7).
template <class E> __host__ __device__ constexpr int heads_per_group() { return 8 / elem_bytes<E>(); }

template <int D> __host__ __device__ constexpr int positions_per_block() { return THREADS / (D / 8); }

// A lane's place: row n of batch b, from the row's number among all B * N.
struct Place {
  unsigned b, n;
};
__device__ __forceinline__ Place place_of(const NormRopeArgs& a, unsigned p) {
  const unsigned b = a.B == 1 ? 0u : p / static_cast<unsigned>(a.N);
  return Place{b, p - b * static_cast<unsigned>(a.N)};
}
template <bool INTER>
__device__ __forceinline__ Turn rotation_at(const NormRopeArgs& a, const Place& at, bool live, int s, bool turn) {
  const long long pos = a.positions && live ? a.positions[at.b * a.pos_stride + at.n] : at.n;
  const bool inside = pos >= 0 && pos < a.max_pos;
  if (turn && live && !inside) atomicOr(&g_status, kStatusBadBlock);
  return rotation<INTER>(a.rope, pos, inside, a.rot, s, turn && live);
}
template <class E>
__device__ __forceinline__ const char* row_at(const void* base, const long long (&stride)[3], const Place& at, int h) {
  return static_cast<const char*>(base) + (at.b * stride[0] + h * stride[1] + at.n * stride[2]) * elem_bytes<E>();
}

// blockIdx.x: the head groups of a run of positions come one after another.
template <class E, int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int L = D / 8, HG = heads_per_group<E>();
  const int s = threadIdx.x % L;
  const unsigned gq = (a.H[0] + HG - 1) / HG, groups = gq + (a.H[1] + HG - 1) / HG;
  const unsigned tile = blockIdx.x / groups, hg = blockIdx.x - tile * groups;
  const int t = hg < gq ? 0 : 1;
  const int h0 = (t ? hg - gq : hg) * HG, heads = min(HG, a.H[t] - h0);
  const unsigned p = tile * positions_per_block<D>() + threadIdx.x / L;
  const bool live = p < static_cast<unsigned>(a.B) * static_cast<unsigned>(a.N);
  const Place at = place_of(a, live ? p : 0u);
  const Lane l = lane_of<E, D, INTER>(s, a.rot);
  wait_for_previous_kernel();
  let_next_kernel_start();

  const char* x = row_at<E>(a.x[t], a.x_stride[t], at, h0);
  const long long xh = a.x_stride[t][1] * elem_bytes<E>();
  typename Raw<E>::type rlo[HG], rhi[HG];
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    rlo[h] = rhi[h] = typename Raw<E>::type{};
    if (live && h < heads) {
      rlo[h] = load4<E>(x + l.lo);
      rhi[h] = load4<E>(x + l.hi);
    }
    x += xh;
  }
  Turn turn = rotation_at<INTER>(a, at, live, s, l.turn);
  if (NORM) turn = weighted<INTER>(turn, load_weight<E, D, INTER>(a.w[t], a.w_f32, s, a.rot));

  char* y = const_cast<char*>(row_at<E>(a.y[t], a.y_stride[t], at, h0));
  const long long yh = a.y_stride[t][1] * elem_bytes<E>();
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    Oct v = unpack<E>(rlo[h], rhi[h]);
    if (NORM) {
      const uint64_t r = f2_both(rsqrt_row(row_sum<L>(dot(v, v)) * (1.f / D) + a.eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = f2_mul(v.p[i], r);
    }
    const Oct z = apply<INTER>(turn, l.turn, v);
    if (live && h < heads) {
      store4<E>(y + l.lo, pack<E>(z.p[0], z.p[1]));
      store4<E>(y + l.hi, pack<E>(z.p[2], z.p[3]));
    }
    y += yh;
  }
}

// Backward.  A persistent grid, the first `blocks_q` blocks for q, the rest for k: each
// block walks its tensor's tiles a grid's share apart and keeps its part of dw in
// registers, so the weight gradients cost one partial row per block, which
// sum_partials_kernel adds in a fixed order (no atomics: the result does not depend on
// timing).  (The next tile's rows copied to shared memory meanwhile, with asynchronous
// copies, measured 67.6 for 64.4 us.)
template <class E, int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(THREADS)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, unsigned tiles, unsigned blocks_q) {
  constexpr int L = D / 8, P = positions_per_block<D>(), HG = heads_per_group<E>();
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int s = threadIdx.x % L;
  const Lane l = lane_of<E, D, INTER>(s, a.rot);
  const int t = blockIdx.x < blocks_q ? 0 : 1;
  const unsigned first = t ? blockIdx.x - blocks_q : blockIdx.x, step = t ? gridDim.x - blocks_q : blocks_q;
  const unsigned groups = (a.H[t] + HG - 1) / HG;
  const long long xh = a.x_stride[t][1] * elem_bytes<E>(), gh = a.g_stride[t][1] * elem_bytes<E>(),
                  yh = a.y_stride[t][1] * elem_bytes<E>();
  Oct w;
  if (NORM) w = load_weight<E, D, INTER>(a.w[t], a.w_f32, s, a.rot);
  uint64_t dw[4] = {0, 0, 0, 0};

  for (unsigned i = first; i < tiles * groups; i += step) {
    const unsigned tile = i / groups;
    const int h0 = (i - tile * groups) * HG, heads = min(HG, a.H[t] - h0);
    const unsigned p = tile * P + threadIdx.x / L;
    const bool live = p < static_cast<unsigned>(a.B) * static_cast<unsigned>(a.N);
    const Place at = place_of(a, live ? p : 0u);
    const char* x = NORM ? row_at<E>(a.x[t], a.x_stride[t], at, h0) : nullptr;
    const char* g = row_at<E>(a.g[t], a.g_stride[t], at, h0);
    typename Raw<E>::type xlo[HG], xhi[HG], glo[HG], ghi[HG];
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      // A dead row or head reads as zeros and adds zeros to dw.
      xlo[h] = xhi[h] = glo[h] = ghi[h] = typename Raw<E>::type{};
      if (live && h < heads) {
        glo[h] = load4<E>(g + l.lo);
        ghi[h] = load4<E>(g + l.hi);
        if (NORM) {
          xlo[h] = load4<E>(x + l.lo);
          xhi[h] = load4<E>(x + l.hi);
        }
      }
      g += gh;
      if (NORM) x += xh;
    }
    const Turn back = transposed(rotation_at<INTER>(a, at, live, s, l.turn));

    char* y = const_cast<char*>(row_at<E>(a.y[t], a.y_stride[t], at, h0));
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      Oct v = apply<INTER>(back, l.turn, unpack<E>(glo[h], ghi[h]));  // g
      if (NORM) {
        const Oct xv = unpack<E>(xlo[h], xhi[h]);
        Oct gx;
#pragma unroll
        for (int e = 0; e < 4; ++e) gx.p[e] = f2_mul(v.p[e], xv.p[e]);
        const float ss = row_sum<L>(dot(xv, xv)), ux = row_sum<L>(dot(gx, w));
        // A dead row's r is 1 / sqrt(eps), infinite for eps = 0: kept out of dw.
        const float r = live && h < heads ? rsqrt_row(ss * (1.f / D) + a.eps) : 0.f;
        // (r ux) first: r^3 leaves float32's range where the product does not (|x| near 1e13 or,
        // with eps = 0, 1e-13).
        const uint64_t r2 = f2_both(r), c2 = f2_both(-(r * ux) * (1.f / D) * r * r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dw[e] = f2_fma(gx.p[e], r2, dw[e]);
          v.p[e] = f2_fma(xv.p[e], c2, f2_mul(v.p[e], f2_mul(w.p[e], r2)));
        }
      }
      if (live && h < heads) {
        store4<E>(y + l.lo, pack<E>(v.p[0], v.p[1]));
        store4<E>(y + l.hi, pack<E>(v.p[2], v.p[3]));
      }
      y += yh;
    }
  }

  if (NORM && a.partials != nullptr) {
    __shared__ alignas(16) float sm[P][D];  // written in 16-byte pieces
    const Lane e = lane_of<F32, D, INTER>(s, a.rot);
    char* row = reinterpret_cast<char*>(sm[threadIdx.x / L]);
    store4<F32>(row + e.lo, pack<F32>(dw[0], dw[1]));
    store4<F32>(row + e.hi, pack<F32>(dw[2], dw[3]));
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) v += sm[i][threadIdx.x];
      a.partials[blockIdx.x * D + threadIdx.x] = v;
    }
  }
}

// dw = the sum of the blocks' partial rows, q's blocks then k's: a block adds 32 columns
// of one of the two, 32 threads to a column, each over every 32nd block.
template <class E>
__global__ void __launch_bounds__(1024) sum_partials_kernel(const __grid_constant__ NormRopeArgs a, int blocks_q, int blocks) {
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5, t = blockIdx.y;
  wait_for_previous_kernel();
  if (a.dw[t] == nullptr) return;
  const int end = t ? blocks : blocks_q;
  float v = 0.f;
#pragma unroll 4
  for (int i = (t ? blocks_q : 0) + part; i < end; i += 32) v += a.partials[i * a.d + col];
  __shared__ float sm[32][33];
  sm[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sm[i][threadIdx.x];
    if (a.w_f32) {
      static_cast<float*>(a.dw[t])[col] = sum;
    } else if constexpr (elem_bytes<E>() == 2) {
      static_cast<unsigned short*>(a.dw[t])[col] = to16<E>(sum);
    }
  }
}

template <class E, int D, bool INTER>
cudaError_t launch(const NormRopeArgs& a, bool backward, cudaStream_t stream) {
  constexpr int HG = heads_per_group<E>();
  const long long positions = static_cast<long long>(a.B) * a.N;
  const long long tiles = (positions + positions_per_block<D>() - 1) / positions_per_block<D>();
  const long long gq = (a.H[0] + HG - 1) / HG, gk = (a.H[1] + HG - 1) / HG;
  if (positions > 0x7fffffffLL || tiles * (gq + gk) > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (!backward) {
    return launch_dependent(a.norm ? norm_rope_kernel<E, D, INTER, true> : norm_rope_kernel<E, D, INTER, false>,
                            dim3(static_cast<unsigned>(tiles * (gq + gk))), dim3(THREADS), 0, stream, a);
  }
  // Blocks in proportion to the tensors' tiles, at least one each.
  const long long all = tiles * (gq + gk) < kNormRopeBlocks ? tiles * (gq + gk) : kNormRopeBlocks;
  long long bk = gk == 0 ? 0 : (all * gk + gq + gk - 1) / (gq + gk);
  if (bk > all - 1) bk = all - 1;
  const unsigned blocks_q = static_cast<unsigned>(all - bk), blocks = static_cast<unsigned>(all);
  const cudaError_t e =
      launch_dependent(a.norm ? norm_rope_bwd_kernel<E, D, INTER, true> : norm_rope_bwd_kernel<E, D, INTER, false>,
                       dim3(blocks), dim3(THREADS), 0, stream, a, static_cast<unsigned>(tiles), blocks_q);
  if (e != cudaSuccess || !a.norm || a.partials == nullptr) return e;
  return launch_dependent(sum_partials_kernel<E>, dim3(D / 32, gk ? 2 : 1), dim3(1024), 0, stream, a,
                          static_cast<int>(blocks_q), static_cast<int>(blocks));
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
