// New tokens' keys and values into a paged cache, the keys (and, asked for, the
// queries) normalised and rotated on the way.
//
// Token t of the packed batch belongs to the sequence b with cu_tokens[b] <= t <
// cu_tokens[b + 1] and takes position p = seqlens[b] - cu_tokens[b + 1] + t, so the
// lengths count the new tokens already, as the decode and chunk attention calls
// want them.  Its keys go to row p % block_size of block block_table[b][p / block_size].
// The arithmetic per row is the norm-and-rotate kernel's (norm_rope.cu).
//
// Bound by memory for many tokens (each row read once and written once), by the
// chain cu_tokens -> seqlens -> block_table -> store for few: the rows' loads are
// issued ahead of that chain, and 16 lanes search cu_tokens together.  Measured: 16384
// tokens of 32 heads in 16-row blocks 83.6 us, 6.5 TB/s (99 % of the copy rate); 64
// single tokens with their queries 3.5 us (4.1 without the dependent launch), nearly all of it launch and that chain.
#include "cache_ops.h"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace fa {
namespace app {

using namespace rows;

constexpr int D = 128;
constexpr int L = D / 8;
constexpr int THREADS = 128;
constexpr int TOKENS = THREADS / L;  // tokens per block
constexpr int HG = 4;                // heads per group of lanes

// Number of i in [0, B) with cu[i + 1] <= t, for a non-decreasing cu: the lanes of the
// row probe 16 places at once.  Every answer lies in [0, B], whatever cu holds.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, long long t, int s) {
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  int lo = 0, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + L - 1) / L;
    const int i = lo + (s + 1) * step - 1;  // last place of this lane's run
    const bool below = i < hi && cu[i + 1] <= t;
    const int runs = __popc(__ballot_sync(mask, below));
    lo = min(hi, lo + runs * step);
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <class E, bool INTER, bool NORM>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendArgs a) {
  const int s = threadIdx.x % L;
  const int gq = a.q ? (a.Hq + HG - 1) / HG : 0, gk = (a.Hkv + HG - 1) / HG;
  const int hg = blockIdx.x % (gq + 2 * gk);
  const long long t = static_cast<long long>(blockIdx.x / (gq + 2 * gk)) * TOKENS + threadIdx.x / L;
  const bool live = t < a.T;
  const int kind = hg < gq ? 0 : hg < gq + gk ? 1 : 2;  // queries, keys, values
  const int h0 = (kind == 0 ? hg : kind == 1 ? hg - gq : hg - gq - gk) * HG;
  const int heads = min(HG, (kind == 0 ? a.Hq : a.Hkv) - h0);
  const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const long long stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
  const Lane l = lane_of<E, D, INTER>(s, a.rot);
  wait_for_previous_kernel();
  let_next_kernel_start();

  uint2 rlo[HG], rhi[HG];
  const char* x = static_cast<const char*>(src) + (t * stride + static_cast<long long>(h0) * D) * 2;
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    rlo[h] = rhi[h] = make_uint2(0u, 0u);
    if (live && h < heads) {
      rlo[h] = load4<E>(x + h * D * 2 + l.lo);
      rhi[h] = load4<E>(x + h * D * 2 + l.hi);
    }
  }
  Oct w;
  if (NORM && kind < 2) w = load_weight<E, D, INTER>(kind == 0 ? a.q_weight : a.k_weight, a.w_f32, s, a.rot);

  // The token's place.  A token past the last sequence has none and writes nothing.
  int b = 0;
  bool placed = false;
  long long pos = -1;
  if (live) {
    if (a.cu_tokens == nullptr) {
      b = static_cast<int>(t);
      placed = true;
      pos = static_cast<long long>(a.seqlens[b]) - 1;
    } else {
      b = sequence_of(a.cu_tokens, a.B, t, s);
      if (b < a.B && a.cu_tokens[b] <= t) {
        placed = true;
        pos = static_cast<long long>(a.seqlens[b]) - a.cu_tokens[b + 1] + t;
      }
    }
  }
  // Checked before anything is read or written through it: the position against the
  // table's rows and the cache's capacity, the block id against the pool.
  const long long cap = static_cast<long long>(a.max_blocks) << a.block_shift;
  bool good = placed && pos >= 0 && pos < cap && (a.rot == 0 || pos < a.max_pos);
  int phys = -1;
  if (good) {  // for queries too: a token has all of its rows or none
    phys = a.block_table[static_cast<long long>(b) * a.max_blocks + (pos >> a.block_shift)];
    good = phys >= 0 && phys < a.num_blocks;
  }
  if (placed && !good && s == 0) atomicOr(&g_status, kStatusBadBlock);

  void* dst = kind == 0 ? a.q_out : kind == 1 ? a.kpool : a.vpool;
  const long long row0 = kind == 0 ? t * a.Hq + h0
                                   : ((static_cast<long long>(phys) * a.Hkv + h0) << a.block_shift) +
                                         (pos & ((1 << a.block_shift) - 1));
  const long long next = (kind == 0 ? 1LL : 1LL << a.block_shift) * (D * 2);
  char* y = static_cast<char*>(dst) + row0 * (D * 2);
  // The query of a token without a place comes out NaN where it is rotated.
  const bool write = kind == 0 ? placed : good;
  Turn turn;
  if (kind < 2) {
    turn = rotation<INTER>(a.rope, pos, good, a.rot, s, l.turn && placed);
    if (NORM) turn = weighted<INTER>(turn, w);
  }
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    if (kind < 2) {
      Oct v = unpack<E>(rlo[h], rhi[h]);
      if (NORM) {
        const uint64_t r = f2_both(rsqrt_row(row_sum<L>(dot(v, v)) * (1.f / D) + a.eps));
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = f2_mul(v.p[i], r);
      }
      if (NORM || l.turn) {
        const Oct z = apply<INTER>(turn, l.turn, v);
        rlo[h] = pack<E>(z.p[0], z.p[1]);
        rhi[h] = pack<E>(z.p[2], z.p[3]);
      }
    }
    if (write && h < heads) {
      store4<E>(y + l.lo, rlo[h]);
      store4<E>(y + l.hi, rhi[h]);
    }
    y += next;
  }
}

template <class E>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  const long long groups = (a.q ? (a.Hq + HG - 1) / HG : 0) + 2LL * ((a.Hkv + HG - 1) / HG);
  const long long blocks = (static_cast<long long>(a.T) + TOKENS - 1) / TOKENS * groups;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kernel = a.interleaved ? (a.norm ? append_kernel<E, true, true> : append_kernel<E, true, false>)
                              : (a.norm ? append_kernel<E, false, true> : append_kernel<E, false, false>);
  return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, stream, a);
}

}  // namespace app

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  return a.f16 ? app::launch<F16>(a, stream) : app::launch<Bf16>(a, stream);
}

cudaError_t take_status_append(unsigned int* out) { return take_local_status(out); }

}  // namespace fa
