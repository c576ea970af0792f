// Launch interface of the kernels around the paged cache: norm and rotation, append,
// chunk attention.  (kernels.h: the attention kernels'.)
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fa {

// Per-head norm and position rotation of q (index 0) and k (index 1), forward and
// backward.  Strides are in elements, (batch, head, row); d is contiguous.
struct NormRopeArgs {
  const void* x[2];             // inputs (k may be null with H[1] = 0)
  const void* g[2];             // backward: gradients of the outputs
  void* y[2];                   // outputs; backward: gradients of the inputs
  const void* w[2];             // weights [d], or null (ones)
  void* dw[2];                  // backward: gradients of the weights, or null
  long long x_stride[2][3], g_stride[2][3], y_stride[2][3];
  const float* rope;            // [max_pos][rot]: rot/2 cosines, rot/2 sines; null with rot = 0
  const int32_t* positions;     // row n of batch b: positions[b * pos_stride + n]; null: n
  long long pos_stride;
  int B, N, H[2], d, rot, max_pos;
  float eps;
  int norm, interleaved;
  int f16, f32, w_f32;
  float* partials;              // backward with dw: [kNormRopeBlocks][d]
};

// Blocks of the backward's persistent grid: 148 SMs x 5 resident blocks of 128 threads.
// A constant, so the order in which the weight gradients are summed is the same everywhere.
// Measured, 4K training shape (16K): 592 blocks 44.7 us (98.9), 740 41.0 (90.8), 1184 47.7 (104).
constexpr int kNormRopeBlocks = 740;

// New tokens' keys and values (and rotated queries) into a paged cache.
struct AppendArgs {
  const void* q;                // [T][Hq][d] at q_stride, or null
  const void* k;
  const void* v;
  void* q_out;                  // [T][Hq][d] contiguous
  void* kpool;
  void* vpool;
  const int32_t* block_table;
  const int32_t* cu_tokens;     // [B + 1], or null: one token per sequence
  const int32_t* seqlens;
  const void* q_weight;
  const void* k_weight;
  const float* rope;
  long long q_stride, k_stride, v_stride;
  int T, B, Hq, Hkv, num_blocks, block_shift, max_blocks, rot, max_pos;
  float eps;
  int norm, interleaved, f16, w_f32;
};

// Attention of packed new tokens over a paged cache.
struct ExtendArgs {
  const void* q;                // [T][Hq][d] at q_stride
  const void* kpool;
  const void* vpool;
  const int32_t* block_table;
  const int32_t* cu_tokens;     // [B + 1], or null: one token per sequence
  const int32_t* seqlens;
  void* o;                      // [T][Hq][d] contiguous
  float* lse;                   // [T][Hq], may be null
  long long q_stride;
  int T, B, Hq, Hkv, num_blocks, block_shift, max_blocks, cap;
  int causal, window;
  float scale, scale_log2;
  int f16;
  // Workspace: pieces of items that several CTAs share.
  struct ExtendDesc* desc;      // [kExtendMaxCtas]
  float* ws_lse;                // [2 kExtendMaxCtas][slot_rows]
  float* ws_o;                  // [2 kExtendMaxCtas][slot_rows][d]
  int slot_rows;
};
// The item that begins in a CTA and ends in CTA `last` (-1: none does).
struct ExtendDesc {
  int tok0, ntok, kvh, last;
};
constexpr int kExtendMaxCtas = 160;

// A 3-D TMA map over 16-bit elements with free strides (bytes; dims, box in elements,
// innermost first): boxes of box[0] = 64 columns (128 bytes, swizzled).
bool make_tmap_3d_half(void* map, const void* base, const long long dims[3], const long long strides[2],
                       const int box[3], int f16);

cudaError_t take_status_norm_rope(unsigned int* out);
cudaError_t take_status_append(unsigned int* out);
cudaError_t take_status_extend(unsigned int* out);
cudaError_t launch_norm_rope(const NormRopeArgs& a, bool backward, cudaStream_t stream);
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream);

}  // namespace fa
