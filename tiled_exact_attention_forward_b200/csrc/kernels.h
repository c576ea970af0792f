// Internal launch interface between the C ABI (fa_api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fa {

struct FwdArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;  // may be null
  int B, H, N, d;     // N: query rows per head
  int causal, window;
  float scale;       // natural units
  float scale_log2;  // scale * log2(e)
  int f16;           // 16-bit inputs/outputs are f16 (else bf16)
  int Nk;            // key rows per head (N for self-attention)
  int q_off;         // position of query row 0 in the key sequence (0 for self-attention)
};

struct DecodeArgs {
  const void* q;
  const void* kcache;
  const void* vcache;
  const int32_t* seqlens;
  void* o;
  float* lse;  // may be null
  int B, H, cap, d;
  float scale, scale_log2;
  float* ws_o;    // [B*H][max_chunks][d] normalised chunk outputs
  float* ws_lse;  // [B*H][max_chunks] chunk logsumexp
  int max_chunks;
  // Paged cache (block_table != null): kcache/vcache are block pools
  // [num_blocks][H][1 << block_shift][d]; key j of sequence b sits in physical
  // block block_table[b * max_blocks + (j >> block_shift)].  cap = max_blocks << block_shift.
  const int32_t* block_table;
  int block_shift, max_blocks, num_blocks;
  int f16;  // q, caches and o are f16 (else bf16)
};

// Device status bit of a paged decode that met a block id outside [0, num_blocks)
// (the block is skipped, never read).
constexpr unsigned kStatusBadBlock = 2u;

struct BwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  int B, H, N, d;
  int causal, window;
  float scale, scale_log2;
  float* ws_delta;  // [B*H*N] rowsum(dO * O)
  float* ws_dq;     // [B*H*N*d] fp32 dQ accumulator
  int f16;          // 16-bit tensors are f16 (else bf16)
};

// Merge of partial results over disjoint key sets (context parallelism).
struct MergeArgs {
  const void* o_parts;     // [S][rows][d] 16-bit (or float32 with f32), each part normalised
  const float* lse_parts;  // [S][rows]; -inf marks a part that saw no key
  void* o;                 // [rows][d], the parts' type
  float* lse;              // [rows], may be null
  long long rows;          // B * H * N
  int S, d;
  int f16;
  int f32;                 // float32 parts and output
};

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

// Decode: keys per split chunk (one CTA each).
constexpr int kDecodeChunk = 512;

inline int decode_max_chunks(int cap) { return (cap + kDecodeChunk - 1) / kDecodeChunk; }

// Host helpers (fa_host.cu).
// A 3-D TMA map over a 16-bit (bf16, or f16 when f16 != 0) [heads][rows_per_head][d]
// array: boxes of 64 columns x box_rows rows, 128-byte swizzle, rows past the end
// read as zero.
bool make_tmap_half_rows(void* map, const void* base, int d, long long rows_per_head,
                         long long heads, int box_rows, int f16);
// The same over a float32 array, boxes of box_cols (32: 128 bytes) x box_rows.
bool make_tmap_f32_rows(void* map, const void* base, int d, long long rows_per_head,
                        long long heads, int box_cols, int box_rows);
// A 3-D TMA map over 16-bit elements with free strides (bytes; dims, box in elements,
// innermost first): boxes of box[0] = 64 columns (128 bytes, swizzled).
bool make_tmap_3d_half(void* map, const void* base, const long long dims[3], const long long strides[2],
                       const int box[3], int f16);
// Launches `kernel` as dependent on the kernel ahead of it in the stream: its launch
// overlaps that one's end (a few microseconds less between them).  The kernel has to call
// wait_for_previous_kernel() before it reads what that one writes.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per device and kernel.
cudaError_t set_max_dynamic_smem(const void* func, size_t bytes);
// Number of SMs of the current device (cached per device).
cudaError_t sm_count(int* out);

// Read and clear the device status word of each source file that has one.
cudaError_t take_status_host(unsigned int* out);
cudaError_t take_status_fwd_tc(unsigned int* out);
cudaError_t take_status_bwd(unsigned int* out);
cudaError_t take_status_decode(unsigned int* out);
cudaError_t take_status_norm_rope(unsigned int* out);
cudaError_t take_status_append(unsigned int* out);
cudaError_t take_status_extend(unsigned int* out);

cudaError_t launch_fwd_tc(const FwdArgs& a, cudaStream_t stream);
cudaError_t launch_fwd_f32(const FwdArgs& a, cudaStream_t stream);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_bwd(const BwdArgs& a, cudaStream_t stream);
cudaError_t launch_norm_rope(const NormRopeArgs& a, bool backward, cudaStream_t stream);
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream);
cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream);
cudaError_t launch_selftest_wait_timeout(long long limit_cycles, cudaStream_t stream);
cudaError_t launch_selftest_exp2_poly(const float* x, float* y, long long n, cudaStream_t stream);

}  // namespace fa
