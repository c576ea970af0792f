// The C ABI declared in include/fa.h: argument validation on the host, then
// one or more kernel launches on the caller's stream.  No device memory is
// allocated here; workspaces come from the caller.
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "cache_ops.h"
#include "common.cuh"
#include "kernels.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

float resolve_scale(float scale, int d) { return scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(d)); }

fa_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  if (e == cudaErrorInvalidValue) return FA_ERR_INVALID;
  return FA_ERR_CUDA;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool sizes_ok(long long B, long long H, long long N) {
  return B >= 1 && H >= 1 && N >= 1 && B * H <= (1LL << 31) / 2 && N <= (1LL << 30);
}

// (batch, head, row) strides against the sizes: multiples of 16 bytes, never
// negative, for outputs never zero where the dimension has more than one entry.
bool strides_ok(const int64_t* st, long long B, long long H, long long N, int elem, bool output) {
  const long long size[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (st[i] < 0 || st[i] > (1LL << 42) || st[i] * elem % 16 != 0 || (output && st[i] == 0)) return false;
  }
  return true;
}

// What the norm and the rotation share among their entry points.
bool rotation_ok(const float* rope, int d, int rot, int max_pos, float eps, int interleaved) {
  if (rot < 0 || rot > d || rot % 16 != 0 || (rot > 0) != (rope != nullptr) || !aligned(rope, 16)) return false;
  if (rot > 0 && max_pos < 1) return false;
  return eps == eps && eps <= 3.4e38f && (interleaved == 0 || interleaved == 1);
}

// Fills the arguments that forward and backward share; FA_OK when they are valid.
fa_status norm_rope_args(fa::NormRopeArgs& a, const void* q_weight, const void* k_weight, const float* rope,
                         const int32_t* positions, long long pos_stride, int B, int Hq, int Hk, int N, int d,
                         int rot, int max_pos, float eps, int interleaved, fa_dtype dtype, fa_dtype weight_dtype) {
  if (!sizes_ok(B, Hq, N) || (Hk != 0 && !sizes_ok(B, Hk, N)) || static_cast<long long>(B) * N > 0x7fffffffLL)
    return FA_ERR_INVALID;
  if (!rotation_ok(rope, d, rot, max_pos, eps, interleaved) || (eps < 0.f && rot == 0)) return FA_ERR_INVALID;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 4) || pos_stride < 0 ||
      pos_stride > (1LL << 42))
    return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16 && dtype != FA_FP32) || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  if (weight_dtype != dtype && weight_dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  a.w[0] = q_weight; a.w[1] = k_weight;
  a.rope = rope; a.positions = positions; a.pos_stride = pos_stride;
  a.B = B; a.N = N; a.H[0] = Hq; a.H[1] = Hk; a.d = d; a.rot = rot; a.max_pos = max_pos;
  a.norm = eps >= 0.f;
  a.eps = eps;
  a.interleaved = interleaved;
  a.f16 = dtype == FA_FP16; a.f32 = dtype == FA_FP32; a.w_f32 = weight_dtype == FA_FP32;
  return FA_OK;
}

int log2_of(int block_size) {
  int s = 0;
  while ((1 << s) < block_size) ++s;
  return s;
}

// The paged cache's geometry, as fa_decode_paged checks it.
bool paged_ok(int B, int H, int num_blocks, int block_size, int max_blocks) {
  if (num_blocks < 1 || max_blocks < 1 || block_size < 1 || block_size > 4096 || (block_size & (block_size - 1)) != 0)
    return false;
  return sizes_ok(B, H, static_cast<long long>(max_blocks) * block_size) &&
         static_cast<long long>(num_blocks) * H <= 0x7fffffffLL;
}

bool token_stride_ok(long long stride, long long row, int T) {
  return T == 1 || (stride >= row && stride % 8 == 0 && stride <= (1LL << 36));
}

// Rows of a workspace slot of the chunk attention: an item's query rows, two tiles of
// 128 rows at most.
int extend_slot_rows(int T, int G) { return T <= 128 / G ? T * G : 256; }

}  // namespace

extern "C" {

int fa_version(void) { return 104; }

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID: return "FA_ERR_INVALID: invalid argument";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED: no kernel for this dtype/head dimension";
    case FA_ERR_CUDA: return "FA_ERR_CUDA: CUDA launch or runtime error";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a kernel gave up waiting on an internal barrier";
  }
  return "unknown fa_status";
}

fa_status fa_forward(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                     int N, int d, float scale, int causal, int window, fa_dtype dtype, void* stream) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID;
  if (!sizes_ok(B, H, N) || window < 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID;
  fa::FwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.B = B; a.H = H; a.N = N; a.d = d;
  a.Nk = N; a.q_off = 0;
  a.causal = causal; a.window = window;
  a.scale = resolve_scale(scale, d);
  a.scale_log2 = a.scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == FA_BF16 || dtype == FA_FP16) {
    if (d != 128) return FA_ERR_UNSUPPORTED;
    a.f16 = dtype == FA_FP16;
    return from_cuda(fa::launch_fwd_tc(a, st));
  }
  if (dtype == FA_FP32) {
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    return from_cuda(fa::launch_fwd_f32(a, st));
  }
  return FA_ERR_UNSUPPORTED;
}

fa_status fa_forward_offset(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                            int H, int Nq, int Nk, int q_offset, int d, float scale, int causal,
                            int window, fa_dtype dtype, void* stream) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID;
  // Positions (row + q_offset, minus window, minus a key index) must stay inside int.
  constexpr int kLimit = 1 << 29;
  if (!sizes_ok(B, H, Nq) || Nk < 1 || Nq > kLimit || Nk > kLimit || q_offset > kLimit ||
      q_offset < -kLimit || window < 0 || window > kLimit || (causal != 0 && causal != 1))
    return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16) || d != 128) return FA_ERR_UNSUPPORTED;
  fa::FwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.B = B; a.H = H; a.N = Nq; a.d = d;
  a.Nk = Nk; a.q_off = q_offset;
  a.causal = causal; a.window = window;
  a.scale = resolve_scale(scale, d);
  a.scale_log2 = a.scale * kLog2e;
  a.f16 = dtype == FA_FP16;
  return from_cuda(fa::launch_fwd_tc(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_merge(const void* o_parts, const float* lse_parts, int S, void* o, float* lse, int B,
                   int H, int N, int d, fa_dtype dtype, void* stream) {
  if (!o_parts || !lse_parts || !o) return FA_ERR_INVALID;
  if (S < 1 || S > (1 << 16) || !sizes_ok(B, H, N)) return FA_ERR_INVALID;
  if (!aligned(o_parts, 16) || !aligned(o, 16) || !aligned(lse_parts, 4) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16 && dtype != FA_FP32) || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  fa::MergeArgs a{};
  a.o_parts = o_parts; a.lse_parts = lse_parts; a.o = o; a.lse = lse;
  a.rows = static_cast<long long>(B) * H * N;
  a.S = S; a.d = d;
  a.f16 = dtype == FA_FP16;
  a.f32 = dtype == FA_FP32;
  return from_cuda(fa::launch_merge(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_decode_workspace_size(int B, int H, int cap, int d) {
  if (B < 1 || H < 1 || cap < 1 || d < 1) return 0;
  const size_t chunks = static_cast<size_t>(fa::decode_max_chunks(cap));
  const size_t rows = static_cast<size_t>(B) * H * chunks;
  return round_up(rows * d * sizeof(float), 256) + round_up(rows * sizeof(float), 256);
}

fa_status fa_decode(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens,
                    void* o, float* lse, int B, int H, int cap, int d, float scale, fa_dtype dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !kcache || !vcache || !seqlens || !o || !workspace) return FA_ERR_INVALID;
  if (!sizes_ok(B, H, cap)) return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kcache, 16) || !aligned(vcache, 16) || !aligned(o, 16) ||
      !aligned(seqlens, 4) || !aligned(workspace, 256) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16) || d != 128) return FA_ERR_UNSUPPORTED;
  if (workspace_bytes < fa_decode_workspace_size(B, H, cap, d)) return FA_ERR_INVALID;
  fa::DecodeArgs a{};
  a.q = q; a.kcache = kcache; a.vcache = vcache; a.seqlens = seqlens; a.o = o; a.lse = lse;
  a.B = B; a.H = H; a.cap = cap; a.d = d;
  a.scale = resolve_scale(scale, d);
  a.scale_log2 = a.scale * kLog2e;
  a.max_chunks = fa::decode_max_chunks(cap);
  a.f16 = dtype == FA_FP16;
  const size_t rows = static_cast<size_t>(B) * H * a.max_chunks;
  a.ws_o = static_cast<float*>(workspace);
  a.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      round_up(rows * d * sizeof(float), 256));
  return from_cuda(fa::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_decode_paged(const void* q, const void* kpool, const void* vpool, const int32_t* block_table,
                          const int32_t* seqlens, void* o, float* lse, int B, int H, int num_blocks,
                          int block_size, int max_blocks, int d, float scale, fa_dtype dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!q || !kpool || !vpool || !block_table || !seqlens || !o || !workspace) return FA_ERR_INVALID;
  if (num_blocks < 1 || max_blocks < 1 || block_size < 1 || block_size > 4096 ||
      (block_size & (block_size - 1)) != 0)
    return FA_ERR_INVALID;
  const long long cap = static_cast<long long>(max_blocks) * block_size;
  if (!sizes_ok(B, H, cap)) return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kpool, 16) || !aligned(vpool, 16) || !aligned(o, 16) ||
      !aligned(block_table, 4) || !aligned(seqlens, 4) || !aligned(workspace, 256) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16) || d != 128) return FA_ERR_UNSUPPORTED;
  if (workspace_bytes < fa_decode_workspace_size(B, H, static_cast<int>(cap), d)) return FA_ERR_INVALID;
  fa::DecodeArgs a{};
  a.q = q; a.kcache = kpool; a.vcache = vpool; a.seqlens = seqlens; a.o = o; a.lse = lse;
  a.B = B; a.H = H; a.cap = static_cast<int>(cap); a.d = d;
  a.scale = resolve_scale(scale, d);
  a.scale_log2 = a.scale * kLog2e;
  a.max_chunks = fa::decode_max_chunks(a.cap);
  a.f16 = dtype == FA_FP16;
  const size_t rows = static_cast<size_t>(B) * H * a.max_chunks;
  a.ws_o = static_cast<float*>(workspace);
  a.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(rows * d * sizeof(float), 256));
  a.block_table = block_table;
  a.block_shift = 0;
  while ((1 << a.block_shift) < block_size) ++a.block_shift;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  return from_cuda(fa::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_backward_workspace_size(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || d < 1) return 0;
  const size_t rows = static_cast<size_t>(B) * H * N;
  return round_up(rows * sizeof(float), 256) + round_up(rows * d * sizeof(float), 256);
}

fa_status fa_backward(const void* q, const void* k, const void* v, const void* o, const void* dout,
                      const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                      float scale, int causal, int window, fa_dtype dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID;
  if (!sizes_ok(B, H, N) || window < 0 || (causal != 0 && causal != 1)) return FA_ERR_INVALID;
  const void* ptrs16[] = {q, k, v, o, dout, dq, dk, dv};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return FA_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(workspace, 256)) return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16) || d != 128) return FA_ERR_UNSUPPORTED;
  if (workspace_bytes < fa_backward_workspace_size(B, H, N, d)) return FA_ERR_INVALID;
  fa::BwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse;
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.B = B; a.H = H; a.N = N; a.d = d;
  a.causal = causal; a.window = window;
  a.scale = resolve_scale(scale, d);
  a.scale_log2 = a.scale * kLog2e;
  a.f16 = dtype == FA_FP16;
  const size_t rows = static_cast<size_t>(B) * H * N;
  a.ws_delta = static_cast<float*>(workspace);
  a.ws_dq = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(rows * sizeof(float), 256));
  return from_cuda(fa::launch_bwd(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const int64_t* strides,
                       const void* q_weight, const void* k_weight, const float* rope, const int32_t* positions,
                       long long pos_stride, int B, int Hq, int Hk, int N, int d, int rot, int max_pos, float eps,
                       int interleaved, fa_dtype dtype, fa_dtype weight_dtype, void* stream) {
  if (!q || !q_out || !strides || (k != nullptr) != (k_out != nullptr) || (k && Hk < 1)) return FA_ERR_INVALID;
  if (!k) Hk = 0;
  const void* ptrs[] = {q, k, q_out, k_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return FA_ERR_INVALID;
  fa::NormRopeArgs a{};
  const fa_status st = norm_rope_args(a, q_weight, k_weight, rope, positions, pos_stride, B, Hq, Hk, N, d, rot, max_pos,
                                      eps, interleaved, dtype, weight_dtype);
  if (st != FA_OK) return st;
  const int elem = dtype == FA_FP32 ? 4 : 2;
  for (int t = 0; t < (k ? 2 : 1); ++t) {
    if (!strides_ok(strides + 3 * t, B, a.H[t], N, elem, false) || !strides_ok(strides + 6 + 3 * t, B, a.H[t], N, elem, true))
      return FA_ERR_INVALID;
    for (int i = 0; i < 3; ++i) {
      a.x_stride[t][i] = strides[3 * t + i];
      a.y_stride[t][i] = strides[6 + 3 * t + i];
    }
  }
  a.x[0] = q; a.x[1] = k; a.y[0] = q_out; a.y[1] = k_out;
  return from_cuda(fa::launch_norm_rope(a, false, static_cast<cudaStream_t>(stream)));
}

size_t fa_norm_rope_backward_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return static_cast<size_t>(fa::kNormRopeBlocks) * d * sizeof(float);
}

fa_status fa_norm_rope_backward(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                const int64_t* strides, const void* q_weight, const void* k_weight, void* dq_weight,
                                void* dk_weight, const float* rope, const int32_t* positions, long long pos_stride, int B,
                                int Hq, int Hk, int N, int d, int rot, int max_pos, float eps, int interleaved,
                                fa_dtype dtype, fa_dtype weight_dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const bool has_k = dk_out != nullptr, norm = eps >= 0.f;
  if (!dq_out || !dq || !strides || has_k != (dk != nullptr) || (has_k && Hk < 1)) return FA_ERR_INVALID;
  if (norm && (!q || (has_k && !k))) return FA_ERR_INVALID;
  if ((dq_weight || dk_weight) && (!norm || !workspace)) return FA_ERR_INVALID;
  if (dk_weight && !has_k) return FA_ERR_INVALID;
  if (!has_k) Hk = 0;
  const void* ptrs[] = {q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return FA_ERR_INVALID;
  if (!aligned(workspace, 256)) return FA_ERR_INVALID;
  fa::NormRopeArgs a{};
  const fa_status st = norm_rope_args(a, q_weight, k_weight, rope, positions, pos_stride, B, Hq, Hk, N, d, rot, max_pos,
                                      eps, interleaved, dtype, weight_dtype);
  if (st != FA_OK) return st;
  if ((dq_weight || dk_weight) && workspace_bytes < fa_norm_rope_backward_workspace_size(d)) return FA_ERR_INVALID;
  const int elem = dtype == FA_FP32 ? 4 : 2;
  for (int t = 0; t < (has_k ? 2 : 1); ++t) {
    if ((norm && !strides_ok(strides + 3 * t, B, a.H[t], N, elem, false)) ||
        !strides_ok(strides + 6 + 3 * t, B, a.H[t], N, elem, false) ||
        !strides_ok(strides + 12 + 3 * t, B, a.H[t], N, elem, true))
      return FA_ERR_INVALID;
    for (int i = 0; i < 3; ++i) {
      a.x_stride[t][i] = strides[3 * t + i];
      a.g_stride[t][i] = strides[6 + 3 * t + i];
      a.y_stride[t][i] = strides[12 + 3 * t + i];
    }
  }
  a.x[0] = q; a.x[1] = k; a.g[0] = dq_out; a.g[1] = dk_out; a.y[0] = dq; a.y[1] = dk;
  a.dw[0] = dq_weight; a.dw[1] = dk_weight;
  a.partials = dq_weight || dk_weight ? static_cast<float*>(workspace) : nullptr;
  return from_cuda(fa::launch_norm_rope(a, true, static_cast<cudaStream_t>(stream)));
}

fa_status fa_append_paged(const void* k, const void* v, const void* q, void* q_out, void* kpool, void* vpool,
                          const int32_t* block_table, const int32_t* cu_tokens, const int32_t* seqlens,
                          long long q_stride, long long k_stride, long long v_stride, const void* q_weight,
                          const void* k_weight, const float* rope, int T, int B, int Hq, int Hkv, int num_blocks,
                          int block_size, int max_blocks, int d, int rot, int max_pos, float eps, int interleaved,
                          fa_dtype dtype, fa_dtype weight_dtype, void* stream) {
  if (!k || !v || !kpool || !vpool || !block_table || !seqlens || (q != nullptr) != (q_out != nullptr)) return FA_ERR_INVALID;
  if (!paged_ok(B, Hkv, num_blocks, block_size, max_blocks) || !sizes_ok(1, Hkv, T) || (q && !sizes_ok(1, Hq, T)))
    return FA_ERR_INVALID;
  if (cu_tokens == nullptr && T != B) return FA_ERR_INVALID;
  const void* ptrs[] = {k, v, q, q_out, kpool, vpool, q_weight, k_weight};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return FA_ERR_INVALID;
  if (!aligned(block_table, 4) || !aligned(cu_tokens, 4) || !aligned(seqlens, 4)) return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16) || d != 128) return FA_ERR_UNSUPPORTED;
  if (weight_dtype != dtype && weight_dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  if (!rotation_ok(rope, d, rot, max_pos, eps, interleaved)) return FA_ERR_INVALID;
  const long long row = static_cast<long long>(Hkv) * d;
  if (!token_stride_ok(k_stride, row, T) || !token_stride_ok(v_stride, row, T) ||
      (q && !token_stride_ok(q_stride, static_cast<long long>(Hq) * d, T)))
    return FA_ERR_INVALID;
  fa::AppendArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_out = q_out; a.kpool = kpool; a.vpool = vpool;
  a.block_table = block_table; a.cu_tokens = cu_tokens; a.seqlens = seqlens;
  a.q_weight = q_weight; a.k_weight = k_weight; a.rope = rope;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.T = T; a.B = B; a.Hq = Hq; a.Hkv = Hkv;
  a.num_blocks = num_blocks; a.block_shift = log2_of(block_size); a.max_blocks = max_blocks;
  a.rot = rot; a.max_pos = max_pos;
  a.norm = eps >= 0.f;
  a.eps = eps;
  a.interleaved = interleaved;
  a.f16 = dtype == FA_FP16; a.w_f32 = weight_dtype == FA_FP32;
  return from_cuda(fa::launch_append(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_extend_paged_workspace_size(int T, int Hq, int Hkv, int d) {
  if (T < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv != 0 || Hq / Hkv > 128) return 0;
  const size_t rows = 2 * static_cast<size_t>(fa::kExtendMaxCtas) * extend_slot_rows(T, Hq / Hkv);
  return round_up(fa::kExtendMaxCtas * sizeof(fa::ExtendDesc), 256) + round_up(rows * sizeof(float), 256) +
         round_up(rows * d * sizeof(float), 256);
}

fa_status fa_extend_paged(const void* q, const void* kpool, const void* vpool, const int32_t* block_table,
                          const int32_t* cu_tokens, const int32_t* seqlens, void* o, float* lse, long long q_stride,
                          int T, int B, int Hq, int Hkv, int num_blocks, int block_size, int max_blocks, int d,
                          float scale, int causal, int window, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (!q || !kpool || !vpool || !block_table || !seqlens || !o || !workspace) return FA_ERR_INVALID;
  constexpr int kLimit = 1 << 29;
  if (!paged_ok(B, Hkv, num_blocks, block_size, max_blocks) || !sizes_ok(1, Hq, T) || T > kLimit ||
      static_cast<long long>(max_blocks) * block_size > kLimit)
    return FA_ERR_INVALID;
  if (Hq % Hkv != 0 || Hq / Hkv > 128 || window < 0 || window > kLimit || (causal != 0 && causal != 1)) return FA_ERR_INVALID;
  if (cu_tokens == nullptr && T != B) return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(kpool, 16) || !aligned(vpool, 16) || !aligned(o, 16) || !aligned(block_table, 4) ||
      !aligned(cu_tokens, 4) || !aligned(seqlens, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
    return FA_ERR_INVALID;
  if ((dtype != FA_BF16 && dtype != FA_FP16) || d != 128) return FA_ERR_UNSUPPORTED;
  if (!token_stride_ok(q_stride, static_cast<long long>(Hq) * d, T)) return FA_ERR_INVALID;
  if (workspace_bytes < fa_extend_paged_workspace_size(T, Hq, Hkv, d)) return FA_ERR_INVALID;
  fa::ExtendArgs a{};
  a.q = q; a.kpool = kpool; a.vpool = vpool; a.block_table = block_table; a.cu_tokens = cu_tokens; a.seqlens = seqlens;
  a.o = o; a.lse = lse;
  a.q_stride = T == 1 ? static_cast<long long>(Hq) * d : q_stride;
  a.T = T; a.B = B; a.Hq = Hq; a.Hkv = Hkv;
  a.num_blocks = num_blocks; a.block_shift = log2_of(block_size); a.max_blocks = max_blocks;
  a.cap = max_blocks * block_size;
  a.causal = causal; a.window = window;
  a.scale = resolve_scale(scale, d);
  a.scale_log2 = a.scale * kLog2e;
  a.f16 = dtype == FA_FP16;
  a.slot_rows = extend_slot_rows(T, Hq / Hkv);
  const size_t rows = 2 * static_cast<size_t>(fa::kExtendMaxCtas) * a.slot_rows;
  char* ws = static_cast<char*>(workspace);
  a.desc = reinterpret_cast<fa::ExtendDesc*>(ws);
  ws += round_up(fa::kExtendMaxCtas * sizeof(fa::ExtendDesc), 256);
  a.ws_lse = reinterpret_cast<float*>(ws);
  a.ws_o = reinterpret_cast<float*>(ws + round_up(rows * sizeof(float), 256));
  return from_cuda(fa::launch_extend(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_selftest_wait_timeout(long long limit_cycles, void* stream) {
  if (limit_cycles < 1 || limit_cycles > 4000000000LL) return FA_ERR_INVALID;
  return from_cuda(fa::launch_selftest_wait_timeout(limit_cycles, static_cast<cudaStream_t>(stream)));
}

fa_status fa_selftest_exp2_poly(const float* x, float* y, long long n, void* stream) {
  if (!x || !y || n < 1 || !aligned(x, 4) || !aligned(y, 4)) return FA_ERR_INVALID;
  return from_cuda(fa::launch_selftest_exp2_poly(x, y, n, static_cast<cudaStream_t>(stream)));
}

fa_status fa_get_device_status(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return FA_ERR_CUDA;
  // Each source file's kernels record into a status word of their own; gather
  // (and clear) all of them.
  unsigned int word = 0;
  for (auto take : {fa::take_status_host, fa::take_status_fwd_tc, fa::take_status_bwd, fa::take_status_decode,
                    fa::take_status_norm_rope, fa::take_status_append, fa::take_status_extend}) {
    unsigned int w = 0;
    e = take(&w);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    word |= w;
  }
  if (word & fa::kStatusTimeout) return FA_ERR_TIMEOUT;
  if (word & fa::kStatusBadBlock) return FA_ERR_INVALID;
  return FA_OK;
}

}  // extern "C"
