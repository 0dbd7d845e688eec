// The paged key-value cache: what its kernels share (internal header).
//
// A cache is k, v [n_pages][n_kv_heads][page_size][head_dim] (pages page_stride
// elements apart, the rest contiguous) in fp16 or bf16: the rows of one head in
// one page lie together, so a wave streams a head's keys as whole lines. Slot t
// of sequence b is row t % page_size of page page_table[b][t / page_size].
#pragma once

#include "common.h"

namespace gptq {

typedef __bf16 bf16_t;
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

// A cache and the sequences in it, as the kernels take them (by value).
struct KvView {
  void* k;
  void* v;
  const int32_t* table;  // [n_seqs][ld_table]
  const int32_t* lens;   // [n_seqs], new tokens counted
  int64_t page_stride;   // elements
  int64_t ld_table;
  int64_t n_pages;
  int32_t n_seqs, n_kv, dim, page_size, page_shift;
  int32_t max_pages;     // table entries a sequence may use
  int32_t bf16;          // 0: fp16

  // lens as the kernels use them: negative reads as 0, beyond the table as its end
  __device__ __forceinline__ int len(int b) const {
    const int n = lens[b], cap = max_pages << page_shift;
    return n < 0 ? 0 : n > cap ? cap : n;
  }
  // element offset of row 0 of head h in page p
  __device__ __forceinline__ int64_t head_base(int p, int h) const {
    return (int64_t)p * page_stride + (int64_t)h * page_size * dim;
  }
  __device__ __forceinline__ bool page_ok(int p) const { return p >= 0 && (int64_t)p < n_pages; }
};

template <typename T>
struct KvType;
template <>
struct KvType<half_t> {
  using x8 = half8;
  static __device__ __forceinline__ float4v mfma16(x8 a, x8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float16v mfma32(x8 a, x8 b, float16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct KvType<bf16_t> {
  using x8 = bf16x8;
  static __device__ __forceinline__ float4v mfma16(x8 a, x8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float16v mfma32(x8 a, x8 b, float16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// The sequence that new-token row i belongs to (cu [n_seqs + 1], ascending):
// the last b with cu[b] <= i, by bisection.
__device__ __forceinline__ int kv_seq_of(const int32_t* cu, int n_seqs, int i) {
  int lo = 0, hi = n_seqs;  // cu[lo] <= i < cu[hi] (i < cu[n_seqs] checked by the caller)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

constexpr float kLog2e = 1.4426950408889634f;

gptq_status_t kv_append_enqueue(const KvView& c, const void* k_new, int64_t ldk, const void* v_new, int64_t ldv,
                                const int32_t* cu, int64_t n_tokens, hipStream_t st);

struct KvAttnArgs {
  const void* q;
  int64_t ldq;  // elements between new tokens
  void* out;
  int64_t ldo;
  float* weights;  // [n_seqs][n_kv][ldw] or NULL
  int64_t ldw;
  float scale;
  int32_t n_heads, window, sinks;
};
size_t kv_token_workspace_bytes(const KvView& c, int64_t n_heads, int64_t window, int64_t sinks, bool weights);
gptq_status_t kv_token_enqueue(const KvView& c, const KvAttnArgs& a, void* ws, hipStream_t st);

// Partial results of rows whose slots are split over blocks: per (row, head, split) the
// running maximum (in powers of two) and the sum, and the unnormalized output.
struct SplitWs {
  float* ml;  // [rows * n_heads][n_splits][2]
  float* o;   // [rows * n_heads][n_splits][dim]
  int n_splits;
};
// Joins them into those of the n_rows rows of out that a sequence of the ragged batch cu has;
// lse [n_heads][n_rows] (optional): log2 of the sum of 2^score.
gptq_status_t kv_join_enqueue(const KvView& c, const KvAttnArgs& a, const SplitWs& w, int64_t n_rows,
                              const int32_t* cu, float* lse, hipStream_t st);

size_t kv_prompt_workspace_bytes(const KvView& c, int64_t n_tokens, int64_t n_heads, int64_t window, int64_t sinks,
                                 bool weights);
gptq_status_t kv_prompt_enqueue(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, void* ws,
                                hipStream_t st);

struct KvEvictArgs {
  const float* weights;
  int64_t ldw;
  int32_t budget, sinks, recent;
  const int32_t* dst;  // [n_seqs][ld_dst]
  int64_t ld_dst;
  int32_t* table_out;  // [n_seqs][ld_out]
  int64_t ld_out;
  int32_t* lens_out;
  float* weights_out;
  int64_t ldw_out;
  int32_t* kept;  // [n_seqs][n_kv][budget]
};
gptq_status_t kv_evict_enqueue(const KvView& c, const KvEvictArgs& a, hipStream_t st);

}  // namespace gptq
