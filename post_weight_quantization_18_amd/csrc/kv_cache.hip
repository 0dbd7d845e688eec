// What changes a paged key-value cache: new rows come in (append), and the rows
// with the smallest accumulated attention weight leave (evict). Both move bytes
// and compute next to nothing: they are bound by HBM, or by latency when small.
#include "kv.h"

namespace gptq {
namespace {

// Append. New token i of sequence b goes to slot lens[b] - n_b + (its index
// among the n_b new ones). One thread per 16 bytes of a token's key or value. A
// row of 256 chunks or more takes grid.y blocks, and its place is found with scalar
// reads; smaller rows are PACKED, `tokens` of them in a block (32000 tokens of one head of
// 64: 6 us packed, 13 with a block each; 1024 tokens of 96 heads of 128: 22 us with reads by
// lane, 17 scalar). Slots or pages outside the table or the cache are skipped.
// Bound by HBM: four prompts of 700 to 2048 tokens, 96 heads of 128 (540 MB) take 96
// us, 5.6 TB/s. One token of each of 16 sequences takes 3 us, three reads that wait for
// one another.
template <bool PACKED>
__global__ __launch_bounds__(256) void append_kernel(KvView c, const uint4v* k_new, int64_t ldk, const uint4v* v_new,
                                                     int64_t ldv, const int32_t* cu, int n_tokens, int tokens) {
  const int per_head = c.dim >> 3, half = c.n_kv * per_head;
  const int in_block = PACKED ? (int)threadIdx.x / (2 * half) : 0;
  const int ch = blockIdx.y * 256 + threadIdx.x - in_block * 2 * half;
  const int i = PACKED ? blockIdx.x * tokens + in_block : blockIdx.x;
  if (ch >= 2 * half || (PACKED && (in_block >= tokens || i >= n_tokens))) return;
  const bool is_v = ch >= half;
  const int rc = is_v ? ch - half : ch;
  const int h = rc / per_head, off = (rc - h * per_head) * 8;
  const uint4v* src = is_v ? v_new : k_new;
  bf16_t* dst = (bf16_t*)(is_v ? c.v : c.k);  // 16-bit elements of either type
  const int cap = c.max_pages << c.page_shift;
  // without branches from here, so that what does not wait for another load is under way together
  const int first = cu ? cu[0] : 0, last = cu ? cu[c.n_seqs] : n_tokens;
  const uint4v x = src[(int64_t)i * ((is_v ? ldv : ldk) >> 3) + rc];
  const bool in = i >= first && i < last;
  const int b = !in ? 0 : cu ? kv_seq_of(cu, c.n_seqs, i) : i;
  int64_t slot = (int64_t)c.lens[b] - (cu ? cu[b + 1] - (int64_t)i : 1);
  if (!in || slot < 0 || slot >= cap) slot = -1;
  const int page = c.table[(int64_t)b * c.ld_table + ((slot < 0 ? 0 : slot) >> c.page_shift)];
  GPTQ_DASSERT(b < c.n_seqs && slot < cap);
  if (slot >= 0 && c.page_ok(page))
    *(uint4v*)(dst + c.head_base(page, h) + (slot & (c.page_size - 1)) * c.dim + off) = x;
}

// Order-preserving key of a sum: larger weight, larger key; a NaN above all, and
// -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64, kBins = 2048;

// x[0] + .. + x[wave - 1] (16 waves), by every lane.
__device__ __forceinline__ uint32_t sum_before(const uint32_t* x, int wave) {
  const int l = threadIdx.x & 15;
  uint32_t v = l < wave ? x[l] : 0u;
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Select: for one sequence and head, the slots that stay, in order. With
// n > budget slots, the first `sinks` and the last `recent` stay, and of those
// between the need = budget - sinks - recent with the largest weights, ties to
// the lower slot. The need-th largest key is found digit by digit (11, 11 and
// 10 bits) from a histogram in LDS; then each wave counts its contiguous part of
// the slots, the waves' counts are summed, and each writes its survivors. Bound by
// latency (five passes over a row that stays in the cache, with barriers): 320 rows of 1500
// to 2048 slots take 11 us, 8 rows of 1333 take 8; keys kept in registers between the passes
// measured the same.
__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(KvView c, KvEvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wave_sum[kSelWaves], wave_eq[kSelWaves];
  __shared__ uint32_t found_digit, found_left;
  const int b = blockIdx.x / c.n_kv, h = blockIdx.x - b * c.n_kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = c.len(b);
  int32_t* kept = a.kept + ((int64_t)b * c.n_kv + h) * a.budget;
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const float* w = a.weights + ((int64_t)b * c.n_kv + h) * a.ldw;
  const int lo = a.sinks, hi = n - a.recent;  // the slots that compete
  const uint32_t need = a.budget - a.sinks - a.recent;
  uint32_t prefix = 0, mask = 0, left = need;
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t key = weight_key(w[t]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // bins from the largest: thread i holds bins 2047 - 2 i and 2046 - 2 i
      const uint32_t h0 = hist[kBins - 1 - 2 * tid], h1 = hist[kBins - 2 - 2 * tid];
      uint32_t incl = h0 + h1;
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(incl, o);
        if (lane >= o) incl += u;
      }
      if (lane == 63) wave_sum[wave] = incl;
      __syncthreads();
      const uint32_t before = incl - h0 - h1 + sum_before(wave_sum, wave);
      if (before < left && before + h0 >= left) {
        found_digit = kBins - 1 - 2 * tid;
        found_left = left - before;
      } else if (before + h0 < left && before + h0 + h1 >= left) {
        found_digit = kBins - 2 - 2 * tid;
        found_left = left - before - h0;
      }
      __syncthreads();
      prefix |= found_digit << shift;
      mask |= ((1u << bits) - 1) << shift;
      left = found_left;
    }
  }
  // slots with key > prefix stay, and the first `left` with key == prefix
  const int per_wave = ((n + 63) / 64 + kSelWaves - 1) / kSelWaves * 64;
  const int t0 = wave * per_wave, t1 = t0 + per_wave < n ? t0 + per_wave : n;
  uint32_t sure = 0, equal = 0;
  for (int r = t0; r < t1; r += 64) {
    const int t = r + lane;
    bool s = false, e = false;
    if (t < t1) {
      s = t < lo || t >= hi;
      if (!s && need > 0) {
        const uint32_t key = weight_key(w[t]);
        s = key > prefix;
        e = key == prefix;
      }
    }
    sure += __popcll(__ballot(s));
    equal += __popcll(__ballot(e));
  }
  __syncthreads();  // wave_sum of the last pass has been read
  if (lane == 0) {
    wave_sum[wave] = sure;
    wave_eq[wave] = equal;
  }
  __syncthreads();
  const uint32_t sure_before = sum_before(wave_sum, wave);
  uint32_t eq_before = sum_before(wave_eq, wave);
  uint32_t base = sure_before + (eq_before < left ? eq_before : left);
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  for (int r = t0; r < t1; r += 64) {
    const int t = r + lane;
    bool s = false, e = false;
    if (t < t1) {
      s = t < lo || t >= hi;
      if (!s && need > 0) {
        const uint32_t key = weight_key(w[t]);
        s = key > prefix;
        e = key == prefix;
      }
    }
    const uint64_t em = __ballot(e);
    if (e && eq_before + __popcll(em & below) < left) s = true;
    eq_before += __popcll(em);
    const uint64_t sm = __ballot(s);
    const uint32_t at = base + __popcll(sm & below);
    if (s && at < (uint32_t)a.budget) kept[at] = t;
    base += __popcll(sm);
  }
}

// Move: the survivors' rows to the new pages, their sums to weights_out (zero
// behind them), the table's row and the length. 16 lanes per row of up to 256
// bytes, key and value together, kMoveRows rows per block. Source and destination
// pages are distinct, so every row moves on its own. Bound by HBM: half of eight
// caches of 1500 to 2048 slots of 40 heads of 128 (336 MB) take 65 us (5.2 TB/s; a
// plain copy reaches 4.9) with 32 rows a block and stores past the caches; 73 with
// ordinary stores, 85 with 64 rows a block.
constexpr int kMoveRows = 32;

__global__ __launch_bounds__(256) void evict_move_kernel(KvView c, KvEvictArgs a, int n_blk) {
  const int blk = blockIdx.x % n_blk, bh = blockIdx.x / n_blk;
  const int b = bh / c.n_kv, h = bh - b * c.n_kv;
  const int tid = threadIdx.x;
  const int n = c.len(b);
  const bool over = n > a.budget;
  const int cap = c.max_pages << c.page_shift, left = over ? a.budget : n;
  const int32_t* kept = a.kept + ((int64_t)b * c.n_kv + h) * a.budget;
  const int32_t* row = c.table + (int64_t)b * c.ld_table;
  const int32_t* dst = a.dst + (int64_t)b * a.ld_dst;
  const int r0 = blk * kMoveRows;
  if (tid < kMoveRows && r0 + tid < cap) {
    const int i = r0 + tid;
    float s = 0.0f;
    if (i < left) s = a.weights[((int64_t)b * c.n_kv + h) * a.ldw + (over ? kept[i] : i)];
    a.weights_out[((int64_t)b * c.n_kv + h) * a.ldw_out + i] = s;
  }
  if (blk == 0 && h == 0) {
    const int nd = (a.budget + c.page_size - 1) >> c.page_shift;
    for (int p = tid; p < c.max_pages; p += 256)
      a.table_out[(int64_t)b * a.ld_out + p] = !over ? row[p] : p < nd ? dst[p] : -1;
    if (tid == 0) a.lens_out[b] = left;
  }
  if (!over || r0 >= a.budget) return;
  const int ch = tid & 15;
  if (ch * 8 >= c.dim) return;
  // stage by stage over the thread's rows, without branches between: each stage's loads (the
  // slot, its page, the row) are under way together (rows past the last repeat it, and a page
  // that is none is read as page 0; neither is stored)
  constexpr int U = kMoveRows / 16;
  int t[U], ps[U], pd[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = r0 + u * 16 + (tid >> 4), j = i < a.budget ? i : a.budget - 1;
    t[u] = kept[j];
    pd[u] = i < a.budget ? dst[j >> c.page_shift] : -1;
    GPTQ_DASSERT(t[u] >= 0 && t[u] < n);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) ps[u] = row[t[u] >> c.page_shift];
  uint4v xk[U], xv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t from =
        c.head_base(c.page_ok(ps[u]) ? ps[u] : 0, h) + (int64_t)(t[u] & (c.page_size - 1)) * c.dim + ch * 8;
    xk[u] = *(const uint4v*)((const bf16_t*)c.k + from);
    xv[u] = *(const uint4v*)((const bf16_t*)c.v + from);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!c.page_ok(ps[u]) || !c.page_ok(pd[u])) continue;
    const int i = r0 + u * 16 + (tid >> 4);
    const int64_t to = c.head_base(pd[u], h) + (int64_t)(i & (c.page_size - 1)) * c.dim + ch * 8;
    // past the caches: what is moved is more than they hold, and the reads behind want the room
    __builtin_nontemporal_store(xk[u], (uint4v*)((bf16_t*)c.k + to));
    __builtin_nontemporal_store(xv[u], (uint4v*)((bf16_t*)c.v + to));
  }
}

}  // namespace

gptq_status_t kv_append_enqueue(const KvView& c, const void* k_new, int64_t ldk, const void* v_new, int64_t ldv,
                                const int32_t* cu, int64_t n_tokens, hipStream_t st) {
  const int64_t row = 2 * (int64_t)c.n_kv * (c.dim >> 3), tokens = 256 / row;
  TraceScope tr(st, GPTQ_TRACE_KV_APPEND);
  if (tokens > 1)
    hipLaunchKernelGGL(append_kernel<true>, dim3((unsigned)ceil_div(n_tokens, tokens)), dim3(256), 0, st, c,
                       (const uint4v*)k_new, ldk, (const uint4v*)v_new, ldv, cu, (int)n_tokens, (int)tokens);
  else
    hipLaunchKernelGGL(append_kernel<false>, dim3((unsigned)n_tokens, (unsigned)ceil_div(row, 256)), dim3(256), 0, st,
                       c, (const uint4v*)k_new, ldk, (const uint4v*)v_new, ldv, cu, (int)n_tokens, 1);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status_t kv_evict_enqueue(const KvView& c, const KvEvictArgs& a, hipStream_t st) {
  const int64_t cap = (int64_t)c.max_pages << c.page_shift;
  // a budget beyond the capacity moves nothing: the blocks cover the capacity's sums
  const int64_t n_blk = ceil_div(cap, kMoveRows), blocks = n_blk * c.n_kv * c.n_seqs;
  if (blocks * 256 >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  TraceScope tr(st, GPTQ_TRACE_KV_EVICT);
  hipLaunchKernelGGL(evict_select_kernel, dim3((unsigned)(c.n_kv * c.n_seqs)), dim3(kSelThreads), 0, st, c, a);
  GPTQ_CHECK_LAUNCH();
  hipLaunchKernelGGL(evict_move_kernel, dim3((unsigned)blocks), dim3(256), 0, st, c, a, (int)n_blk);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace gptq
