// Attention of one new token per sequence over the paged cache:
//   s_t = scale q . k_t over the visible slots t, w = softmax(s), out = sum_t w_t v_t
// and, if asked for, weights[t] += w_t summed over the heads that share a key.
//
// Every visible key and value is read once; with G heads to a key there are 2 G
// flops per element read, so it is bound by HBM. The matrix cores take the
// products all the same, because they cost less issue than vector code even
// with one head to a key (15 of 16 columns idle): a wave's 32 slots x 128 are
// 16 matrix instructions, 256 cycles for 16 KB, against a share of about 4 bytes
// per cycle and SIMD of HBM bandwidth.
//
// One pass with a running maximum and sum. A wave takes 32 slots at a time, as
// S^T = K Q^T (two 16 x 16 tiles) and O^T = V^T P^T, all in registers:
//  - lane l = 16 g + c. K rows are assigned to the rows m of tile a as slot
//    8 (m / 4) + 4 a + m % 4, so the scores a lane ends up with (rows 4 g + r)
//    are slots 8 g .. 8 g + 7 of head c: exactly the P^T operand it must hold.
//  - V rows 8 g .. 8 g + 7 are read along the row (elements c VEC ...), and an
//    8 x VEC block is turned over inside each lane (32 byte permutes for 64
//    elements), so no shared memory and no lane exchange lies in the loop.
//  - the next 32 slots are loaded while the current ones are computed, and the
//    page numbers one step further ahead.
// The maximum is only raised when a score passes it by 2^8 (then every lane of
// the wave rescales): weights stay below 2^8, well inside fp16, and the usual
// step needs no exchange between lanes.
//
// The slots are split over the waves of a block and over n_splits blocks; a
// block's waves are joined through LDS, the blocks by a second kernel (which also
// turns the stored scores into weights).
//
// 32 sequences of 37 to 2048 slots, 96 heads, with weights (1.67 GB): 295 us, 5.7 TB/s;
// three of 9001 to 32768 slots, 64 heads on 8, bf16 (257 MB): 57 us, 4.5 TB/s with the join;
// 700 slots of 32 heads of 80: 9.7 us, latency.
#include <algorithm>

#include "kv.h"

namespace gptq {
namespace {

constexpr int kTile = 32;     // slots per wave and step
constexpr int NW = 4;         // waves per block: 8 stream no faster (a compute unit's misses are the limit)
constexpr float kRaise = 8.0f;  // in powers of two

// The slots a token sees, as steps of kTile slots: the steps that hold sinks, then
// those from the window's first slot on.
struct Steps {
  int n, first, sink_steps, total;  // slots, first slot of the window, steps before the gap, steps
  int jump;                         // step number of the first step after the gap
  __device__ __forceinline__ Steps(int len, int window, int sinks) {
    n = len;
    first = window > 0 && window < len ? len - window : 0;
    const int all = (len + kTile - 1) / kTile;
    const int sk = first > 0 ? (sinks < first ? sinks : first) : 0;
    sink_steps = (sk + kTile - 1) / kTile;
    jump = first / kTile;
    if (jump < sink_steps) jump = sink_steps;
    total = sink_steps + all - jump;
  }
  __device__ __forceinline__ int slot0(int s) const { return (s < sink_steps ? s : s - sink_steps + jump) * kTile; }
};

// The i-th longest sequence (equal lengths in order), of up to 64; i itself of more. Blocks
// start in order, and with the long sequences first the last ones to end are short.
__device__ __forceinline__ int longest(const KvView& c, int i) {
  if (c.n_seqs == 1 || c.n_seqs > 64) return i;
  const int lane = threadIdx.x & 63;
  const int n = lane < c.n_seqs ? c.len(lane) : -1;
  int rank = 0;
  for (int j = 0; j < c.n_seqs; ++j) {
    const int m = __builtin_amdgcn_readlane(n, j);
    rank += m > n || (m == n && j < lane);
  }
  return __builtin_ctzll(__ballot(rank == i && lane < c.n_seqs));
}

// The workspace: the splits' partial results (rows are sequences), then the scores by step.
struct TokenWs {
  SplitWs parts;
  float* scores;  // [n_seqs * n_heads][n_scores]
  int n_scores;
  bool join;  // a second kernel
  bool lds;   // scores in LDS
};

// weights += 2^(score - m) / l, summed over the heads of a group, for the steps [s0,
// s1) of one sequence and key head; sh holds m and 1 / l of each head. U slots per
// thread at a time: fetch() starts the reads of the first lot's old weights (they take
// longest) and add() does the work.
template <int U, bool LDS = false>
struct AddWeights {
  const KvView& c;
  const KvAttnArgs& a;
  const TokenWs& w;
  const Steps& st;
  const float* sp;
  const GPTQ_LDS float* lds = nullptr;
  float* wt;
  int k0, end, threads, group;
  float old[U];
  int t[U];
  __device__ __forceinline__ AddWeights(const KvView& c, const KvAttnArgs& a, const TokenWs& w, const Steps& st, int b,
                                        int kvh, int s0, int s1, int threads)
      : c(c), a(a), w(w), st(st), threads(threads), group(a.n_heads / c.n_kv) {
    sp = w.scores + ((int64_t)b * a.n_heads + kvh * group) * w.n_scores;
    wt = a.weights + ((int64_t)b * c.n_kv + kvh) * a.ldw;
    k0 = s0 * kTile + threadIdx.x;
    end = (s1 < st.total ? s1 : st.total) * kTile;
  }
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = k0 + threads * i;
      t[i] = -1;
      if (k < end) {
        const int slot = st.slot0(k / kTile) + k % kTile;
        if (slot < st.n && (slot >= st.first || slot < a.sinks)) t[i] = slot;
      }
      old[i] = wt[t[i] < 0 ? 0 : t[i]];
    }
  }
  __device__ __forceinline__ void add(const float* sh) {
    while (true) {
      float sum[U];
#pragma unroll
      for (int i = 0; i < U; ++i) sum[i] = 0.0f;
      for (int h = 0; h < group; ++h) {
        float x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = t[i] < 0 ? 0 : k0 + threads * i;
          if constexpr (LDS)
            x[i] = lds[h * w.n_scores + k];
          else
            x[i] = sp[(int64_t)h * w.n_scores + k];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) sum[i] += __builtin_amdgcn_exp2f(x[i] - sh[2 * h]) * sh[2 * h + 1];
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (t[i] >= 0) wt[t[i]] = old[i] + sum[i];
      k0 += U * threads;
      if (k0 - (int)threadIdx.x >= end) return;
      fetch();
    }
  }
};

template <typename T, int KS, int VEC>
struct TokenRegs {
  typename KvType<T>::x8 k[2][KS];
  uint32_t v[8][VEC / 2];
};

// Where the scores of a call with weights are kept until the normalizer is known: in LDS
// where one block holds all of a key head's scores and they fit (no write travels with the
// cache's reads: 297 us instead of 316 for 32 sequences of up to 2048 slots and 96 heads), else
// in the workspace.
constexpr int kScoresGlobal = 1, kScoresLds = 2;
constexpr size_t kScoresLdsBytes = 32 << 10;

// KS: steps of 32 along the head for the scores; VEC: output elements per lane
// (16 VEC >= dim). SPLIT: partial results to the workspace. SCORES: they
// are kept too.
template <typename T, int KS, int VEC, bool SPLIT, int SCORES>
__global__ __launch_bounds__(64 * NW, 2) void token_kernel(KvView c, KvAttnArgs a, TokenWs w) {
  using KT = KvType<T>;
  using x8 = typename KT::x8;
  const int lane = threadIdx.x & 63, g = lane >> 4, cl = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int group = a.n_heads / c.n_kv, qt = (group + 15) / 16;  // heads in tiles of 16
  int id = blockIdx.x;
  const int split = id % w.parts.n_splits;
  id /= w.parts.n_splits;
  const int h0 = (id % qt) * 16;
  id /= qt;
  const int kvh = id % c.n_kv, b = longest(c, id / c.n_kv);
  const int n_h = group - h0 < 16 ? group - h0 : 16;
  const int head = kvh * group + h0 + (cl < n_h ? cl : 0);  // this lane's column
  constexpr int kPitch = 16 * VEC + 4;
  extern __shared__ __attribute__((aligned(16))) float so[];  // [NW][n_h][kPitch], then scores [n_h][n_scores]
  GPTQ_LDS float* lds_scores = (GPTQ_LDS float*)so + NW * n_h * kPitch;

  const Steps st(c.len(b), a.window, a.sinks);
  const int per = (st.total + w.parts.n_splits - 1) / w.parts.n_splits;
  const int s_end = (split + 1) * per < st.total ? (split + 1) * per : st.total;
  const int32_t* table = c.table + (int64_t)b * c.ld_table;
  const int chunks = c.dim >> 3;

  x8 q[KS];
  const T* qp = (const T*)a.q + (int64_t)b * a.ldq + (int64_t)head * c.dim;
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const bool ok = 4 * i + g < chunks && cl < n_h;
    x8 z = *(const x8*)(qp + 8 * (4 * i + g < chunks ? 4 * i + g : 0));
#pragma unroll
    for (int e = 0; e < 8; ++e) q[i][e] = ok ? z[e] : (T)0.0f;
  }
  const float sc = a.scale * kLog2e;

  float4v o[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = (float4v){0, 0, 0, 0};
  float m = -INFINITY, lsum = 0.0f;  // of this lane's column; lsum over this lane's own slots

  // page of the octet of 8 slots whose keys (o_k) or values (o_v) this lane loads, -1 if none
  struct Pages {
    int k, v;
  };
  auto pages = [&](int s) __attribute__((always_inline)) {
    Pages p = {-1, -1};
    if (s < s_end) {
      const int t0 = st.slot0(s), tk = t0 + 8 * (cl >> 2), tv = t0 + 8 * g;
      if (tk < st.n) p.k = table[tk >> c.page_shift];
      if (tv < st.n) p.v = table[tv >> c.page_shift];
    }
    return p;
  };
  using Regs = TokenRegs<T, KS, VEC>;
  const T* kbase = (const T*)c.k + (int64_t)kvh * c.page_size * c.dim;
  const T* vbase = (const T*)c.v + (int64_t)kvh * c.page_size * c.dim;
  const int vch = cl * VEC < c.dim ? cl * VEC : 0;
  auto load = [&](int s, Pages p, Regs& r) __attribute__((always_inline)) {
    const int t0 = st.slot0(s);
    const int pk = c.page_ok(p.k) ? p.k : 0, pv = c.page_ok(p.v) ? p.v : 0;
    const int rk = (t0 + 8 * (cl >> 2) + (cl & 3)) & (c.page_size - 1), rv = (t0 + 8 * g) & (c.page_size - 1);
    GPTQ_DASSERT(pk >= 0 && pk < c.n_pages && pv >= 0 && pv < c.n_pages && t0 >= 0 && t0 < st.n);
    const T* kp = kbase + (int64_t)pk * c.page_stride + rk * c.dim;
    const T* vp = vbase + (int64_t)pv * c.page_stride + rv * c.dim + vch;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < KS; ++i)
        r.k[t][i] = *(const x8*)(kp + 4 * t * c.dim + 8 * (4 * i + g < chunks ? 4 * i + g : 0));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (VEC == 8) {
        const uint4v x = *(const uint4v*)(vp + j * c.dim);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.v[j][e] = x[e];
      } else {
        const uint2v x = *(const uint2v*)(vp + j * c.dim);
        r.v[j][0] = x[0];
        r.v[j][1] = x[1];
      }
    }
  };
  auto compute = [&](int s, Pages p, Regs& r) __attribute__((always_inline)) {
    const int t0 = st.slot0(s);
    // elements beyond the head in the last chunks: the row behind, not this one's
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      if (KS > 2 && i < KS - 1) continue;
      const bool ok = 4 * i + g < chunks;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint4v z = __builtin_bit_cast(uint4v, r.k[t][i]);
        r.k[t][i] = __builtin_bit_cast(x8, (uint4v){ok ? z[0] : 0u, ok ? z[1] : 0u, ok ? z[2] : 0u, ok ? z[3] : 0u});
      }
    }
    float x[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float4v acc = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < KS; ++i) acc = KT::mfma16(r.k[t][i], q[i], acc);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * t + e] = acc[e] * sc;
    }
    // slots past the end, before the window or on no page: out of the scores, and their
    // values zeroed (0 x NaN is not 0)
    const bool whole = t0 + kTile <= st.n && (t0 >= st.first || t0 + kTile <= a.sinks);
    const bool vok = c.page_ok(p.v);
    if (!whole || __any(!vok)) {
      const int tv = t0 + 8 * g;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool ok = vok && tv + j < st.n && (tv + j >= st.first || tv + j < a.sinks);
        x[j] = ok ? x[j] : -INFINITY;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) r.v[j][e] = ok ? r.v[j][e] : 0u;
      }
    }
    if constexpr (SCORES == kScoresLds) {
      if (cl < n_h) {
        GPTQ_LDS float* sp = lds_scores + cl * w.n_scores + s * kTile + 8 * g;
        *(GPTQ_LDS float4v*)sp = (float4v){x[0], x[1], x[2], x[3]};
        *(GPTQ_LDS float4v*)(sp + 4) = (float4v){x[4], x[5], x[6], x[7]};
      }
    }
    if constexpr (SCORES == kScoresGlobal) {
      if (cl < n_h) {
        float* sp = w.scores + ((int64_t)b * a.n_heads + head) * w.n_scores + s * kTile + 8 * g;
        *(float4v*)sp = (float4v){x[0], x[1], x[2], x[3]};
        *(float4v*)(sp + 4) = (float4v){x[4], x[5], x[6], x[7]};
      }
    }
    float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    if (__any(top > m + kRaise)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float nm = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.0f : exp2f(m - nm);
      m = nm;
      lsum *= f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] *= f;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float pr[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      pr[j] = __builtin_amdgcn_exp2f(x[j] - base);
      lsum += pr[j];
    }
    // P in the cache's type for the matrix cores. bf16 keeps 8 bits, fewer than the
    // output's rounding hides behind, so its remainder goes through a second product
    // (the matrix cores have the time); fp16 keeps 11.
    x8 ph, pl;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ph[j] = (T)pr[j];
      if constexpr (__is_same(T, bf16_t)) pl[j] = (T)(pr[j] - (float)ph[j]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      uint4v vt;
#pragma unroll
      for (int jp = 0; jp < 4; ++jp)
        vt[jp] = __builtin_amdgcn_perm(r.v[2 * jp + 1][i / 2], r.v[2 * jp][i / 2], (i & 1) ? 0x07060302u : 0x05040100u);
      const x8 va = __builtin_bit_cast(x8, vt);
      o[i] = KT::mfma16(va, ph, o[i]);
      if constexpr (__is_same(T, bf16_t)) o[i] = KT::mfma16(va, pl, o[i]);
    }
  };

  Regs ra, rb;
  int s = split * per + wave;
  if (s < s_end) {
    Pages pa = pages(s), pb = pages(s + NW);
    load(s, pa, ra);
    while (true) {
      // Page numbers two steps ahead, then the next step's rows (the last step loads itself
      // again, unused). In this order: loads return in order, and a wait for the page numbers
      // must not be one for the rows behind them.
      const bool more = s + NW < s_end;
      const Pages pc = pages(s + 2 * NW);
      asm volatile("" ::: "memory");
      load(more ? s + NW : s, more ? pb : pa, rb);
      asm volatile("" ::: "memory");
      compute(s, pa, ra);
      if (!more) break;
      s += NW;
      const bool more2 = s + NW < s_end;
      const Pages pd = pages(s + 2 * NW);
      asm volatile("" ::: "memory");
      load(more2 ? s + NW : s, more2 ? pc : pb, ra);
      asm volatile("" ::: "memory");
      compute(s, pb, rb);
      if (!more2) break;
      s += NW;
      pa = pc;
      pb = pd;
    }
  }

  AddWeights<8, SCORES == kScoresLds> aw(c, a, w, st, b, kvh, 0, st.total, 64 * NW);
  if constexpr (SCORES && !SPLIT) {
    aw.lds = lds_scores;
    if (st.total > 0) aw.fetch();  // under way while the waves are joined
  }
  // join the waves of the block
  lsum += __shfl_xor(lsum, 16);
  lsum += __shfl_xor(lsum, 32);
  __shared__ float sm[NW][16], sl[NW][16], fin[32];
  if (g == 0) {
    sm[wave][cl] = m;
    sl[wave][cl] = lsum;
  }
  if (cl < n_h) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) so[(wave * n_h + cl) * kPitch + (4 * g + r) * VEC + i] = o[i][r];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < n_h * c.dim; k += 64 * NW) {
    const int hh = k / c.dim, e = k - hh * c.dim;
    float mm = -INFINITY;
#pragma unroll
    for (int u = 0; u < NW; ++u) mm = fmaxf(mm, sm[u][hh]);
    float l = 0.0f, v = 0.0f;
#pragma unroll
    for (int u = 0; u < NW; ++u) {
      const float f = sm[u][hh] == -INFINITY ? 0.0f : exp2f(sm[u][hh] - mm);
      // a wave without a visible slot holds zeros
      l += f * sl[u][hh];
      v += f * so[(u * n_h + hh) * kPitch + e];
    }
    const int64_t bh = (int64_t)b * a.n_heads + kvh * group + h0 + hh;
    if constexpr (SPLIT) {
      const int64_t part = bh * w.parts.n_splits + split;
      w.parts.o[part * c.dim + e] = v;
      if (e == 0) {
        w.parts.ml[2 * part] = mm;
        w.parts.ml[2 * part + 1] = l;
      }
    } else {
      ((T*)a.out)[(int64_t)b * a.ldo + (int64_t)(kvh * group + h0 + hh) * c.dim + e] = (T)(l == 0.0f ? 0.0f : v / l);
      if (SCORES && e == 0) {
        fin[2 * hh] = mm == -INFINITY ? 0.0f : mm;
        fin[2 * hh + 1] = l == 0.0f ? 0.0f : 1.0f / l;
      }
    }
  }
  if constexpr (SCORES && !SPLIT) {
    // this block has seen all scores of its key head: its own writes, read back
    __syncthreads();
    if (st.total > 0) aw.add(fin);
  }
}

// Maximum and sum of one head over its splits, by a wave (every lane returns them).
__device__ __forceinline__ void join_ml(const float* ml, int n_splits, float* m, float* l) {
  const int lane = threadIdx.x & 63;
  float mm = -INFINITY, ll = 0.0f;
  for (int s = lane; s < n_splits; s += 64) mm = fmaxf(mm, ml[2 * s]);
  for (int o = 32; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
  const float base = mm == -INFINITY ? 0.0f : mm;
  for (int s = lane; s < n_splits; s += 64) ll += __builtin_amdgcn_exp2f(ml[2 * s] - base) * ml[2 * s + 1];
  for (int o = 32; o > 0; o >>= 1) ll += __shfl_xor(ll, o);
  *m = base;
  *l = ll;
}

// Joins the splits of one row and head, one per block: 8 groups of threads take every eighth
// split, 4 elements a thread.
template <typename T>
__device__ __forceinline__ void join_row(const KvView& c, const KvAttnArgs& a, const SplitWs& w, int64_t bh, float* lse,
                                         float* sh) {
  const int tid = threadIdx.x;
  const float* ml = w.ml + bh * w.n_splits * 2;
  float m, l;
  join_ml(ml, w.n_splits, &m, &l);
  const int g = tid >> 5, e = (tid & 31) * 4;
  const bool in = e < c.dim;
  const float* o = w.o + bh * w.n_splits * c.dim + (in ? e : 0);
  float4v v = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = g; s < w.n_splits; s += 8)
    if (ml[2 * s] != -INFINITY)
      v += __builtin_amdgcn_exp2f(ml[2 * s] - m) * *(const float4v*)(o + (int64_t)s * c.dim);
  *(float4v*)(sh + 4 * tid) = v;
  __syncthreads();
  if (g == 0 && in) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += *(const float4v*)(sh + 4 * (tid + 32 * k));
    const int64_t row = bh / a.n_heads, h = bh - row * a.n_heads;
    typedef T x4 __attribute__((ext_vector_type(4)));
    x4 y;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = (T)(l == 0.0f ? 0.0f : v[k] / l);
    *(x4*)((T*)a.out + row * a.ldo + h * c.dim + e) = y;
  }
  if (lse && tid == 0) *lse = l == 0.0f ? INFINITY : m + log2f(l);
}

// Row and head bh belong to a sequence of the ragged batch (rows behind the last one, say, stay
// as they were): each of n threads looks at its share of the sequences.
__device__ __forceinline__ bool owned(const KvView& c, const int32_t* cu, int n_rows, int row, int i, int n) {
  bool any = false;
  for (int s = i; s < c.n_seqs; s += n) {
    const int c0 = cu[s], c1 = cu[s + 1];
    any |= c0 >= 0 && c0 <= row && row < c1 && c1 <= n_rows;
  }
  return any;
}

// Joins the splits of all rows of a ragged batch, bound by reading them: many splits of few rows
// with a block for each row and head; up to 16 of them (as many lanes hold their maxima) by half
// a wave, which goes through all. 512 queries, 32 heads of 128, 712 slots in 3 splits: the call
// takes 48 us with a block each, 28 with half a wave.
constexpr int kJoinFew = 16;

template <typename T, bool FEW>
__global__ __launch_bounds__(256) void join_rows_kernel(KvView c, KvAttnArgs a, SplitWs w, const int32_t* cu,
                                                        int n_rows, float* lse) {
  if constexpr (!FEW) {
    __shared__ float sh[1024];
    if (__syncthreads_or(owned(c, cu, n_rows, blockIdx.x / a.n_heads, threadIdx.x, 256)))
      join_row<T>(c, a, w, blockIdx.x,
                  lse ? lse + (int64_t)(blockIdx.x % a.n_heads) * n_rows + blockIdx.x / a.n_heads : nullptr, sh);
  } else {
    const int64_t bh = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, row = (int)(bh / a.n_heads), n = w.n_splits;
    const uint64_t hit = __ballot(row < n_rows && owned(c, cu, n_rows, row, lane, 32));
    if ((uint32_t)(hit >> (threadIdx.x & 32)) == 0) return;
    const float* ml = w.ml + bh * n * 2;
    const int mine = lane & (kJoinFew - 1);
    const float ms = mine < n ? ml[2 * mine] : -INFINITY, ls = mine < n ? ml[2 * mine + 1] : 0.0f;
    float m = ms;
#pragma unroll
    for (int o = kJoinFew / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (m == -INFINITY) m = 0.0f;
    const float f = __builtin_amdgcn_exp2f(ms - m);
    float l = f * ls;
#pragma unroll
    for (int o = kJoinFew / 2; o > 0; o >>= 1) l += __shfl_xor(l, o);
    const int e = 4 * lane;
    const bool in = e < c.dim;
    const float* op = w.o + bh * n * c.dim + (in ? e : 0);
    float4v v = {0, 0, 0, 0};
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float ms_ = __shfl(ms, s, 32), fs = __shfl(f, s, 32);
      if (ms_ != -INFINITY) v += fs * *(const float4v*)(op + (int64_t)s * c.dim);
    }
    const int h = (int)(bh - (int64_t)row * a.n_heads);
    if (in) {
      typedef T x4 __attribute__((ext_vector_type(4)));
      x4 y;
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = (T)(l == 0.0f ? 0.0f : v[k] / l);
      *(x4*)((T*)a.out + (int64_t)row * a.ldo + h * c.dim + e) = y;
    }
    if (lse && lane == 0) lse[(int64_t)h * n_rows + row] = l == 0.0f ? INFINITY : m + log2f(l);
  }
}

// The same after the one-token kernel: the first n_seqs n_heads blocks the outputs, the
// others the weights of kJoinSteps steps of one key head.
constexpr int kJoinSteps = 32;

template <typename T>
__global__ __launch_bounds__(256) void token_join_kernel(KvView c, KvAttnArgs a, TokenWs w, int n_parts) {
  extern __shared__ float sh[];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < c.n_seqs * a.n_heads) {
    join_row<T>(c, a, w.parts, blockIdx.x, nullptr, sh);
    return;
  }
  const int group = a.n_heads / c.n_kv;
  int id = blockIdx.x - c.n_seqs * a.n_heads;
  const int part = id % n_parts;
  id /= n_parts;
  const int kvh = id % c.n_kv, b = id / c.n_kv;
  const Steps st(c.len(b), a.window, a.sinks);
  if (part * kJoinSteps >= st.total) return;
  AddWeights<4> aw(c, a, w, st, b, kvh, part * kJoinSteps, (part + 1) * kJoinSteps, 256);
  aw.fetch();
  const int64_t bh0 = (int64_t)b * a.n_heads + kvh * group;
  for (int h = tid >> 6; h < group; h += 4) {
    float m, l;
    join_ml(w.parts.ml + (bh0 + h) * w.parts.n_splits * 2, w.parts.n_splits, &m, &l);
    if ((tid & 63) == 0) {
      sh[2 * h] = m;
      sh[2 * h + 1] = l == 0.0f ? 0.0f : 1.0f / l;
    }
  }
  __syncthreads();
  aw.add(sh);
}

int64_t max_steps(const KvView& c, int64_t window, int64_t sinks) {
  const int64_t cap = (int64_t)c.max_pages << c.page_shift, all = ceil_div(cap, kTile);
  if (window <= 0 || window >= cap) return all;
  const int64_t some = ceil_div(sinks < cap ? sinks : cap, kTile) + window / kTile + 2;
  return some < all ? some : all;
}

// Blocks per (sequence, key head, tile of heads). One compute unit streams about 45
// GB/s, so a call that has fewer blocks than there are compute units splits its
// sequences until there is one each: a sequence of 2048 slots and 8 key heads takes
// 23.8 us unsplit, 9.8 split by 16. Sequences of different lengths get twice as many
// where that is many (three of 9001 to 32768 slots: 62.9 us at 10 splits each, 57.5 at
// 21; eight of one length 27.3 and 27.6). A block of up to 256 KB stays whole, since the
// second kernel costs more than splitting gives (300 slots of 80, 32 key heads: 7.0 us
// whole, 9.0 split by 2), and so do more pairs than half the compute units (160 of 2048
// slots: 28.3 us whole, 35.4 split by 2).
int64_t splits_of(const KvView& c, int64_t n_heads, int64_t window, int64_t sinks) {
  const int64_t base = (int64_t)c.n_seqs * c.n_kv * ceil_div(n_heads / c.n_kv, 16);
  const int64_t steps = max_steps(c, window, sinks);
  if (steps * kTile * c.dim * 4 <= (256 << 10)) return 1;
  int64_t s = 256 / base;
  if (c.n_seqs > 1 && s >= 4) s = 512 / base;
  return std::max<int64_t>(1, std::min<int64_t>(s, ceil_div(steps, NW)));
}

TokenWs layout(const KvView& c, int64_t n_heads, int64_t window, int64_t sinks, bool weights, void* ws, size_t* bytes) {
  TokenWs w{};
  w.parts.n_splits = (int)splits_of(c, n_heads, window, sinks);
  w.join = w.parts.n_splits > 1 || (weights && n_heads / c.n_kv > 16);
  w.n_scores = (int)(max_steps(c, window, sinks) * kTile);
  const int64_t rows = (int64_t)c.n_seqs * n_heads;
  float* f = (float*)ws;
  size_t n = 0;
  w.lds = weights && !w.join && (size_t)(n_heads / c.n_kv) * w.n_scores * sizeof(float) <= kScoresLdsBytes;
  w.scores = f;  // multiples of 4 floats each: all 16-byte aligned
  if (weights && !w.lds) n += (size_t)rows * w.n_scores;
  if (w.join) {
    w.parts.o = f + n;
    n += (size_t)rows * w.parts.n_splits * c.dim;
    w.parts.ml = f + n;
    n += (size_t)rows * w.parts.n_splits * 2;
  }
  if (bytes) *bytes = n * sizeof(float);
  return w;
}

template <typename T, int KS, int VEC>
gptq_status_t launch(const KvView& c, const KvAttnArgs& a, const TokenWs& w, hipStream_t st) {
  const int64_t group = a.n_heads / c.n_kv;
  const int64_t blocks = (int64_t)c.n_seqs * c.n_kv * ceil_div(group, 16) * w.parts.n_splits;
  if (blocks * 64 * NW >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), blk(64 * NW);
  const size_t lds = NW * (size_t)std::min<int64_t>(group, 16) * (16 * VEC + 4) * sizeof(float);
  if (a.weights && w.join)
    hipLaunchKernelGGL((token_kernel<T, KS, VEC, true, kScoresGlobal>), grid, blk, lds, st, c, a, w);
  else if (a.weights && w.lds)
    hipLaunchKernelGGL((token_kernel<T, KS, VEC, false, kScoresLds>), grid, blk,
                       lds + group * w.n_scores * sizeof(float), st, c, a, w);
  else if (a.weights)
    hipLaunchKernelGGL((token_kernel<T, KS, VEC, false, kScoresGlobal>), grid, blk, lds, st, c, a, w);
  else if (w.join)
    hipLaunchKernelGGL((token_kernel<T, KS, VEC, true, 0>), grid, blk, lds, st, c, a, w);
  else
    hipLaunchKernelGGL((token_kernel<T, KS, VEC, false, 0>), grid, blk, lds, st, c, a, w);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <typename T>
gptq_status_t token_enqueue(const KvView& c, const KvAttnArgs& a, void* ws, hipStream_t st) {
  const TokenWs w = layout(c, a.n_heads, a.window, a.sinks, a.weights != nullptr, ws, nullptr);
  const int64_t parts = a.weights ? ceil_div(w.n_scores / kTile, kJoinSteps) : 1;
  const int64_t jblocks = (int64_t)c.n_seqs * (a.n_heads + (a.weights ? c.n_kv * parts : 0));
  if (jblocks * 256 >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  const gptq_status_t rc = c.dim <= 64   ? launch<T, 2, 4>(c, a, w, st)
                           : c.dim <= 96 ? launch<T, 3, 8>(c, a, w, st)
                                         : launch<T, 4, 8>(c, a, w, st);
  if (rc != GPTQ_OK || !w.join) return rc;
  hipLaunchKernelGGL(token_join_kernel<T>, dim3((unsigned)jblocks), dim3(256),
                     std::max<size_t>(4096, 2 * sizeof(float) * (a.n_heads / c.n_kv)), st, c, a, w, (int)parts);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace

size_t kv_token_workspace_bytes(const KvView& c, int64_t n_heads, int64_t window, int64_t sinks, bool weights) {
  size_t bytes = 0;
  layout(c, n_heads, window, sinks, weights, nullptr, &bytes);
  return bytes;
}

template <typename T>
static gptq_status_t join_enqueue(const KvView& c, const KvAttnArgs& a, const SplitWs& w, int64_t n_rows,
                                  const int32_t* cu, float* lse, hipStream_t st) {
  const bool few = w.n_splits <= kJoinFew;
  const int64_t blocks = few ? ceil_div(n_rows * a.n_heads, 8) : n_rows * a.n_heads;
  if (blocks * 256 >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  if (few)
    hipLaunchKernelGGL((join_rows_kernel<T, true>), dim3((unsigned)blocks), dim3(256), 0, st, c, a, w, cu, (int)n_rows,
                       lse);
  else
    hipLaunchKernelGGL((join_rows_kernel<T, false>), dim3((unsigned)blocks), dim3(256), 0, st, c, a, w, cu, (int)n_rows,
                       lse);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status_t kv_join_enqueue(const KvView& c, const KvAttnArgs& a, const SplitWs& w, int64_t n_rows,
                              const int32_t* cu, float* lse, hipStream_t st) {
  return c.bf16 ? join_enqueue<bf16_t>(c, a, w, n_rows, cu, lse, st)
                : join_enqueue<half_t>(c, a, w, n_rows, cu, lse, st);
}

gptq_status_t kv_token_enqueue(const KvView& c, const KvAttnArgs& a, void* ws, hipStream_t st) {
  TraceScope tr(st, GPTQ_TRACE_KV_ATTENTION);
  return c.bf16 ? token_enqueue<bf16_t>(c, a, ws, st) : token_enqueue<half_t>(c, a, ws, st);
}

}  // namespace gptq
