// Causal attention of a ragged batch of prompts, or of the next chunk of longer
// ones, over the paged cache (the new tokens' rows are in it already): query i of
// sequence b stands at position p = lens[b] - n_b + i and sees the slots t <= p
// with t > p - window (or any, window 0) or t < sinks.
//
// One pass with a running maximum and sum over tiles of 64 slots. A block takes
// 128 queries of one head, a wave 32 of them:
//   S^T [64 slots, 32 queries] = K Q^T,  O^T [dim, 32 queries] += V^T P^T
// on 32 x 32 matrix instructions. A lane holds one query's column of S^T, so the
// softmax needs no exchange between lanes but one (the two halves of the
// column), and only when the running maximum is raised, which waits until a
// score passes it by 2^8. K rows are assigned to the rows of S^T such that a
// lane's scores are the P^T operand of the second product as they stand.
// K is staged in LDS as it is, V turned over (4 x 8 blocks in registers), both
// padded so that the operand reads meet no bank twice.
#include <atomic>

#include "kv.h"

namespace gptq {
namespace {

constexpr int kQ = 128, kT = 64;
constexpr float kRaise = 8.0f;

// The slots some query of a block sees, as tiles of kT.
struct Tiles {
  int n, first, sink_tiles, total, jump;
  __device__ __forceinline__ Tiles(int end, int first_slot, int sinks) {
    n = end;
    first = first_slot;
    const int all = (end + kT - 1) / kT;
    const int sk = first > 0 ? (sinks < first ? sinks : first) : 0;
    sink_tiles = (sk + kT - 1) / kT;
    jump = first / kT;
    if (jump < sink_tiles) jump = sink_tiles;
    total = sink_tiles + (all > jump ? all - jump : 0);
  }
  __device__ __forceinline__ int slot0(int s) const { return (s < sink_tiles ? s : s - sink_tiles + jump) * kT; }
};

// Block t of the ragged batch's blocks of kQ queries: its sequence and first
// query there; sequences in order. b = -1 behind the last one.
struct Where {
  int b, i0, n_b, row0;  // sequence, first query in it, its queries, its first row
  __device__ __forceinline__ Where(const int32_t* cu, int n_seqs, int t, int n_rows) {
    const int lane = threadIdx.x & 63;
    b = -1;
    int before = 0;
    for (int base = 0; base < n_seqs; base += 64) {
      const int s = base + lane;
      int c0 = 0, n = 0;
      if (s < n_seqs) {
        c0 = cu[s];
        const int c1 = cu[s + 1];
        // rows outside the q tensor are not there, whatever cu says
        n = c0 >= 0 && c1 > c0 && c1 <= n_rows ? c1 - c0 : 0;
      }
      int incl = (n + kQ - 1) / kQ;
      const int own = incl;
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(incl, o);
        if (lane >= o) incl += u;
      }
      const int start = before + incl - own;
      const uint64_t hit = __ballot(t >= start && t < start + own);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        b = base + l;
        i0 = (t - __shfl(start, l)) * kQ;
        n_b = __shfl(n, l);
        row0 = __shfl(c0, l);
        break;
      }
      before += __shfl(incl, 63);
    }
    if (b >= 0) {
      b = __builtin_amdgcn_readfirstlane(b);
      i0 = __builtin_amdgcn_readfirstlane(i0);
      n_b = __builtin_amdgcn_readfirstlane(n_b);
      row0 = __builtin_amdgcn_readfirstlane(row0);
    }
  }
};

// Slot (within 32) of row m of S^T: rows 8 q + 4 f + r belong to lane half f.
__device__ __forceinline__ int slot_of_row(int m) {
  return 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);
}

__device__ __forceinline__ uint32_t finite_only(uint32_t x, uint32_t exp_mask, bool* bad) {
  // two 16-bit values: one with all exponent bits set is replaced by 0
  uint32_t lo = (x & exp_mask & 0xffffu) == (exp_mask & 0xffffu) ? 0u : x & 0xffffu;
  uint32_t hi = (x & exp_mask & 0xffff0000u) == (exp_mask & 0xffff0000u) ? 0u : x & 0xffff0000u;
  *bad |= (lo | hi) != x;
  return lo | hi;
}

template <typename T, int DHP>
struct PromptShared {
  static constexpr int KP = DHP + 8, VP = kT + 8;  // row pitches, elements
  T k[2][kT * KP];
  T v[2][DHP * VP];
  // by tile modulo 3 (one is read, one written, one cleared), a bit per slot:
  uint32_t there[3][2];  // lies on a page
  uint32_t odd[3][2];    // its values hold an infinity or NaN (masked tiles only)
};

// LSE: the row's log2 of the sum of 2^score goes to lse [n_tokens][n_heads].
template <typename T, int DHP, bool LSE>
__global__ __launch_bounds__(256, 2) void prompt_kernel(KvView c, KvAttnArgs a, const int32_t* cu, int n_rows,
                                                        int n_blk, float* lse) {
  using KT = KvType<T>;
  using x8 = typename KT::x8;
  using Sh = PromptShared<T, DHP>;
  constexpr int CH = DHP / 8, NK = kT * CH / 256, QS = DHP / 16, NO = DHP / 32;
  constexpr uint32_t kExp = __is_same(T, half_t) ? 0x7c007c00u : 0x7f807f80u;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Sh& sh = *(Sh*)smem;
  const int id = xcd_logical_block(blockIdx.x, gridDim.x);
  const int h = id / n_blk;
  const Where at(cu, c.n_seqs, n_blk - 1 - (id - h * n_blk), n_rows);  // late queries see most: first
  if (at.b < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int kvh = h / (a.n_heads / c.n_kv);
  const int len = c.len(at.b);
  const int p0 = len - at.n_b + at.i0;                                   // position of the block's first query
  const int rows = at.n_b - at.i0 < kQ ? at.n_b - at.i0 : kQ;            // its queries
  const int first = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
  const int end = p0 + rows > 0 ? p0 + rows : 0;
  const Tiles tl(end, first < end ? first : end, a.sinks);
  const int32_t* table = c.table + (int64_t)at.b * c.ld_table;
  const int chunks = c.dim >> 3;

  const int qi = wave * 32 + col, pos = p0 + qi;  // this lane's query
  const bool q_ok = qi < rows;
  x8 q[QS];
  {
    const T* qp = (const T*)a.q + (int64_t)(at.row0 + at.i0 + (q_ok ? qi : 0)) * a.ldq + (int64_t)h * c.dim;
#pragma unroll
    for (int i = 0; i < QS; ++i) {
      const int ch = 2 * i + half;
      const bool ok = ch < chunks;
      const uint4v z = *(const uint4v*)(qp + 8 * (ok ? ch : 0));
      q[i] = __builtin_bit_cast(x8, (uint4v){ok ? z[0] : 0u, ok ? z[1] : 0u, ok ? z[2] : 0u, ok ? z[3] : 0u});
    }
  }
  const float sc = a.scale * kLog2e;
  float16v o[NO];
#pragma unroll
  for (int i = 0; i < NO; ++i) o[i] = (float16v){0};
  float m = -INFINITY, lsum = 0.0f;

  // this wave's queries: positions w0 .. w1
  const int w0 = p0 + wave * 32, w1 = w0 + 31 < end - 1 ? w0 + 31 : end - 1;

  const T* kb = (const T*)c.k + (int64_t)kvh * c.page_size * c.dim;
  const T* vb = (const T*)c.v + (int64_t)kvh * c.page_size * c.dim;
  const int vquad = tid & 15, vchunk = tid >> 4;  // V: 4 slots x 8 elements
  struct Pages {
    int k[NK], v;
  };
  auto pages = [&](int s) __attribute__((always_inline)) {
    Pages p;
    const int t0 = tl.slot0(s);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int t = t0 + (tid + 256 * i) / CH;
      p.k[i] = s < tl.total && t < tl.n ? table[t >> c.page_shift] : -1;
    }
    const int t = t0 + 4 * vquad;
    p.v = s < tl.total && t < tl.n ? table[t >> c.page_shift] : -1;
    return p;
  };
  struct Stage {
    uint4v k[NK], v[4];
  };
  auto load = [&](int s, const Pages& p, Stage& r) __attribute__((always_inline)) {
    const int t0 = tl.slot0(s);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int it = tid + 256 * i, row = it / CH, ch = it - row * CH;
      r.k[i] = (uint4v){0, 0, 0, 0};
      if (c.page_ok(p.k[i]) && ch < chunks)
        r.k[i] = *(const uint4v*)(kb + (int64_t)p.k[i] * c.page_stride + ((t0 + row) & (c.page_size - 1)) * c.dim + ch * 8);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.v[j] = (uint4v){0, 0, 0, 0};
      const int t = t0 + 4 * vquad + j;
      if (c.page_ok(p.v) && t < tl.n && vchunk < chunks)
        r.v[j] = *(const uint4v*)(vb + (int64_t)p.v * c.page_stride + (t & (c.page_size - 1)) * c.dim + vchunk * 8);
    }
  };
  // whether every query of the block sees every slot of tile s
  auto whole = [&](int s) __attribute__((always_inline)) {
    const int t0 = tl.slot0(s), t1 = t0 + kT - 1;
    const int low = a.window > 0 ? p0 + rows - 1 - a.window + 1 : 0;  // first slot of the last query's window
    return t1 <= p0 && (t0 >= low || t1 < a.sinks);
  };
  auto store = [&](int s, int buf, int bits, const Pages& p, Stage& r) __attribute__((always_inline)) {
    const bool masked = !whole(s);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int it = tid + 256 * i, row = it / CH, ch = it - row * CH;
      *(uint4v*)&sh.k[buf][row * Sh::KP + ch * 8] = r.k[i];
    }
    if (vchunk == 0 && !c.page_ok(p.v)) {
      const int t = 4 * vquad;
      atomicAnd(&sh.there[bits][t >> 5], ~(0xfu << (t & 31)));
    }
    if (masked) {
      // a value that is not finite must not reach the queries that do not see its slot
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) r.v[j][e] = finite_only(r.v[j][e], kExp, &bad);
        const int t = 4 * vquad + j;
        if (bad) atomicOr(&sh.odd[bits][t >> 5], 1u << (t & 31));
      }
    }
    if (vchunk < CH) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
        uint2v x;
        x[0] = __builtin_amdgcn_perm(r.v[1][e / 2], r.v[0][e / 2], sel);
        x[1] = __builtin_amdgcn_perm(r.v[3][e / 2], r.v[2][e / 2], sel);
        *(uint2v*)&sh.v[buf][(vchunk * 8 + e) * Sh::VP + 4 * vquad] = x;
      }
    }
  };
  auto clear = [&](int bits) __attribute__((always_inline)) {
    if (tid < 2) {
      sh.there[bits][tid] = ~0u;
      sh.odd[bits][tid] = 0u;
    }
  };
  auto sees = [&](int t) __attribute__((always_inline)) {
    return t <= pos && (a.window <= 0 || t > pos - a.window || t < a.sinks);
  };

  auto compute = [&](int s, int buf, int bits) __attribute__((always_inline)) {
    const int t0 = tl.slot0(s);
    const bool off_page = (sh.there[bits][0] & sh.there[bits][1]) != ~0u;
    // nothing of this tile for any query of this wave
    if (t0 > w1 || w0 >= end || w1 < 0) return;
    if (a.window > 0 && t0 + kT - 1 <= w0 - a.window && t0 >= a.sinks) return;
    float16v sv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      sv[u] = (float16v){0};
      const T* kp = &sh.k[buf][(32 * u + slot_of_row(col)) * Sh::KP + 8 * half];
#pragma unroll
      for (int i = 0; i < QS; ++i) sv[u] = KT::mfma32(*(const x8*)(kp + 16 * i), q[i], sv[u]);
    }
    const bool all = !off_page && t0 + kT - 1 <= w0 && (a.window <= 0 || t0 > w1 - a.window || t0 + kT <= a.sinks);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) sv[u][r] *= sc;
    if (!all) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t there = sh.there[bits][u];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int k = 16 * (r >> 3) + 8 * half + (r & 7), t = t0 + 32 * u + k;
          sv[u][r] = sees(t) && ((there >> k) & 1) ? sv[u][r] : -INFINITY;
        }
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, sv[u][r]);
    if (__any(top > m + kRaise)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float nm = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.0f : exp2f(m - nm);
      m = nm;
      lsum *= f;
#pragma unroll
      for (int i = 0; i < NO; ++i) o[i] *= f;
    }
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        sv[u][r] = __builtin_amdgcn_exp2f(sv[u][r] - base);
        lsum += sv[u][r];
      }
    // P in the cache's type: its rounding (2^-12 or 2^-9 of each weight at most) averages out
    // over the slots and stays below that of the output
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x8 pf;
#pragma unroll
        for (int j = 0; j < 8; ++j) pf[j] = (T)sv[u][8 * k + j];
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          const x8 va = *(const x8*)&sh.v[buf][(32 * i + col) * Sh::VP + 32 * u + 16 * k + 8 * half];
          o[i] = KT::mfma32(va, pf, o[i]);
        }
      }
    if ((sh.odd[bits][0] | sh.odd[bits][1]) != 0u) {
      // rare: the values that are not finite, for the queries that see them
      for (int k = 0; k < kT; ++k) {
        if (!((sh.odd[bits][k >> 5] >> (k & 31)) & 1)) continue;
        float pk = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (32 * u + 16 * (r >> 3) + 8 * half + (r & 7) == k) pk = sv[u][r];
        const float other = __shfl_xor(pk, 32);
        if (((k >> 3) & 1) != half) pk = other;
        if (!sees(t0 + k)) continue;
        const int t = t0 + k, pg = table[t >> c.page_shift];
        if (!c.page_ok(pg)) continue;
        const T* vp = vb + (int64_t)pg * c.page_stride + (t & (c.page_size - 1)) * c.dim;
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int e = 32 * i + 8 * (r >> 2) + 4 * half + (r & 3);
            if (e >= c.dim) continue;
            const float x = (float)vp[e];
            if (!(__builtin_fabsf(x) < INFINITY)) o[i][r] += pk * x;
          }
      }
    }
  };

  if (tl.total > 0) {
    Stage st;
    Pages pa = pages(0);
    clear(0);
    clear(1);
    load(0, pa, st);
    Pages pb = pages(1);
    __syncthreads();
    store(0, 0, 0, pa, st);
    __syncthreads();
    int bits = 0;  // s modulo 3
    for (int s = 0; s < tl.total; ++s) {
      const int buf = s & 1, next = bits == 2 ? 0 : bits + 1;
      if (s + 1 < tl.total) load(s + 1, pb, st);
      pa = pb;
      pb = pages(s + 2);
      clear(next == 2 ? 0 : next + 1);  // tile s + 2's, read last by tile s - 1
      compute(s, buf, bits);
      if (s + 1 < tl.total) store(s + 1, buf ^ 1, next, pa, st);
      __syncthreads();
      bits = next;
    }
  }

  lsum += __shfl_xor(lsum, 32);
  if (!q_ok) return;
  const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
  const int64_t row = at.row0 + at.i0 + qi;
  T* op = (T*)a.out + row * a.ldo + (int64_t)h * c.dim;
#pragma unroll
  for (int i = 0; i < NO; ++i)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int e = 32 * i + 8 * r4 + 4 * half;
      if (e < c.dim) {
        typedef T x4 __attribute__((ext_vector_type(4)));
        x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = lsum == 0.0f ? (T)0.0f : (T)(o[i][4 * r4 + r] * inv);
        *(x4*)(op + e) = y;
      }
    }
  if constexpr (LSE) {
    // a row without a weight: +infinity, so that 2^(score - lse) is 0
    if (half == 0) lse[row * a.n_heads + h] = lsum == 0.0f ? INFINITY : m + log2f(lsum);
  }
}

// weights[b][g][t] += sum over the queries of b and the heads of group g of
// 2^(score - lse): the scores once more (half the products of the attention),
// as S^T tiles whose rows, the slots, are summed along. One block owns 128 slots
// of one key head (a wave 32, its keys in registers) and goes over all queries
// that may see them, 32 at a time, so every sum has one owner and one order.
template <typename T, int DHP>
__global__ __launch_bounds__(256, 2) void prompt_weights_kernel(KvView c, KvAttnArgs a, const int32_t* cu, int n_rows,
                                                               int n_tiles, const float* lse) {
  using KT = KvType<T>;
  using x8 = typename KT::x8;
  constexpr int QS = DHP / 16, CH = DHP / 8, QP = DHP + 8, NQ = 64;
  __shared__ __attribute__((aligned(16))) T qs[NQ * QP];
  __shared__ float ls[NQ];
  const int id = xcd_logical_block(blockIdx.x, gridDim.x);
  const int tile = id % n_tiles, bg = id / n_tiles;
  const int kvh = bg % c.n_kv, b = bg / c.n_kv;
  const int r0 = cu[b], r1 = cu[b + 1];
  const int len = c.len(b);
  const int n_b = r0 >= 0 && r1 > r0 && r1 <= n_rows ? r1 - r0 : 0;
  const int t00 = tile * 128;
  if (n_b == 0 || t00 >= len) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int t0 = t00 + 32 * wave;
  const int group = a.n_heads / c.n_kv, chunks = c.dim >> 3;
  const int32_t* table = c.table + (int64_t)b * c.ld_table;
  const float sc = a.scale * kLog2e;

  x8 k[QS];
  {
    const int t = t0 + slot_of_row(col);
    const int pg = t < len ? table[t >> c.page_shift] : -1;
    const T* kp = (const T*)c.k + (c.page_ok(pg) ? c.head_base(pg, kvh) + (int64_t)(t & (c.page_size - 1)) * c.dim : 0);
#pragma unroll
    for (int i = 0; i < QS; ++i) {
      const int ch = 2 * i + half;
      const bool ok = ch < chunks && c.page_ok(pg);
      const uint4v z = *(const uint4v*)(kp + 8 * (ok ? ch : 0));
      k[i] = __builtin_bit_cast(x8, (uint4v){ok ? z[0] : 0u, ok ? z[1] : 0u, ok ? z[2] : 0u, ok ? z[3] : 0u});
    }
  }
  float16v acc = (float16v){0};
  // queries at positions p >= t, and, unless a slot of the block is a sink, p < t + window
  const int base = len - n_b;  // position of query 0
  int i_lo = t00 - base, i_hi = n_b;
  if (i_lo < 0) i_lo = 0;
  if (a.window > 0 && t00 >= a.sinks) {
    const int64_t last = (int64_t)t00 + 127 + a.window - base;  // first query that no longer sees slot t00 + 127
    if (last < i_hi) i_hi = (int)last;
  }
  i_lo &= ~(NQ - 1);
  const T* qb = (const T*)a.q + (int64_t)r0 * a.ldq;
  for (int hh = 0; hh < group; ++hh) {
    const int h = kvh * group + hh;
    for (int i0 = i_lo; i0 < i_hi; i0 += NQ) {
      __syncthreads();
      for (int it = tid; it < NQ * CH; it += 256) {
        const int row = it / CH, ch = it - row * CH;
        uint4v z = (uint4v){0, 0, 0, 0};
        if (i0 + row < n_b && ch < chunks) z = *(const uint4v*)(qb + (int64_t)(i0 + row) * a.ldq + (int64_t)h * c.dim + ch * 8);
        *(uint4v*)&qs[row * QP + ch * 8] = z;
      }
      if (tid < NQ) ls[tid] = i0 + tid < n_b ? lse[(int64_t)(r0 + i0 + tid) * a.n_heads + h] : INFINITY;
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NQ / 32; ++u) {
        float16v sv = (float16v){0};
#pragma unroll
        for (int i = 0; i < QS; ++i) sv = KT::mfma32(k[i], *(const x8*)&qs[(32 * u + col) * QP + 16 * i + 8 * half], sv);
        const int pos = base + i0 + 32 * u + col;
        const float l = ls[32 * u + col];
        const int lowest = base + i0 + 32 * u;
        const bool all = t0 + 31 <= lowest && (a.window <= 0 || t0 > lowest + 31 - a.window || t0 + 32 <= a.sinks);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int t = t0 + 16 * (r >> 3) + 8 * half + (r & 7);
          const bool ok = all || (t <= pos && (a.window <= 0 || t > pos - a.window || t < a.sinks));
          const float p = __builtin_amdgcn_exp2f(sv[r] * sc - l);
          acc[r] += ok ? p : 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r)
    for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor(acc[r], o);
  if (col == 0) {
    float* wt = a.weights + ((int64_t)b * c.n_kv + kvh) * a.ldw;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int t = t0 + 16 * (r >> 3) + 8 * half + (r & 7);
      if (t < len && c.page_ok(table[t >> c.page_shift])) wt[t] += acc[r];
    }
  }
}

template <typename T, int DHP>
gptq_status_t launch(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, float* lse,
                     hipStream_t st) {
  const int64_t n_blk = n_tokens / kQ + c.n_seqs;  // at least the ragged batch's blocks
  const int64_t blocks = n_blk * a.n_heads;
  const int64_t cap = (int64_t)c.max_pages << c.page_shift, n_tiles = ceil_div(cap, 128);
  const int64_t wblocks = n_tiles * c.n_kv * c.n_seqs;
  if (blocks * 256 >= (int64_t)1 << 32 || wblocks * 256 >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  const size_t lds = sizeof(PromptShared<T, DHP>);
  const void* fn = a.weights ? (const void*)prompt_kernel<T, DHP, true> : (const void*)prompt_kernel<T, DHP, false>;
  // more than 64 KB of LDS has to be asked for, once per device and kernel
  static std::atomic<uint64_t> asked[2];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return GPTQ_ERR_HIP;
  std::atomic<uint64_t>& flags = asked[a.weights ? 1 : 0];
  if (!((flags.load(std::memory_order_acquire) >> dev) & 1)) {
    if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess) return GPTQ_ERR_HIP;
    flags.fetch_or(1ull << dev, std::memory_order_release);
  }
  if (a.weights)
    hipLaunchKernelGGL((prompt_kernel<T, DHP, true>), dim3((unsigned)blocks), dim3(256), lds, st, c, a, cu,
                       (int)n_tokens, (int)n_blk, lse);
  else
    hipLaunchKernelGGL((prompt_kernel<T, DHP, false>), dim3((unsigned)blocks), dim3(256), lds, st, c, a, cu,
                       (int)n_tokens, (int)n_blk, lse);
  GPTQ_CHECK_LAUNCH();
  if (a.weights) {
    hipLaunchKernelGGL((prompt_weights_kernel<T, DHP>), dim3((unsigned)wblocks), dim3(256), 0, st, c, a, cu,
                       (int)n_tokens, (int)n_tiles, lse);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

template <typename T>
gptq_status_t prompt_enqueue(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, float* lse,
                             hipStream_t st) {
  if (c.dim <= 64) return launch<T, 64>(c, a, cu, n_tokens, lse, st);
  if (c.dim <= 96) return launch<T, 96>(c, a, cu, n_tokens, lse, st);
  return launch<T, 128>(c, a, cu, n_tokens, lse, st);
}

}  // namespace

size_t kv_prompt_workspace_bytes(int64_t n_tokens, int64_t n_heads, bool weights) {
  return weights ? (size_t)n_tokens * n_heads * sizeof(float) : 0;
}

gptq_status_t kv_prompt_enqueue(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, void* ws,
                                hipStream_t st) {
  TraceScope tr(st, GPTQ_TRACE_KV_ATTENTION);
  return c.bf16 ? prompt_enqueue<bf16_t>(c, a, cu, n_tokens, (float*)ws, st)
                : prompt_enqueue<half_t>(c, a, cu, n_tokens, (float*)ws, st);
}

}  // namespace gptq
