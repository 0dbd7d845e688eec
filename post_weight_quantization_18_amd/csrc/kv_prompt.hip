// Causal attention of a ragged batch of prompts, or of the next chunk of longer
// ones, over the paged cache (the new tokens' rows are in it already): query i of
// sequence b stands at position p = lens[b] - n_b + i and sees the slots t <= p
// with t > p - window (or any, window 0) or t < sinks.
//
// One pass with a running maximum and sum over tiles of 64 slots. A block takes
// 128 queries of one head, each of its four waves 32 of them, as
//   S^T [32 slots, 32 queries] = K Q^T,  O^T [dim, 32 queries] += V^T P^T
// on 32 x 32 matrix instructions. A lane holds one query's column of S^T, so the
// softmax needs no exchange between lanes but one (the two halves of the
// column), and only when the running maximum is raised, which waits until a
// score passes it by 2^8. K rows are assigned to the rows of S^T such that a
// lane's scores are the P^T operand of the second product as they stand.
//
// K and V go from memory to LDS by DMA as they lie (a page's rows of a head are
// contiguous), the next tile while the current one is used, and no registers
// hold staged data. The chunks of 16 bytes are swizzled on the memory side such
// that the operand reads meet no bank twice. V's operand needs 8 slots of one
// element per lane: transpose reads give it. Two blocks share a compute unit:
// the matrix products of one run beside the softmax of the other (three blocks with
// tiles of 32 slots take 365 us where this takes 285; 64 queries a wave do not fit the
// registers).
//
// Two 2048-token sequences of 96 heads of 128: 284 us, 726 TFLOP/s of the pairs that are
// seen; two chunks of 4096 tokens with a window of 2048, 32 heads on 8: 317 us, 857. A tile of
// 128 queries and 64 slots takes 4.1 ns of the whole card (1022 TFLOP/s); the rest, about 85
// us of the first, goes with the number of blocks: their first reads and last stores, and the
// tiles on the diagonal, half of which is masked.
#include <algorithm>

#include "kv.h"

namespace gptq {
namespace {

constexpr int kQ = 128;     // queries per block
constexpr int kT = 64;      // slots per tile
constexpr int kRing = 2;    // tiles in LDS
constexpr int kLeast = 4;   // tiles per block where they are split
constexpr int kW = 64;      // queries at a time in the weights' kernel
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

// Sum over the lanes up to this one (row shifts, then the rows' last lanes broadcast).
__device__ __forceinline__ int scan64(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast 15, 31
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// The ragged batch as pieces of kQ queries (or, SLOTS, its sequences' slots as pieces of kQ of
// them), and where piece t lies: of up to 64 sequences (one per lane) the pieces with the highest
// number in their sequence, which see most (the lowest, which most queries see), come first; of
// more, the sequences in order, each from its end (its start).
template <bool SLOTS>
struct Pieces {
  const KvView& c;
  const int32_t* cu;
  int n_rows, total, most;
  int c0, n, len, own;  // of sequence `lane`: first row, queries, slots, pieces
  __device__ __forceinline__ void load(int s) {
    c0 = n = len = 0;
    if (s < c.n_seqs) {
      len = c.len(s);
      c0 = cu[s];
      const int c1 = cu[s + 1];
      // rows outside the q tensor are not there, whatever cu says
      n = c0 >= 0 && c1 > c0 && c1 <= n_rows ? c1 - c0 : 0;
    }
    own = ((SLOTS && n > 0 ? len : n) + kQ - 1) / kQ;
  }
  __device__ __forceinline__ Pieces(const KvView& c, const int32_t* cu, int n_rows) : c(c), cu(cu), n_rows(n_rows) {
    const int lane = threadIdx.x & 63;
    total = 0;
    for (int base = 0; base < c.n_seqs; base += 64) {
      load(base + lane);
      total += __builtin_amdgcn_readlane(scan64(own), 63);
    }
    if (!SLOTS) total = min(total, n_rows / kQ + c.n_seqs);  // (more only if cu is not ascending)
    most = own;
    for (int o = 32; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o));
  }
  int b, i0, n_b, row0, len_b;
  __device__ __forceinline__ void find(int t) {
    const int lane = threadIdx.x & 63;
    int at = 0, base = 0, piece = 0;
    if (c.n_seqs <= 64) {
      // the highest level with more than t pieces at or above it
      int lo = 0, hi = most;  // holds at lo, not at hi
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__builtin_amdgcn_readlane(scan64(max(own - mid, 0)), 63) > t)
          lo = mid;
        else
          hi = mid;
      }
      const int above = __builtin_amdgcn_readlane(scan64(max(own - lo - 1, 0)), 63);
      const bool in = own > lo;
      const int rank = scan64(in ? 1 : 0) - 1;
      at = __builtin_ctzll(__ballot(in && rank == t - above));
      piece = lo;
    } else {
      int before = 0;
      for (;; base += 64) {
        load(base + lane);
        const int incl = scan64(own), start = before + incl - own;
        const uint64_t hit = __ballot(t >= start && t < start + own);
        if (hit || base + 64 >= c.n_seqs) {
          at = hit ? __builtin_ctzll(hit) : 0;
          piece = __shfl(own, at) - 1 - (t - __shfl(start, at));
          break;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
      }
    }
    b = __builtin_amdgcn_readfirstlane(base + at);
    if (SLOTS) piece = __shfl(own, at) - 1 - piece;
    i0 = __builtin_amdgcn_readfirstlane(piece * kQ);
    n_b = __builtin_amdgcn_readfirstlane(__shfl(n, at));
    row0 = __builtin_amdgcn_readfirstlane(__shfl(c0, at));
    len_b = __builtin_amdgcn_readfirstlane(__shfl(len, at));
  }
};

// Slot (within 32) of row m of S^T: rows 8 q + 4 f + r belong to lane half f.
__device__ __forceinline__ int slot_of_row(int m) {
  return 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);
}

// 16 bytes per lane from base + off (base wave-uniform) to LDS [lds + 16 lane, ...),
// see dma16 for the M0 handling.
__device__ __forceinline__ void dma16_from(const void* base, uint32_t off, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, %3\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}
// The same, 4 bytes per lane.
__device__ __forceinline__ void dma4_from(const void* base, uint32_t off, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %2, %3\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}
// Eight rows of K and of V in one go, N transfers each, 1 KB apart in LDS.
template <int N>
__device__ __forceinline__ void dma16_octet(const void* kb, const void* vb, const uint32_t (&ok)[N],
                                            const uint32_t (&ov)[N], uint32_t lds_k, uint32_t lds_v) {
  uint32_t saved;
  if constexpr (N == 1) {
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %3, %5\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %4, %6\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds_k), "s"(lds_v), "v"(ok[0]), "v"(ov[0]), "s"(kb), "s"(vb)
        : "memory");
  } else {
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %5, %9\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %6, %9\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %7, %10\n\t"
        "s_mov_b32 m0, %4\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %8, %10\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds_k), "s"(lds_k + 1024), "s"(lds_v), "s"(lds_v + 1024), "v"(ok[0]), "v"(ok[1]), "v"(ov[0]), "v"(ov[1]),
          "s"(kb), "s"(vb)
        : "memory");
  }
}

// The lowest n bits (none below 0, all from 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Eight bits for each of the lowest four.
__device__ __forceinline__ uint32_t octet_bits(uint32_t b) {
  return ((b & 1) ? 0xffu : 0u) | ((b & 2) ? 0xff00u : 0u) | ((b & 4) ? 0xff0000u : 0u) | ((b & 8) ? 0xff000000u : 0u);
}

// A wave-uniform value the compiler cannot see to be one, in scalar registers.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uni(int64_t x) {
  return ((int64_t)uni((int)(x >> 32)) << 32) | (uint32_t)uni((int)x);
}

__device__ __forceinline__ short4v lds_tr(const GPTQ_LDS char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((GPTQ_LDS short4v*)p);
}

// LDS: per tile K then V, kT rows of kPitch bytes.
template <int QS>
struct Ring {
  static constexpr int kPitch = QS <= 4 ? 128 : 256, kLpr = kPitch / 16;  // lanes (16 bytes) per row
  static constexpr int kHalf = kT * kPitch, kTileBytes = 2 * kHalf, kBytes = kRing * kTileBytes;
  // where chunk c (16 bytes) of row r lies in its row: c ^ these
  static constexpr __device__ int fk(int r) { return QS <= 4 ? (r >> 1) & 7 : r & 15; }
  static constexpr __device__ int fv(int r) { return QS <= 4 ? 4 * ((r >> 1) & 1) : 4 * (r & 3); }
};

// What a block leaves: its rows of out; with them the rows' log2 of the sum of 2^score in
// lse [n_heads][n_tokens] (the weights' kernel reads 64 rows of one head at a time); or, where
// a piece's tiles are split over n_splits blocks, the unnormalized sums with their maximum and
// weight in parts [n_tokens][n_heads][n_splits].
constexpr int kOut = 0, kOutLse = 1, kParts = 2;

// QS: steps of 16 along the head for the scores (16 QS >= dim).
template <typename T, int QS, int MODE>
__global__ __launch_bounds__(256, 2) void prompt_kernel(KvView c, KvAttnArgs a, const int32_t* cu, int n_rows,
                                                        float* lse, SplitWs parts) {
  using KT = KvType<T>;
  using x8 = typename KT::x8;
  using R = Ring<QS>;
  constexpr int NO = (QS + 1) / 2;
  constexpr int kRows = 64 / R::kLpr, kDma = 8 / kRows;  // rows per transfer, transfers per octet
  constexpr uint32_t kExp = __is_same(T, half_t) ? 0x7c00u : 0x7f80u;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ uint32_t odd[4][2];  // by tile modulo 4, a bit per slot: its values hold an infinity or NaN
  const GPTQ_LDS char* lds = (const GPTQ_LDS char*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  Pieces<false> at(c, cu, n_rows);
  // All heads' pieces, head by head, in eight parts, one for each XCD (neighbours in a head
  // share its L2); the blocks that are too many come last.
  const int n_splits = MODE == kParts ? parts.n_splits : 1;
  const int real = at.total * a.n_heads * n_splits, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  if (slot >= real / 8 + (xcd < real % 8 ? 1 : 0)) return;
  int item = xcd * (real / 8) + min(xcd, real % 8) + slot;
  const int split = MODE == kParts ? item % n_splits : 0;
  if constexpr (MODE == kParts) item /= n_splits;
  const int h = uni(item / at.total);
  at.find(item - h * at.total);
  const bool exact = c.dim == 16 * QS;
  const int kvh = h / (a.n_heads / c.n_kv);
  // (opaque, as a per-lane value: as a scalar the compiler unrolls what hangs on it into more
  // registers than there are)
  int p0 = at.len_b - at.n_b + at.i0;                          // position of the block's first query
  asm volatile("" : "+v"(p0));
  const int rows = at.n_b - at.i0 < kQ ? at.n_b - at.i0 : kQ;  // its queries
  const int first = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
  const int end = p0 + rows > 0 ? p0 + rows : 0;
  Tiles tl(end, first < end ? first : end, a.sinks);
  tl.n = uni(tl.n);
  tl.sink_tiles = uni(tl.sink_tiles);
  tl.jump = uni(tl.jump);
  tl.total = uni(tl.total);
  const int32_t* table = c.table + (int64_t)at.b * c.ld_table;
  const int chunks = c.dim >> 3;

  // a negative scale is the queries' sign; a zero one is next to it (equal weights either way)
  const float sc = fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1e-30f), raise = kRaise / sc;
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
  const int qi = wave * 32 + col, pos = p0 + qi;  // this lane's query
  x8 q[QS];
  {
    const T* qp = (const T*)a.q + (int64_t)(at.row0 + at.i0 + (qi < rows ? qi : 0)) * a.ldq + (int64_t)h * c.dim;
#pragma unroll
    for (int i = 0; i < QS; ++i) {
      const int ch = 2 * i + half;
      const bool ok = ch < chunks;
      const uint4v z = *(const uint4v*)(qp + 8 * (ok ? ch : 0)) ^ (uint4v){flip, flip, flip, flip};
      q[i] = __builtin_bit_cast(x8, (uint4v){ok ? z[0] : 0u, ok ? z[1] : 0u, ok ? z[2] : 0u, ok ? z[3] : 0u});
    }
  }
  float16v o[NO];
#pragma unroll
  for (int i = 0; i < NO; ++i) o[i] = (float16v){0};
  float m = -INFINITY, lsum = 0.0f;  // largest score seen, before the scale; sum of this lane's weights

  // Tile numbers. Those before sink_tiles are always gone through slot by slot; behind them
  // this wave (queries at w0 .. w1) sees something of the tiles [vis_lo, vis_hi) (and of
  // earlier ones that still hold sinks); every query
  // of the block sees all of [all_lo, all_hi).
  const int w0 = p0 + wave * 32, w1 = w0 + 31 < end - 1 ? w0 + 31 : end - 1;
  const int to_s = tl.sink_tiles - tl.jump;  // tile number of slot 0, were there no gap
  const int all_hi = to_s + ((p0 - kT + 1) >> 6) + 1;
  int all_lo = tl.sink_tiles, vis_lo = 0, vis_hi = to_s + (w1 >> 6) + 1;
  if (a.window > 0) {
    const int alo = to_s + ((p0 + rows - 1 - a.window) >> 6) + 1;
    if (alo > all_lo) all_lo = alo;
    vis_lo = to_s + ((w0 - a.window - kT + 1) >> 6) + 1;
  }
  const bool idle = w0 >= end || w1 < 0;  // a wave without queries, or whose queries stand before slot 0
  auto hidden = [&](int s) __attribute__((always_inline)) {
    return idle || (s >= tl.sink_tiles && ((s < vis_lo && tl.slot0(s) >= a.sinks) || s >= vis_hi));
  };

  // this wave's 16 rows of every tile: two octets
  const int lrow = lane / R::kLpr, lpos = lane % R::kLpr;
  uint32_t off_k[2][kDma], off_v[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
#pragma unroll
    for (int oc = 0; oc < 2; ++oc) {
      const int r = 8 * oc + kRows * i + lrow, ch = lpos ^ R::fk(r);
      off_k[oc][i] = ((r & 7) * c.dim + (ch < chunks ? ch : 0) * 8) * 2;
    }
    const int ch = lpos ^ R::fv(lrow);
    off_v[i] = ((kRows * i + lrow) * c.dim + (ch < chunks ? ch : 0) * 8) * 2;
  }
  // dim = 16 QS: no product reads a chunk behind the head's end, and what lands there is not
  // looked at. Otherwise these chunks stay cleared.
  const T* kb = (const T*)c.k + (int64_t)kvh * c.page_size * c.dim;
  const T* vb = (const T*)c.v + (int64_t)kvh * c.page_size * c.dim;
  // pages of the octets of eight tiles, one per lane
  auto pages = [&](int s8) __attribute__((always_inline)) {
    const int s = 8 * s8 + (lane >> 3), t = tl.slot0(s) + 8 * (lane & 7);
    return s < tl.total && t < tl.n ? table[t >> c.page_shift] : -1;
  };
  auto stage = [&](int s, int pg) __attribute__((always_inline)) {
    const uint32_t to = lds0 + (s & 1) * R::kTileBytes + 16 * wave * R::kPitch;
    const int row0 = tl.slot0(s) + 16 * wave;
#pragma unroll
    for (int oc = 0; oc < 2; ++oc) {
      const int p = __builtin_amdgcn_readlane(pg, 8 * (s & 7) + 2 * wave + oc);
      const uint32_t to_oc = to + 8 * oc * R::kPitch;
      if ((uint32_t)p < (uint32_t)c.n_pages) {
        const int64_t from = uni((int64_t)p * c.page_stride + ((row0 + 8 * oc) & (c.page_size - 1)) * c.dim);
        if (exact) {
          dma16_octet<kDma>(kb + from, vb + from, off_k[oc], off_v, to_oc, to_oc + R::kHalf);
        } else {
          int lp = lpos, chunks = c.dim >> 3;
          asm volatile("" : "+v"(lp));
          asm volatile("" : "+s"(chunks));
#pragma unroll
          for (int i = 0; i < kDma; ++i) {
            if ((lp ^ R::fk(8 * oc + kRows * i + lrow)) < chunks) dma16_from(kb + from, off_k[oc][i], to_oc + 1024 * i);
            if ((lp ^ R::fv(lrow)) < chunks) dma16_from(vb + from, off_v[i], to_oc + 1024 * i + R::kHalf);
          }
        }
      } else {
        // no such slots: nothing may reach the second product from here
        for (int i = 0; i < kDma; ++i)
          *(GPTQ_LDS uint4v*)(lds + (to_oc - lds0) + 1024 * i + R::kHalf + 16 * lane) = (uint4v){0, 0, 0, 0};
      }
    }
  };
  // In a tile that is hidden in part from some query, a value that is not finite must not
  // reach the queries that do not see its slot (0 x NaN): each wave looks through its own
  // rows, replaces these by 0 and notes the slots; the queries that see them get them
  // afterwards.
  auto clean = [&](int s) __attribute__((always_inline)) {
    const int t0 = tl.slot0(s);
    GPTQ_LDS char* v = (GPTQ_LDS char*)lds + (s & 1) * R::kTileBytes + R::kHalf + 16 * wave * R::kPitch + 16 * lane;
    typedef unsigned short u2 __attribute__((ext_vector_type(2)));
    u2 most = (u2){0, 0};  // largest magnitude, as bits
#pragma unroll
    for (int i = 0; i < 2 * kDma; ++i) {
      const uint4v x = *(GPTQ_LDS uint4v*)(v + 1024 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = x[e] & 0x7fff7fffu;
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u2, w));
      }
    }
    if (!__any(most[0] >= kExp || most[1] >= kExp)) return;
    for (int i = 0; i < 2 * kDma; ++i) {
      GPTQ_LDS uint4v* at_v = (GPTQ_LDS uint4v*)(v + 1024 * i);
      const uint4v x = *at_v;
      uint4v y;
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = (x[e] & kExp) == kExp ? 0u : x[e] & 0xffffu;
        const uint32_t hi = ((x[e] >> 16) & kExp) == kExp ? 0u : x[e] & 0xffff0000u;
        y[e] = lo | hi;
      }
      if (y[0] != x[0] || y[1] != x[1] || y[2] != x[2] || y[3] != x[3]) {
        *at_v = y;
        const int k = 16 * wave + kRows * i + lrow;
        if (t0 + k < tl.n && (lpos ^ R::fv(lrow)) < chunks) atomicOr(&odd[s & 3][k >> 5], 1u << (k & 31));
      }
    }
  };
  // bit k: this lane's query sees slot t0 + k
  auto seen = [&](int t0) __attribute__((always_inline)) {
    uint32_t see = low_bits(pos + 1 - t0);
    if (a.window > 0) see &= ~low_bits(pos + 1 - a.window - t0) | low_bits(a.sinks - t0);
    return see;
  };

  // operand addresses within a tile
  const int krow = slot_of_row(col);
  uint32_t at_k[QS], at_v[NO];
#pragma unroll
  for (int i = 0; i < QS; ++i) at_k[i] = krow * R::kPitch + (((2 * i + half) ^ R::fk(krow)) * 16);
  {
    const int j = lane & 15, r = 8 * half + (j >> 2);
#pragma unroll
    for (int i = 0; i < NO; ++i)
      at_v[i] =
          R::kHalf + r * R::kPitch + (((4 * i + 2 * ((lane >> 4) & 1) + ((j & 3) >> 1)) ^ R::fv(r)) * 16) + 8 * (j & 1);
  }
  // Operands are read from LDS well before the products that take them: a read takes longer
  // than a product, and left to itself the compiler waits for each in turn.
  struct Keys {
    x8 f[QS];
  };
  struct Values {
    x8 f[2][NO];
  };
  auto keys = [&](const GPTQ_LDS char* b, int u) __attribute__((always_inline)) {
    Keys k;
#pragma unroll
    for (int i = 0; i < QS; ++i) k.f[i] = *(const GPTQ_LDS x8*)(b + at_k[i] + 32 * u * R::kPitch);
    return k;
  };
  auto scores = [&](const Keys& k) __attribute__((always_inline)) {
    float16v x = (float16v){0};
#pragma unroll
    for (int i = 0; i < QS; ++i) x = KT::mfma32(k.f[i], q[i], x);
    return x;
  };
  auto mask = [&](float16v& x, int t0, uint32_t page_bits) __attribute__((always_inline)) {
    asm volatile("" : "+v"(t0));  // (or its arithmetic is taken out in front of the branch to here)
    const uint32_t see = (seen(t0) & page_bits) >> (8 * half);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint32_t keep = (uint32_t)((int)(see << (31 - 16 * (r >> 3) - (r & 7))) >> 31);
      const float v = x[r];  // (a bit cast of the vector's element itself would take element 0)
      x[r] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, v) & keep) | (0xff800000u & ~keep));
    }
  };
  auto softmax = [&](const float16v& x, float base, x8(&pf)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float p = __builtin_amdgcn_exp2f(fmaf(x[r], sc, -base));
      lsum += p;
      // P in the cache's type: its rounding (2^-11 or 2^-8 of each weight at most) averages
      // out over the slots and stays below that of the output
      pf[r >> 3][r & 7] = (T)p;
    }
  };
  auto values = [&](const GPTQ_LDS char* b, int u) __attribute__((always_inline)) {
    Values v;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const GPTQ_LDS char* p = b + at_v[i] + (32 * u + 16 * k) * R::kPitch;
        const short4v lo = lds_tr(p), hi = lds_tr(p + 4 * R::kPitch);
        v.f[k][i] = __builtin_bit_cast(x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    return v;
  };
  auto weigh = [&](const Values& v, const x8(&pf)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NO; ++i) o[i] = KT::mfma32(v.f[k][i], pf[k], o[i]);
  };
  // rare: values of a tile that are not finite, for the queries that see them (their weight is
  // positive, so the sum is what the value is)
  auto add_odd = [&](int t0, uint32_t bits) __attribute__((always_inline)) {
    int at0 = t0, dim = c.dim;
    asm volatile("" : "+v"(at0));
    asm volatile("" : "+s"(dim));
    const uint32_t see = seen(at0);
    for (int k = 0; k < 32; ++k) {
      if (!((bits >> k) & 1)) continue;
      const int t = t0 + k, pg = t < tl.n ? table[t >> c.page_shift] : -1;
      if (!c.page_ok(pg)) continue;
      const T* vp = vb + (int64_t)pg * c.page_stride + (int64_t)(t & (c.page_size - 1)) * c.dim + 4 * half;
#pragma unroll
      for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          typedef T x4 __attribute__((ext_vector_type(4)));
          x4 z = (x4){0, 0, 0, 0};
          if (32 * i + 8 * r4 < dim) z = *(const x4*)(vp + 32 * i + 8 * r4);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            o[i][4 * r4 + r] += ((see >> k) & 1) && !(__builtin_fabsf((float)z[r]) < INFINITY) ? (float)z[r] : 0.0f;
          asm volatile("" ::: "memory");  // one load at a time: no registers for more
        }
    }
  };

  // this block's tiles
  const int per = MODE == kParts ? max(kLeast, (tl.total + n_splits - 1) / n_splits) : tl.total;
  const int s0 = uni(split * per), s1 = uni(min(s0 + per, tl.total));
  if (s0 < s1) {
    if (tid < 8) odd[tid >> 1][tid & 1] = 0u;
    // elements between the head's end and the row's are never transferred: zeros once and for all
    if (!exact)
      for (int i = tid; i < R::kBytes / 16; i += 256) *(GPTQ_LDS uint4v*)(lds + 16 * i) = (uint4v){0, 0, 0, 0};
    int pg = pages(s0 >> 3), pg_next = pages((s0 >> 3) + 1);
    __syncthreads();
    stage(s0, pg);
    // raises the running maximum to those of x and y if a score is far above it
    auto raise_to = [&](const float16v& x, const float16v& y) __attribute__((always_inline)) {
      float top = fmaxf(x[0], y[0]);
#pragma unroll
      for (int r = 1; r < 16; ++r) top = fmaxf(fmaxf(top, x[r]), y[r]);
      if (__any(top > m + raise)) {
        const float nm = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)));
        const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - nm) * sc);
        m = nm;
        lsum *= f;
#pragma unroll
        for (int i = 0; i < NO; ++i) o[i] *= f;
      }
      return m == -INFINITY ? 0.0f : m * sc;
    };
    for (int s = s0; s < s1; ++s) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // this wave's rows of tile s have landed
      const bool in_part = s < all_lo || s >= all_hi;
      if (in_part) clean(s);
      if (tid < 2) odd[(s + 2) & 3][tid] = 0u;  // read last by tile s - 2, written next two barriers from here
      lds_barrier();  // tile s is in LDS for every wave, tile s - 1 is read by none
      const uint64_t good = __ballot(c.page_ok(pg));
      const uint32_t on_page = (uint32_t)(good >> (8 * (s & 7))) & 0xffu;
      if ((s & 7) == 7) {
        pg = pg_next;
        pg_next = pages((s >> 3) + 2);
      }
      if (s + 1 < s1) stage(s + 1, pg);
      const GPTQ_LDS char* b = lds + (s & 1) * R::kTileBytes;
      x8 px[2], py[2];
      if (!in_part && on_page == 0xffu) {
        // every query sees all of it: one straight piece of code
        const Keys k0 = keys(b, 0), k1 = keys(b, 1);
        __builtin_amdgcn_sched_barrier(0);
        float16v x = scores(k0), y = scores(k1);
        const float base = raise_to(x, y);
        const Values v0 = values(b, 0);
        __builtin_amdgcn_sched_barrier(0);
        softmax(x, base, px);
        __builtin_amdgcn_sched_barrier(0);
        const Values v1 = values(b, 1);
        weigh(v0, px);
        softmax(y, base, py);
        weigh(v1, py);
      } else if (!hidden(s)) {
        const int t0 = tl.slot0(s);
        float16v x = scores(keys(b, 0)), y = scores(keys(b, 1));
        mask(x, t0, octet_bits(on_page));
        mask(y, t0 + 32, octet_bits(on_page >> 4));
        const float base = raise_to(x, y);
        softmax(x, base, px);
        weigh(values(b, 0), px);
        softmax(y, base, py);
        weigh(values(b, 1), py);
        const uint32_t o0 = uni((int)odd[s & 3][0]), o1 = uni((int)odd[s & 3][1]);
        if (o0) add_odd(t0, o0);
        if (o1) add_odd(t0 + 32, o1);
      }
    }
  }

  lsum += __shfl_xor(lsum, 32);
  if (qi < rows) {
    int dim = c.dim;
    asm volatile("" : "+s"(dim));  // (or sixteen comparisons with it are kept from piece to piece)
    const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
    const int64_t row = at.row0 + at.i0 + qi;
    if constexpr (MODE == kParts) {
      const int64_t part = (row * a.n_heads + h) * n_splits + split;
      float* pp = parts.o + part * dim;
      // (a maximum of -infinity says that the sums are not there)
#pragma unroll
      for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int e = 32 * i + 8 * r4 + 4 * half;
          if (s0 < s1 && e < dim)
            *(float4v*)(pp + e) = (float4v){o[i][4 * r4], o[i][4 * r4 + 1], o[i][4 * r4 + 2], o[i][4 * r4 + 3]};
        }
      if (half == 0) {
        parts.ml[2 * part] = m == -INFINITY ? -INFINITY : m * sc;
        parts.ml[2 * part + 1] = lsum;
      }
      return;
    }
    T* op = (T*)a.out + row * a.ldo + (int64_t)h * c.dim;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int e = 32 * i + 8 * r4 + 4 * half;
        if (e < dim) {
          typedef T x4 __attribute__((ext_vector_type(4)));
          x4 z;
#pragma unroll
          for (int r = 0; r < 4; ++r) z[r] = lsum == 0.0f ? (T)0.0f : (T)(o[i][4 * r4 + r] * inv);
          *(x4*)(op + e) = z;
        }
      }
    if constexpr (MODE == kOutLse) {
      // a row without a weight: +infinity, so that 2^(score - lse) is 0
      if (half == 0)
        lse[(int64_t)h * n_rows + row] = lsum == 0.0f ? INFINITY : (m == -INFINITY ? 0.0f : m * sc) + log2f(lsum);
    }
  }
}

// weights[b][g][t] += sum over the queries of b and the heads of group g of
// 2^(score - lse): the scores once more (half the products of the attention),
// as S^T tiles whose rows, the slots, are summed along. One block owns 128 slots
// of one key head (a wave 32, its keys in registers) and goes over all queries
// that may see them, 64 at a time through LDS (DMA, the next 64 while these are
// used; a third buffer costs one of the four blocks on a compute unit: 61 us instead of 57), so
// every sum has one owner and one order. Bound by the vector unit, which is busy 70 % of
// the time: per score an exponential (16 cycles a wave), a multiply-add and a sum,
// against 2 QS cycles of products. Six OPT-2.7B prompts of 65 to 1999 tokens, 32
// heads of 80: 53 us; two of 2048, 96 heads: 116.
template <typename T, int QS>
__global__ __launch_bounds__(256, 2) void prompt_weights_kernel(KvView c, KvAttnArgs a, const int32_t* cu, int n_rows,
                                                               const float* lse) {
  using KT = KvType<T>;
  using x8 = typename KT::x8;
  using R = Ring<QS>;
  constexpr int kRows = 64 / R::kLpr, kDma = 16 / kRows, kBytes = kW * R::kPitch;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kBytes];
  __shared__ float lse_of[4][2][kW];  // of each wave's own transfer
  const GPTQ_LDS char* lds = (const GPTQ_LDS char*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  Pieces<true> at(c, cu, n_rows);
  const int kvh = blockIdx.x % c.n_kv;  // (with 8 n heads, those of an XCD are its own)
  if ((int)(blockIdx.x / c.n_kv) >= at.total) return;
  at.find(blockIdx.x / c.n_kv);
  const int b = at.b, r0 = at.row0, len = at.len_b, n_b = at.n_b, t00 = at.i0;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int t0 = t00 + 32 * wave;
  const int group = a.n_heads / c.n_kv, chunks = c.dim >> 3;
  const int32_t* table = c.table + (int64_t)b * c.ld_table;
  const float sc = fmaxf(__builtin_fabsf(a.scale) * kLog2e, 1e-30f);
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;

  float16v acc = (float16v){0};
  // queries at positions p >= t, and, unless a slot of the block is a sink, p < t + window
  const int base = len - n_b;  // position of query 0
  int i_lo = t00 - base, i_hi = n_b;
  if (i_lo < 0) i_lo = 0;
  if (a.window > 0 && t00 >= a.sinks) {
    const int64_t last = (int64_t)t00 + 127 + a.window - base;  // first query that no longer sees slot t00 + 127
    if (last < i_hi) i_hi = (int)last;
  }
  i_lo &= ~(kW - 1);
  const int steps = i_hi > i_lo ? (i_hi - i_lo + kW - 1) / kW : 0, total = steps * group;

  // this wave's 16 rows of every 64 queries; rows behind the last repeat it (and are masked)
  const int lrow = lane / R::kLpr, lpos = lane % R::kLpr;
  const bool exact = c.dim == 16 * QS;
  const T* qb = (const T*)a.q + (int64_t)r0 * a.ldq + (int64_t)kvh * group * c.dim;
  // 64 queries of one head: the head and the first query
  struct At {
    int hh, i;
  };
  auto after = [&](At p) __attribute__((always_inline)) {
    return p.i + kW < i_hi ? At{p.hh, p.i + kW} : At{p.hh + 1, i_lo};
  };
  uint32_t off[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int r = kRows * i + lrow, ch = lpos ^ R::fk(r);
    off[i] = ((uint32_t)r * (uint32_t)a.ldq + (ch < chunks ? ch : 0) * 8) * 2;
  }
  auto stage = [&](int buf, At p) __attribute__((always_inline)) {
    const int i0 = p.i + 16 * wave;
    const uint32_t to = lds0 + buf * kBytes + 16 * wave * R::kPitch;
    const T* from = qb + uni((int64_t)(i0 < n_b ? i0 : n_b - 1) * a.ldq + (int64_t)p.hh * c.dim);
    const float* from_lse = lse + uni((int64_t)(kvh * group + p.hh) * n_rows + r0 + p.i);
    const uint32_t to_lse = (uint32_t)(uintptr_t)(const GPTQ_LDS char*)&lse_of[wave][buf][0];
    if (exact && p.i + kW <= n_b) {
#pragma unroll
      for (int i = 0; i < kDma; ++i) dma16_from(from, off[i], to + 1024 * i);
      dma4_from(from_lse, 4 * lane, to_lse);
    } else {
      const int left = i0 < n_b ? n_b - 1 - i0 : 0, left_lse = n_b - 1 - p.i;  // last rows that are there
#pragma unroll
      for (int i = 0; i < kDma; ++i) {
        const int r = kRows * i + lrow, ch = lpos ^ R::fk(r);
        const uint32_t of = (uint32_t)((r < left ? r : left) * (uint32_t)a.ldq + (ch < chunks ? ch : 0) * 8) * 2;
        if (exact || ch < chunks) dma16_from(from, of, to + 1024 * i);
      }
      dma4_from(from_lse, 4 * (lane < left_lse ? lane : left_lse), to_lse);
    }
  };
  uint32_t at_q[QS];
#pragma unroll
  for (int i = 0; i < QS; ++i) at_q[i] = col * R::kPitch + (((2 * i + half) ^ R::fk(col)) * 16);
  struct Queries {
    x8 f[QS];
  };
  auto queries = [&](const GPTQ_LDS char* buf, int u) __attribute__((always_inline)) {
    Queries z;
#pragma unroll
    for (int i = 0; i < QS; ++i) z.f[i] = *(const GPTQ_LDS x8*)(buf + at_q[i] + 32 * u * R::kPitch);
    return z;
  };

  At now = {0, i_lo};
  if (total > 0) {
    if (!exact) {
      for (int i = tid; i < 2 * kBytes / 16; i += 256) *(GPTQ_LDS uint4v*)(lds + 16 * i) = (uint4v){0, 0, 0, 0};
      __syncthreads();
    }
    stage(0, now);
  }
  // While these are under way: this wave's keys, and the weight that this lane will add to (at
  // the end, row r's sum is in lanes 2 r and 2 r + 1).
  const int r = col >> 1, tw = t0 + 16 * (r >> 3) + 8 * half + (r & 7), tk = t0 + slot_of_row(col);
  const int pg = tk < len ? table[tk >> c.page_shift] : -1, pw = tw < len ? table[tw >> c.page_shift] : -1;
  float* const wt = a.weights + ((int64_t)b * c.n_kv + kvh) * a.ldw + (c.page_ok(pw) ? tw : t00);
  const float old = *wt;
  x8 k[QS];
  {
    const T* kp =
        (const T*)c.k + (c.page_ok(pg) ? c.head_base(pg, kvh) + (int64_t)(tk & (c.page_size - 1)) * c.dim : 0);
#pragma unroll
    for (int i = 0; i < QS; ++i) {
      const int ch = 2 * i + half;
      const bool ok = ch < chunks && c.page_ok(pg);
      const uint4v z = *(const uint4v*)(kp + 8 * (ok ? ch : 0)) ^ (uint4v){flip, flip, flip, flip};
      k[i] = __builtin_bit_cast(x8, (uint4v){ok ? z[0] : 0u, ok ? z[1] : 0u, ok ? z[2] : 0u, ok ? z[3] : 0u});
    }
  }
  auto scores = [&](const Queries& z) __attribute__((always_inline)) {
    float16v x = (float16v){0};
#pragma unroll
    for (int i = 0; i < QS; ++i) x = KT::mfma32(k[i], z.f[i], x);
    return x;
  };

  for (int s = 0; s < total; ++s) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // this wave's rows of step s have landed
    lds_barrier();  // for every wave, and step s - 1 is read by none
    const int i0 = now.i, lowest = base + i0;
    now = after(now);
    if (s + 1 < total) stage((s + 1) & 1, now);
    const GPTQ_LDS char* buf = lds + (s & 1) * kBytes;
    const float l0 = lse_of[wave][s & 1][col], l1 = lse_of[wave][s & 1][32 + col];
    if (t0 + 31 <= lowest && i0 + kW <= n_b &&
        (a.window <= 0 || t0 > lowest + kW - 1 - a.window || t0 + 32 <= a.sinks)) {
      // every query sees all of this wave's slots: one straight piece of code
      const Queries z0 = queries(buf, 0), z1 = queries(buf, 1);
      __builtin_amdgcn_sched_barrier(0);
      const float16v x = scores(z0), y = scores(z1);
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] += __builtin_amdgcn_exp2f(fmaf(x[r], sc, -l0));
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] += __builtin_amdgcn_exp2f(fmaf(y[r], sc, -l1));
    } else {
      for (int u = 0; u < 2; ++u) {
        const int low = lowest + 32 * u;  // position of the first of 32 queries
        if (low + 31 < t0 || (a.window > 0 && t0 + 31 <= low - a.window && t0 >= a.sinks)) continue;  // none sees any
        const float16v x = scores(queries(buf, u));
        const float l = u ? l1 : l0;
        const int pos = low + col;
        uint32_t see = low_bits(pos + 1 - t0);
        if (a.window > 0) see &= ~low_bits(pos + 1 - a.window - t0) | low_bits(a.sinks - t0);
        if (i0 + 32 * u + col >= n_b) see = 0;
        see >>= 8 * half;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float p = __builtin_amdgcn_exp2f(fmaf(x[r], sc, -l));
          acc[r] += (see >> (16 * (r >> 3) + (r & 7))) & 1 ? p : 0.0f;
        }
      }
    }
  }
  // Sums along the rows: at every step a lane passes on half of the sums it holds, so that
  // lanes 2 r and 2 r + 1 (of each half) end up with row r's, and one lane reads and writes each
  // weight.
#pragma unroll
  for (int n = 8, o = 16; n > 0; n >>= 1, o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float lo = acc[i], hi = acc[i + n];
      const bool up = col & o;
      acc[i] = (up ? hi : lo) + __shfl_xor(up ? lo : hi, o);
    }
  const float sum = acc[0] + __shfl_xor(acc[0], 1);
  if ((col & 1) == 0 && c.page_ok(pw)) *wt = old + sum;
}

int64_t pieces_of(const KvView& c, int64_t n_tokens, int64_t n_heads) {
  return (n_tokens / kQ + c.n_seqs) * n_heads;
}

// Blocks per piece. Few queries over a long cache are few pieces with many tiles: they are
// split until there are two blocks for each compute unit, at least kLeast tiles each (512
// queries, 8 heads of 128, 8512 slots: 184 us whole, 41 split; 128 queries, 32 heads, 30128
// slots: 637 and 95). A tile takes 1.3 us, with two blocks on a compute unit half as much again;
// partial results and their join cost three tiles' time, and one more per 7000 rows of them.
// Where that is more than what splitting saves, pieces stay whole (512 queries, 64 heads, 1012
// slots: 31 us whole, 38 split; 8512 slots: 184 and 165).
int64_t splits_of(const KvView& c, int64_t n_tokens, int64_t n_heads, int64_t window, int64_t sinks) {
  const int64_t cap = (int64_t)c.max_pages << c.page_shift, all = ceil_div(cap, kT);
  int64_t tiles = all;
  if (window > 0 && window < cap)
    tiles = std::min(all, ceil_div(std::min(sinks, cap), kT) + (window + kQ) / kT + 2);
  const int64_t pieces = c.n_seqs * ceil_div(ceil_div(n_tokens, c.n_seqs), kQ) * n_heads;  // were all of one length
  const int64_t s = std::min(512 / pieces, tiles / kLeast);
  if (s <= 1) return 1;
  const int64_t saved = tiles * (2 * s - (pieces * s > 256 ? 3 : 2)) / (2 * s);
  return saved < 3 + n_tokens * n_heads * s / 7000 ? 1 : s;
}

struct PromptWs {
  float* lse;
  SplitWs parts;
};
PromptWs layout(const KvView& c, int64_t n_tokens, int64_t n_heads, int64_t window, int64_t sinks, bool weights,
                void* ws, size_t* bytes) {
  PromptWs w{};
  const int64_t rows = n_tokens * n_heads;
  float* f = (float*)ws;
  size_t n = 0;
  w.parts.n_splits = (int)splits_of(c, n_tokens, n_heads, window, sinks);
  if (w.parts.n_splits > 1) {
    w.parts.o = f + n;
    n += (size_t)rows * w.parts.n_splits * c.dim;
    w.parts.ml = f + n;
    n += (size_t)rows * w.parts.n_splits * 2;
  }
  w.lse = f + n;
  if (weights) n += (size_t)rows;
  if (bytes) *bytes = n * sizeof(float);
  return w;
}

template <typename T, int QS, int MODE>
gptq_status_t launch_rows(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, float* lse,
                          const SplitWs& parts, hipStream_t st) {
  // at least the ragged batch's pieces; blocks in eights, one for each XCD
  const int64_t blocks = ceil_div(pieces_of(c, n_tokens, a.n_heads) * parts.n_splits, 8) * 8;
  if (blocks * 256 >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((prompt_kernel<T, QS, MODE>), dim3((unsigned)blocks), dim3(256), Ring<QS>::kBytes, st, c, a, cu,
                     (int)n_tokens, lse, parts);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <typename T, int QS>
gptq_status_t launch(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, const PromptWs& w,
                     hipStream_t st) {
  const int64_t cap = (int64_t)c.max_pages << c.page_shift, n_tiles = ceil_div(cap, 128);
  const int64_t wblocks = n_tiles * c.n_kv * c.n_seqs;
  if (wblocks * 256 >= (int64_t)1 << 32) return GPTQ_ERR_UNSUPPORTED;
  float* lse = w.lse;
  gptq_status_t rc;
  if (w.parts.n_splits > 1) {
    rc = launch_rows<T, QS, kParts>(c, a, cu, n_tokens, lse, w.parts, st);
    if (rc == GPTQ_OK) rc = kv_join_enqueue(c, a, w.parts, n_tokens, cu, a.weights ? lse : nullptr, st);
  } else {
    rc = a.weights ? launch_rows<T, QS, kOutLse>(c, a, cu, n_tokens, lse, w.parts, st)
                   : launch_rows<T, QS, kOut>(c, a, cu, n_tokens, lse, w.parts, st);
  }
  if (rc != GPTQ_OK || !a.weights) return rc;
  hipLaunchKernelGGL((prompt_weights_kernel<T, QS>), dim3((unsigned)wblocks), dim3(256), 0, st, c, a, cu,
                     (int)n_tokens, lse);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

// Steps along the head: 5 is OPT-2.7B's head of 80, which 6 would slow by a sixth.
template <typename T>
gptq_status_t prompt_enqueue(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens,
                             const PromptWs& w, hipStream_t st) {
  if (c.dim <= 64) return launch<T, 4>(c, a, cu, n_tokens, w, st);
  if (c.dim <= 80) return launch<T, 5>(c, a, cu, n_tokens, w, st);
  if (c.dim <= 96) return launch<T, 6>(c, a, cu, n_tokens, w, st);
  return launch<T, 8>(c, a, cu, n_tokens, w, st);
}

}  // namespace

size_t kv_prompt_workspace_bytes(const KvView& c, int64_t n_tokens, int64_t n_heads, int64_t window, int64_t sinks,
                                 bool weights) {
  size_t bytes = 0;
  layout(c, n_tokens, n_heads, window, sinks, weights, nullptr, &bytes);
  return bytes;
}

gptq_status_t kv_prompt_enqueue(const KvView& c, const KvAttnArgs& a, const int32_t* cu, int64_t n_tokens, void* ws,
                                hipStream_t st) {
  TraceScope tr(st, GPTQ_TRACE_KV_ATTENTION);
  const PromptWs w = layout(c, n_tokens, a.n_heads, a.window, a.sinks, a.weights != nullptr, ws, nullptr);
  return c.bf16 ? prompt_enqueue<bf16_t>(c, a, cu, n_tokens, w, st) : prompt_enqueue<half_t>(c, a, cu, n_tokens, w, st);
}

}  // namespace gptq
