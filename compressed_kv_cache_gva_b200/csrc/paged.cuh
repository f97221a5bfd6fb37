// Device helpers of the paged attention kernels: a sequence's query rows, the row
// blocks a kernel cuts the batch into, and the walk of one CTA over its pieces.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace gva {

// Order of a call's kernels on the stream.  A kernel waits for the work before it, then
// lets the next one launch.  The second kernel of a call that has two (`beside`) shares
// nothing with the first but its inputs: it launched after every CTA of the first had
// passed its wait, so those are in place, and it runs at the same time.  It waits for
// the first only before it ends, so that whoever waits for it has waited for both.
__device__ __forceinline__ void pdl_enter(const PagedArgs& a) {
  if (!a.beside) pdl_wait();
  pdl_trigger();
}
__device__ __forceinline__ void pdl_leave(const PagedArgs& a) {
  if (a.beside) pdl_wait();
}

// Query rows [r0, r0 + n) and cached length of sequence b; n = 0 where the sequence
// is inconsistent or belongs to the other kernel of the call.
struct SeqRows {
  int r0, n, L;
  bool bad;
};

__device__ __forceinline__ SeqRows seq_rows(const PagedArgs& a, int b) {
  SeqRows s;
  s.r0 = __ldg(a.q_start + b);
  const int r1 = __ldg(a.q_start + b + 1);
  s.L = __ldg(a.seq_len + b);
  // (a length above num_slots cannot be right, and would overflow token indices)
  s.bad = s.r0 < 0 || r1 < s.r0 || r1 > a.n_rows || r1 - s.r0 > a.max_new || s.L < 0 || s.L > a.num_slots;
  s.n = s.bad ? 0 : r1 - s.r0;
  const int cols = s.n * a.hpr;   // n_rows * H fits 32 bits
  if (cols <= a.lo_rows || cols > a.hi_rows) s.n = 0;
  return s;
}

// The batch by one warp (B <= 32): lane b holds sequence b and the units before it.
// No block barrier and no second look at the lengths, on the critical path of short calls
// (8 x 4096 decode 11.2 -> 10.6 us on the device).
constexpr int kLaneBatch = 32;
struct LaneBatch {
  SeqRows s;          // this lane's sequence (n = 0 past the batch)
  int before, units;  // exclusive prefix of the units; this sequence's
  long long total;
};
template <class F>
__device__ __forceinline__ LaneBatch lane_batch(const PagedArgs& a, F&& units_of) {
  LaneBatch t;
  const int lane = threadIdx.x & 31;
  t.s = SeqRows{0, 0, 0, false};
  if (lane < a.B) t.s = seq_rows(a, lane);
  const long long u = t.s.n > 0 ? units_of(t.s) : 0;
  long long x = u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  t.total = __shfl_sync(0xffffffffu, x, 31);
  const bool fits = t.total < (1ll << 31);
  t.before = fits ? (int)(x - u) : 0;
  t.units = fits ? (int)u : 0;
  return t;
}
__device__ __forceinline__ SeqRows shfl_rows(const SeqRows& s, int b) {
  return SeqRows{__shfl_sync(0xffffffffu, s.r0, b), __shfl_sync(0xffffffffu, s.n, b),
                 __shfl_sync(0xffffffffu, s.L, b), false};
}

// One CTA reports what is inconsistent in the batch (whole block).
__device__ inline void flag_bad_sequences(const PagedArgs& a) {
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const SeqRows s = seq_rows(a, b);
    if (s.bad || (s.L > 0 && (long long)a.max_pages * a.page < s.L))
      atomicOr(a.status, GVA_DEVERR_RANGE);
  }
}

// Cache row of position t of sequence b; num_slots (a row outside the cache: TMA reads
// zeros there) behind its end, or where the table is wrong (flagged).
__device__ __forceinline__ int slot_of(const PagedArgs& a, const int* row, int t, int L) {
  if (t >= L) return a.num_slots;
  const int col = t / a.page;
  int pg = -1;
  if (col < a.max_pages) pg = __ldg(row + col);
  if (pg < 0 || pg >= a.num_pages) {
    atomicOr(a.status, GVA_DEVERR_RANGE);
    return a.num_slots;
  }
  return pg * a.page + (t - col * a.page);
}

// ---------------------------------------------------------------------------
// Row blocks.  The n * H/G query rows (token x head) of a value group of a sequence
// are cut into blocks of M; block rb sees keys [0, kv_end) and takes
// nt = max(1, ceil(kv_end / TK)) tiles (one masked tile where it sees none, which
// yields its zeros).  Besides, a piece of a block costs about OV tiles (queries in,
// outputs out), so a block counts as OV + nt units, its tiles the last nt of them: with
// tiles alone, a CTA whose share was many short blocks ran 1.5 times as long as the rest.
// Units are numbered by sequence, block and group, and CTA i takes units
// [i, i+1) * NT / grid; a block whose tiles fall to several CTAs is merged from their
// pieces.
// ---------------------------------------------------------------------------
// Terms floor(j / h) over j < x: q = floor(x / h) whole steps of h equal terms 0 .. q-1, and
// the rest at height q.
template <typename U>
__device__ __forceinline__ unsigned long long steps_below(U x, U h) {
  const U q = x / h;
  const unsigned long long w = q;
  return h * (w * (w - (w > 0)) / 2) + w * (x - q * h);
}
// The same over every second j from c on, n of them.  Added up with its neighbour j + 1 each
// term counts twice, except where j + 1 is a multiple of h and the neighbour is one higher.
// For even h the pair (2i, 2i + 1) shares one term.  For odd h the multiples in question are
// those of c + 1's parity, every second one: y0 mod 2h.
template <typename U>
__device__ inline unsigned long long alternate_steps(U c, U n, U h) {
  if (h % 2 == 0) return steps_below<U>(c / 2 + n, h / 2) - steps_below<U>(c / 2, h / 2);
  const U last = c + 2 * n, y0 = c % 2 ? 0 : h, p = 2 * h;
  const U higher = (last + p - y0) / p - (c + p - y0) / p;
  return (steps_below<U>(last, h) - steps_below<U>(c, h) - higher) / 2;
}
// Sum over i in [0, n) of floor((M i + b) / (h TK)): M and TK are powers of two, so the quotient
// by the smaller one is exact and leaves a staircase of steps h TK / M, or h at every second place.
// Out of line: inlined in every prologue it cost a step of drafts 30.2 -> 30.9 us.
template <int M, int TK, typename U>
__device__ __noinline__ unsigned long long line_floors(U n, U h, unsigned long long b) {
  static_assert(TK % M == 0 || M == 2 * TK, "tiles of these kernels");
  if constexpr (TK % M == 0) {
    const U c = (U)(b / M), p = h * (TK / M);
    return steps_below<U>(c + n, p) - steps_below<U>(c, p);
  } else {
    return alternate_steps<U>((U)(b / TK), n, h);
  }
}

template <int M, int TK, int OV>
struct RowBlocks {
  const PagedArgs& a;
  __device__ __forceinline__ int blocks(const SeqRows& s) const {
    return (int)((unsigned)(s.n * a.hpr + M - 1) / M);
  }
  __device__ __forceinline__ int kv_end(const SeqRows& s, int rb) const {
    const int last = min(s.n - 1, (int)((unsigned)((rb + 1) * M - 1) / (unsigned)a.hpr));
    return max(0, s.L - s.n + last + 1);
  }
  __device__ __forceinline__ int tiles(const SeqRows& s, int rb) const {
    return max(1, (int)((unsigned)(kv_end(s, rb) + TK - 1) / TK));
  }
  __device__ long long units(const SeqRows& s) const {
    const int nb = blocks(s);
    if (nb == 0) return 0;
    long long u = tiles(s, nb - 1);
    if (nb <= 4 || s.L < s.n) {
      for (int rb = 0; rb < nb - 1; ++rb) u += tiles(s, rb);
    } else {
      // full blocks: ceil((L - n + floor(((rb + 1) M - 1) / hpr) + 1) / TK), one floor
      // of a line in rb
      const unsigned long long h = a.hpr, b = M - 1 + h * (unsigned long long)(s.L - s.n + TK);
      u += b + (unsigned long long)M * nb < (1ull << 31) && h * TK < (1ull << 31)
               ? (long long)line_floors<M, TK, unsigned>(nb - 1, (unsigned)h, b)
               : (long long)line_floors<M, TK, unsigned long long>(nb - 1, h, b);
    }
    return (u + (long long)OV * nb) * a.G;
  }
  __device__ long long units(int b) const { return units(seq_rows(a, b)); }
};

// A piece: tiles [k0, k1) of block rb of group g of sequence b, which has nt tiles.
struct RowPiece {
  int b, g, rb, k0, k1, nt;
};

// The pieces of a CTA's units [u, end), in order.  first() is called by whole warps,
// next() by any thread that called first().
template <int M, int TK, int OV>
struct RowWalk {
  RowBlocks<M, TK, OV> rb;
  const int* prefix;   // units before each sequence [B + 1], read by first() only
  int u, end;          // first unit of the piece's block; end of the CTA's units
  RowPiece p;
  SeqRows s;
  // first piece; false if the CTA has none
  __device__ bool first(int from) {
    if (from >= end) return false;
    p.b = seq_at(prefix, rb.a.B, from);
    s = seq_rows(rb.a, p.b);
    return seek(from, from - prefix[p.b]);
  }
  // the same from one warp's batch
  __device__ bool first(int from, const LaneBatch& t) {
    if (from >= end) return false;
    const unsigned over = __ballot_sync(0xffffffffu, t.before + t.units > from);
    p.b = __ffs(over) - 1;
    s = shfl_rows(t.s, p.b);
    return seek(from, from - __shfl_sync(0xffffffffu, t.before, p.b));
  }
  __device__ bool seek(int from, int rem) {
    // the block that holds unit `from`: lanes take consecutive blocks
    const int nb = rb.blocks(s), lane = threadIdx.x & 31;
    for (int base = 0;; base += 32) {
      const int i = base + lane;
      const int mine = i < nb ? rb.a.G * (rb.tiles(s, i) + OV) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned over = __ballot_sync(0xffffffffu, incl > rem);
      if (over || base + 32 >= nb) {
        const int l = over ? __ffs(over) - 1 : 31;
        rem -= __shfl_sync(0xffffffffu, incl - mine, l);
        p.rb = base + l;
        break;
      }
      rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    p.nt = rb.tiles(s, p.rb);
    p.g = (unsigned)rem / (unsigned)(p.nt + OV);
    rem -= p.g * (p.nt + OV);
    u = from - rem;
    p.k0 = max(0, rem - OV);
    return clip();
  }
  // tiles of the block before the CTA's end; none where that lies in its overhead
  __device__ __forceinline__ bool clip() {
    p.k1 = min(p.nt, end - u - OV);
    return p.k1 > p.k0;
  }
  __device__ bool next() {
    u += OV + p.nt;
    if (u >= end) return false;
    p.k0 = 0;
    if (++p.g == rb.a.G) {
      p.g = 0;
      if (++p.rb == rb.blocks(s)) {
        p.rb = 0;
        do s = seq_rows(rb.a, ++p.b); while (s.n == 0 && p.b + 1 < rb.a.B);
      }
      p.nt = rb.tiles(s, p.rb);
    }
    return clip();
  }
};

// Record of a block that this CTA starts and does not end: the number of its pieces (up
// to the CTA of its last tile), and its rows (q row of its sequence, query rows of it).
template <int M, int TK, int OV>
__device__ __forceinline__ void write_row_meta(const PagedArgs& a, const TileSplit& ts,
                                               const RowWalk<M, TK, OV>& w) {
  const RowPiece& p = w.p;
  if (p.k0 > 0 || p.k1 == p.nt) return;
  const int pieces = ts.cta_of(w.u + OV + p.nt - 1) - (int)blockIdx.x + 1;
  a.meta[2 * blockIdx.x] = make_int4(pieces, p.b, p.g, p.rb);
  a.meta[2 * blockIdx.x + 1] = make_int4(w.s.r0, w.s.n * a.hpr - p.rb * M, 0, 0);
}

// Where a piece's partial state goes: a CTA leaves at most one block that it did not
// start (slot 2 cta) and one that it started and does not end (slot 2 cta + 1).
__device__ __forceinline__ int piece_slot(const RowPiece& p, int cta) {
  return 2 * cta + (p.k0 == 0 ? 1 : 0);
}

}  // namespace gva
