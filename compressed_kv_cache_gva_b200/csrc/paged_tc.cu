// Paged attention of blocks of query rows on the fifth-generation tensor cores:
// prompt chunks, and drafts too wide for the mma.sync kernel.
//
// A block is M = 128 query rows (new token x head of a value group) of one sequence:
//   S[M x TK] = Q~_hi V^T + Q~_lo V^T + Qr_hi Kr^T + Qr_lo Kr^T   (tcgen05, TMEM)
//   online softmax of the rows, fp32, base 2                       (4 or 8 warps)
//   O[M x d_h] = alpha O + P V                                     (tcgen05, TMEM)
// The fp32 query is split in bf16 hi + lo, so the scores keep ~16 bits.  P is bf16
// where the output is (each term off by at most 2^-8 of itself, as the output's own
// rounding, and their errors average out) and hi + lo where the output is float32.
//
// Work: the tiles of all blocks, numbered in order, are cut evenly over a fixed grid
// (paged.cuh).  A long chunk gives every CTA the same number of tiles although its
// causal blocks differ in length; a few drafts on a long cache, which are one block
// per group, are split over the keys as well.  A CTA walks its pieces; a block that
// several CTAs share leaves partial states that the merge kernel joins.
//
// Roles: warp 0 streams tiles with 2-D TMA loads, one box per page (or part of one),
// its lanes holding the cache rows of the next 32 boxes; one thread of warp 1 issues
// every MMA; warps 2 and 3 (and the last four, where there are 16) load the queries of
// the next piece; the warps from 4 on (one or two per TMEM lane quarter) do the softmax,
// write P back to tensor memory (the A operand of the value product) and rescale O only
// when a row's maximum grew by more than 8 (log2 units).  While they exponentiate tile k,
// the MMA thread has the scores of tile k + 1 computed.  All ring and buffer barriers
// count tiles over the whole CTA, so they run on across pieces.
//
// Bound by hand-offs between the roles: a chunk of 8 x 512 tokens on 4096 (d_h = 64, bf16
// output) takes 156 us, its products 54 to 67 us and its exponentials 62 to 76 us by the
// clock; with 88 registers for the loading warps the d_h = 64 kernels spill up to 412 bytes
// a thread (d_r > 16; 144 for d_r <= 16), in the copy of the positional queries.
#include <atomic>

#include "launch.h"
#include "paged.cuh"
#include "tc.cuh"

namespace gva {

namespace {

template <int D_H_, int DRP_, bool HILO_, int MS_>
struct PtCfg {
  static constexpr int D_H = D_H_, DRP = DRP_;
  // Query rows kept in shared memory.  Where no block has more than 32 rows (drafts)
  // only those are stored; the MMA's other rows read whatever lies behind them, which
  // no one looks at, and the ring gets the memory: with 3 instead of 2 stages a draft
  // step no longer waits a DRAM latency per tile.
  static constexpr int MS = MS_;
  static constexpr bool HILO = HILO_;        // P in two bf16 halves (float32 output)
  static constexpr int M = kPagedTcRows;
  // Keys per tile and score buffers, by what tensor memory holds (512 columns an SM):
  // d_h = 64: S 128, P 64, O 64 in the 256 columns of one of two CTAs per SM (S 64, P 32
  // + 32 where P has two halves); d_h = 128: 2 x S 128, P 64 (+ 64), O 128 of one CTA.
  // 128-key tiles: the score products of 64 keys read 6 KB of shared memory for 32
  // clocks of arithmetic, above its 128 bytes a clock; those of 128 keys do not.
  static constexpr int TK = D_H == 64 && HILO ? 64 : 128;
  static constexpr int NS = D_H == 64 ? 1 : 2;
  // Softmax warps per 32 rows.  The one CTA of d_h = 128 needs two, half of the keys
  // each, to keep up with the products (mixed d_h = 128 step 105 -> 95 us); with two CTAs
  // an SM one each does as well and costs no exchange (d_h = 64 chunk 168 against 174 us).
  static constexpr int NH = D_H == 64 ? 1 : 2;
  static constexpr int HK = TK / NH, HD = D_H / NH;   // keys and output columns of a softmax warp
  static constexpr int OV = D_H == 64 ? 3 : 4;   // cost of a piece, in tiles
  static constexpr int CB = D_H / 64, KS = D_H / 16, RS = DRP / 16;
  static constexpr int QB = MS * D_H * 2;    // q~ hi (or lo): CB blocks of MS rows x 128 B
  static constexpr int QRB = DRP ? (MS * DRP * 2 + 1023) / 1024 * 1024 : 0;
  static constexpr int VB = CB * TK * 128;
  static constexpr int KRB = DRP * TK * 2;
  static constexpr int STAGE = VB + (KRB + 1023) / 1024 * 1024;
  static constexpr int OFF_QR = 2 * QB, OFF_RING = OFF_QR + 2 * QRB;
  // as many stages as fit beside the CTAs of an SM
  static constexpr int PER_SM = D_H == 64 ? 2 : 1;
  static constexpr int ROOM = (PER_SM == 2 ? 113 : 227) * 1024 - 4096;
  static constexpr int STAGES_RAW = (ROOM - OFF_RING) / STAGE;
  static constexpr int STAGES = STAGES_RAW > 6 ? 6 : STAGES_RAW;
  static constexpr int OFF_BAR = OFF_RING + STAGES * STAGE;
  // full[S], empty[S], s_full[2], s_free[2], p_full, pv_done, q_full, q_free, fin
  static constexpr int NBAR = 2 * STAGES + 9;
  // the unit prefix of the prologue lies where the queries and the ring are later
  static constexpr int SMEM = 1024 + OFF_BAR + NBAR * 8 + 8;
  static_assert(OFF_BAR >= (int)sizeof(int) * (2 * kMaxBatch + 1) + 16 + 33 * 8, "unit prefix");
  // rows past MS are read up to a full block's size behind each operand
  static_assert(SMEM - 1024 >= 2 * QB + 2 * QRB + M * 128, "operand reads stay inside");
  static_assert(STAGES >= 2 && SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t S_COL = 0, P_COL = NS * TK, P_COLS = TK / 2;
  static constexpr uint32_t O_COL = P_COL + P_COLS * (HILO ? 2 : 1);
  static constexpr uint32_t TMEM_COLS = 512 / PER_SM;
  static_assert(O_COL + D_H <= TMEM_COLS, "tensor memory");
  static constexpr uint32_t TX = VB + KRB;
  // Warps that load queries: 2 and 3, and four more where a CTA has the SM to itself and
  // 128 registers a thread suffice.
  static constexpr int LW = NH == 2 && PER_SM == 1 && !HILO ? 6 : 2;
  static constexpr int QT = 32 * (LW + 4 * NH);             // with the softmax warps
  static constexpr int THREADS = 64 + QT;
  static constexpr uint32_t SW_R = DRP == 32 ? tc::kSw64 : tc::kSw32;
  static constexpr uint32_t SBO_R = DRP * 2 * 8;
  // Two CTAs of 256 threads leave 128 registers a thread; a softmax warp holds 128 scores
  // a lane, so those warps take registers from the other four (88 + 168 = 2 x 128).
  static constexpr bool SPLIT_REGS = PER_SM == 2 && HK == 128;
};

// 16-byte chunk of a row in a swizzled K-major tile (rows of 128, 64 or 32 bytes).
__device__ __forceinline__ uint32_t sw128(int r, int chunk) {
  return (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4));
}
template <int DRP>
__device__ __forceinline__ uint32_t sw_pos(int r, int chunk) {
  return DRP == 32 ? (uint32_t)(r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4))
                   : (uint32_t)(r * 32 + ((chunk ^ ((r >> 2) & 1)) << 4));
}

// x = hi + lo in two bf16 each (pairs share a conversion: those queue behind the
// exponentials of the softmax warps).
__device__ __forceinline__ uint4 split_bf16(const float* x, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    l[i] = pack_bf16(x[2 * i] - __uint_as_float(h[i] << 16), x[2 * i + 1] - __uint_as_float(h[i] & 0xffff0000u));
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// Two packed fp32 additions (one instruction on sm_100).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Queries of a piece -> shared memory: bf16 hi and lo halves, swizzled K-major rows; by
// threads tid of nthr.  A chunk of 8 fp32 elements takes the room of its two halves, so
// its two 16-byte parts are first copied there raw, all of them in flight at once
// (asynchronous copies hold no registers), and each thread then splits its own chunks in
// place.  (Through registers, a group of rows at a time, two warps took 10 us for the
// next piece's queries; a load's latency is ~1 us beside the stream.)
template <class C, bool POS, int NTHR>
struct QueryPart {
  static constexpr int W = (POS ? C::DRP : C::D_H) / 8;   // chunks of a row
  static constexpr int HALF = POS ? C::QRB : C::QB;       // from the hi to the lo half
  static constexpr int STEP = NTHR / W, N = (C::MS + STEP - 1) / STEP;   // rows apart; rows of a thread at most
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    return POS ? C::OFF_QR + sw_pos<C::DRP>(r, c) : (uint32_t)((c / 8) * (C::MS * 128)) + sw128(r, c % 8);
  }
  __device__ static __forceinline__ void copy(const float* base, int rows, unsigned row0, int hpr, long long token,
                                              int dq, int width, uint32_t sb, int tid) {
    const int c = tid % W, r0 = tid / W;
    const unsigned R = row0 + r0;
    int h = R % (unsigned)hpr;
    const float* src = base + (R / (unsigned)hpr) * token + h * dq + c * 8;
    const int dh = STEP % hpr;   // the next row of this thread: STEP rows on
    const long long step = (STEP / hpr) * token + dh * dq, wrap = token - (long long)hpr * dq;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int r = r0 + i * STEP;
      if (N * STEP == C::MS || r < C::MS) {
        const bool on = r < rows && c * 8 < width;
        const uint32_t dst = sb + at(r, c), n = on ? 16 : 0;   // 0: zeros, nothing is read
        const float* from = on ? src : base;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(n) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + HALF), "l"(on ? src + 4 : base), "r"(n)
                     : "memory");
      }
      src += step;
      h += dh;
      if (h >= hpr) {
        h -= hpr;
        src += wrap;
      }
    }
  }
  __device__ static __forceinline__ void split(uint8_t* sm, int tid) {
    const int c = tid % W, r0 = tid / W;
    constexpr int U = N < 2 ? N : 2;   // chunks at once: their chains overlap
#pragma unroll 1
    for (int i = 0; i < N; i += U) {
      float4 x[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + (i + u) * STEP;
        if (r < C::MS) {
          x[u] = *reinterpret_cast<const float4*>(sm + at(r, c));
          y[u] = *reinterpret_cast<const float4*>(sm + at(r, c) + HALF);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + (i + u) * STEP;
        if (r < C::MS) {
          const float v[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
          uint4 lo;
          *reinterpret_cast<uint4*>(sm + at(r, c)) = split_bf16(v, lo);
          *reinterpret_cast<uint4*>(sm + at(r, c) + HALF) = lo;
        }
      }
    }
  }
};
template <class C, int NTHR>
__device__ __forceinline__ void load_queries(const PagedArgs& a, const RowPiece& p, const SeqRows& s, uint8_t* sm,
                                             int tid) {
  const int row0 = p.rb * C::M, rows = min(C::MS, s.n * a.hpr - row0), dq = C::D_H + a.d_r;
  const float* base = a.q_abs + ((long long)s.r0 * a.H + p.g * a.hpr) * dq;
  const long long token = (long long)a.H * dq;
  QueryPart<C, false, NTHR>::copy(base, rows, row0, a.hpr, token, dq, C::D_H, smem_u32(sm), tid);
  if constexpr (C::DRP > 0)
    QueryPart<C, true, NTHR>::copy(base + C::D_H, rows, row0, a.hpr, token, dq, a.d_r, smem_u32(sm), tid);
  asm volatile("cp.async.wait_all;" ::: "memory");
  QueryPart<C, false, NTHR>::split(sm, tid);
  if constexpr (C::DRP > 0) QueryPart<C, true, NTHR>::split(sm, tid);
  fence_proxy_async_smem();   // the queries are read by the tensor core (async proxy)
}
// Ask L2 for the queries of a piece that is loaded later.
template <class C>
__device__ __forceinline__ void prefetch_queries(const PagedArgs& a, const RowPiece& p, const SeqRows& s, int tid,
                                                 int nthr) {
  const int row0 = p.rb * C::M, rows = min(C::MS, s.n * a.hpr - row0), dq = C::D_H + a.d_r;
  for (int r = tid; r < rows; r += nthr) {
    const unsigned R = row0 + r, qi = R / (unsigned)a.hpr;
    const float* src = a.q_abs + ((long long)(s.r0 + (int)qi) * a.H + p.g * a.hpr + (int)(R - qi * a.hpr)) * dq;
    for (int i = 0; i < dq; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
  }
}

// 32 bytes of a row per lane, as one store where the buffers are 32-byte aligned: rows
// lie apart, so each lane fills a whole sector instead of halves by two instructions.
__device__ __forceinline__ void store_32b(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A softmax warp's place in the walk over the CTA's pieces.
struct SoftmaxPiece {
  RowPiece p;
  SeqRows s;
  int u, end;
  bool more;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM)
    paged_tc_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_kr) {
  extern __shared__ unsigned char smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(sm);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  const uint32_t full = smem_u32(bars), empty = full + 8 * C::STAGES;
  const uint32_t s_full = empty + 8 * C::STAGES, s_free = s_full + 16;
  const uint32_t p_full = s_free + 16, pv_done = p_full + 8, q_full = pv_done + 8;
  const uint32_t q_free = q_full + 8, fin = q_free + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  int* prefix = reinterpret_cast<int*>(sm);
  long long* wtmp = reinterpret_cast<long long*>(
      (reinterpret_cast<uintptr_t>(prefix + 2 * a.B + 1) + 15) & ~uintptr_t(15));
  int* units = prefix + a.B + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hpr = a.hpr;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(s_free + 8 * i, 4 * C::NH);
    }
    mbar_init(p_full, 4 * C::NH);
    mbar_init(pv_done, 1);
    mbar_init(q_full, C::LW);
    mbar_init(q_free, 1);
    mbar_init(fin, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tc::relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_v);
    if (C::DRP) prefetch_tmap(&tm_kr);
  }
  // queries, lengths, tables and cache rows may come from the kernels before
  pdl_enter(a);
  if (blockIdx.x == 0 && a.flag_errors) flag_bad_sequences(a);
  const RowBlocks<C::M, C::TK, C::OV> blocks{a};
  // Every role walks the CTA's pieces by itself.
  RowWalk<C::M, C::TK, C::OV> walk{blocks, prefix, 0, 0, {}, {}};
  TileSplit ts;
  long long total;
  bool more;
  if (a.B <= kLaneBatch) {
    const LaneBatch t = lane_batch(a, [&](const SeqRows& s) { return blocks.units(s); });
    total = t.total;
    ts = make_split(total < (1ll << 31) ? (int)total : 0, (int)gridDim.x, 0);
    walk.end = ts.first(blockIdx.x + 1);
    more = walk.first(ts.first(blockIdx.x), t);
  } else {
    const int per = (a.B + C::THREADS - 1) / C::THREADS;   // as block_scan deals them out
    for (int b = threadIdx.x * per; b < min((int)(threadIdx.x + 1) * per, a.B); ++b)
      units[b] = (int)min(blocks.units(b), 0x7fffffffll);
    total = block_scan(a.B, [&](int b) { return (long long)units[b]; }, prefix, wtmp);
    ts = make_split(prefix[a.B], (int)gridDim.x, 0);
    walk.end = ts.first(blockIdx.x + 1);
    more = walk.first(ts.first(blockIdx.x));
  }
  if (threadIdx.x == 0) {
    if (total >= (1ll << 31)) atomicOr(a.status, GVA_DEVERR_RANGE);
    a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();   // the prefix was read where TMA writes the ring
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const RowPiece& p = walk.p;
  const SeqRows& s = walk.s;

  // kt: tiles of this CTA before the piece; all barrier phases count from it.
  // ok: false once a bounded wait gave up: skip work, keep the order.
  int kt = 0;
  bool ok = true;
  // ------------------------------------------------------------ queries of the next piece
  auto loader = [&]() {
    const int tid = warp < 4 ? threadIdx.x - 64 : threadIdx.x - 64 - 128 * C::NH;
    for (int i = 0; more; more = walk.next(), ++i) {
      if (i > 0) {
        prefetch_queries<C>(a, p, s, tid, 32 * C::LW);
        ok = ok && mbar_wait_warp(q_free, (i - 1) & 1, a.status);
        load_queries<C, 32 * C::LW>(a, p, s, sm, tid);
      } else {   // the softmax warps have nothing else to do yet, and help
        load_queries<C, C::QT>(a, p, s, sm, tid);
        named_bar_sync(5, C::QT);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
  };
  if (warp < 4) {
    if constexpr (C::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      int issued = 0;
      const int per_tile = C::TK >> a.box_log2;
      for (; more; more = walk.next()) {
        const int nk = p.k1 - p.k0, end = p.k1 * per_tile;
        if (lane == 0) write_row_meta(a, ts, walk);
        const int* row = a.table + (long long)p.b * a.table_stride;
        int base = p.k0 * per_tile;
        auto look = [&](int i) { return i < end ? slot_of(a, row, i << a.box_log2, s.L) : a.num_slots; };
        int y_now = look(base + lane), y_next = look(base + 32 + lane);
        for (int k = 0; k < nk && ok; ++k) {
          const int box0 = (p.k0 + k) * per_tile;
          if (box0 - base >= 32) {
            base += 32;
            y_now = y_next;
            y_next = look(base + 32 + lane);
          }
          const int kk = kt + k, sg = kk % C::STAGES;
          if (kk >= C::STAGES) ok = mbar_wait_warp(empty + 8 * sg, ((kk / C::STAGES) - 1) & 1, a.status);
          if (!ok) break;
#ifdef GVA_TEST_WITHHOLD_TILE
          // Failure-detection test builds only: this tile of every CTA is never requested
          // (nothing is armed, no copy is in flight for it), so bounded waits run out.
          if (kk == GVA_TEST_WITHHOLD_TILE) continue;
#endif
          const uint32_t fb = full + 8 * sg, st = sb + C::OFF_RING + sg * C::STAGE;
          if (lane == 0) mbar_arrive_expect_tx(fb, C::TX);
          __syncwarp();
          for (int j = 0; j < per_tile; ++j) {
            const int y = __shfl_sync(0xffffffffu, y_now, box0 + j - base);
            if (lane == 0) {
              const uint32_t r = (uint32_t)j << a.box_log2;
#pragma unroll
              for (int c = 0; c < C::CB; ++c)
                tma_load_2d(st + c * C::TK * 128 + r * 128, &tm_v, p.g * C::D_H + c * 64, y, fb);
              if constexpr (C::DRP > 0) tma_load_2d(st + C::VB + r * C::DRP * 2, &tm_kr, 0, y, fb);
            }
          }
          issued = kk + 1;
        }
        kt += nk;
      }
      // no copy in flight may outlive the CTA
      for (int kk = max(0, issued - C::STAGES); kk < issued; ++kk)
        mbar_wait(full + 8 * (kk % C::STAGES), (kk / C::STAGES) & 1, a.status);
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issue
      if (lane == 0) {
        constexpr uint32_t idS = tc::idesc_bf16(C::M, C::TK, 0, 0);   // Q (K-major) x V^T (K-major)
        constexpr uint32_t idO = tc::idesc_bf16(C::M, C::D_H, 0, 1);  // P (tensor memory) x V (MN-major)
        for (int i = 0; more; more = walk.next(), ++i) {
          const int nk = p.k1 - p.k0;
          ok = ok && mbar_wait(q_full, i & 1, a.status);
          for (int k = 0; k <= nk; ++k) {
            if (k < nk) {
              const int kk = kt + k, sg = kk % C::STAGES;
              ok = ok && mbar_wait(full + 8 * sg, (kk / C::STAGES) & 1, a.status);
              const int sb_ = kk % C::NS;   // score buffer
              if (kk >= C::NS) ok = ok && mbar_wait(s_free + 8 * sb_, (kk / C::NS - 1) & 1, a.status);
              tc::fence_after();
              if (ok) {
                const uint32_t d = tmem + C::S_COL + sb_ * C::TK, vt = sb + C::OFF_RING + sg * C::STAGE;
#pragma unroll
                for (int ks = 0; ks < C::KS; ++ks) {
                  const uint32_t kb = (ks >> 2) * (C::MS * 128) + (ks & 3) * 32;
                  const uint64_t bq =
                      tc::smem_desc(vt + (ks >> 2) * (C::TK * 128) + (ks & 3) * 32, 16, 1024, tc::kSw128);
                  tc::mma_bf16(d, tc::smem_desc(sb + kb, 16, 1024, tc::kSw128), bq, idS, ks > 0);
                  tc::mma_bf16(d, tc::smem_desc(sb + C::QB + kb, 16, 1024, tc::kSw128), bq, idS, 1);
                }
#pragma unroll
                for (int rs = 0; rs < C::RS; ++rs) {
                  const uint64_t bk = tc::smem_desc(vt + C::VB + rs * 32, 16, C::SBO_R, C::SW_R);
                  tc::mma_bf16(d, tc::smem_desc(sb + C::OFF_QR + rs * 32, 16, C::SBO_R, C::SW_R), bk, idS, 1);
                  tc::mma_bf16(d, tc::smem_desc(sb + C::OFF_QR + C::QRB + rs * 32, 16, C::SBO_R, C::SW_R), bk,
                               idS, 1);
                }
              }
              tc::commit(s_full + 8 * sb_);
              if (k == nk - 1) tc::commit(q_free);   // the piece's queries have been read
            }
            if (k >= 1) {   // P.V of the tile before
              const int kp = kt + k - 1, sp = kp % C::STAGES;
              ok = ok && mbar_wait(p_full, kp & 1, a.status);
              tc::fence_after();
              if (ok) {
                const uint32_t vt = sb + C::OFF_RING + sp * C::STAGE;
#pragma unroll
                for (int h = 0; h < (C::HILO ? 2 : 1); ++h)
#pragma unroll
                  for (int kk = 0; kk < C::TK / 16; ++kk)
                    tc::mma_bf16_ts(tmem + C::O_COL, tmem + C::P_COL + h * C::P_COLS + kk * 8,
                                    tc::smem_desc(vt + kk * 16 * 128, C::TK * 128, 1024, tc::kSw128), idO,
                                    (k > 1 || h > 0 || kk > 0) ? 1u : 0u);
              }
              tc::commit(pv_done);
              tc::commit(empty + 8 * sp);
            }
          }
          kt += nk;
        }
        // every MMA has completed before the tensor memory is freed
        tc::commit(fin);
        mbar_wait(fin, 0, a.status);
      }
      __syncwarp();
    } else {
      loader();
    }
  } else if (warp >= 4 + 4 * C::NH) {
    loader();
  } else {
    if constexpr (C::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    // One warp per lane quarter, or two that share its 32 rows, half of a tile's keys and
    // of the output columns each.
    const int quarter = warp & 3, half = (warp - 4) >> 2, r = 32 * quarter + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
    __shared__ float row_x[2][C::NH][C::M];   // exchange between two halves: [tile parity][half][row]
    // A row of scores takes most of the registers: the walk waits in shared memory.
    __shared__ SoftmaxPiece pieces[4 * C::NH];
    SoftmaxPiece& sp = pieces[warp - 4];
    if (more) {
      load_queries<C, C::QT>(a, p, s, sm, 32 * C::LW + threadIdx.x - 128);
      named_bar_sync(5, C::QT);
      if (lane == 0) sp = SoftmaxPiece{walk.p, walk.s, walk.u, walk.end};
    }
    __syncwarp();
    while (more) {
      const int nk = sp.p.k1 - sp.p.k0, k0 = sp.p.k0, row0 = sp.p.rb * C::M;
      const int L = sp.s.L, first_lim = sp.s.L - sp.s.n, rows = min(C::M, sp.s.n * hpr - row0);
      // ---------------------------------------------------------- softmax, P, O rescale, output
      // idle: no row of this quarter counts.  A row of P meets only its own row of O, so
      // what idle lanes of the tensor memory hold does not matter.
      const bool valid = r < rows, idle = 32 * quarter >= rows;
      const int lim = first_lim + (row0 + r) / hpr;                // last key of this row
      const int kv_all = first_lim + row0 / hpr + 1;               // keys every row sees
      float m = -INFINITY, l = 0.f;   // the row's reference; this half's sum
      for (int k = 0; k < nk; ++k) {
        const int kk = kt + k, sbuf = kk % C::NS, t0 = (k0 + k) * C::TK;
        ok = ok && mbar_wait_warp(s_full + 8 * sbuf, (kk / C::NS) & 1, a.status);
        tc::fence_after();
        if (!idle) {
          float x[C::HK];
#pragma unroll
          for (int q = 0; q < C::HK / 32; ++q)
            tc::ld32(trow + C::S_COL + sbuf * C::TK + half * C::HK + q * 32, x + q * 32);
          tc::wait_ld();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + 8 * sbuf);
          // four running maxima (and sums below): one dependent chain would cost more
          // than the operations themselves
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (!ok || t0 + C::TK > kv_all) {   // some row does not see the whole tile
            const int vis = (ok && valid ? min(lim + 1, L) - t0 : 0) - half * C::HK;
#pragma unroll
            for (int j = 0; j < C::HK; ++j) x[j] = j < vis ? x[j] : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < C::HK; j += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx4[i] = max3(mx4[i], x[j + 2 * i], x[j + 2 * i + 1]);
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          if constexpr (C::NH == 2) {
            row_x[kk & 1][half][r] = mx;
            named_bar_sync(1 + quarter, 64);
            mx = fmaxf(mx, row_x[kk & 1][half ^ 1][r]);
          }
          // a row keeps the maximum its exponentials are taken against until a tile
          // exceeds it by more than 8 (log2 units): P <= 2^8, and O is touched only then
          const bool grow = mx > m + 8.f;
          const float mn = grow ? mx : m;
          const float ms = mn == -INFINITY ? 0.f : mn;
          const float alpha = ex2(m - ms);
          m = mn;
          const float2 neg = make_float2(-ms, -ms);
          float2 sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int q = 0; q < C::HK / 16; ++q) {   // 16 keys at a time
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 e = add2(make_float2(x[16 * q + 2 * i], x[16 * q + 2 * i + 1]), neg);
              e = make_float2(ex2(e.x), ex2(e.y));
              sum[i & 3] = add2(sum[i & 3], e);
              hi[i] = pack_bf16(e.x, e.y);
              if constexpr (C::HILO)
                lo[i] = pack_bf16(e.x - __uint_as_float(hi[i] << 16), e.y - __uint_as_float(hi[i] & 0xffff0000u));
            }
            if (q == 0 && kk >= 1) {   // P is free, and O still, once the P.V before has completed
              ok = ok && mbar_wait_warp(pv_done, (kk - 1) & 1, a.status);
              tc::fence_after();
            }
            const uint32_t pc = trow + C::P_COL + half * (C::HK / 2) + q * 8;
            tc::st8u(pc, hi);
            if constexpr (C::HILO) tc::st8u(pc + C::P_COLS, lo);
          }
          l = l * alpha + (((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
                           ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y)));
          // O *= alpha before this tile's P.V
          if (k >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int q4 = 0; q4 < C::HD / 16; ++q4) {
              float o[16];
              const uint32_t oc = trow + C::O_COL + half * C::HD + q4 * 16;
              tc::ld16(oc, o);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              tc::st16(oc, o);
            }
          }
          tc::wait_st();
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + 8 * sbuf);
          // keep step with the warps that write P: an arrival for this tile must not
          // count for the one before
          if (kk >= 1) ok = ok && mbar_wait_warp(pv_done, (kk - 1) & 1, a.status);
        }
        // value rows behind the sequence meet P = 0 but may hold anything (NaN): zero
        // them before the P.V product reads them
        if (t0 + C::TK > L) {
          uint8_t* vt = sm + C::OFF_RING + (kk % C::STAGES) * C::STAGE;
          const int r_lo = max(L - t0, 0), nz = (C::TK - r_lo) * 8;   // 16-byte chunks per block
          for (int e = (int)threadIdx.x - 128; e < nz * C::CB; e += 128 * C::NH) {
            const int c = e / nz, i = e % nz;
            *reinterpret_cast<uint4*>(vt + c * C::TK * 128 + (r_lo + i / 8) * 128 + (i % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();   // the zeroed rows are read by the tensor core
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      {   // the last P.V of the piece (and with it every MMA before) has completed
        const int kl = kt + nk - 1;
        ok = ok && mbar_wait_warp(pv_done, kl & 1, a.status);
        tc::fence_after();
      }
      if (!idle) {
        if constexpr (C::NH == 2) {   // the halves' sums, through the buffer of the next tile
          const int xb = (kt + nk) & 1;
          row_x[xb][half][r] = l;
          named_bar_sync(1 + quarter, 64);
          l += row_x[xb][half ^ 1][r];
          named_bar_sync(1 + quarter, 64);
        }
        const bool whole = nk == sp.p.nt;
        const int R = row0 + r, qi = R / hpr, head = sp.p.g * hpr + R % hpr;
        const long long orow = (long long)(sp.s.r0 + qi) * a.H + head;
        const long long prt = (long long)piece_slot(sp.p, blockIdx.x) * C::M + r;
        const float inv = norm_of(l);
        const int d0 = half * C::HD;
#pragma unroll
        for (int q = 0; q < C::HD / 32; ++q) {
          float o[32];
          tc::ld32(trow + C::O_COL + d0 + q * 32, o);
          tc::wait_ld();
          if (valid && ok) {
            if (!whole || !a.out_bf16) {
              const float f = whole ? inv : 1.f;
              float* dst = whole ? reinterpret_cast<float*>(a.out) + orow * C::D_H + d0 + q * 32
                                 : a.part_o + prt * C::D_H + d0 + q * 32;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(o[i + j] * f);
                store_32b(dst + i, w, a.wide);
              }
            } else {
              __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + orow * C::D_H + d0 + q * 32;
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pack_bf16(o[i + 2 * j] * inv, o[i + 2 * j + 1] * inv);
                store_32b(dst + i, w, a.wide);
              }
            }
          }
        }
        if (valid && ok && half == 0) {
          if (!whole) a.part_ml[prt] = make_float2(m, l);
          else if (a.lse) a.lse[orow] = natural_lse(m, l);
        }
      }
      kt += nk;
      __syncwarp();
      if (lane == 0) {
        RowWalk<C::M, C::TK, C::OV> w{blocks, nullptr, sp.u, sp.end, sp.p, sp.s};
        sp.more = w.next();
        sp.p = w.p;
        sp.s = w.s;
        sp.u = w.u;
      }
      __syncwarp();
      more = sp.more;
      tc::fence_before();   // O has been read: the P of the next piece orders its first P.V behind
    }
  }

  // ---- every role is done with the tensor memory: free it
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, C::TMEM_COLS);
  }
  pdl_leave(a);
}

// Visit the configuration of (d_h, padded d_r, output type, rows of a block).
template <class F>
bool dispatch(const gva_shape_t& sh, int max_new, F&& f) {
  const int drp = sh.d_r == 0 ? 0 : (sh.d_r <= 16 ? 16 : (sh.d_r <= 32 ? 32 : -1));
  const bool hilo = sh.out_dtype == GVA_F32, few = (long long)max_new * (sh.H / sh.G) <= 32;
#define GVA_PT(DH, DRP, HILO)                                   \
  if (sh.d_h == DH && drp == DRP && hilo == HILO) {             \
    if (few) f(PtCfg<DH, DRP, HILO, 32>{});                     \
    else f(PtCfg<DH, DRP, HILO, kPagedTcRows>{});               \
    return true;                                                \
  }
#define GVA_PT_DR(DH, HILO) GVA_PT(DH, 0, HILO) GVA_PT(DH, 16, HILO) GVA_PT(DH, 32, HILO)
  GVA_PT_DR(64, false)
  GVA_PT_DR(64, true)
  GVA_PT_DR(128, false)
  GVA_PT_DR(128, true)
#undef GVA_PT_DR
#undef GVA_PT
  return false;
}

}  // namespace

bool paged_tc_supported(const gva_shape_t& sh, int page) {
  return sh.cache_dtype == GVA_BF16 && page % 8 == 0 && sh.d_r % 8 == 0 && dispatch(sh, 1, [](auto) {});
}

int paged_tc_tile(const gva_shape_t& sh) {
  int tk = 0;
  dispatch(sh, 1, [&](auto c) { tk = decltype(c)::TK; });
  return tk;
}

int paged_tc_grid(const gva_shape_t& sh, int n_rows, int max_new, int num_sms, long long max_total) {
  int tk = 64, per_sm = 1;
  dispatch(sh, max_new, [&](auto c) {
    tk = decltype(c)::TK;
    per_sm = decltype(c)::PER_SM;
  });
  // no more CTAs than blocks x tiles could be
  const long long blocks = ((long long)n_rows * (sh.H / sh.G) + kPagedTcRows - 1) / kPagedTcRows + sh.B;
  const long long want = blocks * sh.G * (max_total / tk + 1);
  const long long grid = (long long)num_sms * per_sm;
  return (int)(want < grid ? want : grid);
}

cudaError_t launch_paged_tc(const gva_shape_t& sh, const PagedArgs& a, const CUtensorMap& tv,
                            const CUtensorMap& tk, cudaStream_t st) {
  cudaError_t err = cudaErrorNotSupported;
  dispatch(sh, a.max_new, [&](auto c) {
    using C = decltype(c);
    const size_t smem = C::SMEM;
    if ((err = ensure_max_smem(paged_tc_kernel<C>, smem)) != cudaSuccess) return;
    if constexpr (C::SPLIT_REGS) {
      // the register split needs the full 128 at launch (it would wait forever on fewer)
      static std::atomic<bool> checked{false};
      if (!checked.load(std::memory_order_relaxed)) {
        cudaFuncAttributes fa;
        if ((err = cudaFuncGetAttributes(&fa, paged_tc_kernel<C>)) != cudaSuccess) return;
        if (fa.numRegs <= 120) {
          err = cudaErrorInvalidConfiguration;
          return;
        }
        checked.store(true, std::memory_order_relaxed);
      }
    }
    err = launch_pdl(paged_tc_kernel<C>, dim3(a.grid), dim3(C::THREADS), smem, st, a, tv, tk);
  });
  return err;
}

}  // namespace gva
