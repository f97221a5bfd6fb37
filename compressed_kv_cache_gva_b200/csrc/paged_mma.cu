// Paged split-KV attention of few query columns per value group (one new token per
// request, or a few drafts), on mma.sync.
//
// A CTA is one consumer warp per value group and 8 of its query columns (two per group
// for 9 to 16 columns) and one producer warp.  The batch's tiles of TT cached tokens are
// numbered in request order and cut evenly over the CTAs; each tile is read once and
// serves every head.  The producer resolves pages: its lanes hold the cache rows of the
// next 32 boxes (table entries loaded one round ahead, so their latency hides behind the
// stream) and one lane issues the 2-D TMA loads of a tile, TT / box boxes per 64
// columns.  A box never crosses a page, lands where the unpaged tile's rows would (8-row
// boxes keep the 128-byte swizzle pattern), and reads zeros where there is no page.
//
// Per tile and group, tokens on M and query columns on N (m16n8k16):
//   S = V Qb (+ kr Qr),  online softmax in fp32 base 2,  O^T += V^T P.
// With 4 columns the 8 of the instruction hold [hi | lo] halves of the fp32 query
// (x = hi + lo in two bf16), with 8 the halves take two instructions; P is split the
// same way, so scores and outputs keep ~16 significand bits.  The score fragment
// becomes the B operand of the second product through movmatrix.
//
// Bound by the cache stream on long batches and by the dependent MMA / softmax chain
// of a tile on short ones.  The thin N is why this is not tcgen05 work: a 128-row
// tensor-memory tile would be 3 % full, and its hand-offs cost more than the products.
#include "launch.h"
#include "paged.cuh"

namespace gva {

namespace {

template <int D_H_, int NG_, int COLS_, int DRP_>
struct PmCfg {
  static constexpr int D_H = D_H_, NG = NG_, COLS = COLS_, DRP = DRP_;
  static constexpr int CPW = COLS < 8 ? COLS : 8;     // query columns of a warp
  static constexpr int NJ = COLS / CPW;               // warps per group
  static constexpr int NC = NG * NJ;                  // consumer warps
  static constexpr int ROW_BYTES = NG * D_H * 2;
  static constexpr int TT_RAW = 16384 / ROW_BYTES;
  static constexpr int TT = TT_RAW >= 64 ? 64 : (TT_RAW >= 32 ? 32 : 16);   // tokens per tile
  static constexpr int VW = D_H < 64 ? D_H : 64;      // columns per box
  static constexpr int VROW = VW * 2;                 // bytes of a box row (= swizzle span)
  static constexpr int CPR = VROW / 16;               // 16-byte chunks per box row
  static constexpr int CB = D_H / VW;                 // column blocks per group
  static constexpr int BOX = TT * VROW;               // one [TT x VW] block of the tile
  static constexpr int XB = NG * CB * BOX;
  static constexpr int KRB = DRP * TT * 2;
  static constexpr int STAGE = XB + (KRB + 1023) / 1024 * 1024;
  // 96 KB of ring for two CTAs per SM, 160 KB for one; the 33 KB tiles of eight 128-wide
  // groups get a third stage (as in the unpaged kernel)
  static constexpr bool ALONE = NJ > 1 && NG >= 4;
  static constexpr int RING = ALONE ? 160 * 1024 : (D_H == 128 && NG == 8) ? 108 * 1024 : 96 * 1024;
  static constexpr int STAGES_RAW = RING / STAGE;
  static constexpr int STAGES = STAGES_RAW < 2 ? 2 : (STAGES_RAW > 12 ? 12 : STAGES_RAW);
  static constexpr int PIPE = STAGES * STAGE;
  static constexpr uint32_t TX = XB + KRB;
  static constexpr int MT = TT / 16;
  static constexpr int THREADS = (NC + 1) * 32;
  static constexpr int NT = CPW == 8 ? 2 : 1;
  static constexpr int KS = D_H / 16, RS = DRP / 16;
  static constexpr int KR_SW = DRP * 2;
  // 8 columns of d_h = 128 keep ~100 values live per consumer thread: one CTA per SM,
  // and so for two warps per group of four (26.8 against 29.9 us with two CTAs, which
  // leave a thread 112 registers)
  static constexpr int MINB = ALONE || (NG >= 8 && COLS == 8 && D_H == 128) ? 1 : 2;
  static size_t smem_bytes(int B) {
    return 1024 + PIPE + 16 * STAGES + sizeof(int) * (B + 1) + 16 + sizeof(long long) * 33;
  }
};

template <class C>
__device__ __forceinline__ void load_query(const PagedArgs& a, const SeqRows& s, int g, int c0, int ncol, int gq,
                                           int t, uint32_t (&qb)[C::NT][C::KS][2],
                                           uint32_t (&qr)[C::NT][C::RS > 0 ? C::RS : 1][2]) {
  const int dq = C::D_H + a.d_r;
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    const int col = c0 + (C::CPW == 8 ? gq : (gq & 3));
    const bool lo = C::CPW == 8 ? nt == 1 : gq >= 4;
    const bool on = col < ncol;   // padding columns carry a zero query
    const float* row =
        a.q_abs + ((long long)(s.r0 + (on ? col / a.hpr : 0)) * a.H + g * a.hpr + (on ? col % a.hpr : 0)) * dq;
    auto part = [&](float x) {
      const float h = bf16_round(x);
      return lo ? x - h : h;
    };
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      const int k0 = ks * 16 + 2 * t;
      const float2 x = on ? *reinterpret_cast<const float2*>(row + k0) : make_float2(0.f, 0.f);
      const float2 y = on ? *reinterpret_cast<const float2*>(row + k0 + 8) : make_float2(0.f, 0.f);
      qb[nt][ks][0] = pack_bf16(part(x.x), part(x.y));
      qb[nt][ks][1] = pack_bf16(part(y.x), part(y.y));
    }
#pragma unroll
    for (int rs = 0; rs < C::RS; ++rs) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = rs * 16 + 2 * t + (e & 1) + (e >> 1) * 8;
        w[e] = on && k < a.d_r ? row[C::D_H + k] : 0.f;
      }
      qr[nt][rs][0] = pack_bf16(part(w[0]), part(w[1]));
      qr[nt][rs][1] = pack_bf16(part(w[2]), part(w[3]));
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MINB)
    paged_mma_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_kr) {
  extern __shared__ unsigned char smraw[];
  uint8_t* pipe =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(pipe + C::PIPE);
  uint64_t* empty = full + C::STAGES;
  int* tp = reinterpret_cast<int*>(empty + C::STAGES);   // tiles before each sequence
  long long* wtmp =
      reinterpret_cast<long long*>((reinterpret_cast<uintptr_t>(tp + a.B + 1) + 15) & ~uintptr_t(15));
  __shared__ int4 batch[kLaneBatch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), C::NC);
    }
    fence_barrier_init();
  }
  if (warp == C::NC && lane == 0) {
    prefetch_tmap(&tm_v);
    if (C::DRP) prefetch_tmap(&tm_kr);
  }
  // queries, lengths, tables and cache rows may come from the kernels before
  pdl_enter(a);
  // tiles of a sequence: one (masked) tile where it has no key
  auto tiles = [](const SeqRows& s) -> long long {
    return s.n == 0 ? 0 : max(1, (s.L + C::TT - 1) / C::TT);
  };
  long long total;
  if (a.B <= kLaneBatch) {
    const LaneBatch t = lane_batch(a, tiles);
    total = t.total;
    if (warp == 0) {
      if (lane < a.B) {
        tp[lane] = t.before;
        batch[lane] = make_int4(t.s.r0, t.s.n, t.s.L, 0);
      }
      if (lane == 0) tp[a.B] = total < (1ll << 31) ? (int)total : 0;
    }
    __syncthreads();
  } else {
    total = block_scan(a.B, [&](int b) { return tiles(seq_rows(a, b)); }, tp, wtmp);
  }
  auto rows_of = [&](int b) -> SeqRows {
    if (a.B > kLaneBatch) return seq_rows(a, b);
    const int4 v = batch[b];
    return SeqRows{v.x, v.y, v.z, false};
  };
  if (total >= (1ll << 31) && threadIdx.x == 0) atomicOr(a.status, GVA_DEVERR_RANGE);
  const TileSplit ts = make_split(tp[a.B], (int)gridDim.x, 0);
  const int T0 = ts.first(blockIdx.x), T1 = ts.first(blockIdx.x + 1);
  if (blockIdx.x == 0) {
    if (a.flag_errors) flag_bad_sequences(a);
    for (int b = threadIdx.x; b < a.B; b += blockDim.x)
      a.meta[b] = tp[b + 1] > tp[b] ? ts.slots(b, tp[b], tp[b + 1], a.B) : make_int4(0, 0, 0, 0);
  }
  if (T1 <= T0) return;
  const int b_first = seq_at(tp, a.B, T0);

  if (warp == C::NC) {
    // ---------------------------------------------------------------- producer
    const uint64_t pol = policy_evict_first();   // the cache is read once per call
    const int per_tile = C::TT >> a.box_log2;
    int k = 0;
    bool ok = true;
    for (int b = b_first; ok && b < a.B && tp[b] < T1; ++b) {
      const int u0 = max(T0, tp[b]) - tp[b], u1 = min(T1, tp[b + 1]) - tp[b];
      if (u1 <= u0) continue;
      const int L = rows_of(b).L;
      const int* row = a.table + (long long)b * a.table_stride;
      int base = u0 * per_tile;
      const int end = u1 * per_tile;
      auto look = [&](int i) { return i < end ? slot_of(a, row, i << a.box_log2, L) : a.num_slots; };
      int y_now = look(base + lane), y_next = look(base + 32 + lane);
      for (int u = u0; u < u1; ++u, ++k) {
        if (u * per_tile - base >= 32) {
          base += 32;
          y_now = y_next;
          y_next = look(base + 32 + lane);
        }
        const int s = k % C::STAGES;
        if (k >= C::STAGES && !mbar_wait_warp(smem_u32(empty + s), ((k / C::STAGES) - 1) & 1, a.status)) {
          ok = false;
          break;
        }
#ifdef GVA_TEST_WITHHOLD_TILE
        // Failure-detection test builds only: this tile of every CTA is never requested
        // (nothing is armed, no copy is in flight for it), so bounded waits run out.
        if (k == GVA_TEST_WITHHOLD_TILE) continue;
#endif
        const uint32_t fb = smem_u32(full + s), st = smem_u32(pipe + s * C::STAGE);
        if (lane == 0) mbar_arrive_expect_tx(fb, C::TX);
        __syncwarp();
        for (int j = 0; j < per_tile; ++j) {
          const int y = __shfl_sync(0xffffffffu, y_now, u * per_tile + j - base);
          if (lane == 0) {
            const uint32_t r = (uint32_t)j << a.box_log2;   // first tile row of the box
#pragma unroll
            for (int c = 0; c < C::NG * C::CB; ++c)
              tma_load_2d_hint(st + c * C::BOX + r * C::VROW, &tm_v, c * C::VW, y, fb, pol);
            if constexpr (C::DRP > 0)
              tma_load_2d_hint(st + C::XB + r * C::DRP * 2, &tm_kr, 0, y, fb, pol);
          }
        }
      }
    }
    // do not leave while a copy into this CTA's shared memory is in flight
    for (int kk = max(0, k - C::STAGES); kk < k; ++kk)
      mbar_wait(smem_u32(full + kk % C::STAGES), (kk / C::STAGES) & 1, a.status);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = warp % C::NG, c0 = warp / C::NG * C::CPW;   // this warp's group and first column
  const int t = lane & 3, gq = lane >> 2, mi = lane >> 3, r8 = lane & 7;
  const int a_row = (mi & 1) * 8 + r8, a_kc = mi >> 1;   // scores A: rows = tokens
  const int v_tok = (mi >> 1) * 8 + r8, v_dc = mi & 1;   // P.V A (trans): rows = tokens
  const bool lo_half = C::CPW == 4 && t >= 2;
  const int hcol = c0 + ((2 * t) & (C::CPW - 1));        // columns hcol, hcol + 1 after hi / lo merge
  const int Hp = a.H * min(a.max_new, C::COLS / a.hpr);  // heads of a partial
  const int qi0 = hcol / a.hpr, qi1 = (hcol + 1) / a.hpr;
  const int head0 = g * a.hpr + hcol % a.hpr, head1 = g * a.hpr + (hcol + 1) % a.hpr;
  bool ok = true;
  int k = 0;
  for (int b = b_first; b < a.B && tp[b] < T1; ++b) {
    const int u0 = max(T0, tp[b]) - tp[b], u1 = min(T1, tp[b + 1]) - tp[b];
    if (u1 <= u0) continue;
    const SeqRows sq = rows_of(b);
    const int ncol = sq.n * a.hpr;
    uint32_t qb[C::NT][C::KS][2], qr[C::NT][C::RS > 0 ? C::RS : 1][2];
    load_query<C>(a, sq, g, c0, ncol, gq, t, qb, qr);
    const int lim0 = sq.L - sq.n + qi0, lim1 = sq.L - sq.n + qi1;   // last key of each column
    float o[C::KS][4];
#pragma unroll
    for (int md = 0; md < C::KS; ++md)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[md][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int u = u0; u < u1; ++u, ++k) {
      const int s = k % C::STAGES, t0 = u * C::TT;
      if (ok) ok = mbar_wait_warp(smem_u32(full + s), (k / C::STAGES) & 1, a.status);
      if (!ok) continue;
      if (C::NJ > 1 && c0 >= ncol) {   // no query of this request is this warp's
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(empty + s));
        continue;
      }
      const int nvalid = min(C::TT, sq.L - t0);
      uint8_t* st = pipe + s * C::STAGE;
      uint8_t* xg = st + g * C::CB * C::BOX;
      const bool ragged = nvalid < C::TT;
      if (ragged) {
        // rows behind the sequence may hold anything (even NaN): zero this group's
        // rows so that p = 0 contributes nothing
        const int nz = C::TT - nvalid;
        for (int e = lane; e < nz * C::CPR * C::CB; e += 32) {
          const int c = e / (nz * C::CPR), rr = nvalid + (e / C::CPR) % nz, ch = e % C::CPR;
          *reinterpret_cast<uint4*>(xg + c * C::BOX + rr * C::VROW + ch * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      const uint32_t xg_u = smem_u32(xg), kr_u = smem_u32(st + C::XB);
      // byte offset of 16-byte chunk `ch` of tile row r in this group's blocks
      auto at = [&](int r, int ch) -> uint32_t {
        return C::VROW == 128 ? (ch >> 3) * C::BOX + r * 128 + (((ch & 7) ^ r8) << 4)
                              : (ch / C::CPR) * C::BOX + swz<C::VROW>(r * C::VROW + (ch % C::CPR) * 16);
      };
      // ---- scores: two accumulator chains per 16 tokens
      float sc[C::MT][4];
#pragma unroll
      for (int mm = 0; mm < C::MT; ++mm) {
        const int arow = a_row + mm * 16;
        float acc[2][C::NT][4];
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c2][nt][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < C::KS; ++ks) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4(xg_u + at(arow, ks * 2 + a_kc), a0, a1, a2, a3);
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt)
            mma_bf16(acc[ks & 1][nt], a0, a1, a2, a3, qb[nt][ks][0], qb[nt][ks][1]);
        }
#pragma unroll
        for (int rs = 0; rs < C::RS; ++rs) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4(kr_u + swz<C::KR_SW>(arow * C::DRP * 2 + (rs * 2 + a_kc) * 16), a0, a1, a2, a3);
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt)
            mma_bf16(acc[(C::KS + rs) & 1][nt], a0, a1, a2, a3, qr[nt][rs][0], qr[nt][rs][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x;
          if constexpr (C::CPW == 8) x = (acc[0][0][e] + acc[1][0][e]) + (acc[0][1][e] + acc[1][1][e]);
          else {
            x = acc[0][0][e] + acc[1][0][e];
            x += __shfl_xor_sync(0xffffffffu, x, 2);
          }
          const int r = mm * 16 + gq + (e >= 2 ? 8 : 0);
          sc[mm][e] = (r < nvalid && t0 + r <= ((e & 1) ? lim1 : lim0)) ? x : -INFINITY;
        }
      }
      // ---- V^T fragments, requested before the softmax so their latency overlaps it
      uint32_t vf[C::MT][C::KS][4];
#pragma unroll
      for (int mm = 0; mm < C::MT; ++mm)
#pragma unroll
        for (int md = 0; md < C::KS; ++md)
          ldsm_x4_t(xg_u + at(v_tok + mm * 16, md * 2 + v_dc), vf[mm][md][0], vf[mm][md][1], vf[mm][md][2],
                    vf[mm][md][3]);
      // ---- online softmax; this thread owns columns hcol, hcol + 1
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int mm = 0; mm < C::MT; ++mm) {
        mx0 = fmaxf(mx0, fmaxf(sc[mm][0], sc[mm][2]));
        mx1 = fmaxf(mx1, fmaxf(sc[mm][1], sc[mm][3]));
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
      }
      const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
      // no key seen yet: exponentiate against 0, so that p = 0 and alpha = 0, never NaN
      const float ms0 = mn0 == -INFINITY ? 0.f : mn0, ms1 = mn1 == -INFINITY ? 0.f : mn1;
      const float al0 = ex2(m0 - ms0), al1 = ex2(m1 - ms1);
      m0 = mn0;
      m1 = mn1;
      float rs0 = 0.f, rs1 = 0.f;
      uint32_t bp[C::MT][C::NT][2];
#pragma unroll
      for (int mm = 0; mm < C::MT; ++mm) {
        const float p0 = ex2(sc[mm][0] - ms0), p1 = ex2(sc[mm][1] - ms1);
        const float p2 = ex2(sc[mm][2] - ms0), p3 = ex2(sc[mm][3] - ms1);
        rs0 += p0 + p2;
        rs1 += p1 + p3;
        const float h0 = bf16_round(p0), h1 = bf16_round(p1), h2 = bf16_round(p2), h3 = bf16_round(p3);
        if constexpr (C::CPW == 8) {
          bp[mm][0][0] = movm_t(pack_bf16(h0, h1));
          bp[mm][0][1] = movm_t(pack_bf16(h2, h3));
          bp[mm][1][0] = movm_t(pack_bf16(p0 - h0, p1 - h1));
          bp[mm][1][1] = movm_t(pack_bf16(p2 - h2, p3 - h3));
        } else {
          bp[mm][0][0] = movm_t(lo_half ? pack_bf16(p0 - h0, p1 - h1) : pack_bf16(h0, h1));
          bp[mm][0][1] = movm_t(lo_half ? pack_bf16(p2 - h2, p3 - h3) : pack_bf16(h2, h3));
        }
      }
      l0 = l0 * al0 + rs0;
      l1 = l1 * al1 + rs1;
#pragma unroll
      for (int md = 0; md < C::KS; ++md) {
        o[md][0] *= al0;
        o[md][1] *= al1;
        o[md][2] *= al0;
        o[md][3] *= al1;
      }
      // ---- O^T += V^T P
#pragma unroll
      for (int mm = 0; mm < C::MT; ++mm)
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int md = 0; md < C::KS; ++md)
            mma_bf16(o[md], vf[mm][md][0], vf[mm][md][1], vf[mm][md][2], vf[mm][md][3], bp[mm][nt][0],
                     bp[mm][nt][1]);
      if (ragged) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(empty + s));
    }

    // ---- end of the piece: final rows where this CTA had the whole sequence
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if constexpr (C::CPW == 4) {
#pragma unroll
      for (int md = 0; md < C::KS; ++md)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[md][e] += __shfl_xor_sync(0xffffffffu, o[md][e], 2);
    }
    if (!ok || lo_half) continue;
    const bool whole = u1 - u0 == tp[b + 1] - tp[b];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (hcol + e >= ncol) continue;
      const int head = e ? head1 : head0, qi = e ? qi1 : qi0;
      const float m = e ? m1 : m0, l = e ? l1 : l0;
      if (whole) {
        const long long orow = (long long)(sq.r0 + qi) * a.H + head;
        const float inv = norm_of(l);
        if (a.out_bf16) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + orow * C::D_H + gq;
#pragma unroll
          for (int md = 0; md < C::KS; ++md) {
            dst[md * 16] = __float2bfloat16_rn(o[md][e] * inv);
            dst[md * 16 + 8] = __float2bfloat16_rn(o[md][e + 2] * inv);
          }
        } else {
          float* dst = reinterpret_cast<float*>(a.out) + orow * C::D_H + gq;
#pragma unroll
          for (int md = 0; md < C::KS; ++md) {
            dst[md * 16] = o[md][e] * inv;
            dst[md * 16 + 8] = o[md][e + 2] * inv;
          }
        }
        if (gq == 0 && a.lse) a.lse[orow] = natural_lse(m, l);
      } else {
        const long long ph = (long long)(blockIdx.x + b) * Hp + qi * a.H + head;
        float* dst = a.part_o + ph * C::D_H + gq;
#pragma unroll
        for (int md = 0; md < C::KS; ++md) {
          dst[md * 16] = o[md][e];
          dst[md * 16 + 8] = o[md][e + 2];
        }
        if (gq == 0) a.part_ml[ph] = make_float2(m, l);
      }
    }
  }
}

// Visit the configuration of (d_h, G, columns, padded d_r); false if there is none.
template <class F>
bool dispatch(const gva_shape_t& sh, int cols, F&& f) {
  const int drp = sh.d_r == 0 ? 0 : (sh.d_r <= 16 ? 16 : (sh.d_r <= 32 ? 32 : -1));
#define GVA_PM(DH, NG, COLS, DRP)                                                \
  if (sh.d_h == DH && sh.G == NG && cols == COLS && drp == DRP) {                \
    f(PmCfg<DH, NG, COLS, DRP>{});                                               \
    return true;                                                                 \
  }
#define GVA_PM_COLS(DH, NG, DRP) GVA_PM(DH, NG, 4, DRP) GVA_PM(DH, NG, 8, DRP)
#define GVA_PM_NG(DH, DRP)                                                       \
  GVA_PM_COLS(DH, 2, DRP) GVA_PM_COLS(DH, 4, DRP) GVA_PM_COLS(DH, 8, DRP) GVA_PM(DH, 2, 16, DRP)
#define GVA_PM_DR(DH) GVA_PM_NG(DH, 0) GVA_PM_NG(DH, 16) GVA_PM_NG(DH, 32)
#define GVA_PM_WIDE(DH) GVA_PM(DH, 4, 16, 0) GVA_PM(DH, 4, 16, 16) GVA_PM(DH, 4, 16, 32)
  GVA_PM_DR(32)
  GVA_PM_WIDE(32)
  GVA_PM_DR(64)
  GVA_PM_WIDE(64)
  GVA_PM_DR(128)
#undef GVA_PM_WIDE
#undef GVA_PM_DR
#undef GVA_PM_NG
#undef GVA_PM_COLS
#undef GVA_PM
  return false;
}

}  // namespace

bool paged_mma_supported(const gva_shape_t& sh, int page) {
  if (sh.cache_dtype != GVA_BF16 || page % 8 || sh.H / sh.G > 8) return false;
  return dispatch(sh, 4, [](auto) {});
}

// Columns of the variant that takes `columns` per group (16: two warps per group, up to 4
// groups and rows of 512 bytes), 0 if they are work for 128-row blocks.  Four new tokens of
// four heads on 16 x 1k-8k and 4 x 512-2k tokens: d_h = 64, 4 groups 26.8 and 12.1 us (row
// blocks 30.8 and 15.7), d_h = 128, 2 groups 25.6 and 12.9 us (32.9 and 16.5); 4 groups of
// d_h = 128 42.4 and 18.0 us (46.3 and 17.0), on 64 x 1k-8k 140 (133).  With three warps per
// group, five tokens took 32.6 us (31.9), on 64 x 1k-8k 100 (80): the split of the query
// doubles products that mma.sync already bounds.
int paged_mma_cols(const gva_shape_t& sh, long long columns) {
  if (columns <= 8) return columns <= 4 ? 4 : 8;
  return columns <= 16 && sh.G <= 4 && sh.G * sh.d_h <= 256 ? 16 : 0;
}

int paged_mma_tile(const gva_shape_t& sh) {
  int tt = 0;
  dispatch(sh, 4, [&](auto c) { tt = decltype(c)::TT; });
  return tt;
}

int paged_mma_grid(const gva_shape_t& sh, int cols, int num_sms, long long max_total, int cap_B) {
  int tt = 16, minb = 2;
  size_t smem = 0;
  dispatch(sh, cols, [&](auto c) {
    tt = decltype(c)::TT;
    minb = decltype(c)::MINB;
    smem = decltype(c)::smem_bytes(cap_B);
  });
  int per_sm = (int)((227 * 1024) / (smem + 1024));
  per_sm = per_sm < 1 ? 1 : (per_sm > minb ? minb : per_sm);
  if (sh.ctas_per_sm > 0) per_sm = sh.ctas_per_sm;
  const long long want = (max_total + tt - 1) / tt + sh.B;   // a sequence may end in a ragged tile
  const long long grid = (long long)num_sms * per_sm;
  return (int)(want < grid ? want : grid);
}

cudaError_t launch_paged_mma(const gva_shape_t& sh, const PagedArgs& a, int cols, const CUtensorMap& tv,
                             const CUtensorMap& tk, cudaStream_t st) {
  cudaError_t err = cudaErrorNotSupported;
  dispatch(sh, cols, [&](auto c) {
    using C = decltype(c);
    const size_t smem = C::smem_bytes(sh.B);
    if ((err = ensure_max_smem(paged_mma_kernel<C>, smem)) != cudaSuccess) return;
    err = launch_pdl(paged_mma_kernel<C>, dim3(a.grid), dim3(C::THREADS), smem, st, a, tv, tk);
  });
  return err;
}

}  // namespace gva
