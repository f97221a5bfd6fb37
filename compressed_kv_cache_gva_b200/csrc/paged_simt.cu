// Paged attention on the CUDA cores: any type, width, page size and number of query
// rows within the limits below (float32 caches, where fp32 products are wanted, and
// the shapes no tensor-core kernel is built for).
//
// Row blocks of 16 query rows, tiles of 32 keys staged as fp32 in shared memory
// (rows padded to an odd stride, so that 16 keys at one column hit 16 banks).
// Thread (r, x) of 16 x 16: scores of row r with keys x and x + 16, online softmax
// over the row's 16 threads, then output columns x, x + 16, ... of row r.
// Bound by the fp32 FMAs and their shared-memory operands, about one load per FMA.
#include <type_traits>

#include "launch.h"
#include "paged.cuh"

namespace gva {

namespace {

constexpr int kM = kPagedSimtRows, kTK = 32, kOV = 1, kThreads = 256;
constexpr int kMaxD = 512;

struct SimtSmem {
  int ldq, ldv, ldr;
  size_t q, v, kr, p, prefix, wtmp, total;
};

__host__ __device__ inline SimtSmem simt_smem(int B, int d_h, int d_r) {
  SimtSmem s;
  s.ldq = (d_h + d_r) | 1;
  s.ldv = d_h | 1;
  s.ldr = d_r | 1;
  size_t o = 0;
  s.q = o; o = align_up(o + 4u * kM * s.ldq, 16);
  s.v = o; o = align_up(o + 4u * kTK * s.ldv, 16);
  s.kr = o; o = align_up(o + 4u * kTK * s.ldr, 16);
  s.p = o; o = align_up(o + 4u * kM * (kTK + 1), 16);
  s.prefix = o; o = align_up(o + 4u * (B + 1), 16);
  s.wtmp = o; o += 8u * 33;
  s.total = o;
  return s;
}

template <typename T, int COLS>   // output columns per thread: d_h <= 16 COLS
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(const PagedArgs a, const SimtSmem S) {
  extern __shared__ __align__(16) unsigned char sm[];
  float* Qs = reinterpret_cast<float*>(sm + S.q);
  float* Vs = reinterpret_cast<float*>(sm + S.v);
  float* Ks = reinterpret_cast<float*>(sm + S.kr);
  float* Ps = reinterpret_cast<float*>(sm + S.p);
  int* prefix = reinterpret_cast<int*>(sm + S.prefix);
  long long* wtmp = reinterpret_cast<long long*>(sm + S.wtmp);
  __shared__ RowPiece piece;
  __shared__ int more;

  const int tid = threadIdx.x, r = tid >> 4, x = tid & 15;
  const int d_h = a.d_h, d_r = a.d_r, dq = d_h + d_r, hpr = a.hpr;
  const T* V = reinterpret_cast<const T*>(a.V);
  const T* KR = reinterpret_cast<const T*>(a.KR);
  // queries, lengths, tables and cache rows may come from the kernels before
  pdl_enter(a);
  if (blockIdx.x == 0 && a.flag_errors) flag_bad_sequences(a);
  const RowBlocks<kM, kTK, kOV> blocks{a};
  TileSplit ts;
  long long total;
  RowWalk<kM, kTK, kOV> walk{blocks, prefix, 0, 0, {}, {}};
  if (a.B <= kLaneBatch) {
    const LaneBatch t = lane_batch(a, [&](const SeqRows& s) { return blocks.units(s); });
    total = t.total;
    ts = make_split(total < (1ll << 31) ? (int)total : 0, (int)gridDim.x, 0);
    walk.end = ts.first(blockIdx.x + 1);
    if (tid < 32) {
      const bool any = walk.first(ts.first(blockIdx.x), t);
      if (tid == 0) {
        more = any;
        piece = walk.p;
      }
    }
  } else {
    total = block_scan(a.B, [&](int b) { return blocks.units(b); }, prefix, wtmp);
    ts = make_split(prefix[a.B], (int)gridDim.x, 0);
    walk.end = ts.first(blockIdx.x + 1);
    if (tid < 32) {
      const bool any = walk.first(ts.first(blockIdx.x));
      if (tid == 0) {
        more = any;
        piece = walk.p;
      }
    }
  }
  if (total >= (1ll << 31) && tid == 0) atomicOr(a.status, GVA_DEVERR_RANGE);
  if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  while (more) {
    const RowPiece p = piece;
    const SeqRows s = seq_rows(a, p.b);
    const int* row = a.table + (long long)p.b * a.table_stride;
    const int row0 = p.rb * kM, rows = min(kM, s.n * hpr - row0);
    for (int e = tid; e < kM * dq; e += kThreads) {
      const int rr = e / dq, c = e - rr * dq;
      const int R = row0 + rr, qi = R / hpr, head = p.g * hpr + R % hpr;
      Qs[rr * S.ldq + c] =
          rr < rows ? a.q_abs[((long long)(s.r0 + qi) * a.H + head) * dq + c] : 0.f;
    }
    const int qi = (row0 + r) / hpr, head = p.g * hpr + (row0 + r) % hpr;
    const int lim = s.L - s.n + qi;   // last key of this row
    float m = -INFINITY, l = 0.f, o[COLS];
#pragma unroll
    for (int i = 0; i < COLS; ++i) o[i] = 0.f;
    for (int k = p.k0; k < p.k1; ++k) {
      const int t0 = k * kTK;
      __syncthreads();   // the previous tile (and this block's queries) are in place / free
      for (int t = tid >> 5; t < kTK; t += kThreads / 32) {   // one warp per key
        const int slot = slot_of(a, row, t0 + t, s.L);
        const bool ok = slot < a.num_slots;
        const T* src = V + ((long long)(ok ? slot : 0) * a.G + p.g) * d_h;
        for (int c = tid & 31; c < d_h; c += 32) Vs[t * S.ldv + c] = ok ? to_f32(src[c]) : 0.f;
        const T* rsrc = KR + (long long)(ok ? slot : 0) * d_r;
        for (int c = tid & 31; c < d_r; c += 32) Ks[t * S.ldr + c] = ok ? to_f32(rsrc[c]) : 0.f;
      }
      __syncthreads();
      float sc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = x + 16 * u;
        const float* q = Qs + r * S.ldq;
        const float* v = Vs + t * S.ldv;
        float acc = 0.f;
        for (int c = 0; c < d_h; ++c) acc = fmaf(q[c], v[c], acc);
        const float* kr = Ks + t * S.ldr;
        for (int c = 0; c < d_r; ++c) acc = fmaf(q[d_h + c], kr[c], acc);
        sc[u] = (r < rows && t0 + t <= lim && t0 + t < s.L) ? acc : -INFINITY;
      }
      float mx = fmaxf(sc[0], sc[1]);
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
      const float al = ex2(m - ms), p0 = ex2(sc[0] - ms), p1 = ex2(sc[1] - ms);
      float sum = p0 + p1;
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      m = mn;
      l = l * al + sum;
      Ps[r * (kTK + 1) + x] = p0;
      Ps[r * (kTK + 1) + x + 16] = p1;
      __syncwarp();   // a row's 16 threads are in one warp
#pragma unroll
      for (int i = 0; i < COLS; ++i) o[i] *= al;
      for (int t = 0; t < kTK; ++t) {
        const float pt = Ps[r * (kTK + 1) + t];
        const float* v = Vs + t * S.ldv + x;
#pragma unroll
        for (int i = 0; i < COLS; ++i)
          if (x + 16 * i < d_h) o[i] = fmaf(pt, v[16 * i], o[i]);
      }
      __syncwarp();
    }
    const bool whole = p.k0 == 0 && p.k1 == p.nt;
    if (r < rows) {
      if (whole) {
        const long long orow = (long long)(s.r0 + qi) * a.H + head;
        const float inv = norm_of(l);
#pragma unroll
        for (int i = 0; i < COLS; ++i) {
          const int c = x + 16 * i;
          if (c >= d_h) break;
          if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[orow * d_h + c] = __float2bfloat16_rn(o[i] * inv);
          else reinterpret_cast<float*>(a.out)[orow * d_h + c] = o[i] * inv;
        }
        if (x == 0 && a.lse) a.lse[orow] = natural_lse(m, l);
      } else {
        const long long slot = piece_slot(p, blockIdx.x);
        float* po = a.part_o + (slot * kM + r) * d_h;
#pragma unroll
        for (int i = 0; i < COLS; ++i) {
          const int c = x + 16 * i;
          if (c >= d_h) break;
          po[c] = o[i];
        }
        if (x == 0) a.part_ml[slot * kM + r] = make_float2(m, l);
      }
    }
    if (tid == 0) {
      write_row_meta(a, ts, walk);
      more = walk.next();
      piece = walk.p;
    }
    __syncthreads();
  }
  pdl_leave(a);
}

}  // namespace

bool paged_simt_supported(const gva_shape_t& sh) {
  return sh.d_h <= kMaxD && simt_smem(sh.B, sh.d_h, sh.d_r).total <= 200 * 1024;
}

int paged_simt_grid(const gva_shape_t& sh, int n_rows, int num_sms, long long max_total, int cap_B) {
  const size_t smem = simt_smem(cap_B, sh.d_h, sh.d_r).total;
  int per_sm = (int)((220 * 1024) / (smem + 1024));
  per_sm = per_sm < 1 ? 1 : (per_sm > 3 ? 3 : per_sm);
  if (sh.ctas_per_sm > 0) per_sm = sh.ctas_per_sm;
  // no more CTAs than blocks x tiles could be
  const long long blocks = ((long long)n_rows * (sh.H / sh.G) + kM - 1) / kM + sh.B;
  const long long want = blocks * sh.G * (max_total / kTK + 1);
  const long long grid = (long long)num_sms * per_sm;
  return (int)(want < grid ? want : grid);
}

cudaError_t launch_paged_simt(const gva_shape_t& sh, const PagedArgs& a, cudaStream_t st) {
  const SimtSmem S = simt_smem(sh.B, sh.d_h, sh.d_r);
  auto go = [&](auto k) {
    const cudaError_t e = ensure_max_smem(k, S.total);
    return e == cudaSuccess ? launch_pdl(k, dim3(a.grid), dim3(kThreads), S.total, st, a, S) : e;
  };
  auto by_type = [&](auto cols) {
    constexpr int COLS = decltype(cols)::value;
    return sh.cache_dtype == GVA_BF16 ? go(paged_simt_kernel<__nv_bfloat16, COLS>)
                                      : go(paged_simt_kernel<float, COLS>);
  };
  if (sh.d_h <= 64) return by_type(std::integral_constant<int, 4>{});
  if (sh.d_h <= 128) return by_type(std::integral_constant<int, 8>{});
  return by_type(std::integral_constant<int, 32>{});
}

}  // namespace gva
