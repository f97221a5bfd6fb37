// Merge of the pieces of the paged attention kernels: pieces c of the same query row
// hold (m_c, l_c, o_c) in base 2,
//   m* = max m_c,  L = sum 2^(m_c - m*) l_c,  out = sum 2^(m_c - m*) o_c / L,
//   lse = (m* + log2 L) ln 2.
// The order is fixed by the piece index, so results do not depend on which CTA was
// first.  Partials are read once, from L2.
#include "launch.h"
#include "paged.cuh"

namespace gva {

namespace {

__device__ __forceinline__ void store_out(const PagedArgs& a, long long orow, int d, float v) {
  if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[orow * a.d_h + d] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(a.out)[orow * a.d_h + d] = v;
}

// Sequences cut by the split-KV kernel: block (b, h of H * rows, z of d_h / 32), 32
// columns x PG piece groups: group pg merges pieces pg, pg + PG, ... (all loads
// requested before the first use), then the groups merge through shared memory.
constexpr int kPieces = 4;   // pieces per thread in flight
__device__ __forceinline__ void merge_seq(const PagedArgs& a, int b, int h, int z, int Hp) {
  __shared__ float sm_m[32][33], sm_l[32][33], sm_o[32][33];
  const int lane = threadIdx.x & 31, d = z * 32 + lane;
  const int pg = threadIdx.x >> 5, npg = blockDim.x >> 5, d_h = a.d_h;
  const int4 meta = a.meta[b];
  const int n = meta.y;
  if (n <= 1) return;                       // nothing here, or written by its one CTA
  const int r0 = a.q_start[b], rows = a.q_start[b + 1] - r0, qi = h / a.H;
  if (qi >= rows) return;
  const bool col = d < d_h;
  const float2* ml = a.part_ml + (size_t)meta.x * Hp + h;
  const float* po = a.part_o + ((size_t)meta.x * Hp + h) * d_h + (col ? d : 0);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int c0 = pg; c0 < n; c0 += kPieces * npg) {
    float2 e[kPieces];
    float x[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int c = c0 + u * npg;
      if (c < n) {
        e[u] = ml[(size_t)c * Hp];
        x[u] = po[(size_t)c * Hp * d_h];
      }
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (c0 + u * npg >= n) break;
      if (e[u].y == 0.f) continue;          // no key of the piece is this query's
      const float mn = fmaxf(m, e[u].x);
      const float f = ex2(m - mn), w = ex2(e[u].x - mn);
      l = l * f + w * e[u].y;
      o = o * f + w * x[u];
      m = mn;
    }
  }
  sm_m[pg][lane] = m;
  sm_l[pg][lane] = l;
  sm_o[pg][lane] = o;
  __syncthreads();
  if (pg != 0) return;
  float M = -INFINITY;
  for (int u = 0; u < npg; ++u) M = fmaxf(M, sm_m[u][lane]);
  float L = 0.f, O = 0.f;
  for (int u = 0; u < npg; ++u) {
    if (sm_l[u][lane] == 0.f) continue;
    const float f = ex2(sm_m[u][lane] - M);
    L = fmaf(f, sm_l[u][lane], L);
    O = fmaf(f, sm_o[u][lane], O);
  }
  const long long orow = (long long)(r0 + qi) * a.H + h % a.H;
  if (col) store_out(a, orow, d, L == 0.f ? 0.f : O / L);
  if (lane == 0 && z == 0 && a.lse) a.lse[orow] = natural_lse(M, L);
}

// Row blocks cut between CTAs: the block that CTA i of the split started and did not end;
// its pieces lie in slots 2 i + 1, 2 (i + 1), 2 (i + 2), ...  A thread merges VEC columns
// of one row: after the block's record, which names its rows, one round of loads fetches
// four pieces.  Many small threads: two dependent latencies are nearly all of the time
// (a warp per row with its piece weights in lanes, or four rows per warp, took 24 and
// 28 us after a chunk of 8 x 512 tokens).
constexpr int kRowThreads = 256;
template <int VEC>
__device__ __forceinline__ void merge_rows(const PagedArgs& a, int i, int y, int M) {
  const int4 meta = a.meta[2 * i], where = a.meta[2 * i + 1];   // pieces, block, group; first row, rows
  const unsigned tpr = a.d_h / VEC, e = (unsigned)y * kRowThreads + threadIdx.x;
  const unsigned r = e / tpr, d = (e - r * tpr) * VEC;
  const int n = meta.x;
  if (n == 0 || (int)r >= min(where.y, M)) return;
  float m = -INFINITY, l = 0.f, o[VEC];
#pragma unroll
  for (int u = 0; u < VEC; ++u) o[u] = 0.f;
  for (int c0 = 0; c0 < n; c0 += kPieces) {
    float2 ml[kPieces];
    float x[kPieces][VEC];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      ml[c] = make_float2(-INFINITY, 0.f);
      if (c0 + c < n) {
        const size_t row = (size_t)(c0 + c == 0 ? 2 * i + 1 : 2 * (i + c0 + c)) * M + r;
        ml[c] = a.part_ml[row];
        if constexpr (VEC == 4) {
          const float4 v = *reinterpret_cast<const float4*>(a.part_o + row * a.d_h + d);
          x[c][0] = v.x; x[c][1] = v.y; x[c][2] = v.z; x[c][3] = v.w;
        } else {
          x[c][0] = a.part_o[row * a.d_h + d];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      if (ml[c].y == 0.f) continue;         // no piece, or none of its keys is this row's
      const float mn = fmaxf(m, ml[c].x);
      const float f = ex2(m - mn), w = ex2(ml[c].x - mn);
      l = l * f + w * ml[c].y;
#pragma unroll
      for (int u = 0; u < VEC; ++u) o[u] = o[u] * f + w * x[c][u];
      m = mn;
    }
  }
  const unsigned R = meta.w * M + r, qi = R / (unsigned)a.hpr;
  const long long orow = (long long)(where.x + (int)qi) * a.H + meta.z * a.hpr + (int)(R - qi * a.hpr);
  const float inv = norm_of(l);
#pragma unroll
  for (int u = 0; u < VEC; ++u) o[u] *= inv;
  if constexpr (VEC == 4) {
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + orow * a.d_h + d) =
          make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + orow * a.d_h + d) =
          make_float4(o[0], o[1], o[2], o[3]);
  } else {
    store_out(a, orow, d, o[0]);
  }
  if (d == 0 && a.lse) a.lse[orow] = natural_lse(m, l);
}

// Both kinds in one launch: blocks [0, seq_blocks) take sequences, the rest row blocks.
// ROWS false: sequences only, with as many warps per block as their pieces want.
template <bool ROWS>
__global__ void __launch_bounds__(ROWS ? kRowThreads : 1024)
    paged_merge_kernel(const PagedArgs s, const PagedArgs r, int seq_blocks, int Hp, int chunks, int rows_y,
                       int M) {
  pdl_trigger();   // successors wait for this kernel before they read its outputs
  pdl_wait();
  int i = blockIdx.x;
  if (!ROWS || i < seq_blocks) {
    const int z = i % chunks;
    i /= chunks;
    merge_seq(s, i / Hp, i % Hp, z, Hp);
  } else if constexpr (ROWS) {
    i -= seq_blocks;
    if (r.d_h % 4 == 0) merge_rows<4>(r, i / rows_y, i % rows_y, M);
    else merge_rows<1>(r, i / rows_y, i % rows_y, M);
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs* s, const PagedArgs* r, int M, cudaStream_t st) {
  int npg = kRowThreads / 32, Hp = 1, chunks = 1, rows_y = 1;
  long long seq_blocks = 0, row_blocks = 0;
  if (s) {
    if (!r) {
      // a sequence has about grid / B + 1 pieces (ragged batches: more for the long ones)
      const int per_seq = s->grid / s->B + 2;
      npg = (per_seq + kPieces - 1) / kPieces;
      npg = npg < 1 ? 1 : (npg > 32 ? 32 : npg);
    }
    Hp = s->H * s->max_new;
    chunks = (s->d_h + 31) / 32;
    seq_blocks = (long long)s->B * Hp * chunks;
  }
  if (r) {
    const long long most = (long long)r->max_new * r->hpr, rows = most < M ? most : M;   // of the fullest block
    const int tpr = r->d_h % 4 == 0 ? r->d_h / 4 : r->d_h;
    rows_y = (int)((rows * tpr + kRowThreads - 1) / kRowThreads);
    row_blocks = (long long)r->grid * rows_y;
  }
  const PagedArgs none{};
  auto go = [&](auto k) {
    return launch_pdl(k, dim3((unsigned)(seq_blocks + row_blocks)), dim3(32 * npg), 0, st, s ? *s : none,
                      r ? *r : none, (int)seq_blocks, Hp, chunks, rows_y, M);
  };
  return r ? go(paged_merge_kernel<true>) : go(paged_merge_kernel<false>);
}

}  // namespace gva
