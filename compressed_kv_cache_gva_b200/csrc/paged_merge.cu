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
      if (e[u].x == -INFINITY) continue;    // a piece past this query's last key
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
    const float mu = sm_m[u][lane];
    if (mu == -INFINITY) continue;
    const float f = ex2(mu - M);
    L = fmaf(f, sm_l[u][lane], L);
    O = fmaf(f, sm_o[u][lane], O);
  }
  const long long orow = (long long)(r0 + qi) * a.H + h % a.H;
  if (col) store_out(a, orow, d, L > 0.f ? O / L : 0.f);
  if (lane == 0 && z == 0 && a.lse) a.lse[orow] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

// Row blocks cut between CTAs: a warp per row.  Block (i, y) merges rows y W .. y W + W-1
// (W warps) of the block that CTA i of the split started and did not end; its pieces lie
// in slots 2 i + 1, 2 (i + 1), 2 (i + 2), ...  A warp holds the piece weights of its row
// one per lane, then walks the pieces.
__device__ __forceinline__ void merge_rows(const PagedArgs& a, int i, int y, int M) {
  const int r = y * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int4 meta = a.meta[i];
  const int n = meta.x;
  if (n == 0 || r >= M) return;
  const int b = meta.y, g = meta.z, R = meta.w * M + r;
  const int r0 = a.q_start[b], rows = (a.q_start[b + 1] - r0) * a.hpr;
  if (R >= rows) return;
  const int d_h = a.d_h;
  auto slot = [&](int c) { return c == 0 ? 2 * i + 1 : 2 * (i + c); };
  float mx = -INFINITY;
  for (int c = lane; c < n; c += 32) mx = fmaxf(mx, a.part_ml[(size_t)slot(c) * M + r].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ms = mx == -INFINITY ? 0.f : mx;
  const int qi = R / a.hpr, head = g * a.hpr + R % a.hpr;
  const long long orow = (long long)(r0 + qi) * a.H + head;
  float L = 0.f;
  for (int d0 = 0; d0 < d_h; d0 += 128) {   // 4 columns per lane and turn
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    L = 0.f;
    for (int c0 = 0; c0 < n; c0 += 32) {
      const int c = c0 + lane;
      float w = 0.f;
      if (c < n) {
        const float2 e = a.part_ml[(size_t)slot(c) * M + r];
        w = ex2(e.x - ms);
        L = fmaf(w, e.y, L);
      }
      const int cn = min(32, n - c0);
      for (int j = 0; j < cn; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float* po = a.part_o + ((size_t)slot(c0 + j) * M + r) * d_h;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int d = d0 + lane + 32 * u;
          if (d < d_h) o[u] = fmaf(wj, po[d], o[u]);
        }
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int d = d0 + lane + 32 * u;
      if (d < d_h) store_out(a, orow, d, o[u] * inv);
    }
  }
  if (lane == 0 && a.lse) a.lse[orow] = L > 0.f ? (mx + log2f(L)) * kLn2 : -INFINITY;
}

// Both kinds in one launch: blocks [0, seq_blocks) take sequences, the rest row blocks.
__global__ void __launch_bounds__(1024)
    paged_merge_kernel(const PagedArgs s, const PagedArgs r, int seq_blocks, int Hp, int chunks, int rows_y,
                       int M) {
  pdl_trigger();   // successors wait for this kernel before they read its outputs
  pdl_wait();
  int i = blockIdx.x;
  if (i < seq_blocks) {
    const int z = i % chunks;
    i /= chunks;
    merge_seq(s, i / Hp, i % Hp, z, Hp);
  } else {
    i -= seq_blocks;
    merge_rows(r, i / rows_y, i % rows_y, M);
  }
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs* s, const PagedArgs* r, int M, cudaStream_t st) {
  int npg = 8, Hp = 1, chunks = 1, rows_y = 1;
  long long seq_blocks = 0, row_blocks = 0;
  if (s) {
    // a sequence has about grid / B + 1 pieces (ragged batches: more for the long ones)
    const int per_seq = s->grid / s->B + 2;
    npg = (per_seq + kPieces - 1) / kPieces;
    npg = npg < 1 ? 1 : (npg > 32 ? 32 : npg);
    if (r && npg < 8) npg = 8;
    Hp = s->H * s->max_new;
    chunks = (s->d_h + 31) / 32;
    seq_blocks = (long long)s->B * Hp * chunks;
  }
  if (r) {
    const long long most = (long long)r->max_new * r->hpr;   // rows of the fullest block
    rows_y = (int)(((most < M ? most : M) + npg - 1) / npg);
    row_blocks = (long long)r->grid * rows_y;
  }
  const PagedArgs none{};
  return launch_pdl(paged_merge_kernel, dim3((unsigned)(seq_blocks + row_blocks)), dim3(32 * npg), 0, st,
                    s ? *s : none, r ? *r : none, (int)seq_blocks, Hp, chunks, rows_y, M);
}

}  // namespace gva
