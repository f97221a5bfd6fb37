// Verification of drafted tokens against the target model's probabilities
// (speculative sampling), from given random numbers.
//
// Request b was fed n = k + 1 tokens, rows q_start[b] .. q_start[b+1]-1: its last
// token and k drafts x_1..x_k.  Row j holds the target's distribution p_j of the
// token after fed token j, and the draft's q_j from which x_{j+1} was drawn (one-hot
// at x_{j+1} where there is no draft model).  In order, draft j+1 is accepted while
//   u_j * q_j(x) < p_j(x);
// with a drafts accepted, one more token follows, drawn from
//   w = max(p_a - q_a, 0)  (a < k: the residual)   or   w = p_a  (a = k)
// by inversion: the first v whose running sum of w exceeds u * sum(w).  Accepted
// tokens and this one are then distributed as the target's own samples.
//
// What bounds it: memory.  Besides k probabilities a request reads one row of each
// model, vocab * 2 * 4 bytes, once.  A cluster of CTAs shares a request: each warp
// sums a contiguous chunk through a ring in shared memory, up to three CTAs per SM,
// the chunk sums meet through distributed shared memory, and the CTA whose chunk
// holds the answer reads it again from L2, an eighth per warp.
// Sums keep 48 bits (64-bit sums of pairs, whose exact rounding errors are summed in
// 32; see chunk_sum_of): with ~10^5 tokens of mass ~10^-5 each, 32-bit running sums are
// off by a good part of a token's mass, and the drawn token would depend on the order
// of the additions.
#include "common.cuh"
#include "launch.h"
#include "paged.h"

namespace gva {

namespace {

constexpr int kVfWarps = 8;
constexpr int kVfThreads = 32 * kVfWarps;
constexpr int kVfMaxCluster = 8;
// A warp's part of the shared-memory ring: units of 512 bytes (a 16-byte vector per lane).
constexpr int kVfUnits = 12;
constexpr int kVfRing = kVfWarps * kVfUnits * 512;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (Both want whole warps together.)
__device__ __forceinline__ void cl_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cl_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A double from the same shared-memory offset of another CTA of the cluster.
__device__ __forceinline__ double ld_cluster_f64(const double* p, uint32_t rank) {
  uint32_t local = smem_u32(p), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote) : "memory");
  return v;
}

// VEC consecutive elements of a row as floats, from element v (which may be < 0 or
// reach past n: those read as 0).  vec: the 16-byte load is aligned.
template <typename T> struct RowVec;
template <> struct RowVec<float> { static constexpr int N = 4; };
template <> struct RowVec<__nv_bfloat16> { static constexpr int N = 8; };

template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int v, int n, bool vec) {
  constexpr int N = RowVec<T>::N;
  if (vec && v >= 0 && v + N <= n) return __ldg(reinterpret_cast<const uint4*>(row + v));
  union { uint4 u; T e[N]; } x;
  x.u = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (v + i >= 0 && v + i < n) x.e[i] = row[v + i];
  return x.u;
}
__device__ __forceinline__ void widen(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void widen(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The weights of one row: p, max(p - q, 0) (q: the draft's row), or p without
// token `skip`.  Anything that is not > 0 (NaN too) counts as 0.
template <typename T>
struct Weights {
  static constexpr int N = RowVec<T>::N;
  const T* p;
  const T* q;      // or null
  int vocab, skip; // skip < 0: none
  bool vec_q;
  __device__ __forceinline__ uint4 load_p(int v) const { return load_vec(p, v, vocab, true); }
  __device__ __forceinline__ uint4 load_q(int v) const {
    return q ? load_vec(q, v, vocab, vec_q) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(int v, const uint4& up, const uint4& uq, double (&w)[N]) const {
    float a[N], b[N];
    widen(up, a);
    widen(uq, b);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double d = q ? (double)a[i] - (double)b[i] : (double)a[i];
      w[i] = (d > 0.0 && v + i != skip) ? d : 0.0;
    }
  }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Exact sum of two floats: their rounded sum, and what the rounding left (Knuth's TwoSum).
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z));
  return s;
}

// Sum of the chunk's weights: lanes take vectors 32 apart.
// A weight is kept as its rounded float and the rounding's exact error (p - q with p > q:
// Dekker's), pairs are added the same way, one value per pair goes to the 64-bit sum, and
// the errors, 2^-24 of the values, are summed in 32 bits (2^-48 of the values).  That
// leaves one conversion to 64 bits per pair instead of two per element, which queue at 16
// a clock and SM (24.5 -> 24.1 us for 64 requests x 131072 tokens by itself).
//
// The vectors pass through the warp's ring by asynchronous copies, 12 of a row (6 of
// each of two) in flight per lane: four in registers left a warp waiting one DRAM latency
// per 1 KB, and took 24.1 us against 19.4 at that size.  A lane reads only what it copied
// itself, so nothing is synchronised.  Vectors that are not aligned or leave the row go
// through registers.
template <typename T>
__device__ __forceinline__ void fetch(const T* row, int v, int n, bool vec, uint32_t dst, uint8_t* at) {
  if (vec && v >= 0 && v + RowVec<T>::N <= n)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(row + v) : "memory");
  else
    *reinterpret_cast<uint4*>(at) = load_vec(row, v, n, false);
}
// The lane's part of a chunk, every weight in 64 bits: where pairs exceed the largest float
// (weights need not be normalised).
template <typename T>
__device__ __noinline__ double lane_sum_wide(const Weights<T> W, int v0, int v1, int lane) {
  constexpr int N = RowVec<T>::N, SEG = 32 * N;
  double sum = 0.0;
  for (int v = v0 + lane * N; v - lane * N < v1; v += SEG) {
    double w[N];
    W.get(v, W.load_p(v), W.load_q(v), w);
    for (int j = 0; j < N; ++j) sum += w[j];
  }
  return sum;
}
template <typename T, bool Q>
__device__ __forceinline__ double chunk_sum_of(const Weights<T>& W, int v0, int v1, uint8_t* ring, int lane) {
  constexpr int N = RowVec<T>::N, SEG = 32 * N, S = Q ? kVfUnits / 2 : kVfUnits;
  ring += lane * 16;
  const uint32_t base = smem_u32(ring);
  auto issue = [&](int i) {
    const int v = v0 + i * SEG + lane * N, slot = i % S * (Q ? 1024 : 512);
    if (v0 + i * SEG < v1) {
      fetch(W.p, v, W.vocab, true, base + slot, ring + slot);
      if constexpr (Q) fetch(W.q, v, W.vocab, W.vec_q, base + slot + 512, ring + slot + 512);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < S - 1; ++i) issue(i);
  double acc = 0.0;
  float rest = 0.f;
  for (int i = 0; v0 + i * SEG < v1; ++i) {
    issue(i + S - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    const int v = v0 + i * SEG + lane * N, slot = i % S * (Q ? 1024 : 512);
    float p[N], q[N];
    widen(*reinterpret_cast<const uint4*>(ring + slot), p);
    if constexpr (Q) widen(*reinterpret_cast<const uint4*>(ring + slot + 512), q);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      float d[2], e[2], t;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float x = p[j + u], y = Q ? q[j + u] : 0.f;
        const float r = __fsub_rn(x, y);
        const bool on = r > 0.f && v + j + u != W.skip;
        d[u] = on ? r : 0.f;
        // a draft's probability is >= 0, so x >= y here and this is exact
        e[u] = Q && on ? __fsub_rn(__fsub_rn(x, r), y) : 0.f;
      }
      acc += (double)two_sum(d[0], d[1], t);
      rest += t + (e[0] + e[1]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");   // the ring is free again
  double sum = acc + (double)rest;
  if (!isfinite(sum)) sum = lane_sum_wide(W, v0, v1, lane);
  return warp_sum(sum);
}
template <typename T>
__device__ __forceinline__ double chunk_sum(const Weights<T>& W, int v0, int v1, uint8_t* ring, int lane) {
  return W.q ? chunk_sum_of<T, true>(W, v0, v1, ring, lane) : chunk_sum_of<T, false>(W, v0, v1, ring, lane);
}

// First v of the chunk whose running sum (from `base`) exceeds t; the last v with a
// positive weight if rounding leaves none (-1 if there is none).  One warp.
template <typename T>
__device__ __forceinline__ int chunk_find(const Weights<T>& W, int v0, int v1, double base, double t,
                                          int lane) {
  constexpr int N = RowVec<T>::N, SEG = 32 * N;
  int last = -1;
  for (int s = v0; s < v1; s += SEG) {
    const int v = s + lane * N;
    double w[N], sum = 0.0;
    W.get(v, W.load_p(v), W.load_q(v), w);
    int mine = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sum += w[i];
      if (w[i] > 0.0) mine = v + i;
    }
    double incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned over = __ballot_sync(0xffffffffu, sum > 0.0 && base + incl > t);
    if (over) {
      const int l = __ffs(over) - 1;
      double run = base + (incl - sum);
      int hit = -1;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        run += w[i];
        if (hit < 0 && w[i] > 0.0 && run > t) hit = v + i;
      }
      if (hit < 0) hit = mine;
      return __shfl_sync(0xffffffffu, hit, l);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    const unsigned pos = __ballot_sync(0xffffffffu, mine >= 0);
    if (pos) last = __shfl_sync(0xffffffffu, mine, 31 - __clz(pos));
  }
  return last;
}

template <typename T>
__global__ void __launch_bounds__(kVfThreads, 4) verify_kernel(const VerifyArgs a, const int cl) {
  __shared__ double sums[kVfWarps], part[kVfWarps];
  __shared__ double all[kVfMaxCluster * kVfWarps];
  __shared__ int s_first;
  extern __shared__ __align__(16) uint8_t vf_ring[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = vf_ring + warp * kVfUnits * 512;
  const int b = (int)blockIdx.x / cl;
  const uint32_t rank = cl > 1 ? cluster_rank() : 0u;
  // probabilities and tokens come from the kernels before
  pdl_wait();
  const int r0 = a.q_start[b], r1 = a.q_start[b + 1];
  const bool good = r0 >= 0 && r1 >= r0 && r1 <= a.n_rows;
  const bool lead = rank == 0 && tid == 0;
  if (!good || r1 == r0) {   // no tokens were fed: nothing to verify (uniform over the cluster)
    if (lead) {
      if (!good && a.err_flag) atomicOr(a.err_flag, GVA_DEVERR_RANGE);
      a.n_accepted[b] = 0;
      if (a.kept_len) a.kept_len[b] = a.seq_len[b];
    }
    __threadfence();
    return;
  }
  const int k = r1 - r0 - 1;
  const T* target = reinterpret_cast<const T*>(a.target);
  const T* draft = reinterpret_cast<const T*>(a.draft);
  if (tid == 0) s_first = k;
  __syncthreads();
  for (int i = tid; i < k; i += kVfThreads) {
    const int x = a.tokens[r0 + i + 1];
    bool yes = false;
    if (x >= 0 && x < a.vocab) {
      const double p = to_f32(target[(long long)(r0 + i) * a.target_stride + x]);
      const double q = draft ? (double)to_f32(draft[(long long)(r0 + i) * a.draft_stride + x]) : 1.0;
      yes = (double)a.u_accept[r0 + i] * q < p;
    } else if (rank == 0 && a.err_flag) {
      atomicOr(a.err_flag, GVA_DEVERR_RANGE);
    }
    if (!yes) atomicMin(&s_first, i);
  }
  __syncthreads();
  const int acc = s_first;
  const bool refused = acc < k;
  const long long row = r0 + acc;
  const int x_no = refused ? a.tokens[row + 1] : -1;

  constexpr int N = RowVec<T>::N, SEG = 32 * N;
  Weights<T> W;
  W.vocab = a.vocab;
  W.p = target + row * a.target_stride;
  W.q = (refused && draft) ? draft + row * a.draft_stride : nullptr;
  W.skip = (refused && !draft) ? x_no : -1;
  // chunks start `mis` elements early, so that the vectors of the target's row are
  // 16-byte aligned whatever the row stride
  const int mis = (int)((reinterpret_cast<uintptr_t>(W.p) / sizeof(T)) % N);
  W.vec_q = W.q && (int)((reinterpret_cast<uintptr_t>(W.q) / sizeof(T)) % N) == mis;
  const int chunks = cl * kVfWarps;
  const int len = ((a.vocab + mis + chunks - 1) / chunks + SEG - 1) / SEG * SEG;
  // in 64 bits, then clipped: the last chunks of a short row start past its end
  const auto edge = [&](int c) { return (int)min((long long)c * len - mis, (long long)a.vocab); };
  const double u = (double)a.u_sample[b];
  int token = -1;
  bool found = false;
  for (int pass = 0; pass < 2; ++pass) {
    const int c = (int)rank * kVfWarps + warp;
    const double s = chunk_sum(W, edge(c), edge(c + 1), ring, lane);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (cl > 1) {
      cl_arrive();
      cl_wait();
    }
    for (int i = tid; i < chunks; i += kVfThreads)
      all[i] = cl > 1 ? ld_cluster_f64(&sums[i % kVfWarps], i / kVfWarps) : sums[i];
    __syncthreads();
    // remote reads done; waited for before the sums change or a CTA leaves
    if (cl > 1) cl_arrive();
    // every warp finds the chunk by itself: lanes hold consecutive pairs of chunk sums
    const double s0 = 2 * lane < chunks ? all[2 * lane] : 0.0;
    const double s1 = 2 * lane + 1 < chunks ? all[2 * lane + 1] : 0.0;
    double incl = s0 + s1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const double total = __shfl_sync(0xffffffffu, incl, 31);
    if (total > 0.0 || pass == 1) {
      const double t = u * total;
      const double e0 = incl - (s0 + s1), e1 = e0 + s0;
      const bool h0 = s0 > 0.0 && e1 > t, h1 = s1 > 0.0 && incl > t;
      const unsigned over = __ballot_sync(0xffffffffu, h0 || h1);
      const unsigned pos = __ballot_sync(0xffffffffu, s0 > 0.0 || s1 > 0.0);
      int ch = -1;
      double base = 0.0;
      if (over) {
        const int l = __ffs(over) - 1;
        ch = __shfl_sync(0xffffffffu, h0 ? 2 * lane : 2 * lane + 1, l);
        base = __shfl_sync(0xffffffffu, h0 ? e0 : e1, l);
      } else if (pos) {   // u >= 1, or rounding: the last chunk with any mass
        const int l = 31 - __clz(pos);
        ch = __shfl_sync(0xffffffffu, s1 > 0.0 ? 2 * lane + 1 : 2 * lane, l);
        base = __shfl_sync(0xffffffffu, s1 > 0.0 ? e1 : e0, l);
      }
      if (ch >= 0 && ch / kVfWarps == (int)rank) {
        // this CTA's warps share the chunk once more: sums of its eighths (from L2),
        // then the one warp whose eighth holds the answer walks it
        const int v0 = edge(ch), sub = (len / kVfWarps + SEG - 1) / SEG * SEG, v1 = edge(ch + 1);
        const int w0 = min(v0 + warp * sub, v1), w1 = min(v0 + (warp + 1) * sub, v1);
        const double sw = chunk_sum(W, w0, w1, ring, lane);
        if (lane == 0) part[warp] = sw;
        __syncthreads();
        int at = -1, last = -1;
        double run = base, from = base;
        for (int w = 0; w < kVfWarps; ++w) {
          const double x = part[w];
          if (x > 0.0) {
            last = w;
            if (at < 0) {
              from = run;
              if (run + x > t) at = w;
            }
          }
          run += x;
        }
        if (at < 0) at = last;
        if (warp == at) {
          token = chunk_find(W, w0, w1, from, t, lane);
          found = true;
        }
      } else if (ch < 0 && c == 0) {   // a row without any probability
        token = a.vocab - 1;
        found = true;
        if (lane == 0 && a.err_flag) atomicOr(a.err_flag, GVA_DEVERR_RANGE);
      }
      break;
    }
    // the residual is empty (p <= q everywhere): draw from p itself
    W.q = nullptr;
    W.skip = -1;
    if (cl > 1) cl_wait();
  }
  if (found && lane == 0) a.out_tokens[row] = token;
  if (rank == 0) {
    for (int i = tid; i <= k; i += kVfThreads)
      if (i != acc) a.out_tokens[r0 + i] = i < acc ? a.tokens[r0 + i + 1] : -1;
    if (tid == 0) {
      a.n_accepted[b] = acc;
      if (a.kept_len) a.kept_len[b] = a.seq_len[b] - (k - acc);
    }
  }
  __threadfence();   // no early trigger: the next step's calls read these lengths
  if (cl > 1) cl_wait();
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  int cl = kVfMaxCluster;
  while (cl > 1 && (long long)a.B * cl > 3ll * num_sms) cl >>= 1;   // (3: 21.4, 4: 22.8 us, 256 requests)
  static_assert(kVfMaxCluster * kVfWarps <= 64, "two chunk sums per lane");
  const dim3 grid((unsigned)(a.B * cl)), block(kVfThreads);
  auto go = [&](auto k) {
    const cudaError_t e = ensure_max_smem(k, kVfRing);
    return e == cudaSuccess ? launch_pdl_cluster(k, grid, block, cl, kVfRing, st, a, cl) : e;
  };
  return bf16 ? go(verify_kernel<__nv_bfloat16>) : go(verify_kernel<float>);
}

}  // namespace gva
