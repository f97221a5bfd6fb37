// Page plan of one serving step: block tables, slots and positions of the new
// tokens, built on the GPU from the requests' lengths.
//
// Request b keeps kept[b] cached tokens and brings n[b] new ones, so it needs
// goal = ceil((kept + n) / page) pages; it holds held[b].  Pages it no longer needs
// (goal < held: drafts rejected, request finished) go on top of the free list in
// request order, then requests that need more take them from its top, again in
// request order.  All of it is prefix sums over the batch:
//   back  = max(held - goal, 0)   pushed at  count + prefix(back)[b] + j
//   need  = max(goal - held, 0)   popped at  top - 1 - (prefix(need)[b] + j)
//   slot of token i of b at position p = kept + i:  page(p / P) * P + p % P
// A page popped in the call may be one pushed in the same call; its id is then read
// from the table entry that returned it.  So every read is of an entry that this
// call does not write (old table columns < held, free-list entries < count, table
// columns >= goal of shrinking requests), and no ordering between threads is needed
// once the per-request inputs are in shared memory.
//
// What bounds it: latency.  A step moves a few hundred KB at most (12 + 16 bytes per
// request, 8 per new token), so the cost is the chain load -> three scans -> binary
// search -> table entry -> store.  One cluster does it in one launch: every CTA scans
// the whole batch (12 bytes a request, from L2) and the expansion over pages and
// tokens is dealt out over the cluster's threads.  A cluster barrier between the
// loads and the stores lets callers update held and free_count in place.
#include "common.cuh"
#include "launch.h"
#include "paged.h"

namespace gva {

namespace {

constexpr int kPlanMaxThreads = 1024;
constexpr int kPlanPer = kMaxBatch / kPlanMaxThreads;   // requests per thread at most
constexpr int kPlanCluster = 16;                        // CTAs of a large step
constexpr int kTok = 4;                                 // new tokens per thread in flight

// (Both want whole warps together: the loops before them let lanes leave early.)
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix over the block of each thread's pair of sums; total in both.
__device__ __forceinline__ void scan_pair(long long& x, long long& y, long long& tx, long long& ty,
                                          longlong2* tmp) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) {
      ix += ux;
      iy += uy;
    }
  }
  if (lane == 31) tmp[w] = make_longlong2(ix, iy);
  __syncthreads();
  // every warp scans the warps' sums, one per lane
  const longlong2 s = lane < nw ? tmp[lane] : make_longlong2(0, 0);
  long long bx = s.x, by = s.y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, bx, o), uy = __shfl_up_sync(0xffffffffu, by, o);
    if (lane >= o) {
      bx += ux;
      by += uy;
    }
  }
  tx = __shfl_sync(0xffffffffu, bx, 31);
  ty = __shfl_sync(0xffffffffu, by, 31);
  x = __shfl_sync(0xffffffffu, bx - s.x, w) + ix - x;
  y = __shfl_sync(0xffffffffu, by - s.y, w) + iy - y;
  __syncthreads();   // tmp free again
}

// Last b in [0, B) with prefix[b] <= v, given prefix[0] = 0 <= v < prefix[B].
__device__ __forceinline__ int owner_of(const int* prefix, int B, int v) {
  int lo = 0, hi = B;   // prefix[lo] <= v < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanMaxThreads) plan_pages_kernel(const PlanArgs a, const int cl) {
  extern __shared__ int plan_sm[];
  __shared__ longlong2 tmp[32];
  const int B = a.B, tid = threadIdx.x, nt = blockDim.x;
  int* qs = plan_sm;            // granted tokens, prefix
  int* np = qs + B + 1;         // granted new pages, prefix
  int* bp = np + B + 1;         // returned pages, prefix
  int* kept = bp + B + 1;
  int* held = kept + B;
  int* goal = held + B;         // = held for a request that gets nothing

  // every input may come from the kernel before: nothing is read before this wait
  pdl_wait();
  const int per = (B + nt - 1) / nt, beg = min(tid * per, B), end = min(beg + per, B);
  const long long count_in = *a.free_count_in;
  int k_[kPlanPer], n_[kPlanPer], h_[kPlanPer], g_[kPlanPer];
  bool fit[kPlanPer];
  bool any_bad = false, any_denied = false;
  long long asked = 0, dummy = 0, t0, t1;
#pragma unroll
  for (int u = 0; u < kPlanPer; ++u) {
    const int b = beg + u;
    k_[u] = n_[u] = h_[u] = g_[u] = 0;
    fit[u] = false;
    if (b >= end) continue;
    k_[u] = a.kept_len[b];
    n_[u] = a.n_new[b];
    h_[u] = a.held_in[b];
    const long long goal_l = ((long long)k_[u] + n_[u] + a.page - 1) / a.page;
    const bool bad = k_[u] < 0 || n_[u] < 0 || h_[u] < 0 || h_[u] > a.max_pages ||
                     goal_l > a.max_pages || k_[u] > (long long)h_[u] * a.page;
    if (bad) {
      any_bad = true;
      k_[u] = 0;
    } else {
      g_[u] = (int)goal_l;
      fit[u] = true;
      asked += n_[u];
    }
  }
  if (cl > 1) {   // all CTAs hold the inputs: the outputs may overwrite them
    cluster_arrive();
    cluster_wait();
  }
  // tokens: a request fits while the tokens asked for so far fit the step's room
  scan_pair(asked, dummy, t0, t1, tmp);
  long long need = 0, back = 0;
#pragma unroll
  for (int u = 0; u < kPlanPer; ++u) {
    if (!fit[u]) continue;
    asked += n_[u];
    if (asked > a.max_new) {
      fit[u] = false;
      any_denied = true;
      continue;
    }
    need += max(g_[u] - h_[u], 0);
    back += max(h_[u] - g_[u], 0);
  }
  // pages: in request order, until the free list (with the returned pages) is empty
  long long need_x = need, back_x = back, need_t, back_t;
  scan_pair(need_x, back_x, need_t, back_t, tmp);
  // a free list that cannot be right: nothing moves
  const bool broken = count_in < 0 || count_in + back_t > a.num_pages;
  const int count = broken ? 0 : (int)count_in;
  const long long top = broken ? -1 : count_in + back_t;
  long long got_pages = 0, got_tokens = 0;
#pragma unroll
  for (int u = 0; u < kPlanPer; ++u) {
    if (!fit[u]) {
      n_[u] = 0;
      g_[u] = h_[u];
      continue;
    }
    const int nd = max(g_[u] - h_[u], 0);
    need_x += nd;
    if (broken || (nd > 0 && need_x > top)) {
      fit[u] = false;
      any_denied = true;
      n_[u] = 0;
      g_[u] = h_[u];
    } else {
      got_pages += nd;
      got_tokens += n_[u];
    }
  }
  long long gp_x = got_pages, gt_x = got_tokens, pages_t, tokens_t;
  scan_pair(gp_x, gt_x, pages_t, tokens_t, tmp);
#pragma unroll
  for (int u = 0; u < kPlanPer; ++u) {
    const int b = beg + u;
    if (b >= end) continue;
    qs[b] = (int)gt_x;
    np[b] = (int)gp_x;
    bp[b] = (int)back_x;
    kept[b] = k_[u];
    held[b] = h_[u];
    goal[b] = g_[u];
    gt_x += n_[u];
    gp_x += max(g_[u] - h_[u], 0);
    back_x += max(h_[u] - g_[u], 0);
  }
  const int n_back = broken ? 0 : (int)back_t, n_pages = (int)pages_t, n_tokens = (int)tokens_t;
  if (tid == 0) {
    qs[B] = n_tokens;
    np[B] = n_pages;
    bp[B] = n_back;
  }
  any_bad = __syncthreads_or(any_bad || broken);
  any_denied = __syncthreads_or(any_denied);

  const int rank = (int)blockIdx.x, gid = rank * nt + tid, gt = cl * nt;
  if (gid == 0) {
    *a.free_count_out = broken ? (int)count_in : (int)(top - pages_t);
    const int e = (any_bad ? GVA_DEVERR_RANGE : 0) | (any_denied ? GVA_DEVERR_PAGES : 0);
    if (e && a.err_flag) atomicOr(a.err_flag, e);
  }
  for (int b = gid; b <= B; b += gt) {
    a.q_start[b] = qs[b];
    if (b == B) continue;
    const int nb = qs[b + 1] - qs[b];
    a.held_out[b] = goal[b];
    a.seq_len[b] = kept[b] + nb;
    a.n_granted[b] = nb;
  }
  auto returned = [&](int k) {   // the k-th returned page
    const int b = owner_of(bp, B, k);
    return a.table[(long long)b * a.table_stride + goal[b] + (k - bp[b])];
  };
  auto page_of_rank = [&](int r) {   // the r-th page handed out
    const int idx = (int)(top - 1 - r);
    return idx < count ? a.free_pages[idx] : returned(idx - count);
  };
  // Tokens, kTok per thread at a time: their searches and table reads are independent
  // chains that overlap.  (These loops step past their ends, so their counters are
  // unsigned: tokens and pages may number 2^31 - 1.)
  const unsigned step = (unsigned)gt, room = (unsigned)a.max_new;
  for (unsigned i0 = gid; i0 < room; i0 += kTok * step) {
    int p[kTok], pg[kTok];
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
      const unsigned i = i0 + u * step;
      p[u] = pg[u] = -1;
      if (i < (unsigned)n_tokens) {
        const int b = owner_of(qs, B, (int)i);
        p[u] = kept[b] + ((int)i - qs[b]);
        const int col = p[u] / a.page;
        pg[u] = col < held[b] ? a.table[(long long)b * a.table_stride + col]
                              : page_of_rank(np[b] + col - held[b]);
      }
    }
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
      const unsigned i = i0 + u * step;
      if (i >= room) break;
      const bool ok = pg[u] >= 0 && pg[u] < a.num_pages;
      if (!ok && i < (unsigned)n_tokens && a.err_flag) atomicOr(a.err_flag, GVA_DEVERR_RANGE);
      a.slot[i] = ok ? pg[u] * a.page + p[u] % a.page : -1;
      a.pos[i] = p[u];
    }
  }
  for (unsigned k = gid; k < (unsigned)n_back; k += step) a.free_pages[count + k] = returned((int)k);
  for (unsigned q = gid; q < (unsigned)n_pages; q += step) {
    const int r = (int)q, b = owner_of(np, B, r);
    a.table[(long long)b * a.table_stride + held[b] + (r - np[b])] = page_of_rank(r);
  }
  // No early trigger: slots, positions and lengths are inputs that the next call's
  // first kernel may read before its own wait.
  __threadfence();
}

}  // namespace

cudaError_t launch_plan_pages(const PlanArgs& a, cudaStream_t st) {
  int threads = 128;
  while (threads < kPlanMaxThreads && threads * 4 < max(a.B * 4, a.max_new)) threads *= 2;
  if (threads * kPlanPer < a.B) threads = kPlanMaxThreads;
  // One CTA for small steps; else a cluster of 16 (the most there is, opt-in): the step
  // of 2048 requests and 39102 new tokens takes 13.4 us with 16 CTAs, 15.8 with 8.
  // (Any size works; a context that cannot hold 16 takes the largest half, quarter, ... of
  // it that fits.)
  int cl = (a.B > 512 || a.max_new > 4096) ? kPlanCluster : 1;
  const size_t smem = sizeof(int) * (size_t)(6 * a.B + 3), most = sizeof(int) * (size_t)(6 * kMaxBatch + 3);
  cudaError_t e = ensure_max_smem(plan_pages_kernel, most);
  if (e != cudaSuccess) return e;
  const void* key = reinterpret_cast<const void*>(plan_pages_kernel);
  const int wide = (int)cudaFuncAttributeNonPortableClusterSizeAllowed;
  if (cl > 8 && !attr_applied(key, wide, 1)) {
    e = cudaFuncSetAttribute(plan_pages_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_record(key, wide, 1);
  }
  if (cl > 1) cl = cluster_that_fits(key, cl, threads, most);
  return launch_pdl_cluster(plan_pages_kernel, dim3(cl), dim3(threads), cl, smem, st, a, cl);
}

}  // namespace gva
