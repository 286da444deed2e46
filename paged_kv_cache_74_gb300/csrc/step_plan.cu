// step_plan.cu -- the bookkeeping of a step on the device: cache blocks for the
// new tokens, block tables, slots, positions and the masks of drafted trees
// (plan_step), and blocks given back (release_blocks).
//
// With B tokens a block, request r at context_lens[r] = c, query_lens[r] = n and
// held_blocks[r] = h has  need_r = max(0, ceil((c + n) / B) - h).  The new blocks
// of the step are numbered request-major, then in logical order; block i comes
// from free_blocks[count - 1 - i].  A release gives back the blocks past
// ceil(keep / B), numbered the same way, block j of F to free_blocks[count + F - 1 - j]:
// what a plan has taken and a release gives back whole leaves the stack as it was.
//
// Each of them is a scan over the requests, then scattered writes whose places
// follow from it: nothing to compute and little to move, so what counts is the
// chain of round trips.  One cluster does all of it in one launch: its CTAs sum
// their slices of the requests, exchange the sums through distributed shared
// memory, and write.  The cluster barrier of the exchange puts the sums and the stack's
// count, which all CTAs need, before the first write; behind it a CTA reads only
// the state of its own slice (again, where that has more requests than a CTA has
// threads) and arrays that the call does not write.  So the state can be
// updated in place without a workspace, a ticket or a second launch.  A second
// cluster barrier puts the block tables before the tokens' slots, which are
// spread evenly over the CTAs whatever the requests' lengths (the request of a
// token by bisection of the row offsets).  Blocks are spread over a CTA's threads the
// same way: with a request's blocks on a warp 67 requests, four of them prompts of up to
// 11000 tokens, took 26.8 + 20.5 us (plan, release), now 17.1 + 5.7; 256 requests with trees of
// 8 to 24 rows 14.5 + 5.5, four small requests 8.4 + 5.0, each alone with cold caches.
#include <cooperative_groups.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kInShared = 4096;  // requests whose row offsets and contexts are kept in shared memory, 32 KB
constexpr int kRows = 4;         // rows of a thread that are in flight together

// Sums over the block of two non-negative values per thread, exclusive prefixes
// in *ea, *eb, totals in *ta, *tb.  (64 bits: lengths come from device data.)
__device__ __forceinline__ void block_scan2(long long a, long long b, long long (*warp_sums)[2], long long* ea,
                                            long long* eb, long long* ta, long long* tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long va = __shfl_up_sync(0xffffffffu, ia, o), vb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += va;
      ib += vb;
    }
  }
  __syncthreads();  // the sums of an earlier scan are read
  if (lane == 31) {
    warp_sums[warp][0] = ia;
    warp_sums[warp][1] = ib;
  }
  __syncthreads();
  long long pa_ = 0, pb = 0, sa = 0, sb = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long xa = warp_sums[w][0], xb = warp_sums[w][1];
    if (w < warp) {
      pa_ += xa;
      pb += xb;
    }
    sa += xa;
    sb += xb;
  }
  *ea = pa_ + ia - a;
  *eb = pb + ib - b;
  *ta = sa;
  *tb = sb;
}

struct Exchange {
  long long rows[kMaxCluster], blocks[kMaxCluster];  // sums of each CTA's slice
  int flags[kMaxCluster];
};

// Shared memory of a CTA that has not started may not be written: every CTA arrives on the
// cluster's barrier first thing and waits there before its first remote store, so that the
// loads and the scan between them cover the wait.
__device__ __forceinline__ void cluster_started(cg::cluster_group& cluster) {
  if (cluster.num_blocks() > 1) cluster_arrive();
}

// This CTA's sums and flag to every CTA of the cluster; gives the sums of the slices
// before this one and of all, and whether any flag is set.  Ends in a cluster barrier.
__device__ __forceinline__ bool exchange(cg::cluster_group& cluster, Exchange* ex, long long rows, long long blocks,
                                         int flag, long long* rows_before, long long* blocks_before,
                                         long long* rows_all, long long* blocks_all) {
  const int rank = static_cast<int>(cluster.block_rank()), n = static_cast<int>(cluster.num_blocks());
  if (n > 1) cluster_wait();  // for cluster_started(): every CTA's shared memory is there
  if (static_cast<int>(threadIdx.x) < n) {
    Exchange* to = cluster.map_shared_rank(ex, threadIdx.x);
    to->rows[rank] = rows;
    to->blocks[rank] = blocks;
    to->flags[rank] = flag;
  }
  cluster.sync();
  long long rb = 0, bb = 0, ra = 0, ba = 0;
  int any = 0;
  for (int c = 0; c < n; ++c) {
    if (c < rank) {
      rb += ex->rows[c];
      bb += ex->blocks[c];
    }
    ra += ex->rows[c];
    ba += ex->blocks[c];
    any |= ex->flags[c];
  }
  *rows_before = rb;
  *blocks_before = bb;
  *rows_all = ra;
  *blocks_all = ba;
  return any != 0;
}

// Runs f(i, j, e) for the entries e = 0 .. total - 1 of the block's kThreads requests, entry
// j of request i: spread evenly over the threads whatever the requests' counts.
// `before`: entries of the requests before this thread's; `start`: shared.
template <typename F>
__device__ __forceinline__ void for_entries(int before, int total, int* start, F f) {
  start[threadIdx.x] = before;
  __syncthreads();
  for (int e = threadIdx.x; e < total; e += kThreads) {
    int lo = 0, hi = kThreads;  // the last request that starts at or before e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= e)
        lo = mid;
      else
        hi = mid;
    }
    f(lo, e - start[lo], e);
  }
}

// What request r asks for.  ok: its lengths are in range.
struct StepNeed {
  long long rows;  // rows it takes up in the packed batch
  int ctx, len, held, blocks;
  bool ok;
};

__device__ __forceinline__ StepNeed step_need(const PlanStepArgs& a, int r, bool report) {
  StepNeed s{0, 0, 0, 0, 0, false};
  const int ctx = __ldcg(a.context_lens + r), n = __ldcg(a.query_lens + r), held = __ldcg(a.held_blocks + r);
  s.rows = max(n, 0);
  s.ctx = ctx;
  s.held = held;
  const long long len = static_cast<long long>(ctx) + n;
  if (n < 0 || (a.words > 0 && n > 64 * a.words)) {
    if (report) record_error(a.status, PA_DEV_BAD_QUERY_LEN, r, n);
    return s;
  }
  if (ctx < 0 || len > static_cast<long long>(a.max_blocks_per_seq) * a.block_size) {
    if (report) record_error(a.status, PA_DEV_BAD_SEQ_LEN, r, ctx < 0 ? ctx : static_cast<int>(min(len, 0x7fffffffll)));
    return s;
  }
  if (held < 0 || held > a.max_blocks_per_seq) {
    if (report) record_error(a.status, PA_DEV_BAD_HELD, r, held);
    return s;
  }
  s.ok = true;
  s.len = static_cast<int>(len);
  s.blocks = max(0, static_cast<int>((len + a.block_size - 1) / a.block_size) - held);
  return s;
}

// Whether `mine` holds for a thread of the cluster.  What a thread has written before is there
// for the others behind it.
__device__ __forceinline__ bool cluster_any(cg::cluster_group& cluster, Exchange* ex, bool mine) {
  __threadfence();
  const int any = __syncthreads_or(mine);
  cluster_started(cluster);  // (every thread has read the sums of the exchange before)
  long long before[2], all[2];
  return exchange(cluster, ex, 0, 0, any, &before[0], &before[1], &all[0], &all[1]);
}

// Depths of the rows in their trees where some are longer than kShortTree (without masks; up
// to there a row walks to its root where its slot is written, 2 to 4 us less): row t's, shifted
// up by 32 bits, into slot_mapping[t], which has its slots only later.  A row walks up
// kWalk parents by itself.  Where that does not end in a root, rows double what they have
// walked: with (ancestor a, steps d) of each row, (a, d) becomes (a's ancestor, d + a's
// steps), until every row has come to its root, ceil(log2(depth / kWalk)) rounds.  A
// pair is one 64-bit word, true at any time, so rows may read each other's while they change.
// Walked to the end by each row a chain of 120000 rows took 264 ms, now 0.29.
// request_of(t): the request of row t and its first row, or -1 where it was refused.
constexpr int kShortTree = 64 * kMaxMaskWords;
constexpr int kWalk = 64;
template <typename F>
__device__ void tree_depths(cg::cluster_group& cluster, Exchange* ex, const PlanStepArgs& a, int live, F request_of) {
  const int stride = static_cast<int>(cluster.num_blocks()) * kThreads;
  const int t0 = static_cast<int>(cluster.block_rank()) * kThreads + threadIdx.x;
  auto pair_of = [](int ancestor, int steps) -> long long {
    return static_cast<long long>(steps) << 32 | static_cast<unsigned>(ancestor);
  };
  bool on = false;
  for (long long t = t0; t < live; t += stride) {
    int first = 0;
    const int r = request_of(t, &first);
    int ancestor = -1, steps = 0;
    if (r >= 0) {
      int node = static_cast<int>(t) - first;
      while (true) {
        const int up = __ldg(a.parents + first + node);
        if (up < -1 || up >= node) record_error(a.status, PA_DEV_BAD_PARENT, r, up);
        if (up < 0 || up >= node) break;
        node = up;
        if (++steps == kWalk) {
          ancestor = first + node;
          on = true;
          break;
        }
      }
    }
    __stcg(reinterpret_cast<long long*>(a.slot_mapping) + t, pair_of(ancestor, steps));
  }
  while (cluster_any(cluster, ex, on)) {
    on = false;
    for (long long t = t0; t < live; t += stride) {
      const long long mine = __ldcg(reinterpret_cast<const long long*>(a.slot_mapping) + t);
      const int ancestor = static_cast<int>(mine);
      if (ancestor < 0) continue;
      const long long other = __ldcg(reinterpret_cast<const long long*>(a.slot_mapping) + ancestor);
      __stcg(reinterpret_cast<long long*>(a.slot_mapping) + t,
             pair_of(static_cast<int>(other), static_cast<int>((mine >> 32) + (other >> 32))));
      on = on || static_cast<int>(other) >= 0;
    }
  }
}

__global__ void __launch_bounds__(kThreads) plan_step_kernel(const PlanStepArgs a) {
  __shared__ long long warp_sums[kThreads / 32][2];
  __shared__ Exchange ex;
  __shared__ int start[kThreads], first[kThreads];
  __shared__ int offsets[kInShared + 1], contexts[kInShared];
  cg::cluster_group cluster = cg::this_cluster();
  cluster_started(cluster);
  griddep_launch_dependents();
  griddep_wait();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x;
  const int S = a.num_seqs;
  const int per = (S + ctas - 1) / ctas;
  const int r0 = min(S, rank * per), r1 = min(S, r0 + per);
  const bool one = r1 - r0 <= kThreads;  // (the slice's state is read and summed once)
  const bool cached = S <= kInShared;
  const bool local = ctas == 1 && one;   // all requests are this CTA's, each a thread's
  const int count = __ldcg(a.free_count);

  // Sums of this CTA's slice.
  long long rows = 0, blocks = 0, e0, e1, ta, tb;
  StepNeed s{0, 0, 0, 0, 0, false};
  bool long_tree = false;
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    s = StepNeed{0, 0, 0, 0, 0, false};
    if (r < r1) s = step_need(a, r, true);
    long_tree = long_tree || s.rows > kShortTree;
    block_scan2(s.rows, s.blocks, warp_sums, &e0, &e1, &ta, &tb);
    rows += ta;
    blocks += tb;
  }
  long long row, block, all_rows, all_blocks;
  int flag = 0;
  if (a.parents != nullptr && a.words == 0) flag = __syncthreads_or(long_tree);
  const bool long_trees = exchange(cluster, &ex, rows, blocks, flag, &row, &block, &all_rows, &all_blocks);
  // All or nothing: a batch that does not fit leaves tables, counts and stack alone.
  const bool fits = all_rows <= a.max_tokens && count >= 0 && count <= a.capacity && all_blocks <= count;
  if (!fits && rank == 0 && tid == 0) {
    if (all_rows > a.max_tokens)
      record_error(a.status, PA_DEV_BAD_QUERY_LEN, S, static_cast<int>(min(all_rows, 0x7fffffffll)));
    else
      record_error(a.status, PA_DEV_OUT_OF_BLOCKS, S, static_cast<int>(min(all_blocks, 0x7fffffffll)));
  }

  // Tables, offsets and lengths.
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    if (!one) {
      s = StepNeed{0, 0, 0, 0, 0, false};
      if (r < r1) s = step_need(a, r, false);
      block_scan2(s.rows, s.blocks, warp_sums, &e0, &e1, &ta, &tb);
    }
    const bool go = fits && s.ok;
    first[tid] = s.held;
    for_entries(static_cast<int>(fits ? e1 : 0), static_cast<int>(fits ? tb : 0), start, [&](int i, int j, int e) {
      const int id = __ldcg(a.free_blocks + (count - 1 - (static_cast<int>(block) + e)));
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks))
        record_error(a.status, PA_DEV_BAD_BLOCK_ID, base + i, id);
      a.block_tables[static_cast<size_t>(base + i) * a.max_blocks_per_seq + first[i] + j] = id;
    });
    if (r < r1) {
      const int at = static_cast<int>(min(row + e0, 0x7fffffffll));
      a.query_start_loc[r] = at;
      a.seq_lens[r] = go ? s.len : 0;
      if (go && s.blocks > 0) a.held_blocks[r] = s.held + s.blocks;
      if (local) {
        offsets[r] = at;
        contexts[r] = go && s.len > 0 ? s.ctx : -1;
      }
    }
    row += ta;
    block += tb;
  }
  if (rank == ctas - 1 && tid == 0) {
    a.query_start_loc[S] = static_cast<int>(min(all_rows, 0x7fffffffll));
    if (local) offsets[S] = static_cast<int>(min(all_rows, 0x7fffffffll));
  }
  if (ctas > 1) {
    __threadfence();
    cluster.sync();
  } else {
    __syncthreads();
  }
  if (rank == 0 && tid == 0 && fits) *a.free_count = count - static_cast<int>(all_blocks);

  // The rows: slots, positions, masks.
  if (cached && !local) {
    for (int r = tid; r <= S; r += kThreads) {
      offsets[r] = __ldcg(a.query_start_loc + r);
      if (r < S) contexts[r] = __ldcg(a.seq_lens + r) > 0 ? __ldcg(a.context_lens + r) : -1;  // -1: refused
    }
    __syncthreads();
  }
  auto first_row = [&](int r) -> int { return cached ? offsets[r] : __ldcg(a.query_start_loc + r); };
  auto context = [&](int r) -> int {
    return cached ? contexts[r] : (__ldcg(a.seq_lens + r) > 0 ? __ldcg(a.context_lens + r) : -1);
  };
  auto request_of = [&](long long t) -> int {  // the last one whose first row is at or before t
    int lo = 0, hi = S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_row(mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };
  const int live = fits ? static_cast<int>(all_rows) : 0;
  const int stride = ctas * kThreads;
  if (long_trees)
    tree_depths(cluster, &ex, a, live, [&](long long t, int* first) -> int {
      const int r = request_of(t);
      *first = first_row(r);
      return context(r) < 0 ? -1 : r;
    });
  for (long long t64 = static_cast<long long>(rank) * kThreads + tid; t64 < a.max_tokens;
       t64 += static_cast<long long>(kRows) * stride) {
    int req[kRows], row_in[kRows], pos[kRows], id[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const long long t = t64 + static_cast<long long>(u) * stride;
      req[u] = -1;
      if (t >= live) continue;
      const int lo = request_of(t);
      const int ctx = context(lo);
      if (ctx < 0) continue;
      req[u] = lo;
      row_in[u] = static_cast<int>(t) - first_row(lo);
      pos[u] = ctx + row_in[u];
      id[u] = __ldcg(a.block_tables + static_cast<size_t>(lo) * a.max_blocks_per_seq + pos[u] / a.block_size);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const long long t = t64 + static_cast<long long>(u) * stride;
      if (t >= a.max_tokens) break;
      long long slot = -1;
      int place = 0;
      unsigned long long mask[kMaxMaskWords] = {0, 0, 0, 0};
      if (req[u] >= 0) {
        const int i = row_in[u];
        if (static_cast<unsigned>(id[u]) < static_cast<unsigned>(a.num_blocks))
          slot = static_cast<long long>(id[u]) * a.block_size + pos[u] % a.block_size;
        else
          record_error(a.status, PA_DEV_BAD_BLOCK_ID, req[u], id[u]);
        place = pos[u];
        if (long_trees) {
          place += static_cast<int>(__ldcg(reinterpret_cast<const long long*>(a.slot_mapping) + t) >> 32) - i;
        } else if (a.parents != nullptr) {
          // Up the tree, kShortTree parents at most: every one comes before its child.
          const int32_t* parents = a.parents + (t - i);
          int depth = 0, node = i;
          while (true) {
#pragma unroll
            for (int w = 0; w < kMaxMaskWords; ++w)
              if (node >> 6 == w) mask[w] |= 1ull << (node & 63);
            const int up = __ldg(parents + node);
            if (up < -1 || up >= node) {
              record_error(a.status, PA_DEV_BAD_PARENT, req[u], up);
              break;
            }
            if (up < 0) break;
            node = up;
            ++depth;
          }
          place += depth - i;
        } else {
          // A chain: row i sees rows 0 .. i.
#pragma unroll
          for (int w = 0; w < kMaxMaskWords; ++w) {
            const int n = i + 1 - 64 * w;
            mask[w] = n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
          }
        }
      }
      a.slot_mapping[t] = slot;
      a.positions[t] = place;
#pragma unroll
      for (int w = 0; w < kMaxMaskWords; ++w)
        if (w < a.words) a.tree_masks[static_cast<size_t>(t) * a.words + w] = mask[w];
    }
  }
}

// Blocks that request r gives back, from logical block `keep` on.
__device__ __forceinline__ int release_need(const ReleaseArgs& a, int r, bool report, int* keep) {
  const int len = __ldcg(a.keep_lens + r), held = __ldcg(a.held_blocks + r);
  *keep = 0;
  if (len < 0) {
    if (report) record_error(a.status, PA_DEV_BAD_SEQ_LEN, r, len);
    return 0;
  }
  if (held < 0 || held > a.max_blocks_per_seq) {
    if (report) record_error(a.status, PA_DEV_BAD_HELD, r, held);
    return 0;
  }
  *keep = static_cast<int>((static_cast<long long>(len) + a.block_size - 1) / a.block_size);
  return max(0, held - *keep);
}

__global__ void __launch_bounds__(kThreads) release_blocks_kernel(const ReleaseArgs a) {
  __shared__ long long warp_sums[kThreads / 32][2];
  __shared__ Exchange ex;
  __shared__ int start[kThreads], first[kThreads];
  cg::cluster_group cluster = cg::this_cluster();
  cluster_started(cluster);
  griddep_launch_dependents();
  griddep_wait();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x;
  const int S = a.num_seqs;
  const int per = (S + ctas - 1) / ctas;
  const int r0 = min(S, rank * per), r1 = min(S, r0 + per);
  const bool one = r1 - r0 <= kThreads;
  const int count = __ldcg(a.free_count);
  long long blocks = 0, e0, e1, ta, tb;
  int keep = 0, n = 0;
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    n = r < r1 ? release_need(a, r, true, &keep) : 0;
    block_scan2(0, n, warp_sums, &e0, &e1, &ta, &tb);
    blocks += tb;
  }
  long long row, block, all_rows, all;
  exchange(cluster, &ex, 0, blocks, 0, &row, &block, &all_rows, &all);
  if (count < 0 || count + all > a.capacity) {  // more blocks than there are: given back twice
    if (rank == 0 && tid == 0)
      record_error(a.status, PA_DEV_OUT_OF_BLOCKS, S, static_cast<int>(min(count + all, 0x7fffffffll)));
    return;  // (every CTA of the cluster; none is read from any more)
  }
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    if (!one) {
      n = r < r1 ? release_need(a, r, false, &keep) : 0;
      block_scan2(0, n, warp_sums, &e0, &e1, &ta, &tb);
    }
    first[tid] = keep;
    for_entries(static_cast<int>(e1), static_cast<int>(tb), start, [&](int i, int j, int e) {
      const int id = __ldcg(a.block_tables + static_cast<size_t>(base + i) * a.max_blocks_per_seq + first[i] + j);
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks))
        record_error(a.status, PA_DEV_BAD_BLOCK_ID, base + i, id);
      a.free_blocks[count + all - 1 - block - e] = id;
    });
    if (n > 0) a.held_blocks[r] = keep;
    block += tb;
  }
  if (rank == 0 && tid == 0 && all > 0) *a.free_count = count + static_cast<int>(all);
}

// CTAs of the cluster.
int cluster_for(int64_t work) { return work > 1024 ? kMaxCluster : 1; }

template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), const Args& a, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_plan_step(const PlanStepArgs& a, cudaStream_t stream) {
  return launch_cluster(plan_step_kernel, a, cluster_for(std::max<int64_t>(a.num_seqs, a.max_tokens)), stream);
}

cudaError_t launch_release_blocks(const ReleaseArgs& a, cudaStream_t stream) {
  return launch_cluster(release_blocks_kernel, a, cluster_for(a.num_seqs), stream);
}

}  // namespace pa
