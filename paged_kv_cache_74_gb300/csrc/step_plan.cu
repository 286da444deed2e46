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
// memory, and write; the cluster barrier orders every read of the lengths, the
// held counts and the stack before the first write, so that the state can be
// updated in place without a workspace, a ticket or a second launch.  A second
// cluster barrier puts the block tables before the tokens' slots, which are
// spread evenly over the CTAs whatever the requests' lengths (the request of a
// token by bisection of the row offsets).
#include <cooperative_groups.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kOffsetsInShared = 8192;  // row offsets bisected in shared memory, 32 KB
constexpr int kAlone = 4;               // blocks of a request that one thread handles by itself

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
};

// This CTA's sums to every CTA of the cluster; returns the sums of the slices
// before this one and of all.  Ends in a cluster barrier.
__device__ __forceinline__ void exchange(cg::cluster_group& cluster, Exchange* ex, long long rows, long long blocks,
                                         long long* rows_before, long long* blocks_before, long long* rows_all,
                                         long long* blocks_all) {
  const int rank = static_cast<int>(cluster.block_rank()), n = static_cast<int>(cluster.num_blocks());
  if (static_cast<int>(threadIdx.x) < n) {
    Exchange* to = cluster.map_shared_rank(ex, threadIdx.x);
    to->rows[rank] = rows;
    to->blocks[rank] = blocks;
  }
  cluster.sync();
  long long rb = 0, bb = 0, ra = 0, ba = 0;
  for (int c = 0; c < n; ++c) {
    if (c < rank) {
      rb += ex->rows[c];
      bb += ex->blocks[c];
    }
    ra += ex->rows[c];
    ba += ex->blocks[c];
  }
  *rows_before = rb;
  *blocks_before = bb;
  *rows_all = ra;
  *blocks_all = ba;
}

// Runs f(r, j, base + j) for entries j = 0 .. n - 1 of each lane's request: a few by
// the lane itself, more by the whole warp.
template <typename F>
__device__ __forceinline__ void for_entries(int r, int n, long long base, int lane, F f) {
  if (n <= kAlone)
    for (int j = 0; j < n; ++j) f(r, j, base + j);
  for (unsigned large = __ballot_sync(0xffffffffu, n > kAlone); large != 0; large &= large - 1) {
    const int src = __ffs(large) - 1;
    const int wr = __shfl_sync(0xffffffffu, r, src), wn = __shfl_sync(0xffffffffu, n, src);
    const long long wb = __shfl_sync(0xffffffffu, base, src);
    for (int j = lane; j < wn; j += 32) f(wr, j, wb + j);
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

__global__ void __launch_bounds__(kThreads) plan_step_kernel(const PlanStepArgs a) {
  __shared__ long long warp_sums[kThreads / 32][2];
  __shared__ Exchange ex;
  __shared__ int offsets[kOffsetsInShared];
  cg::cluster_group cluster = cg::this_cluster();
  griddep_launch_dependents();
  griddep_wait();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x, lane = tid & 31;
  const int S = a.num_seqs;
  const int per = (S + ctas - 1) / ctas;
  const int r0 = min(S, rank * per), r1 = min(S, r0 + per);

  // Sums of this CTA's slice.
  long long rows = 0, blocks = 0, e0, e1;
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    StepNeed s{0, 0, 0, 0, 0, false};
    if (r < r1) s = step_need(a, r, true);
    long long ta, tb;
    block_scan2(s.rows, s.blocks, warp_sums, &e0, &e1, &ta, &tb);
    rows += ta;
    blocks += tb;
  }
  const int count = __ldcg(a.free_count);
  long long row, block, all_rows, all_blocks;
  exchange(cluster, &ex, rows, blocks, &row, &block, &all_rows, &all_blocks);
  // All or nothing: a batch that does not fit leaves tables, counts and stack alone.
  const bool fits = all_rows <= a.max_tokens && count >= 0 && count <= a.capacity && all_blocks <= count;
  if (!fits && rank == 0 && tid == 0) {
    if (all_rows > a.max_tokens)
      record_error(a.status, PA_DEV_BAD_QUERY_LEN, S, static_cast<int>(min(all_rows, 0x7fffffffll)));
    else
      record_error(a.status, PA_DEV_OUT_OF_BLOCKS, S, static_cast<int>(min(all_blocks, 0x7fffffffll)));
  }

  // Tables, offsets and lengths.  (The slices' state has been read.)
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    StepNeed s{0, 0, 0, 0, 0, false};
    if (r < r1) s = step_need(a, r, false);
    long long ta, tb;
    block_scan2(s.rows, s.blocks, warp_sums, &e0, &e1, &ta, &tb);
    const bool go = fits && s.ok;
    for_entries(r, go ? s.blocks : 0, block + e1, lane, [&](int wr, int j, long long i) {
      const int id = __ldcg(a.free_blocks + (count - 1 - i));
      const int h = __ldcg(a.held_blocks + wr);
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks))
        record_error(a.status, PA_DEV_BAD_BLOCK_ID, wr, id);
      a.block_tables[static_cast<size_t>(wr) * a.max_blocks_per_seq + h + j] = id;
    });
    __syncwarp();  // the warp has read its requests' held counts
    if (r < r1) {
      a.query_start_loc[r] = static_cast<int>(min(row + e0, 0x7fffffffll));
      a.seq_lens[r] = go ? s.len : 0;
      if (go && s.blocks > 0) a.held_blocks[r] = s.held + s.blocks;
    }
    row += ta;
    block += tb;
  }
  if (rank == ctas - 1 && tid == 0) a.query_start_loc[S] = static_cast<int>(min(all_rows, 0x7fffffffll));
  __threadfence();
  cluster.sync();
  if (rank == 0 && tid == 0 && fits) *a.free_count = count - static_cast<int>(all_blocks);

  // The rows: slots, positions, masks.
  const bool cached = S < kOffsetsInShared;
  if (cached) {
    for (int r = tid; r <= S; r += kThreads) offsets[r] = __ldcg(a.query_start_loc + r);
    __syncthreads();
  }
  auto first_row = [&](int r) -> int { return cached ? offsets[r] : __ldcg(a.query_start_loc + r); };
  const int live = fits ? static_cast<int>(all_rows) : 0;
  for (long long t64 = static_cast<long long>(rank) * kThreads + tid; t64 < a.max_tokens;
       t64 += static_cast<long long>(ctas) * kThreads) {
    const int t = static_cast<int>(t64);
    long long slot = -1;
    int pos = 0;
    unsigned long long mask[kMaxMaskWords] = {0, 0, 0, 0};
    if (t < live) {
      int lo = 0, hi = S;  // the last request whose first row is at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_row(mid) <= t)
          lo = mid;
        else
          hi = mid;
      }
      const int r = lo;
      const int f = first_row(r);
      const int i = t - f;
      const int len = __ldcg(a.seq_lens + r);
      if (len > 0) {  // 0: the request was refused
        const int ctx = __ldcg(a.context_lens + r);
        const int p = ctx + i;
        const int id = __ldcg(a.block_tables + static_cast<size_t>(r) * a.max_blocks_per_seq + p / a.block_size);
        if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
          slot = static_cast<long long>(id) * a.block_size + p % a.block_size;
        else
          record_error(a.status, PA_DEV_BAD_BLOCK_ID, r, id);
        pos = p;
        if (a.parents != nullptr) {
          // Up the tree: every parent comes before its child, so the walk ends.
          int depth = 0, node = i;
          while (true) {
#pragma unroll
            for (int w = 0; w < kMaxMaskWords; ++w)
              if (node >> 6 == w) mask[w] |= 1ull << (node & 63);
            const int up = __ldg(a.parents + f + node);
            if (up < -1 || up >= node) {
              record_error(a.status, PA_DEV_BAD_PARENT, r, up);
              break;
            }
            if (up < 0) break;
            node = up;
            ++depth;
          }
          pos = ctx + depth;
        } else {
          // A chain: row i sees rows 0 .. i.
#pragma unroll
          for (int w = 0; w < kMaxMaskWords; ++w) {
            const int n = i + 1 - 64 * w;
            mask[w] = n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
          }
        }
      }
    }
    a.slot_mapping[t] = slot;
    a.positions[t] = pos;
#pragma unroll
    for (int w = 0; w < kMaxMaskWords; ++w)
      if (w < a.words) a.tree_masks[static_cast<size_t>(t) * a.words + w] = mask[w];
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
  cg::cluster_group cluster = cg::this_cluster();
  griddep_launch_dependents();
  griddep_wait();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x, lane = tid & 31;
  const int S = a.num_seqs;
  const int per = (S + ctas - 1) / ctas;
  const int r0 = min(S, rank * per), r1 = min(S, r0 + per);
  long long blocks = 0, e0, e1, ta, tb;
  int keep = 0;
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    block_scan2(0, r < r1 ? release_need(a, r, true, &keep) : 0, warp_sums, &e0, &e1, &ta, &tb);
    blocks += tb;
  }
  const int count = __ldcg(a.free_count);
  long long row, block, all_rows, all;
  exchange(cluster, &ex, 0, blocks, &row, &block, &all_rows, &all);
  if (count < 0 || count + all > a.capacity) {  // more blocks than there are: given back twice
    if (rank == 0 && tid == 0)
      record_error(a.status, PA_DEV_OUT_OF_BLOCKS, S, static_cast<int>(min(count + all, 0x7fffffffll)));
    return;  // (every CTA of the cluster; none is read from any more)
  }
  for (int base = r0; base < r1; base += kThreads) {
    const int r = base + tid;
    const int n = r < r1 ? release_need(a, r, false, &keep) : 0;
    block_scan2(0, n, warp_sums, &e0, &e1, &ta, &tb);
    for_entries(r, n, block + e1, lane, [&](int wr, int j, long long i) {
      const int first = (__ldcg(a.keep_lens + wr) + a.block_size - 1ll) / a.block_size;
      const int id = __ldcg(a.block_tables + static_cast<size_t>(wr) * a.max_blocks_per_seq + first + j);
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks))
        record_error(a.status, PA_DEV_BAD_BLOCK_ID, wr, id);
      a.free_blocks[count + all - 1 - i] = id;
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
