// prefill_masked.cu -- the chunked-prefill kernel with modified scores (tanh
// cap, distance bias, prefix and first-key masks): the plan of its work, and
// the launchers of the instantiations of prefill_kernel.cuh.
//
// A query tile (128 rows of a request) reads the 128-key steps that hold a key
// some of its rows sees: those of [0, prefix) and of [lo, hi), where lo is the
// least first key of its rows that see one and hi the last such row's position
// + 1; of these steps the 16-token blocks with such a key (visible_keys.cuh).  All
// of it comes from the rows' key_starts and has no closed form: one CTA
// computes them, a warp per tile, and scans them, and the tile kernel finds
// its range of steps in the scan.  The tile kernel's CTAs start meanwhile and
// wait for it.  (8 to 10 us alone from cold caches, 12 where rows see nothing and
// the unseen keys are worked out; with the requests and scans held in shared
// memory it was no faster: its time is the arrival of its instructions and three
// dependent loads.)
//
// Measured, one GB300, call after call (L2 flushed before each call: 11 us more):
// four long chunks with a 4096-key window (32 q, 8 kv heads of 128, bf16) 246 us,
// with a cap of 30 289 us, with slopes 307 us, capped over e4m3 417 us (249 GFLOP
// on visible pairs: 0.54, 0.46, 0.43 and 0.32 of the bf16 peak); a 512-token chunk
// with a cap before 63 decode rows 234 us (1.1 GB of K/V, 0.69 of the copy peak),
// over e4m3 170 us (0.48).
#include "prefill_kernel.cuh"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the CTA; *total: the sum.  `sums` holds 33 values.
__device__ __forceinline__ long long block_scan(long long v, long long* sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const long long w = sums[lane];
    long long wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += u;
    }
    sums[lane] = wi - w;
    if (lane == 31) sums[32] = wi;
  }
  __syncthreads();
  const long long before = sums[warp] + incl - v;
  *total = sums[32];
  __syncthreads();  // sums may be written again
  return before;
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_prefill_kernel(const PrefillArgs a) {
  __shared__ long long sums[33];
  __shared__ unsigned long long decode_tiles;  // 16-token tiles of the decode rows (per kv head)
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const PrefillPlan& pl = a.plan;
  if (tid == 0) decode_tiles = 0;
  if (a.partition) {
    __syncthreads();
    for (int r = tid; r < a.num_seqs; r += kPlanThreads) {
      const int q0 = __ldg(a.query_start_loc + r), len = __ldg(a.seq_lens + r);
      if (decode_row_tiles(q0, __ldg(a.query_start_loc + r + 1), len, row_limits(a)) > 0)
        atomicAdd(&decode_tiles, static_cast<unsigned long long>(tile_span(a.mods, r, q0, len).nb));
    }
  }
  // First tile of each request.
  long long tiles = 0;
  for (int base = 0; base < a.num_seqs; base += kPlanThreads) {
    const int r = base + tid;
    long long total;
    const long long before = block_scan(prefill_req(a, r).ntq, sums, &total);
    if (r < a.num_seqs)
      pl.first[r] = static_cast<int>(min(tiles + before, static_cast<long long>(pl.max_tiles)));
    tiles += total;
  }
  // (requests that share rows, which no valid query_start_loc has, may count more)
  if (tiles > pl.max_tiles) {
    if (tid == 0) record_error(a.status, PA_DEV_BAD_QUERY_LEN, a.num_seqs - 1, a.total_q);
    tiles = pl.max_tiles;
  }
  const int n = static_cast<int>(tiles);
  __syncthreads();
  for (int t = warp; t < n; t += kPlanThreads / 32) {
    const int r = warp_search_last(a.num_seqs, lane, [&](int i) { return pl.first[i] <= t; });
    const PReq p = prefill_req(a, r);
    const int row0 = max(0, p.ntq - 1 - (t - pl.first[r])) * 128;
    const int rows = min(128, p.q_len - row0);
    const int own = p.ctx + row0;  // position of the tile's first row
    int lo = 0, last = rows - 1;   // the least first key, and the last row that sees one of its run
    uint32_t seen[4] = {0, 0, 0, 0}, blocks = 0xffffffffu;
    if (a.mods.key_starts != nullptr) {
      // Row 32 w + lane: its first key, if it sees one of its run.
      int start[4];
      uint32_t see[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int i = 32 * w + lane;
        start[w] = i < rows ? max(0, __ldg(a.mods.key_starts + p.q0 + row0 + i)) : 0x7fffffff;
      }
      lo = 0x7fffffff;
      last = -1;
      int seeing = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (start[w] > own + 32 * w + lane) start[w] = 0x7fffffff;
        lo = min(lo, start[w]);
        see[w] = __ballot_sync(0xffffffffu, start[w] != 0x7fffffff);
        if (see[w] != 0) last = 32 * w + 31 - __clz(see[w]);
        seeing += __popc(see[w]);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      bool gap = false;  // some key before that of row `last` is seen neither by its own nor by the next row
      if (seeing <= last) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int behind = w < 3 ? __shfl_sync(0xffffffffu, start[w + 1 < 4 ? w + 1 : 3], 0) : 0x7fffffff;
          int next = __shfl_down_sync(0xffffffffu, start[w], 1);
          if (lane == 31) next = behind;
          const int k = 32 * w + lane;
          gap |= k < last && start[w] == 0x7fffffff && next > own + k;
        }
        gap = __any_sync(0xffffffffu, gap) != 0;
      }
      if (gap) {
        // Key own + k is seen by a row i >= k that starts at or before it.
        int least = 0x7fffffff;  // first key of the rows behind word w
        bool holes = false;
#pragma unroll 1
        for (int w = 3; w >= 0; --w) {
          int m = w == 0 ? start[0] : w == 1 ? start[1] : w == 2 ? start[2] : start[3];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int next = __shfl_down_sync(0xffffffffu, m, o);
            if (lane + o < 32) m = min(m, next);
          }
          m = min(m, least);
          least = __shfl_sync(0xffffffffu, m, 0);
          const int k = 32 * w + lane;
          const uint32_t word = __ballot_sync(0xffffffffu, m <= own + k);
          if (w == 0) seen[0] = word;
          if (w == 1) seen[1] = word;
          if (w == 2) seen[2] = word;
          if (w == 3) seen[3] = word;
          holes |= __any_sync(0xffffffffu, k <= last && m > own + k) != 0;
        }
        if (holes) blocks = __ballot_sync(0xffffffffu, lane < 9 && own_block_seen(seen, own, lo, lane));
      }
    }
    if (lane != 0) continue;
    const int prefix =
        a.mods.prefix_lens != nullptr ? min(max(__ldg(a.mods.prefix_lens + r), 0), p.seq_len) : 0;
    const int hi = last >= 0 ? own + last + 1 : 0;
    PlanTile w;
    w.r = r;
    w.q0 = p.q0;
    w.row0 = row0;
    w.rows = rows;
    w.ctx = p.ctx;
    w.kv_end = max(prefix, hi);
    w.prefix = prefix;
    w.lo = lo;
    w.hi = hi;
    // Steps [0, n1) hold the prefix; those of the run that are not among them
    // follow after a gap.
    const int n1 = (prefix + 127) / 128;
    const int second = hi > 0 ? max(n1, lo / 128) : n1;
    w.gap = second - n1;
    w.blocks = blocks;
    for (int u = 0; u < 4; ++u) w.seen[u] = seen[u];
    w.steps = n1 + max(0, (hi + 127) / 128 - second);
    if (w.steps == 0) {  // no row sees a key: one step without data writes the zeros
      w.steps = 1;
      w.gap = 0;
    }
    pl.tiles[t] = w;
  }
  __syncthreads();
  long long steps = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int t = base + tid;
    long long total;
    const long long before = block_scan(t < n ? pl.tiles[t].steps : 0, sums, &total);
    if (t < n) pl.cum[t] = steps + before;
    steps += total;
  }
  if (tid == 0) {
    pl.head->tiles = n;
    pl.head->steps = steps;
    // The split of the SMs with the decode rows.
    const long long pairs = static_cast<long long>(a.num_kv_heads) * ((a.group + 1) / 2);
    pl.head->tile_ctas =
        a.partition ? masked_tile_sms((kCostStep * steps + kCostUnit * n) * pairs,
                                      static_cast<long long>(decode_tiles) * a.num_kv_heads, a.num_ctas,
                                      a.partition == 2)
                    : a.num_ctas;
  }
}

template <int MOD>
cudaError_t launch_tiles(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, int head_dim, bool kv8, cudaStream_t stream) {
  if (head_dim == 128)
    return kv8 ? launch_prefill_impl<128, true, MOD>(a, qmap, kmap, vmap, stream)
               : launch_prefill_impl<128, false, MOD>(a, qmap, kmap, vmap, stream);
  if (head_dim == 64)
    return kv8 ? launch_prefill_impl<64, true, MOD>(a, qmap, kmap, vmap, stream)
               : launch_prefill_impl<64, false, MOD>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_prefill_masked(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                  const CUtensorMap& vmap, int head_dim, bool kv8, cudaStream_t stream) {
  const cudaError_t err = launch_overlapped(plan_prefill_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (err != cudaSuccess) return err;
  return a.mods.cap_log2 > 0.f ? launch_tiles<kModsCap>(a, qmap, kmap, vmap, head_dim, kv8, stream)
                               : launch_tiles<kMods>(a, qmap, kmap, vmap, head_dim, kv8, stream);
}

}  // namespace pa
