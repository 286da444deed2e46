// commit_tokens.cu -- K and V of the accepted tokens of a drafted tree, moved to
// the slots behind the context, in every layer's cache.
//
// With context length c and accepted nodes a_0 < a_1 < .. < a_{n-1}, row c + i of
// the request becomes row c + a_i, for i ascending.  As a_i >= i, the row written
// for i is never one that a later i reads (a_j >= j > i), so rows may be taken in
// batches, all loads of a batch before its stores, batches in order.
//
// Pure data movement: each row that moves is read and written once (at most
// num_kv_heads * head_dim * 2 bytes, 2 KB at 8 x 128 in bf16).  A warp owns 512 bytes of the
// rows of one request and cache in some of the layers, for the whole path, so its
// order is the only one needed.  It looks the path up once and then keeps kBatch pieces in
// flight, whichever layers they are of; rows that stay where they are are not touched.
#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 8;
constexpr int kWarpsInFlight = 152 * 24;  // about what the device holds of this kernel's

__global__ void __launch_bounds__(kWarps * 32) commit_tokens_kernel(const CommitArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int segs = (a.row_chunks + 31) / 32;
  const int groups = (a.num_layers + a.warp_layers - 1) / a.warp_layers;
  const int r = static_cast<int>(w / (2ll * segs * groups));
  if (r >= a.num_seqs) return;
  const int rest = static_cast<int>(w - static_cast<long long>(r) * (2ll * segs * groups));
  const int layer0 = rest / (2 * segs) * a.warp_layers;
  const int layers = min(a.warp_layers, a.num_layers - layer0);
  const int part = rest % (2 * segs);
  const bool first = rest == 0;  // reports, and writes the new length
  const int ctx = __ldg(a.context_lens + r), rows = __ldg(a.query_lens + r), n = __ldg(a.accept_lens + r);
  const bool planned = a.seq_lens == nullptr || __ldg(a.seq_lens + r) == static_cast<long long>(ctx) + rows;
  const int32_t* path = a.accepted + static_cast<size_t>(r) * a.max_accepted;
  const int first_node = lane < a.max_accepted ? __ldg(path + lane) : -1;  // (before the lengths are known)
  const int32_t* table = a.block_tables + static_cast<size_t>(r) * a.max_blocks_per_seq;

  // The slot of position p, or -1.
  auto slot_of = [&](long long p) -> long long {
    const int id = __ldg(table + p / a.block_size);
    return static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks)
               ? static_cast<long long>(id) * a.block_size + p % a.block_size
               : -1;
  };
  // The whole path is looked at before any row moves.
  int bad = PA_DEV_OK, what = 0;
  const long long end = static_cast<long long>(ctx) + rows;
  if (ctx < 0 || rows < 0 || end > static_cast<long long>(a.max_blocks_per_seq) * a.block_size) {
    bad = PA_DEV_BAD_SEQ_LEN;
    what = ctx < 0 ? ctx : rows;
  } else if (n < 0 || n > a.max_accepted || n > rows) {
    bad = PA_DEV_BAD_PATH;
    what = n;
  } else if (!planned && n > 0) {
    // The plan refused the request: the table's entries behind the held blocks are not its own.
    bad = PA_DEV_BAD_SEQ_LEN;
    what = __ldg(a.seq_lens + r);
  }
  long long src = -1, dst = -1;
  for (int base = 0; bad == PA_DEV_OK && base < n; base += 32) {
    const int i = base + lane;
    int code = PA_DEV_OK, node = 0;
    int prev = __shfl_up_sync(0xffffffffu, first_node, 1);
    if (lane == 0) prev = -1;
    if (i < n) {
      if (base > 0) prev = __ldg(path + i - 1);
      node = base == 0 ? first_node : __ldg(path + i);
      if (node <= prev || node >= rows) {
        code = PA_DEV_BAD_PATH;
      } else if (node != i) {
        src = slot_of(static_cast<long long>(ctx) + node);
        dst = slot_of(static_cast<long long>(ctx) + i);
        if (src < 0 || dst < 0) code = PA_DEV_BAD_BLOCK_ID;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, code != PA_DEV_OK);
    if (hit != 0) {
      bad = __shfl_sync(0xffffffffu, code, __ffs(hit) - 1);
      what = __shfl_sync(0xffffffffu, node, __ffs(hit) - 1);
    }
  }
  if (first && lane == 0) {
    if (bad != PA_DEV_OK) record_error(a.status, bad, r, what);
    if (a.new_lens != nullptr) a.new_lens[r] = bad == PA_DEV_OK ? ctx + n : ctx;
  }
  if (bad != PA_DEV_OK) return;

  const bool value = part >= segs;
  const int col = (value ? part - segs : part) * 32 + lane;
  const bool active = col < a.row_chunks;
  uint4* cache = (value ? a.value_cache : a.key_cache) + static_cast<size_t>(layer0) * a.layer_chunks + col;
  __shared__ long long places[kWarps][32][2];
  long long (*place)[2] = places[threadIdx.x >> 5];
  for (int base = 0; base < n; base += 32) {
    if (n > 32) {  // (up to 32 the loop above has left them)
      const int i = base + lane;
      src = dst = -1;
      if (i < n) {
        const int node = __ldg(path + i);
        if (node != i) {
          src = slot_of(static_cast<long long>(ctx) + node);
          dst = slot_of(static_cast<long long>(ctx) + i);
        }
      }
    }
    // The moving rows, in order; then their pieces in all layers, layer by layer.
    const unsigned moving = __ballot_sync(0xffffffffu, dst >= 0);
    const int m = __popc(moving);
    __syncwarp();
    if (dst >= 0) {
      const int k = __popc(moving & ((1u << lane) - 1u));
      place[k][0] = src * a.row_chunks;
      place[k][1] = dst * a.row_chunks;
    }
    __syncwarp();
    if (!active || m == 0) continue;
    int layer = 0, k = 0;
    while (layer < layers) {
      uint4 held[kBatch];
      uint4* to[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        to[u] = nullptr;
        if (layer < layers) {
          uint4* base_of = cache + static_cast<size_t>(layer) * a.layer_chunks;
          held[u] = base_of[place[k][0]];
          to[u] = base_of + place[k][1];
          if (++k == m) {
            k = 0;
            ++layer;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (to[u] != nullptr) *to[u] = held[u];
    }
  }
}

}  // namespace

cudaError_t launch_commit_tokens(const CommitArgs& args, cudaStream_t stream) {
  CommitArgs a = args;
  const int segs = (a.row_chunks + 31) / 32;
  // As many layers a warp as leave one wave of warps: the lookup of the path is three round
  // trips (64 requests, 32 layers of 2 KB rows, caches cold: 12.6 us with a layer a warp, 9.9 to 10.8 so).
  const long long warps = 2ll * segs * a.num_seqs;
  a.warp_layers = static_cast<int>(std::min<long long>(
      a.num_layers, std::max<long long>(1, (warps * a.num_layers + kWarpsInFlight - 1) / kWarpsInFlight)));
  const long long blocks = (warps * ((a.num_layers + a.warp_layers - 1) / a.warp_layers) + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_overlapped(commit_tokens_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace pa
