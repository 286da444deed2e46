// qk_norm_rope.cu -- a step's new tokens made ready for attention in one
// launch: the norm of every q and k head, the position rotation, and the
// write of K and V into the cache blocks (what pa_append_tokens does with
// keys that are already normed and rotated).
//
// Mathematics.  For one head x of D values at rotation position p:
//   y = x * (sum(x^2) / D + eps)^(-1/2) * w          (w absent: y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)
// for the rot_dim / 2 pairs (a, b) of the head's first rot_dim values, with
// cos and sin of pair i from row p of the caller's table; pair i is
// (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1).  Everything is fp32
// from the bf16 inputs to the one rounding of each stored value (bf16, or
// e4m3 of the quotient by the scale).
//
// The kernel is bound by memory: at 32 q and 8 kv heads of 128 values a token
// reads 12 KB, writes 12 KB and takes about 60 K operations.  A lane holds 16
// values of a head as two 16-byte chunks chosen so that both members of every
// pair sit in the same lane: chunks (j, j + rot_dim / 16) of the rotated part
// and neighbouring chunks of the rest, so that the rotation needs no shuffle
// and the norm log2(D / 16) of them.  A warp covers 512 / D heads (1 KB) in a
// pass; passes arrive through a ring of four slots in shared memory that its
// lanes fill with asynchronous copies, three passes ahead, without holding
// registers for what is in flight.
//
// Measured on 24065 prompt tokens (32 q and 8 kv heads of 128, bf16): 99 us call
// after call, 6.0 TB/s, 0.89 of the copy peak; with L2 flushed before each call 105
// us, 0.84, and there with one pass ahead in registers 136 us, ring slots 3, 6, 8:
// 109, 107, 115 us, 64 registers (four CTAs per SM): 126 us.  Over e4m3 caches 101 us
// call after call (80 by the bytes); 16 q heads and 1 kv head 54 (33), 32 and 2 over
// e4m3 83 (64): there the padded k and v passes and the division per stored value
// show.  Few tokens: the time is the chain launch, query_start_loc and
// seq_lens, block id and cos / sin, write: one token 9 us, 575 tokens 13 us.
#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeDepth = 4;  // passes of a warp in flight or at work

// Two floats to two e4m3 codes (low byte = lo): nearest even, magnitudes
// beyond 448 saturated, NaN kept.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 8 values (four pairs) as e4m3 of their quotient by the scale, or as bf16.
__device__ __forceinline__ uint2 e4m3_chunk(const float2* y, float scale) {
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = e4m3_pair(__fdiv_rn(y[e].x, scale), __fdiv_rn(y[e].y, scale));
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
__device__ __forceinline__ uint4 bf16_chunk(const float2* y) {
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(y[e].x, y[e].y);
    p[e] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ void unpack_pairs(const uint4& v, float2* y) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = make_float2(bf16_lo(w[e]), bf16_hi(w[e]));
}

// N consecutive floats (a multiple of 4, 16-byte aligned) as pairs.
template <int N>
__device__ __forceinline__ void load_pairs(const float* src, float2* dst) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(src + e));
    dst[e / 2] = make_float2(a.x, a.y);
    dst[e / 2 + 1] = make_float2(a.z, a.w);
  }
}

// The request that owns flattened token t (the largest r with
// query_start_loc[r] <= t, if t also lies before query_start_loc[r + 1]; r = -1 for
// a token of no request), its range and its length.  Down to 127 requests by a
// 32-way search, then all their entries and lengths in one round of loads.
struct TokenRequest {
  int r, q0, q1, seq_len;
};
__device__ __forceinline__ TokenRequest request_of_token(const int32_t* qsl, const int32_t* seq_lens,
                                                         int num_seqs, int t, int lane) {
  int lo = 0, n = num_seqs;  // the answer lies in [lo, lo + n)
  while (n > 127) {
    const int stride = (n - 1) / 32 + 1;
    const bool holds =
        lane == 0 || (static_cast<long long>(lane) * stride < n && __ldg(qsl + lo + lane * stride) <= t);
    const int last = __popc(__ballot_sync(0xffffffffu, holds)) - 1;
    n = min(stride, n - last * stride);
    lo += last * stride;
  }
  int start[4], len[4], count = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 32 * u + lane;
    start[u] = i <= n ? __ldg(qsl + lo + i) : 0x7fffffff;
    len[u] = i < n ? __ldg(seq_lens + lo + i) : 0;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    count += __popc(__ballot_sync(0xffffffffu, 32 * u + lane < n && start[u] <= t));
  const int i = count - 1;  // of the entries from lo on
  TokenRequest q{-1, 0, 0, 0};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int a = __shfl_sync(0xffffffffu, start[u], i & 31);
    const int b = __shfl_sync(0xffffffffu, start[u], (i + 1) & 31);
    const int l = __shfl_sync(0xffffffffu, len[u], i & 31);
    if (i >> 5 == u) {
      q.q0 = a;
      q.seq_len = l;
    }
    if ((i + 1) >> 5 == u) q.q1 = b;
  }
  if (i >= 0 && q.q0 <= t && t < q.q1) q.r = lo + i;
  return q;
}

template <int D, bool KV8, bool IL>
__global__ void __launch_bounds__(kRopeWarps * 32, 3)
qk_norm_rope_append_kernel(const NormRopeArgs a) {
  constexpr int LPH = D / 16;      // lanes per head
  constexpr int HPW = 32 / LPH;    // heads per warp and pass
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t token64 = g / a.warps_per_token;
  if (token64 >= a.total_tokens) return;
  const int token = static_cast<int>(token64);
  const int part = static_cast<int>(g - token64 * a.warps_per_token);

  // Passes over HPW heads each: q heads, then k heads, then v heads.
  const int nq = (a.num_heads + HPW - 1) / HPW, nk = (a.num_kv_heads + HPW - 1) / HPW;
  const int passes = nq + 2 * nk;
  const int sub = lane % LPH, hl = lane / LPH;
  const int rc = a.rot_dim / 16;
  const bool rotates = sub < rc;
  const int c0 = rotates ? sub : 2 * sub;       // this lane's two 16-byte chunks of a head
  const int c1 = rotates ? sub + rc : 2 * sub + 1;
  const __nv_bfloat16* rows[3] = {a.q + token * a.q_stride, a.key + token * a.key_stride,
                                  a.value + token * a.value_stride};
  // Pass p of the warp goes through slot k of its ring in shared memory: every
  // lane copies and later reads its own two chunks.
  __shared__ uint4 ring[kRopeWarps][kRopeDepth][2][32];
  uint4(*mine)[2][32] = ring[threadIdx.x >> 5];
  auto fetch = [&](int p, int k) {
    if (p < passes) {
      const int kind = p < nq ? 0 : (p < nq + nk ? 1 : 2);
      const int h = (p - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * HPW + hl;
      if (h < (kind == 0 ? a.num_heads : a.num_kv_heads)) {
        const uint4* src =
            reinterpret_cast<const uint4*>((kind == 0 ? rows[0] : (kind == 1 ? rows[1] : rows[2])) +
                                           static_cast<int64_t>(h) * D);
        cp_async_16(smem_u32(&mine[k][0][lane]), src + c0, 16);
        cp_async_16(smem_u32(&mine[k][1][lane]), src + c1, 16);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kRopeDepth - 1; ++k) fetch(part + k * a.warps_per_token, k);  // not tied to the request

  if (g == 0 && lane == 0 && __ldg(a.query_start_loc + a.num_seqs) > a.total_tokens)
    record_error(a.status, PA_DEV_BAD_QUERY_LEN, a.num_seqs - 1, a.query_start_loc[a.num_seqs]);
  const TokenRequest req = request_of_token(a.query_start_loc, a.seq_lens, a.num_seqs, token, lane);
  const int r = req.r, seq_len = req.seq_len;
  if (r < 0) {  // a row behind the last request: left as it is
    cp_async_wait_all();
    return;
  }
  const int64_t pos = static_cast<int64_t>(seq_len) - req.q1 + token;
  const int64_t rpos = a.positions != nullptr ? a.positions[token] : pos;
  int64_t slot = -1;
  {
    const int64_t logical = pos >= 0 ? pos / a.block_size : -1;
    if (logical < 0 || logical >= a.max_blocks_per_seq) {
      if (lane == 0 && part == 0) record_error(a.status, PA_DEV_BAD_SEQ_LEN, r, seq_len);
    } else {
      const int32_t phys = __ldg(a.block_tables + static_cast<int64_t>(r) * a.max_blocks_per_seq + logical);
      if (phys < 0 || phys >= a.num_blocks) {
        if (lane == 0 && part == 0) record_error(a.status, PA_DEV_BAD_BLOCK_ID, r, phys);
      } else {
        slot = static_cast<int64_t>(phys) * a.block_size + (pos - logical * a.block_size);
      }
    }
  }
  const bool in_table = rpos >= 0 && rpos < a.max_position;
  if (!in_table) {
    if (lane == 0 && part == 0) record_error(a.status, PA_DEV_BAD_POSITION, r, static_cast<int>(rpos));
    slot = -1;
  }
  if (a.slot_mapping != nullptr && lane == 0 && part == 0) a.slot_mapping[token] = slot;
  if (!in_table) {
    cp_async_wait_all();  // no copy outlives the CTA
    return;
  }

  // cos and sin of this lane's pairs: pair e of the half-split form is
  // (chunk 0 value e, chunk 1 value e); interleaved, pairs 0-3 are in chunk 0
  // and 4-7 in chunk 1.
  float2 cs[4], sn[4];
  if (rotates) {
    const float* row = a.cos_sin + rpos * a.rot_dim;
    const int half = a.rot_dim / 2;
    if constexpr (IL) {
      load_pairs<4>(row + 4 * c0, cs);
      load_pairs<4>(row + 4 * c1, cs + 2);
      load_pairs<4>(row + half + 4 * c0, sn);
      load_pairs<4>(row + half + 4 * c1, sn + 2);
    } else {
      load_pairs<8>(row + 8 * c0, cs);
      load_pairs<8>(row + half + 8 * c0, sn);
    }
  }

  int slot_k = 0;
  for (int p = part; p < passes; p += a.warps_per_token) {
    cp_async_wait<kRopeDepth - 2>();
    const uint4 x0 = mine[slot_k][0][lane], x1 = mine[slot_k][1][lane];
    fetch(p + (kRopeDepth - 1) * a.warps_per_token, (slot_k + kRopeDepth - 1) % kRopeDepth);
    slot_k = (slot_k + 1) % kRopeDepth;
    const int kind = p < nq ? 0 : (p < nq + nk ? 1 : 2);
    const int h = (p - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * HPW + hl;
    float2 y[8];
    unpack_pairs(x0, y);
    unpack_pairs(x1, y + 4);
    if (kind < 2) {
      const float* weight = kind == 0 ? a.q_weight : a.k_weight;
      if (weight != nullptr) {
        float2 w[8];
        load_pairs<8>(weight + 8 * c0, w);
        load_pairs<8>(weight + 8 * c1, w + 4);
        float2 s2 = make_float2(0.f, 0.f), s3 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s2 = __ffma2_rn(y[e], y[e], s2);
          s3 = __ffma2_rn(y[e + 4], y[e + 4], s3);
        }
        float ss = (s2.x + s2.y) + (s3.x + s3.y);
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fmul2_rn(__fmul2_rn(y[e], make_float2(inv, inv)), w[e]);
      }
      if (rotates) {
        if constexpr (IL) {
          // pair e of cs is that of y[2 e] and y[2 e + 1]
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float c = e & 1 ? cs[e / 2].y : cs[e / 2].x, v = e & 1 ? sn[e / 2].y : sn[e / 2].x;
            y[e] = make_float2(fmaf(y[e].x, c, -(y[e].y * v)), fmaf(y[e].y, c, y[e].x * v));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = y[e], v = y[e + 4];
            y[e] = __ffma2_rn(v, make_float2(-sn[e].x, -sn[e].y), __fmul2_rn(u, cs[e]));
            y[e + 4] = __ffma2_rn(u, sn[e], __fmul2_rn(v, cs[e]));
          }
        }
      }
    }
    if (kind == 0) {
      if (h < a.num_heads) {
        uint4* dst = reinterpret_cast<uint4*>(a.q_out + (static_cast<int64_t>(token) * a.num_heads + h) * D);
        dst[c0] = bf16_chunk(y);
        dst[c1] = bf16_chunk(y + 4);
      }
    } else if (slot >= 0 && h < a.num_kv_heads) {
      const int64_t row = (slot * a.num_kv_heads + h) * (D / 8);  // in chunks of 8 values
      void* cache = kind == 1 ? a.key_cache : a.value_cache;
      if constexpr (KV8) {
        const float scale = kind == 1 ? a.k_scale : a.v_scale;
        uint2* dst = static_cast<uint2*>(cache) + row;
        dst[c0] = e4m3_chunk(y, scale);
        dst[c1] = e4m3_chunk(y + 4, scale);
      } else {
        uint4* dst = static_cast<uint4*>(cache) + row;
        dst[c0] = kind == 1 ? bf16_chunk(y) : x0;
        dst[c1] = kind == 1 ? bf16_chunk(y + 4) : x1;
      }
    }
  }
}

template <int D>
cudaError_t launch_qk_norm_rope_d(NormRopeArgs& a, bool kv8, bool interleaved, cudaStream_t stream) {
  constexpr int HPW = 512 / D;
  const int passes = (a.num_heads + HPW - 1) / HPW + 2 * ((a.num_kv_heads + HPW - 1) / HPW);
  // One warp per token when the tokens alone fill the GPU; fewer tokens are
  // spread over more warps each, one pass per warp at most.
  constexpr int64_t kWarpsWanted = 152 * 48;
  a.warps_per_token = static_cast<int>(std::min<int64_t>(
      passes, std::max<int64_t>(1, (kWarpsWanted + a.total_tokens - 1) / a.total_tokens)));
  const int64_t warps = static_cast<int64_t>(a.total_tokens) * a.warps_per_token;
  const int64_t grid = (warps + kRopeWarps - 1) / kRopeWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto* kernel = kv8 ? (interleaved ? qk_norm_rope_append_kernel<D, true, true>
                                    : qk_norm_rope_append_kernel<D, true, false>)
                     : (interleaved ? qk_norm_rope_append_kernel<D, false, true>
                                    : qk_norm_rope_append_kernel<D, false, false>);
  return launch_overlapped(kernel, dim3(static_cast<unsigned>(grid)), dim3(kRopeWarps * 32), 0, stream, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(NormRopeArgs a, int head_dim, bool kv8, bool interleaved,
                                cudaStream_t stream) {
  if (head_dim == 128) return launch_qk_norm_rope_d<128>(a, kv8, interleaved, stream);
  if (head_dim == 64) return launch_qk_norm_rope_d<64>(a, kv8, interleaved, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
