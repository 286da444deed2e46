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
// and the norm log2(D / 16) of them.  A warp covers 512 / D heads at a time
// (1 KB); the next heads' loads are in flight while it works on these.
#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "warp_search.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 8;

// Two floats to two e4m3 codes (low byte = lo): nearest even, magnitudes
// beyond 448 saturated, NaN kept.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 e4m3_chunk(const float* y, float scale) {
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    p[e] = e4m3_pair(__fdiv_rn(y[2 * e], scale), __fdiv_rn(y[2 * e + 1], scale));
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
__device__ __forceinline__ uint4 bf16_chunk(const float* y) {
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
    p[e] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

__device__ __forceinline__ void load_floats8(const float* src, float* dst) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(src));
  const float4 b = __ldg(reinterpret_cast<const float4*>(src) + 1);
  dst[0] = a.x; dst[1] = a.y; dst[2] = a.z; dst[3] = a.w;
  dst[4] = b.x; dst[5] = b.y; dst[6] = b.z; dst[7] = b.w;
}

// The request that owns flattened token t: the largest r with
// query_start_loc[r] <= t, if t also lies before query_start_loc[r + 1]; -1 for
// a token of no request.
__device__ __forceinline__ int request_of_token(const int32_t* qsl, int num_seqs, int t, int lane,
                                                int* q0, int* q1) {
  const int lo = warp_search_last(num_seqs, lane, [&](int i) { return __ldg(qsl + i) <= t; });
  *q0 = __ldg(qsl + lo);
  *q1 = __ldg(qsl + lo + 1);
  return *q0 <= t && t < *q1 ? lo : -1;
}

template <int D, bool KV8, bool IL>
__global__ void __launch_bounds__(kRopeWarps * 32)
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
  auto fetch = [&](int p, uint4& x0, uint4& x1) {
    const int kind = p < nq ? 0 : (p < nq + nk ? 1 : 2);
    const int h = (p - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * HPW + hl;
    x0 = x1 = make_uint4(0u, 0u, 0u, 0u);
    if (p < passes && h < (kind == 0 ? a.num_heads : a.num_kv_heads)) {
      const uint4* src = reinterpret_cast<const uint4*>((kind == 0 ? rows[0] : (kind == 1 ? rows[1] : rows[2])) +
                                                        static_cast<int64_t>(h) * D);
      x0 = src[c0];
      x1 = src[c1];
    }
  };
  uint4 x0, x1;
  fetch(part, x0, x1);  // does not depend on the request

  if (g == 0 && lane == 0 && __ldg(a.query_start_loc + a.num_seqs) > a.total_tokens)
    record_error(a.status, PA_DEV_BAD_QUERY_LEN, a.num_seqs - 1, a.query_start_loc[a.num_seqs]);
  int q0, q1;
  const int r = request_of_token(a.query_start_loc, a.num_seqs, token, lane, &q0, &q1);
  if (r < 0) return;  // a row behind the last request: left as it is
  const int seq_len = __ldg(a.seq_lens + r);
  const int64_t pos = static_cast<int64_t>(seq_len) - q1 + token;
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
  if (!in_table) return;

  // cos and sin of this lane's pairs: pair e of the half-split form is
  // (chunk 0 value e, chunk 1 value e); interleaved, pairs 0-3 are in chunk 0
  // and 4-7 in chunk 1.
  float cs[8], sn[8];
  if (rotates) {
    const float* row = a.cos_sin + rpos * a.rot_dim;
    const int half = a.rot_dim / 2;
    if constexpr (IL) {
      const float4 u0 = __ldg(reinterpret_cast<const float4*>(row + 4 * c0));
      const float4 u1 = __ldg(reinterpret_cast<const float4*>(row + 4 * c1));
      const float4 v0 = __ldg(reinterpret_cast<const float4*>(row + half + 4 * c0));
      const float4 v1 = __ldg(reinterpret_cast<const float4*>(row + half + 4 * c1));
      cs[0] = u0.x; cs[1] = u0.y; cs[2] = u0.z; cs[3] = u0.w;
      cs[4] = u1.x; cs[5] = u1.y; cs[6] = u1.z; cs[7] = u1.w;
      sn[0] = v0.x; sn[1] = v0.y; sn[2] = v0.z; sn[3] = v0.w;
      sn[4] = v1.x; sn[5] = v1.y; sn[6] = v1.z; sn[7] = v1.w;
    } else {
      load_floats8(row + 8 * c0, cs);
      load_floats8(row + half + 8 * c0, sn);
    }
  }

  float w[16];
  int weights_of = -1;  // 0: w holds the q weights, 1: the k weights
  for (int p = part; p < passes; p += a.warps_per_token) {
    uint4 n0, n1;
    fetch(p + a.warps_per_token, n0, n1);
    const int kind = p < nq ? 0 : (p < nq + nk ? 1 : 2);
    const int h = (p - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * HPW + hl;
    float y[16];
    unpack8(x0, y);
    unpack8(x1, y + 8);
    if (kind < 2) {
      const float* weight = kind == 0 ? a.q_weight : a.k_weight;
      if (weight != nullptr) {
        if (weights_of != kind) {
          load_floats8(weight + 8 * c0, w);
          load_floats8(weight + 8 * c1, w + 8);
          weights_of = kind;
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = y[e] * inv * w[e];
      }
      if (rotates) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& u = IL ? y[2 * e] : y[e];
          float& v = IL ? y[2 * e + 1] : y[e + 8];
          const float ua = u, va = v;
          u = fmaf(ua, cs[e], -(va * sn[e]));
          v = fmaf(va, cs[e], ua * sn[e]);
        }
      }
    }
    if (kind == 0) {
      if (h < a.num_heads) {
        uint4* dst = reinterpret_cast<uint4*>(a.q_out + (static_cast<int64_t>(token) * a.num_heads + h) * D);
        dst[c0] = bf16_chunk(y);
        dst[c1] = bf16_chunk(y + 8);
      }
    } else if (slot >= 0 && h < a.num_kv_heads) {
      const int64_t row = (slot * a.num_kv_heads + h) * (D / 8);  // in chunks of 8 values
      void* cache = kind == 1 ? a.key_cache : a.value_cache;
      if constexpr (KV8) {
        const float scale = kind == 1 ? a.k_scale : a.v_scale;
        uint2* dst = static_cast<uint2*>(cache) + row;
        dst[c0] = e4m3_chunk(y, scale);
        dst[c1] = e4m3_chunk(y + 8, scale);
      } else {
        uint4* dst = static_cast<uint4*>(cache) + row;
        dst[c0] = kind == 1 ? bf16_chunk(y) : x0;
        dst[c1] = kind == 1 ? bf16_chunk(y + 8) : x1;
      }
    }
    x0 = n0;
    x1 = n1;
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
