// tree_attention.cu -- attention of drafted token trees over the paged cache, on
// the sm_103a tensor cores (tcgen05).
//
// Request r has n new tokens (the nodes of its trees) behind a context of c tokens,
// K and V of all of them in the cache.  Node i sees keys 0 .. c - 1 and the keys c + k
// of the nodes k that its mask names:
//   O_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j) over the seen keys j,
// 128 keys at a time with an online softmax (m, l, O) per row; S and P never
// reach HBM.  Pieces of a row's keys computed by different CTAs are merged by
// m = max m_p, O = sum O_p 2^(m_p - m), l = sum l_p 2^(m_p - m).
//
// What bounds it.  Each K/V byte serves all nodes and all q heads of its kv head,
// n * group query rows.  A 128-key step reads 64 KB at head_dim 128 in bf16 (1.47 us of an SM's
// share of the copy bandwidth) and takes 0.33 us of the SM's tensor core per 128 rows for each
// of the two products: up to 256 rows a kv head the keys' bytes are the bound.
// That holds to one tile of rows; what two tiles take in practice is the exponentials, maxima
// and conversions of 256 x 128 scores a step (1.7 us with the products, not hidden by each other
// entirely) and a unit's end.  Measured, bf16 in us a call: 64 requests x 16 nodes, 32 / 8 heads,
// 512 to 4096 keys 114 (0.85 of the copy peak), 32 x 64 nodes 87 (832 TFLOP/s), 8 x 32768 keys
// 172 (0.92); e4m3, 96 x up to 16 nodes, 64 / 8 heads, up to 4099 keys 142.
// So the design reads the keys once for all rows:
// * The rows of a kv head are packed, row = node * group + head: one TMA box
//   {64, group, 128 / group} of q lands as the 128-row operand of the products.  A
//   tile of rows is one slot, up to two slots share every K/V step of a work
//   unit (request, kv head, two tiles of rows).
// * A unit of one tile would leave the softmax of its only slot between its two
//   products; there both slots take the same rows and alternate key steps, each with
//   its own (m, l, O) in TMEM, joined at the end.
// * Persistent grid, one CTA per SM: the 128-key steps of all units are numbered
//   (request, kv head, tile pair, step) and cut into equal contiguous ranges by
//   cost (a unit's start counts kUnitCost / kStepCost steps).  A unit that a range boundary
//   cuts leaves its pieces as fp32 records, which a second kernel merges with the whole
//   device: the last contributor alone would read up to 152 records of 64 KB by itself
//   where few long contexts are split over every SM.
// * Warps: 0-3 softmax of slot 0, 4-7 of slot 1 (thread = row, two passes over its scores
//   in TMEM); 8 range walk, Q and K copies (TMA); 9 and 11 MMA issue of a slot each; 10 V
//   copies; over e4m3 caches 12-15 split q and turn landed V steps into f16.
// * e4m3 keys are the operand as they lie in the cache: q is the exact sum of two e4m3
//   operands (split_q), two products.  V has to become f16: the
//   weights need more bits than an e4m3 number or two have.
// A step that holds nodes takes its mask from the row's words; V of keys that no
// row of the unit sees is zeroed before the product (a zero weight does not
// cancel a NaN inside the MMA).  Every wait is bounded; a timeout records
// PA_DEV_WAIT_TIMEOUT.
#include <algorithm>

#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "work_split.cuh"

namespace pa {
namespace {

constexpr float kLowest = -1e30f;     // finite stand-in for -inf in running maxima
constexpr float kRescaleSlack = 8.0f;  // log2 units: the reference of a row moves lazily
// What a step and a unit's start and end take, relative to each other.  10 to 16 per unit are
// alike; 24 and 32 cost 2 and 5 % on 32 trees of 64 nodes, 5 % each on ragged trees.
constexpr long long kStepCost = 4;
constexpr long long kUnitCost = 12;

// How a segment's result is written.
constexpr int kWhole = 0;  // the whole unit: bf16 output
constexpr int kHead = 1;   // continues a unit begun by an earlier CTA: record 0
constexpr int kTail = 2;   // begins a unit finished by later CTAs: record 1
constexpr int kEnd = 3;    // no more work

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int D, bool KV8>
struct TreeCfg {
  static constexpr int BM = 128, BN = 128;          // rows of a slot, keys of a step
  static constexpr int HALVES = D / 64;             // 128-byte column chunks of head_dim
  static constexpr int CHUNK = 128 * 128;
  static constexpr int QBYTES = HALVES * CHUNK;     // Q of one slot
  static constexpr int TBYTES = HALVES * CHUNK;     // K (or V) of one step
  static constexpr int BLOCK_BYTES = HALVES * 16 * 128;  // K (or V) of 16 tokens
  // 16-token blocks land as [8-key group][head_dim half][8 keys][128 B].
  static constexpr int GSTRIDE = HALVES * 1024;
  // A V stage is held from its copy to the end of its step, a K stage only to S.
  // e4m3: K lands as the operand; landed V bytes have stages of their own, free again
  // once converted.  NK is even (see the MMA issue).
  static constexpr int NK = KV8 ? (D == 128 ? 4 : 6) : (D == 128 ? 2 : 4);
  static constexpr int NV = KV8 ? (D == 128 ? 2 : 4) : (D == 128 ? 3 : 6);
  static constexpr int NR = KV8 ? (D == 128 ? 2 : 4) : 0;  // raw V stages
  static constexpr int RAW_BLOCK = 16 * D;
  static constexpr int RAW_BYTES = 128 * D;
  static constexpr int KBYTES = KV8 ? RAW_BYTES : TBYTES;
  static constexpr int K_BLOCK = KV8 ? RAW_BLOCK : BLOCK_BYTES;
  static constexpr int SEGS = 4;                    // segment records in flight
  static constexpr int OFF_Q = 0;                   // [2 slots]
  static constexpr int OFF_K = 2 * QBYTES;
  static constexpr int OFF_V = OFF_K + NK * KBYTES;
  static constexpr int OFF_VRAW = OFF_V + NV * TBYTES;
  static constexpr int OFF_SEG = OFF_VRAW + NR * RAW_BYTES;
  static constexpr int OFF_XCH = OFF_SEG + SEGS * 64;   // [2 slots][128 rows] (m, l)
  static constexpr int OFF_EXP = OFF_XCH + 2 * 128 * 8;  // e4m3: [2 slots][128 rows] exponents of q
  static constexpr int OFF_BAR = OFF_EXP + (KV8 ? 2 * 128 : 0);
  // Barriers
  static constexpr int KFULL = 0;                // [NK] K step landed
  static constexpr int KFREE = KFULL + NK;       // [NK] the S products that read it are done (both slots)
  static constexpr int VFULL = KFREE + NK;       // [NV] V step landed (e4m3: converted)
  static constexpr int VFREE = VFULL + NV;       // [NV] the P.V products that read it are done
  static constexpr int QFULL = VFREE + NV;       // [2] Q of a slot landed
  static constexpr int QFREE = QFULL + 2;        // the last S product of a segment is done
  static constexpr int SFULL = QFREE + 1;        // [2] S of a slot in TMEM
  static constexpr int PFULL = SFULL + 2;        // [2] P of a slot in TMEM (4 warps)
  static constexpr int PHALF = PFULL + 2;        // [2] P of its first 64 keys, O rescaled
  static constexpr int OFULL = PHALF + 2;        // the last P.V product of a segment is done
  static constexpr int OFREE = OFULL + 1;        // O read at a segment's end (8 warps)
  static constexpr int SEGFULL = OFREE + 1;      // [SEGS]
  static constexpr int SEGFREE = SEGFULL + SEGS; // [SEGS] every role is done with it
  static constexpr int SYNC = SEGFREE + SEGS;    // the 8 softmax warps
  static constexpr int DRAIN = SYNC + 1;         // [2] an MMA warp's last commit
  static constexpr int TURN = DRAIN + 2;         // [2] a slot's turn to issue (two tiles)
  static constexpr int QCONV = TURN + 2;         // e4m3: Q split (4 warps)
  static constexpr int EXPFREE = QCONV + 1;      // e4m3: the rows' exponents read (8 warps)
  static constexpr int VRAW = EXPFREE + 1;       // [NR] e4m3 step landed
  static constexpr int VRAWFREE = VRAW + NR;     // [NR] ... and read by the four warps
  static constexpr int NBAR = VRAWFREE + NR;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 64;
  static constexpr int CONVERTERS = KV8 ? 4 : 0;    // a quarter of a V step each
  static constexpr int THREADS = (12 + CONVERTERS) * 32;
  static constexpr int SEG_USERS = 11 + CONVERTERS;  // 2 MMA, 8 softmax, V producer
  static constexpr uint32_t TMEM_COLS = 512;        // S0 0, S1 128, O0 256, O1 256 + D
  // (The descriptor bits of e4m3 in kind::f8f6f4 are those of f16 in kind::f16.)
  static constexpr uint32_t IDESC_S = KV8 ? idesc_f16_f32(BM, BN, 0) : idesc_bf16_f32(BM, BN, 0);
  static constexpr uint32_t IDESC_O = KV8 ? idesc_f16_f32(BM, D, 1) : idesc_bf16_f32(BM, D, 1);
  static_assert(SMEM <= 227 * 1024 && OFF_BAR % 8 == 0 && NK % 2 == 0, "shared memory");
};

// A request's rows, or tiles = 0 where it has none or a length is out of range.
struct TreeReq {
  int q0, n, len, tiles;
};

__device__ __forceinline__ TreeReq make_req(const TreeArgs& a, int q0, int q1, int len) {
  TreeReq p{0, 0, 0, 0};
  const int n = q1 - q0;
  if (n < 1 || n > len || n > a.max_query_len || n > 32 * a.words32 || q0 < 0 || q0 > a.total_q - n ||
      len > a.max_seq_len || len > a.max_blocks_per_seq * a.block_size)
    return p;
  p.q0 = q0;
  p.n = n;
  p.len = len;
  p.tiles = (n + 2 * a.slot_nodes - 1) / (2 * a.slot_nodes);
  return p;
}

__device__ __forceinline__ TreeReq tree_req(const TreeArgs& a, int r) {
  if (r >= a.num_seqs) return TreeReq{0, 0, 0, 0};
  return make_req(a, __ldg(a.query_start_loc + r), __ldg(a.query_start_loc + r + 1), __ldg(a.seq_lens + r));
}

__device__ __forceinline__ int req_steps(const TreeReq& p) { return (p.len + 127) / 128; }

__device__ void report_bad_requests(const TreeArgs& a, int lane) {
  for (int r = lane; r < a.num_seqs; r += 32) {
    const int q0 = __ldg(a.query_start_loc + r), n = __ldg(a.query_start_loc + r + 1) - q0;
    const int len = __ldg(a.seq_lens + r);
    if (n == 0) continue;
    if (n < 0 || n > len || n > a.max_query_len || n > 32 * a.words32 || q0 < 0 || q0 > a.total_q - n)
      record_error(a.status, PA_DEV_BAD_QUERY_LEN, r, n);
    else if (len > a.max_seq_len || len > a.max_blocks_per_seq * a.block_size)
      record_error(a.status, PA_DEV_BAD_SEQ_LEN, r, len);
  }
}

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// Whether a barrier's phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Holds the registers of an asynchronous TMEM load until its wait.
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 8)
    asm volatile("" : "+r"(r[e]), "+r"(r[e + 1]), "+r"(r[e + 2]), "+r"(r[e + 3]), "+r"(r[e + 4]),
                      "+r"(r[e + 5]), "+r"(r[e + 6]), "+r"(r[e + 7]));
}

// A segment: steps [j0, j1) of one unit inside this CTA's range.
struct TreeSeg {
  int r, q0, node0, nodes;  // q0: the request's first row; the unit's nodes
  int ctx, n_new, j0, j1;
  int kvh, kind;
  int pad[6];
};
static_assert(sizeof(TreeSeg) == 64, "segment record");

// 32 bits of a row's view of the keys from 32 * i behind the context on: the
// context (i < 0), the nodes its mask names, nothing behind the last one.
__device__ __forceinline__ uint32_t view_word(const uint32_t* mask, int words32, int n_new, int i) {
  if (i < 0) return 0xffffffffu;
  const int left = n_new - 32 * i;
  if (left <= 0 || i >= words32) return 0u;
  return __ldg(mask + i) & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
}

// A part of an e4m3 V step (16-token blocks [b0, b1) of head_dim bytes a token at
// `raw`) written as f16, exactly, in the operand layout of the bf16 copies ([8-key
// group][head_dim half][8 keys][128 B], 128-byte swizzle).  Run by one warp, an
// 8-key group at a time.  A raw 16-byte chunk becomes two f16 chunks; lanes
// of the upper head_dim half store them in the other order, so that the eight lanes
// of a key hit eight bank groups.
template <int D, bool KV8>
__device__ __forceinline__ void convert_v(uint32_t raw, uint32_t stage, int b0, int b1, int lane) {
  using C = TreeCfg<D, KV8>;
  constexpr int CPR = D / 16;     // 16-byte raw chunks per key row
  constexpr int KPI = 32 / CPR;   // key rows per warp-wide load
  constexpr int NLD = 8 / KPI;    // loads per lane per 8-key group
  const int c = lane % CPR;
  const uint32_t half = (c / 4) * 1024;
  const int cc = 2 * (c % 4), swap = c / 4;
#pragma unroll 1
  for (int g8 = 2 * b0; g8 < 2 * b1; ++g8) {
    uint4 w[NLD];
#pragma unroll
    for (int k = 0; k < NLD; ++k) w[k] = ld_shared_v4(raw + (g8 * 8 + lane / CPR + KPI * k) * D + c * 16);
#pragma unroll
    for (int k = 0; k < NLD; ++k) {
      const int r = lane / CPR + KPI * k;
      const uint32_t row = stage + g8 * C::GSTRIDE + half + r * 128;
      const uint4 x = w[k];
      const uint32_t a0 = swap ? x.z : x.x, a1 = swap ? x.w : x.y, b0w = swap ? x.x : x.z, b1w = swap ? x.y : x.w;
      st_shared_v4(row + (((cc + swap) ^ r) * 16),
                   make_uint4(e4m3x2_to_f16x2(a0), e4m3x2_to_f16x2(a0 >> 16), e4m3x2_to_f16x2(a1),
                              e4m3x2_to_f16x2(a1 >> 16)));
      st_shared_v4(row + (((cc + 1 - swap) ^ r) * 16),
                   make_uint4(e4m3x2_to_f16x2(b0w), e4m3x2_to_f16x2(b0w >> 16), e4m3x2_to_f16x2(b1w),
                              e4m3x2_to_f16x2(b1w >> 16)));
    }
  }
}

// Two floats rounded to e4m3 (nearest even, saturating), packed low / high.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// q of a slot as two e4m3 operands, q 2^e = h + l with h = e4m3(q 2^e) and l = e4m3(q 2^e - h):
// bf16 has eight significant bits, h takes four and what it leaves has at most four.  e is
// the row's own, its largest value lands in [128, 256); so l is exact for all values down to
// 2^-9 of the row's largest, and off by at most 2^-10 (2^-17 of the largest) below.  S = h K^T
// + l K^T then takes K as it lies in the cache: K is not converted (and has no second place in
// shared memory, and all converting warps work on V).
// In place: h takes the place of the rows' first halves, l of the second (head_dim 64:
// within the row).  Warp w4 of four, a row by four lanes.
template <int D, bool KV8>
__device__ __forceinline__ void split_q(uint32_t q, int8_t* exps, int exp_max, int w4, int lane) {
  using C = TreeCfg<D, KV8>;
  constexpr int NCH = D / 32;  // 16-byte chunks of a lane
  const int part = lane >> 3;
#pragma unroll 1
  for (int r0 = w4 * 8; r0 < 128; r0 += 32) {
    const int r = r0 + (lane & 7), sw = lane & 7;
    const uint32_t row = q + r * 128;
    uint4 w[NCH];
    uint32_t m2 = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      w[c] = ld_shared_v4(row + (D == 128 ? (part >> 1) * C::CHUNK + ((((part & 1) * 4 + c) ^ sw) * 16) : ((2 * part + c) ^ sw) * 16));
      m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu),
                                 __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu)));
    }
    m2 = max(m2 & 0xffffu, m2 >> 16);
    m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, 8));
    m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, 16));  // (all of the warp's rows are read)
    // (Beyond 2^47 a row saturates; rows of zeros and of values below 2^-93 take the last step,
    // or exp_max, which keeps scale 2^-e a normal number.)
    const int e = min(max(134 - static_cast<int>(m2 >> 7), -40), exp_max);
    // (A row with an infinity or a NaN becomes NaNs: e4m3 numbers saturate, so it would come out finite.)
    const float s = __int_as_float(m2 >= 0x7f80u ? 0x7fffffff : (e + 127) << 23);
    if (part == 0) exps[r] = static_cast<int8_t>(e);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < NCH; c += 2) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = w[c + i / 2];
        const uint32_t p0 = i % 2 ? x.z : x.x, p1 = i % 2 ? x.w : x.y;
        const float a = bf16_lo(p0) * s, b = bf16_hi(p0) * s, c2 = bf16_lo(p1) * s, d = bf16_hi(p1) * s;
        const uint32_t h0 = pack_e4m3x2(a, b), h1 = pack_e4m3x2(c2, d);
        const uint32_t f0 = e4m3x2_to_f16x2(h0), f1 = e4m3x2_to_f16x2(h1);
        const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&f0));
        const float2 g1 = __half22float2(*reinterpret_cast<const __half2*>(&f1));
        h[i] = h0 | h1 << 16;
        l[i] = pack_e4m3x2(a - g0.x, b - g0.y) | pack_e4m3x2(c2 - g1.x, d - g1.y) << 16;
      }
      const int at = part * (NCH / 2) + c / 2;  // chunk of the row's e4m3 values
      st_shared_v4(row + (at ^ sw) * 16, make_uint4(h[0], h[1], h[2], h[3]));
      st_shared_v4(D == 128 ? row + C::CHUNK + (at ^ sw) * 16 : row + ((4 + at) ^ sw) * 16,
                   make_uint4(l[0], l[1], l[2], l[3]));
    }
  }
}

// D (TMEM) = A * B (+ D if accumulate), e4m3 operands in shared memory, 32 of K.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// sdesc_sw128's neighbour for rows of 64 bytes (64-byte swizzle, groups of eight rows
// 512 bytes apart).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (4ull << 61);
}

// Exchanges half of two 16-byte pieces with lane ^ bit: a 2 x 2 transpose.
__device__ __forceinline__ void swap_pieces(uint4& x, uint4& y, int bit, int lane) {
  const bool up = lane & bit;
  uint32_t* a = &x.x;
  uint32_t* b = &y.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a[i] : b[i], bit);
    (up ? a[i] : b[i]) = got;
  }
}

// Records of a cut unit: (CTA, piece, slot) holds (m, l) of 128 rows and their
// unnormalised O as [D / 4][128 rows][4 columns], so that a warp's 16-byte accesses to
// one column group are 512 contiguous bytes.  Piece 1: a unit's first CTA, else 0.
__device__ __forceinline__ size_t record_of(int cta, int piece, int slot) {
  return (static_cast<size_t>(cta) * 2 + piece) * 2 + slot;
}

template <int D, bool KV8>
__global__ void __launch_bounds__(TreeCfg<D, KV8>::THREADS, 1)
tree_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
  using C = TreeCfg<D, KV8>;
  const int cta = blockIdx.x;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t q_s = sbase + C::OFF_Q;
  const uint32_t k_s = sbase + C::OFF_K;
  const uint32_t v_s = sbase + C::OFF_V;
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto bar = [&](int k) -> uint32_t { return bar0 + 8 * k; };
  TreeSeg* segs = reinterpret_cast<TreeSeg*>(smem + C::OFF_SEG);
  float2* xch = reinterpret_cast<float2*>(smem + C::OFF_XCH);
  int8_t* exps = reinterpret_cast<int8_t*>(smem + C::OFF_EXP);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  volatile int* fail_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* n_k_issued = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  volatile int* n_v_issued = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 12);
  volatile int* n_q_issued = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);  // [2]

  // The swizzled copies need 1024-byte aligned tiles; the dynamic shared-memory base
  // always is on this GPU, but never issue a copy if it were not.
  if (sbase & 1023) {
    griddep_wait();
    if (tid == 0) record_error(a.status, PA_DEV_WAIT_TIMEOUT, cta, 6);
    if (tid == 0) a.splits[cta].c1 = -1;
    return;
  }
  if (tid == 0) {
    for (int k = 0; k < C::NBAR; ++k) {
      int count = 1;
      if (k >= C::PFULL && k < C::PHALF + 2) count = 4;
      if (KV8 && ((k >= C::VFULL && k < C::VFULL + C::NV) || k == C::QCONV || k >= C::VRAWFREE)) count = 4;
      if (k == C::OFREE || k == C::SYNC || (KV8 && k == C::EXPFREE)) count = 8;
      if ((k >= C::KFREE && k < C::KFREE + C::NK) || (k >= C::VFREE && k < C::VFREE + C::NV) || k == C::QFREE ||
          k == C::OFULL)
        count = 2;  // both slots
      if (k >= C::SEGFREE && k < C::SEGFREE + C::SEGS) count = C::SEG_USERS;
      mbar_init(bar(k), count);
    }
    *fail_flag = 0;
    *n_k_issued = 0;
    *n_v_issued = 0;
    n_q_issued[0] = 0;
    n_q_issued[1] = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the cache write of this step's tokens
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int G = a.group, NPS = a.slot_nodes;
  auto give_up = [&](int where) {
    record_error(a.status, PA_DEV_WAIT_TIMEOUT, cta, where);
    *fail_flag = 1;
  };
  // A wait by the whole warp (the same answer for all its lanes).
  auto warp_wait = [&](int k, uint32_t parity, int where) -> bool {
    if (*fail_flag) return false;
    const bool good = __all_sync(0xffffffffu, mbar_wait(bar(k), parity) ? 1 : 0) != 0;
    if (!good && lane == 0) give_up(where);
    return good;
  };
  // Cache row of 16-token tile t8 + lane (lane < 8) of request r; an id outside the
  // pool is reported (if `report`) and read as wholly out of bounds (zeros).
  auto tile_rows = [&](int r, int t8, int nblk, bool report) -> int {
    const int t16 = t8 + lane;
    if (lane >= 8 || t16 >= nblk) return 0;
    const int id = __ldg(a.block_tables + static_cast<size_t>(r) * a.max_blocks_per_seq + (t16 >> a.tile_shift));
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) {
      if (report) record_error(a.status, PA_DEV_BAD_BLOCK_ID, r, id);
      return a.num_blocks * a.block_size;
    }
    return id * a.block_size + (t16 & ((1 << a.tile_shift) - 1)) * kBlockSize;
  };

  if (warp < 8) {
    // ============================================================ softmax
    // Warps 0-3 serve slot 0, 4-7 slot 1; warp w owns TMEM lanes 32 (w % 4) .. + 31.
    const int b = warp >> 2;
    const int i_row = (warp & 3) * 32 + lane;
    auto node_of = [&](int row) -> int { return row * a.group_inv >> 16; };  // row / group
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tm_s = lane_base + b * C::BN;
    const uint32_t tm_o = lane_base + 256;
    float sl2 = a.scale_log2;
    bool ok = true;
    int sc = 0, g = 0;
    uint32_t sync_phase = 0;
    for (int seg = 0; ok; ++seg) {
      const int slot = seg % C::SEGS;
      if (!(ok = warp_wait(C::SEGFULL + slot, (seg / C::SEGS) & 1, 81))) break;
      const volatile TreeSeg& sg = segs[slot];
      if (sg.kind == kEnd) break;
      const int n = sg.j1 - sg.j0;
      const int nodes = sg.nodes, ctx = sg.ctx, n_new = sg.n_new;
      const bool two = nodes > NPS;
      if constexpr (KV8) {
        // The row's scores carry 2^e of its q.
        if (!(ok = warp_wait(C::QCONV, seg & 1, 79))) break;
        sl2 = a.scale_log2 * __int_as_float((127 - exps[(two ? b * 128 : 0) + i_row]) << 23);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::EXPFREE));
      }
      // Rows of this slot; whether this warp has some.
      const bool live = (warp & 3) * 32 < (two ? (b ? nodes - NPS : NPS) : nodes) * G;
      for (int i = lane; i < nodes; i += 32)  // read in the last steps
        prefetch_l1(a.masks + static_cast<size_t>(sg.q0 + sg.node0 + i) * a.words32);
      float m_ref = kLowest, l_run = 0.f;
      bool first = true;
      const int k0 = two ? 0 : (g ^ b) & 1;  // this slot's first step
      for (int k = k0; k < n; k += two ? 1 : 2) {
        const int key0 = (sg.j0 + k) * C::BN;
        const bool masked = key0 + C::BN > ctx;  // the step holds nodes, or ends behind the keys
        // Before S is there: what the row sees of the step, and whether some row of the
        // unit sees the key that this lane looks after.
        uint32_t seen[4];
        bool dead = false;
        if (masked) {
          const int off = key0 - ctx;
          const int sh = off & 31, w0 = off >> 5;
          if (live) {
            // (rows behind the slot's last take the unit's last node)
            const int node = min((two && b ? NPS : 0) + node_of(i_row), nodes - 1);
            const uint32_t* mask = a.masks + static_cast<size_t>(sg.q0 + sg.node0 + node) * a.words32;
            uint32_t w[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = view_word(mask, a.words32, n_new, w0 + i);
#pragma unroll
            for (int i = 0; i < 4; ++i) seen[i] = __funnelshift_r(w[i], w[i + 1], sh);
          }
          // (two words hold this warp's 32 keys)
          const uint32_t* mk = a.masks + static_cast<size_t>(sg.q0 + sg.node0) * a.words32;
          uint32_t lo = 0, hi = 0;
          for (int i = lane; i < nodes; i += 32) {
            lo |= view_word(mk + static_cast<size_t>(i) * a.words32, a.words32, n_new, w0 + (warp & 3));
            hi |= view_word(mk + static_cast<size_t>(i) * a.words32, a.words32, n_new, w0 + (warp & 3) + 1);
          }
          lo = __reduce_or_sync(0xffffffffu, lo);
          hi = __reduce_or_sync(0xffffffffu, hi);
          dead = !(__funnelshift_r(lo, hi, sh) >> lane & 1u);
        }
        if (!(ok = warp_wait(C::SFULL + b, sc++ & 1, 82))) break;
        tc_fence_after();
        constexpr int W = KV8 ? 32 : 64;
        if (live) {
          if (masked) {
            // Scores of unseen keys become -inf in place, 32 columns at a time (a loop of
            // its own: code that few steps run is fetched anew each time).
#pragma unroll 1
            for (int c = 0; c < C::BN; c += 32) {
              const uint32_t w = seen[0];
              seen[0] = seen[1];
              seen[1] = seen[2];
              seen[2] = seen[3];
              if (__all_sync(0xffffffffu, w == 0xffffffffu)) continue;
              uint32_t x[32];
              tmem_ld32_async(tm_s + c, x);
              tmem_wait_ld();
              pin(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = w >> e & 1u ? x[e] : 0xff800000u;
              tmem_st32_async(tm_s + c, x);
            }
            tmem_wait_st();
          }
          // Two passes over the scores in TMEM, W columns at a time.  The loops' code is what
          // counts: with all 128 scores of a row in registers and nothing rolled the warps'
          // code outgrew the instruction caches (e4m3, five roles at once: 206 -> 154 us on a
          // batch of 96 requests, W = 32; 64: 162.  bf16: 64 is the better one, 102 against 107
          // us on 32 trees of 64 nodes).
          // The row's maximum; the reference moves before any weight.
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < C::BN; c += W) {
            uint32_t sr[W];
#pragma unroll
            for (int e = 0; e < W; e += 32) tmem_ld32_async(tm_s + c + e, sr + e);
            tmem_wait_ld();
            pin(sr);
#pragma unroll
            for (int e = 0; e < W; e += 2)
              mx[(e / 2) % 4] = fmax3(mx[(e / 2) % 4], __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
          }
          const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
          const bool moved = m_tile > m_ref + kRescaleSlack;
          float alpha = 1.f;
          if (moved) {
            alpha = fast_exp2(m_ref - m_tile);
            l_run *= alpha;
            m_ref = m_tile;
          }
          if (__any_sync(0xffffffffu, moved) && !first) {
            // S of this step is done, so the slot's P V before it is too.
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float ov[16];
              tmem_ld16(tm_o + b * D + c * 16, ov);
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] *= alpha;
              tmem_st16(tm_o + b * D + c * 16, ov);
            }
          }
        }
        first = false;
        // V of keys that no row of the unit sees may hold anything: zeros instead, before the
        // slot's product reads the step.  (Two tiles: by each slot, for its own product.)
        if (masked) {
          const int stg = (g + k) % C::NV;
          if (!(ok = warp_wait(C::VFULL + stg, ((g + k) / C::NV) & 1, 83))) break;
          if (dead) {
#pragma unroll 1
            for (int c = 0; c < C::HALVES * 8; ++c)  // (eight lanes hit eight bank groups)
              st_shared_v4(v_s + stg * C::TBYTES + (i_row >> 4) * C::BLOCK_BYTES + ((i_row >> 3) & 1) * C::GSTRIDE +
                               (c >> 3) * 1024 + (i_row & 7) * 128 + ((c ^ i_row) & 7) * 16,
                           make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        // The first half of P V starts while the second half of P is worked out (32 trees
        // of 64 nodes: 89.9 -> 87.5 us).
        auto half_done = [&]() {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::PHALF + b));
        };
        if (live) {
          // The weights, 16 bits each, over the scores' columns.
          const float2 sl = make_float2(sl2, sl2), mm = make_float2(-m_ref, -m_ref);
          float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int c = 0; c < C::BN; c += W) {
            uint32_t sr[W], pk[W / 2];
#pragma unroll
            for (int e = 0; e < W; e += 32) tmem_ld32_async(tm_s + c + e, sr + e);
            tmem_wait_ld();
            pin(sr);
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sl, mm);
              const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
              pk[e / 2] = KV8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
              sum[(e / 2) % 4] = __fadd2_rn(sum[(e / 2) % 4], make_float2(p0, p1));
            }
#pragma unroll
            for (int e = 0; e < W / 2; e += 16) tmem_st16_async(tm_s + c / 2 + e, pk + e);
            if (c + W == C::BN / 2) half_done();
          }
          const float2 ps = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
          l_run += ps.x + ps.y;
        } else {
          half_done();
        }
        tmem_wait_st();
        tc_fence_before();  // P and O precede the next products
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::PFULL + b));
      }
      if (!ok) break;
      g += n;
      // ---- the segment's end
      if (!(ok = warp_wait(C::OFULL, seg & 1, 84))) break;
      tc_fence_after();
      // (What the loop needed of the record is read again here: registers.)
      const int kind = sg.kind, e_nodes = sg.nodes, e_n = sg.j1 - sg.j0;
      const bool e_two = e_nodes > NPS;
      const bool has_own = !first;                          // this slot took a step
      const bool has_other = !e_two && (e_n > 1 || first);  // ... and the other one, of the same rows
      // One tile: (m, l) of the two halves of its keys, joined.
      float w_other = 0.f, w_own = 1.f;
      if (!e_two) {
        xch[b * 128 + i_row] = make_float2(m_ref, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::SYNC));
        if (!(ok = warp_wait(C::SYNC, sync_phase++ & 1, 80))) break;
        const float2 other = xch[(b ^ 1) * 128 + i_row];
        const float m = fmaxf(m_ref, other.x);
        w_own = fast_exp2(m_ref - m);
        w_other = fast_exp2(other.x - m);
        m_ref = m;
        l_run = l_run * w_own + other.y * w_other;
      }
      const int e_rows = (e_two ? (b ? e_nodes - NPS : NPS) : e_nodes) * G;
      if ((warp & 3) * 32 < e_rows) {
        const bool mine = i_row < e_rows;
        const size_t rec = record_of(cta, kind == kTail ? 1 : 0, e_two ? b : 0);
        // A quad's lanes take 16 bytes each of one row at a time: whole sectors (kWhole).
        __nv_bfloat16* dst = a.out + (static_cast<size_t>(sg.q0 + sg.node0 + (e_two && b ? NPS : 0)) * a.num_heads +
                                      sg.kvh * G) * D + (lane & 3) * 8;
        const int row0 = i_row & ~3;
        float4* part = reinterpret_cast<float4*>(a.part_o + rec * (D * 128)) + i_row;
        if (kind != kWhole && mine && (e_two || b == 0))
          *reinterpret_cast<float2*>(a.part_ml + (rec * 128 + i_row) * 2) = make_float2(m_ref, l_run);
        const float inv = kind != kWhole ? 1.f : (l_run > 0.f ? a.o_scale / l_run : 0.f);
        const float f_own = w_own * inv, f_other = w_other * inv;
        // Two tiles: the slot's columns; one: half the columns each, of both slots' O.
        constexpr int E = 32;
        const int c_first = e_two ? 0 : b * (D / 2);
#pragma unroll 1
        for (int c = c_first; c < (e_two ? D : c_first + D / 2); c += E) {
          uint32_t o[E];
          tmem_ld32_async(tm_o + b * D + c, o);
          uint32_t x[E];
          if (has_other) tmem_ld32_async(tm_o + (b ^ 1) * D + c, x);
          tmem_wait_ld();
          pin(o);
          if (has_other) pin(x);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float v = has_own ? __uint_as_float(o[e]) * f_own : 0.f;
            if (has_other) v = fmaf(__uint_as_float(x[e]), f_other, v);
            o[e] = __float_as_uint(v);
          }
          auto f = [&](int e) { return __uint_as_float(o[e]); };
          if (kind == kWhole) {
            uint4 p[4];
#pragma unroll
            for (int e = 0; e < E; e += 8)
              p[e / 8] = make_uint4(pack_bf16x2(f(e), f(e + 1)), pack_bf16x2(f(e + 2), f(e + 3)),
                                    pack_bf16x2(f(e + 4), f(e + 5)), pack_bf16x2(f(e + 6), f(e + 7)));
            swap_pieces(p[0], p[1], 1, lane);
            swap_pieces(p[2], p[3], 1, lane);
            swap_pieces(p[0], p[2], 2, lane);
            swap_pieces(p[1], p[3], 2, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = row0 + j, node = node_of(row);
              if (row < e_rows)
                *reinterpret_cast<uint4*>(dst + (node * a.num_heads + row - node * G) * D + c) = p[j];
            }
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < E; e += 4)
              part[((c + e) / 4) * 128] = make_float4(f(e), f(e + 1), f(e + 2), f(e + 3));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::OFREE));
        mbar_arrive(bar(C::SEGFREE + slot));
      }
    }
    if (!ok && lane == 0) *fail_flag = 1;
  } else {
    if (warp == 8) {
      // ====================================== range walk, Q and K producer
      const uint64_t policy = l2_policy_evict_first();
      if (lane == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        a.splits[cta].c1 = -1;  // no unit cut at the end of this range so far
      }
      const int H = a.num_kv_heads;
      // 128 requests at a time, their loads in flight together.
      int tiles[4], steps[4];
      auto load_requests = [&](int rc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const TreeReq p = tree_req(a, rc + 32 * i + lane);
          tiles[i] = p.tiles;
          steps[i] = req_steps(p);
        }
      };
      long long st = 0, un = 0;
      for (int rc = 0; rc < a.num_seqs; rc += 128) {
        load_requests(rc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          un += tiles[i];
          st += static_cast<long long>(tiles[i]) * steps[i];
        }
      }
      const long long n_steps = warp_sum64(st) * H, n_units = warp_sum64(un) * H;
      const long long Cw = kStepCost * n_steps + kUnitCost * n_units;
      // By cost only where every share holds a unit's start and a step, so that every
      // CTA between a unit's first and last has one of its steps; else by steps.
      const bool by_cost = div_ll(Cw, a.num_ctas) >= kStepCost + kUnitCost;
      const long long CT = by_cost ? kStepCost : 1, CS = by_cost ? kUnitCost : 0;
      const long long Ctot = by_cost ? Cw : n_steps;
      const long long x0 = Ctot > 0 ? range_lo(Ctot, a.num_ctas, cta) : 0;
      const long long x1 = Ctot > 0 ? range_lo(Ctot, a.num_ctas, cta + 1) : 0;
      int seg = 0, g = 0, nq[2] = {0, 0};
      bool ok = true;
      // Steps [j, ..) of a unit whose cost starts at cb: step j starts at cb + CS + CT j.
      auto first_step_at = [&](long long cb, long long x) -> long long {
        return x <= cb + CS ? 0 : div_ll(x - cb - CS + CT - 1, CT);
      };
      if (x0 < x1) {
        // The request that holds x0, and the cost before it.
        int r = -1;
        long long cb = 0;
        for (int rc = 0; rc < a.num_seqs && r < 0; rc += 128) {
          if (a.num_seqs > 128) load_requests(rc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (r >= 0) continue;
            const long long cost = (CS + CT * steps[i]) * tiles[i] * H;
            long long incl = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const long long v = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, cb + incl > x0);
            if (hit != 0) {
              const int first = __ffs(hit) - 1;
              cb += __shfl_sync(0xffffffffu, incl - cost, first);
              r = rc + 32 * i + first;
            } else {
              cb += __shfl_sync(0xffffffffu, incl, 31);
            }
          }
        }
        TreeReq p = tree_req(a, r);
        int n_u = req_steps(p);
        int u = static_cast<int>(div_ll(x0 - cb, CS + CT * n_u));  // unit: kv head, then tile pair
        cb += u * (CS + CT * n_u);
        long long j = first_step_at(cb, x0);
        while (ok) {
          if (j >= n_u) {  // no step of this unit starts in the range: the next one
            cb += CS + CT * n_u;
            j = 0;
            if (cb + CS >= x1) break;  // (before looking for a unit that the range does not reach)
            if (++u == H * p.tiles) {
              u = 0;
              // The next request with rows (idle ones may be most of a batch of fixed slots), 32 at a
              // time: 30000 of them between four live requests 3.35 ms one by one, 0.58 ms so, in front of
              // them 0.71.  (128 at a time, unrolled: 1 to 3 % slower on batches without idle ones, code.)
              TreeReq c;
              unsigned hit;
              do {
                c = tree_req(a, r + 1 + lane);
                hit = __ballot_sync(0xffffffffu, c.tiles > 0);
                r += hit != 0 ? __ffs(hit) : 32;
              } while (hit == 0 && r < a.num_seqs);
              if (hit == 0) break;  // no more work
              const int from = __ffs(hit) - 1;
              p.q0 = __shfl_sync(0xffffffffu, c.q0, from);
              p.n = __shfl_sync(0xffffffffu, c.n, from);
              p.len = __shfl_sync(0xffffffffu, c.len, from);
              p.tiles = __shfl_sync(0xffffffffu, c.tiles, from);
              n_u = req_steps(p);
            }
          }
          if (cb + CS + CT * j >= x1) break;
          const int j0 = static_cast<int>(j);
          const int j1 = static_cast<int>(min(static_cast<long long>(n_u), first_step_at(cb, x1)));
          const int kvh = u / p.tiles, node0 = (u - kvh * p.tiles) * 2 * NPS;
          const int nodes = min(2 * NPS, p.n - node0);
          const int nsl = nodes > NPS ? 2 : 1;
          if (seg >= C::SEGS && !(ok = warp_wait(C::SEGFREE + seg % C::SEGS, ((seg / C::SEGS) - 1) & 1, 60))) break;
          if (lane == 0) {
            TreeSeg sg{};
            sg.r = r;
            sg.q0 = p.q0;
            sg.node0 = node0;
            sg.nodes = nodes;
            sg.ctx = p.len - p.n;
            sg.n_new = p.n;
            sg.j0 = j0;
            sg.j1 = j1;
            sg.kvh = kvh;
            sg.kind = (j0 == 0 && j1 == n_u) ? kWhole : (j0 > 0 ? kHead : kTail);
            segs[seg % C::SEGS] = sg;
            mbar_arrive(bar(C::SEGFULL + seg % C::SEGS));
            if (sg.kind == kTail) {
              TreeSplit sp;
              sp.c1 = cta_of_tile(Ctot, a.num_ctas, cb + CS + CT * (n_u - 1));
              sp.row0 = p.q0 + node0;
              sp.nodes = nodes;
              sp.kvh = kvh;
              a.splits[cta] = sp;
            }
          }
          // Q of both slots, once the last S product of the previous segment is done.
          if (seg > 0 && !(ok = warp_wait(C::QFREE, (seg - 1) & 1, 61))) break;
          if (lane == 0) {
            for (int b = 0; b < nsl; ++b) {
              mbar_arrive_expect_tx(bar(C::QFULL + b), C::HALVES * G * NPS * 128);
#pragma unroll
              for (int h = 0; h < C::HALVES; ++h)
                tma_load_3d(q_s + b * C::QBYTES + h * C::CHUNK, &qmap, bar(C::QFULL + b), 64 * h, kvh * G,
                            p.q0 + node0 + b * NPS, policy);
              n_q_issued[b] = ++nq[b];
            }
          }
          __syncwarp();
          const int nblk = (p.len + kBlockSize - 1) / kBlockSize;
          int rowc = tile_rows(r, j0 * 8, nblk, true);
          for (int jj = j0; jj < j1; ++jj) {
            const int stg = g % C::NK;
            if (g >= C::NK && !(ok = warp_wait(C::KFREE + stg, ((g / C::NK) - 1) & 1, 62))) break;
            const int nb = min(8, nblk - jj * 8);
            if (lane == 0) mbar_arrive_expect_tx(bar(C::KFULL + stg), nb * C::K_BLOCK);
            __syncwarp();
            if (lane < nb) {
              const uint32_t dst = k_s + stg * C::KBYTES + lane * C::K_BLOCK;
              if constexpr (KV8)
                tma_load_3d(dst, &kmap, bar(C::KFULL + stg), 0, kvh, rowc, policy);
              else
                tma_load_5d(dst, &kmap, bar(C::KFULL + stg), 0, 0, 0, rowc / 8, kvh, policy);
            }
            ++g;
            if (lane == 0) *n_k_issued = g;
            if (jj + 1 < j1) rowc = tile_rows(r, (jj + 1) * 8, nblk, true);
          }
          ++seg;
          if (!ok || j1 < n_u) break;  // the range ends inside this unit
          j = n_u;
        }
      }
      if (ok && seg >= C::SEGS) ok = warp_wait(C::SEGFREE + seg % C::SEGS, ((seg / C::SEGS) - 1) & 1, 67);
      if (ok && lane == 0) {
        segs[seg % C::SEGS].kind = kEnd;
        mbar_arrive(bar(C::SEGFULL + seg % C::SEGS));
      }
      if (!ok && lane == 0) *fail_flag = 1;
      if (cta == 0) report_bad_requests(a, lane);
    } else if (warp == 10) {
      // =========================================================== V producer
      const uint64_t policy = l2_policy_evict_first();
      if (lane == 0) tma_prefetch_desc(&vmap);
      bool ok = true;
      int g = 0;
      for (int seg = 0; ok; ++seg) {
        const int slot = seg % C::SEGS;
        if (!(ok = warp_wait(C::SEGFULL + slot, (seg / C::SEGS) & 1, 63))) break;
        const TreeSeg sg = segs[slot];
        if (sg.kind == kEnd) break;
        const int nblk = (sg.ctx + sg.n_new + kBlockSize - 1) / kBlockSize;
        int rowc = tile_rows(sg.r, sg.j0 * 8, nblk, false);
        for (int jj = sg.j0; jj < sg.j1; ++jj) {
          constexpr int NS = KV8 ? C::NR : C::NV;
          const int stg = g % NS;
          if (g >= NS && !(ok = warp_wait((KV8 ? C::VRAWFREE : C::VFREE) + stg, ((g / NS) - 1) & 1, 64))) break;
          const int nb = min(8, nblk - jj * 8);
          const int full = (KV8 ? C::VRAW : C::VFULL) + stg;
          if (lane == 0) mbar_arrive_expect_tx(bar(full), nb * (KV8 ? C::RAW_BLOCK : C::BLOCK_BYTES));
          __syncwarp();
          if (lane < nb) {
            if constexpr (KV8)
              tma_load_3d(sbase + C::OFF_VRAW + stg * C::RAW_BYTES + lane * C::RAW_BLOCK, &vmap, bar(full), 0, sg.kvh,
                          rowc, policy);
            else
              tma_load_5d(v_s + stg * C::TBYTES + lane * C::BLOCK_BYTES, &vmap, bar(full), 0, 0, 0, rowc / 8, sg.kvh,
                          policy);
          }
          ++g;
          if (lane == 0) *n_v_issued = g;
          if (jj + 1 < sg.j1) rowc = tile_rows(sg.r, (jj + 1) * 8, nblk, false);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(C::SEGFREE + slot));
      }
      if (!ok && lane == 0) *fail_flag = 1;
    } else if (warp == 9 || warp == 11) {
      // =========================== MMA issue of slot 0 (warp 9) and 1 (warp 11)
      // A warp each: one thread that issues for both slots is busy longer with its
      // waits, fences and commits than the tensor core with the products.
      if (lane == 0) {
        const int b = warp == 9 ? 0 : 1;
        bool ok = true;
        int g = 0, pc = 0, qc[2] = {0, 0}, turns = 0;
        auto wait = [&](int k, uint32_t parity, int where) -> bool {
          if (*fail_flag) return false;
          if (!mbar_wait(bar(k), parity)) {
            give_up(where);
            return false;
          }
          return true;
        };
        // Operand descriptors differ by their start addresses alone, the low word's low
        // bits: one is built for each operand, offsets are added.
        const uint64_t qd = sdesc_sw128(q_s, 16, 1024);
        const uint64_t kd = !KV8 ? sdesc_sw128(k_s, 16, C::GSTRIDE)
                                 : (D == 128 ? sdesc_sw128(k_s, 16, 1024) : sdesc_sw64(k_s, 16, 512));
        const uint64_t vd = sdesc_sw128(v_s, 1024, C::GSTRIDE);
        const uint32_t ts = tmem + b * C::BN, to = tmem + 256 + b * D;
        // Whether K step gk has landed.
        auto k_there = [&](int gk) -> bool {
          return mbar_test(bar(C::KFULL + gk % C::NK), (gk / C::NK) & 1);
        };
        auto k_wait = [&](int gk) -> bool {
          if (!wait(C::KFULL + gk % C::NK, (gk / C::NK) & 1, 72)) return false;
          tc_fence_after();
          return true;
        };
        // S = Q (buffer qb) K^T of K step gk, into the slot's columns.  `pass_on`: the other
        // slot's turn begins early enough that it wakes as the last products are issued.
        auto issue_s = [&](int qb, int gk, bool pass_on) {
          const uint64_t q0 = qd + qb * (C::QBYTES >> 4);
          const uint64_t k0 = kd + (gk % C::NK) * (C::KBYTES >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            if constexpr (KV8) {  // q's upper parts, then its lower ones
              const int part = ks / (D / 32), k32 = ks % (D / 32) * 32;
              umma_e4m3(ts, q0 + ((part * (D == 128 ? C::CHUNK : 64) + k32) >> 4), k0 + (k32 >> 4), C::IDESC_S, ks > 0);
            } else {
              umma_bf16(ts, q0 + (((ks / 4) * C::CHUNK + (ks % 4) * 32) >> 4),
                        k0 + (((ks / 4) * 1024 + (ks % 4) * 32) >> 4), C::IDESC_S, ks > 0);
            }
            if (ks == 1 && pass_on) mbar_arrive(bar(C::TURN + (b ^ 1)));
          }
          umma_commit(bar(C::SFULL + b));
        };
        // The step's K stage is free when S is done; a step that only this slot takes
        // is freed for the other one as well.
        auto free_k = [&](int gk, bool both) {
          umma_commit(bar(C::KFREE + gk % C::NK));
          if (!both) mbar_arrive(bar(C::KFREE + gk % C::NK));
        };
        // O += P V of V step gv (P: 16 bits in the slot's S columns).
        auto issue_pv = [&](int gv, bool acc, bool in_turn) -> bool {
          if (!wait(C::VFULL + gv % C::NV, (gv / C::NV) & 1, 73) || !wait(C::PHALF + b, pc & 1, 75)) return false;
          if (in_turn && (b == 1 || turns > 0) && !wait(C::TURN + b, (b == 1 ? turns : turns - 1) & 1, 77)) return false;
          tc_fence_after();
          const uint64_t v0 = vd + (gv % C::NV) * (C::TBYTES >> 4);
          umma_tmem_a(to, ts, v0, C::IDESC_O, acc ? 1u : 0u);
#pragma unroll
          for (int ks = 1; ks < C::BN / 32; ++ks)
            umma_tmem_a(to, ts + ks * 8, v0 + ((ks * C::BLOCK_BYTES) >> 4), C::IDESC_O, 1u);
          if (!wait(C::PFULL + b, pc++ & 1, 75)) return false;
          tc_fence_after();
#pragma unroll
          for (int ks = C::BN / 32; ks < C::BN / 16; ++ks)
            umma_tmem_a(to, ts + ks * 8, v0 + ((ks * C::BLOCK_BYTES) >> 4), C::IDESC_O, 1u);
          return true;
        };
        for (int seg = 0; ok; ++seg) {
          const int slot = seg % C::SEGS;
          if (!(ok = wait(C::SEGFULL + slot, (seg / C::SEGS) & 1, 70))) break;
          const TreeSeg sg = segs[slot];
          if (sg.kind == kEnd) break;
          const int n = sg.j1 - sg.j0;
          const bool two = sg.nodes > NPS;
          // Two tiles: both slots take every step; one: those of their parity (of the
          // CTA's step count g + k, so that a K stage always has the same owner).  Both
          // slots wait for and free every V step, in order: a barrier's parity names a
          // phase only to who has seen the one before.  With two tiles they issue in
          // turn: at the same time their products share the tensor core, both softmaxes start
          // together when they are done, and the core idles meanwhile (32 trees of 64 nodes:
          // 127 us without, 106 with turns).  A slot without a step still waits for the segment's Q
          // and the end of the one before, so that its arrivals count for this one.
          const int k0 = two ? 0 : (g ^ b) & 1, dk = two ? 1 : 2;
          const int qb = two ? b : 0;
          ok = KV8 ? wait(C::QCONV, seg & 1, 71) : wait(C::QFULL + qb, qc[qb] & 1, 71);
          ++qc[0];
          if (two) ++qc[1];
          if (!ok) break;
          if (k0 < n) {
            if (!(ok = k_wait(g + k0))) break;
            issue_s(qb, g + k0, false);
            free_k(g + k0, two);
          }
          if (k0 + dk >= n) {  // the last S of the segment
            if (k0 < n)
              umma_commit(bar(C::QFREE));
            else
              mbar_arrive(bar(C::QFREE));
          }
          if (seg > 0 && !(ok = wait(C::OFREE, (seg - 1) & 1, 76))) break;
          for (int k = 0; k < n; ++k) {
            if (!two && ((k ^ k0) & 1)) {
              if (!(ok = wait(C::VFULL + (g + k) % C::NV, ((g + k) / C::NV) & 1, 74))) break;
              mbar_arrive(bar(C::VFREE + (g + k) % C::NV));
              continue;
            }
            // The next step's K usually has landed: known before, S follows P V without a
            // wait, and all commits come behind both (each takes as long as a product's part).
            const int gv = g + k;
            const bool more = k + dk < n;
            const bool there = more && k_there(gv + dk);
            if (!(ok = issue_pv(gv, k > k0, two))) break;
            if (more) {
              if (!there) {
                umma_commit(bar(C::VFREE + gv % C::NV));
                if (!(ok = k_wait(gv + dk))) break;
              }
              issue_s(qb, gv + dk, two);
            }
            if (two && !more) mbar_arrive(bar(C::TURN + (b ^ 1)));
            turns += two;
            if (more) free_k(gv + dk, two);
            if (there || !more) umma_commit(bar(C::VFREE + gv % C::NV));
            if (more && k + 2 * dk >= n) umma_commit(bar(C::QFREE));
          }
          if (!ok) break;
          if (k0 < n)
            umma_commit(bar(C::OFULL));
          else
            mbar_arrive(bar(C::OFULL));
          g += n;
          mbar_arrive(bar(C::SEGFREE + slot));
        }
        if (!ok) *fail_flag = 1;
        // Every MMA issued has completed before TMEM can be released.
        umma_commit(bar(C::DRAIN + b));
        (void)mbar_wait(bar(C::DRAIN + b), 0);
      }
      __syncwarp();
    } else if (warp >= 12) {
      // ============================= e4m3: q split, V to f16 (a quarter of a step each)
      if constexpr (KV8) {
        const int w4 = warp - 12;
        bool ok = true;
        int g = 0, qn[2] = {0, 0};
        for (int seg = 0; ok; ++seg) {
          const int slot = seg % C::SEGS;
          if (!(ok = warp_wait(C::SEGFULL + slot, (seg / C::SEGS) & 1, 68))) break;
          const TreeSeg sg = segs[slot];
          if (sg.kind == kEnd) break;
          const int nblk = (sg.ctx + sg.n_new + kBlockSize - 1) / kBlockSize, n = sg.j1 - sg.j0;
          const int nsl = sg.nodes > NPS ? 2 : 1;
          if (seg > 0 && !(ok = warp_wait(C::EXPFREE, (seg - 1) & 1, 78))) break;
          for (int qb = 0; qb < nsl && ok; ++qb)
            if ((ok = warp_wait(C::QFULL + qb, qn[qb]++ & 1, 65)))
              split_q<D, KV8>(q_s + qb * C::QBYTES, exps + qb * 128, a.exp_max, w4, lane);
          if (!ok) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::QCONV));
          for (int k = 0; k < n; ++k, ++g) {
            const int rs = g % C::NR, st = g % C::NV;
            if (!(ok = warp_wait(C::VRAW + rs, (g / C::NR) & 1, 66))) break;
            if (g >= C::NV && !(ok = warp_wait(C::VFREE + st, (g / C::NV - 1) & 1, 69))) break;
            convert_v<D, KV8>(sbase + C::OFF_VRAW + rs * C::RAW_BYTES, v_s + st * C::TBYTES, 2 * w4,
                              min(2 * w4 + 2, nblk - (sg.j0 + k) * 8), lane);
            fence_proxy_async_smem();  // the f16 step is read by the tensor core, the raw one overwritten by a copy
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(C::VFULL + st));
              mbar_arrive(bar(C::VRAWFREE + rs));
            }
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(bar(C::SEGFREE + slot));
        }
        if (!ok && lane == 0) *fail_flag = 1;
      }
    }
  }

  __syncthreads();
  if (*fail_flag && tid == 0) {
    // Let copies still in flight land before TMEM is released and the CTA leaves (bounded).
    const int nk = *n_k_issued, nv = *n_v_issued;
    const int vb = KV8 ? C::VRAW : C::VFULL;
    constexpr int SV = KV8 ? C::NR : C::NV;
    for (int i = max(0, nk - C::NK); i < nk; ++i) (void)mbar_wait(bar(C::KFULL + i % C::NK), (i / C::NK) & 1);
    for (int i = max(0, nv - SV); i < nv; ++i) (void)mbar_wait(bar(vb + i % SV), (i / SV) & 1);
    for (int b = 0; b < 2; ++b)
      if (n_q_issued[b] > 0) (void)mbar_wait(bar(C::QFULL + b), (n_q_issued[b] - 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merges the units that range boundaries cut (151 of them: 8 us over 64 requests x 16 nodes,
// 13 over two tiles a unit, 40 MB, caches cold).  Block (c, b, z): slot b of the unit
// that CTA c began and did not finish.  A warp takes 8 rows x 32 columns, a thread two
// groups of 4 columns, over the contributors in order, four at a time with all their loads
// in flight: a unit mostly has two, and what counts is the chain of round trips.
constexpr int kMergeWarps = 8;
constexpr int kMergeBatch = 4;
template <int D>
constexpr int merge_blocks() { return 16 * (D / 32) / kMergeWarps; }  // a task a warp
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const TreeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int c0 = blockIdx.x, b = blockIdx.y;
  const int4 rec = __ldcg(reinterpret_cast<const int4*>(a.splits + c0));
  const int c1 = rec.x, row0 = rec.y, nodes = rec.z, kvh = rec.w;
  if (c1 < 0) return;
  const int NPS = a.slot_nodes, G = a.group;
  const bool two = nodes > NPS;
  if (b == 1 && !two) return;
  const int rows = (two ? (b ? nodes - NPS : NPS) : nodes) * G;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.z * kMergeWarps + (threadIdx.x >> 5);
  const int i = t / (D / 32) * 8 + (lane & 7);
  const int c4 = t % (D / 32) * 8 + (lane >> 3);  // column groups of 4: this one and the fourth from it
  if (i >= rows) return;
  float m = kLowest, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f), o2 = o;
  auto add = [](float4& s, const float4& x, float w) {
    s = make_float4(fmaf(x.x, w, s.x), fmaf(x.y, w, s.y), fmaf(x.z, w, s.z), fmaf(x.w, w, s.w));
  };
  for (int c = c0; c <= c1; c += kMergeBatch) {
    float2 ml[kMergeBatch];
    float4 x[kMergeBatch], x2[kMergeBatch];
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      ml[u] = make_float2(kLowest, 0.f);
      x[u] = x2[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + u > c1) continue;
      const size_t rid = record_of(c + u, c + u == c0 ? 1 : 0, b);
      const float4* part = reinterpret_cast<const float4*>(a.part_o + rid * (D * 128)) + c4 * 128 + i;
      ml[u] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (rid * 128 + i) * 2));
      x[u] = __ldcg(part);
      x2[u] = __ldcg(part + 4 * 128);
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) top = fmaxf(top, ml[u].x);
    const float w0 = fast_exp2(m - top);
    m = top;
    l *= w0;
    o = make_float4(o.x * w0, o.y * w0, o.z * w0, o.w * w0);
    o2 = make_float4(o2.x * w0, o2.y * w0, o2.z * w0, o2.w * w0);
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const float w = fast_exp2(ml[u].x - m);
      l = fmaf(ml[u].y, w, l);
      add(o, x[u], w);
      add(o2, x2[u], w);
    }
  }
  const float inv = l > 0.f ? a.o_scale / l : 0.f;
  const int node = i * a.group_inv >> 16;
  __nv_bfloat16* dst = a.out + (static_cast<size_t>(row0 + (two && b ? NPS : 0) + node) * a.num_heads + kvh * G +
                                (i - node * G)) * D + c4 * 4;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  *reinterpret_cast<uint2*>(dst + 16) =
      make_uint2(pack_bf16x2(o2.x * inv, o2.y * inv), pack_bf16x2(o2.z * inv, o2.w * inv));
}

template <int D, bool KV8>
cudaError_t launch_impl(const TreeArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        cudaStream_t stream) {
  using C = TreeCfg<D, KV8>;
  static bool attr_set[64] = {false};  // per device: set once
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    const cudaError_t err =
        cudaFuncSetAttribute(tree_attention_kernel<D, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (err != cudaSuccess) return err;
    attr_set[dev] = true;
  }
  const cudaError_t err = launch_overlapped(tree_attention_kernel<D, KV8>, dim3(a.num_ctas), dim3(C::THREADS), C::SMEM,
                                            stream, qmap, kmap, vmap, a);
  // Units of one step are never cut.
  if (err != cudaSuccess || a.max_seq_len <= 128) return err;
  return launch_overlapped(tree_merge_kernel<D>, dim3(a.num_ctas, 2, merge_blocks<D>()), dim3(kMergeWarps * 32), 0, stream,
                           a);
}

}  // namespace

size_t tree_record_floats(int head_dim) { return 4 * 128 * static_cast<size_t>(head_dim); }

cudaError_t launch_tree_attention(const TreeArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                  const CUtensorMap& vmap, int head_dim, bool kv8, cudaStream_t stream) {
  if (head_dim == 128)
    return kv8 ? launch_impl<128, true>(a, qmap, kmap, vmap, stream) : launch_impl<128, false>(a, qmap, kmap, vmap, stream);
  return kv8 ? launch_impl<64, true>(a, qmap, kmap, vmap, stream) : launch_impl<64, false>(a, qmap, kmap, vmap, stream);
}

}  // namespace pa
