// pa_decode_fp4 — paged decode attention over a 4-bit cache (format:
// pa_fp4.cuh), sm_100a.
//
// What it computes: pa_decode's softmax(scale q K^T) V (vLLM blog §"关键细节"
// 2; study notes ch.05 §4) with the K and V values that the 4-bit pools hold;
// on request each row's log normaliser, and each token's scores for the
// accumulated attention weights (pa_weights.cu).
//
// What bounds it.  A (token, kv head) pair is 2 x 9/16 D bytes (144 at D =
// 128), which at the card's copy rate arrives about every 6 cycles on an SM;
// in that time 2 D codes become halves (one conversion and one multiply by
// the scale for two of them).  Expanding K and V into shared memory or
// tensor memory for tcgen05 would move 512 bytes more per pair through
// memories that carry 128 bytes a cycle, twice (write and operand read); so
// the codes go from shared memory into registers, are expanded there and
// enter mma.sync as the A operand straight from those registers.  The thin
// products (at most 8 query rows) need a third of that path's rate.  Not tried:
// K alone as the packed operand of a block-scaled tcgen05.mma, which takes e2m1
// with an e4m3 scale per 16 elements along the contraction as they lie here, and
// q as several e2m1 digits.  V's scales run along the output's rows, so V would
// be expanded as now.
//
// Rows (the kernel: pa_thin_decode.cuh).  p enters as a half and the half of its
// rounding residual.  A half alone, off by up to 2^-11 of each weight, would do
// for most bf16 outputs (half a step is 2^-8), but not where they nearly cancel;
// it saves 3 % of the ragged batch below, and 7 % with 8 query heads a kv head.
// q is rounded to half after each row is scaled by a power of two to at most
// 2^15: exact for fp16, and for bf16 exact but for elements under 2^-29 of the
// row's largest, whose rounding is below fp32's own.  code * scale is exact in
// half (pa_fp4.cuh), so the products are those of the stored values, summed
// in fp32.
//
// Fragments without exchange.  A thread's A elements of K are two bytes of
// one row's codes (neighbours along d), with d permuted so that it reads one
// contiguous piece of the row; q is permuted alike.  V's pairs run along
// tokens instead: the codes of two token rows are interleaved by nibbles (4
// operations for 16 codes) before they are expanded.  p^T is transposed by
// movmatrix.
//
// Measured (B200, one launch, D = 128, in a captured graph): 8 sequences of 32k
// tokens x 40 kv heads, G = 1, fp16: 275 us, 5.5 TB/s (0.84 of the copy rate;
// under the power cap of a long loop through the entry point 323); 256 sequences
// of log-normal lengths (median 1024) x 8, G = 4, bf16: 93 us, 4.2 TB/s, 99
// through the entry point; one sequence of 1027 tokens x 8, G = 4: 10.  What is
// left of the roof goes to instructions: about 320 for 16 tokens and a kv head,
// issued at 0.58 a clock, with the pipe of the conversions half busy and the
// tensor pipe a quarter.  The warps do not wait for memory: 3 CTAs an SM (168
// registers, no spills) took 274 us where 2 took 298, 4 took 280 and 5 (96
// registers) twice as much; copies by TMA instead of cp.async and ranges weighted
// by the CTAs' age measured slower (294 and 334 us where 4 CTAs took 280 and 290).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pa_decode_host.h"
#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"
#include "pa_thin_decode.cuh"

namespace pa {
namespace fp4 {

using namespace thin;

// The 4-bit format of the thin decode.
template <int D>
struct Fp4 {
  static constexpr int kD = D, kCtasPerSm = 3;
  static constexpr bool kBf16P = false;
  static constexpr int kCodeRow = code_row_bytes(D), kScaleRow = scale_row_bytes(D);
  static constexpr int kKXor = 0, kVXor = 32;
  static constexpr int kCodes = kStepTok * code_row_bytes(D);
  static constexpr int kScales = kStepTok * scale_row_bytes(D);
  static constexpr int kK = 0, kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
  static constexpr int kBytes = 2 * (kCodes + kScales);
  // V's 16-byte pieces are placed so that the reads of a warp (8 bytes of
  // rows 2t, or 4 bytes at D = 64) fall into different banks: the piece's
  // index in its 128-byte line, exclusive-or with the line's number
  __device__ static __forceinline__ int v_at(int row, int piece) {
    constexpr int kPieces = code_row_bytes(D) / 16;     // of a row
    constexpr int kRows = 8 / kPieces;                  // of a line
    const int line = row / kRows;
    const int p8 = (row % kRows) * kPieces + piece;
    return kV + line * 128 + ((p8 ^ (2 * (line & (D == 128 ? 3 : 1)))) << 4);
  }

  // q's fragments for the unit's rows (B operand, each lane's d's) from its
  // query rows, which have arrived: rounded to half after scaling each row by a
  // power of two.  One warp.
  template <bool kEight, int kRows>
  __device__ static __forceinline__ void prepare(const ThinParams& p, int lane, Unit<D, kRows>& unit) {
    uint32_t qf[D / 8];
    const int g = lane >> 2, t = lane & 3;
    const int row = kEight ? g : (g & 3);
    float inv = 1.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 w = row < p.G ? unit.raw[row * (D / 8) + t * (D / 32) + i] : make_uint4(0, 0, 0, 0);
      qf[4 * i] = w.x;
      qf[4 * i + 1] = w.y;
      qf[4 * i + 2] = w.z;
      qf[4 * i + 3] = w.w;
    }
    if (p.bf16) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float a, b;
        unpack2<true>(qf[i], a, b);
        top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e with top * 2^e in [2^14, 2^15); rows of zeros or with an infinity
      // keep their values
      float up = 1.f;
      if (top > 0.f && top <= 3.4e38f) {
        const int e = 14 - max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
        up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float a, b;
        unpack2<true>(qf[i], a, b);
        qf[i] = pack2<false>(a * up, b * up);
      }
    }
    const float f = p.d.scale_log2 * inv;
    // the row of column 2t is held by the lanes with g = 2t
    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    unit.f[lane] = make_float2(f0, f1);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) unit.q[w][lane] = make_uint4(qf[4 * w], qf[4 * w + 1], qf[4 * w + 2], qf[4 * w + 3]);
  }

  // S^T of a step's two halves: c[half] += K q^T.
  template <int kRows>
  __device__ static __forceinline__ void scores(const uint8_t* slot, int lane, const Unit<D, kRows>& unit,
                                                float (&c)[2][4]) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int kW = D / 32;  // words of codes a thread reads of each row
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t k[2][kW], s[2][D / 64];  // two rows, and their scales, twice each
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r + 16 * half;
        if constexpr (D == 128) {
          *reinterpret_cast<uint4*>(k[r]) = *reinterpret_cast<const uint4*>(slot + kK + row * 64 + t * 16);
          const uint32_t x = halves_of_e4m3(*reinterpret_cast<const uint16_t*>(slot + kKs + row * 8 + t * 2));
          s[r][0] = __byte_perm(x, x, 0x1010);
          s[r][1] = __byte_perm(x, x, 0x3232);
        } else {
          *reinterpret_cast<uint2*>(k[r]) = *reinterpret_cast<const uint2*>(slot + kK + row * 32 + t * 8);
          const uint32_t x = halves_of_e4m3(slot[kKs + row * 4 + t]);
          s[r][0] = __byte_perm(x, x, 0x1010);
        }
      }
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const uint4 q = unit.q[w][lane];
        uint32_t a[4], b[4];
        halves_of_e2m1(k[0][w], a);
        halves_of_e2m1(k[1][w], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = hmul2(a[i], s[0][w / 2]);
          b[i] = hmul2(b[i], s[1][w / 2]);
        }
        mma_f16(c[half], a[0], b[0], a[1], b[1], q.x, q.y);
        mma_f16(c[half], a[2], b[2], a[3], b[3], q.z, q.w);
      }
    }
  }

  // O^T += V^T p^T of 16 tokens, rows `at` of the slot.  This thread's tokens
  // are 2t, 2t + 1, 2t + 8, 2t + 9, its d's D/8 neighbours; tile i's rows g and
  // g + 8 are their pair 2i, 2i + 1.  b: p, and its residual where that is a
  // second product.
  template <int kParts>
  __device__ static __forceinline__ void values(const uint8_t* slot, int at, int lane, const uint32_t (&b)[kParts][2],
                                                float (&acc)[D / 16][4]) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int kVW = D / 64;  // words of codes a thread reads of each row
    uint32_t v[4][kVW], sv[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int tok = at + 2 * t + (k & 1) + 8 * (k >> 1);
      if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(v[k]) = *reinterpret_cast<const uint2*>(slot + v_at(tok, g >> 1) + (g & 1) * 8);
      } else {
        v[k][0] = *reinterpret_cast<const uint32_t*>(slot + v_at(tok, g >> 2) + (g & 3) * 4);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t* s = slot + kVs + (at + 2 * t + 8 * k) * scale_row_bytes(D) + (D == 128 ? g : g >> 1);
      sv[k] = halves_of_e4m3(s[0] | (static_cast<uint32_t>(s[scale_row_bytes(D)]) << 8));
    }
#pragma unroll
    for (int w = 0; w < kVW; ++w) {
      uint32_t lo[4], hi[4], lo8[4], hi8[4];
      const uint32_t m = 0x0f0f0f0fu;
      halves_of_e2m1((v[0][w] & m) | ((v[1][w] << 4) & ~m), lo);
      halves_of_e2m1(((v[0][w] >> 4) & m) | (v[1][w] & ~m), hi);
      halves_of_e2m1((v[2][w] & m) | ((v[3][w] << 4) & ~m), lo8);
      halves_of_e2m1(((v[2][w] >> 4) & m) | (v[3][w] & ~m), hi8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = hmul2(lo[j], sv[0]), a1 = hmul2(hi[j], sv[0]);
        const uint32_t a2 = hmul2(lo8[j], sv[1]), a3 = hmul2(hi8[j], sv[1]);
#pragma unroll
        for (int i = 0; i < kParts; ++i) mma_f16(acc[4 * w + j], a0, a1, a2, a3, b[i][0], b[i][1]);
      }
    }
  }

  // Column j of a thread's O^T: its D/8 neighbouring d's.
  __device__ static __forceinline__ void put(float* row, int g, int j, const float (&acc)[D / 16][4]) {
    float* to = row + g * (D / 8);
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      *reinterpret_cast<float4*>(to + 2 * i) = make_float4(acc[i][j], acc[i][j + 2], acc[i + 1][j], acc[i + 1][j + 2]);
    }
  }
};

template <int D, bool kScores>
static ThinKernel pick_rows(int G, Variant& v) {
  using F = Fp4<D>;
  return G == 8 ? thin_kernel<F, true, kScores>(G, v) : thin_kernel<F, false, kScores>(G, v);
}

static ThinKernel select_fp4(const pa_pool_desc& pool, int G, bool scores, Variant& v) {
  if (G != 1 && G != 2 && G != 4 && G != 8) return nullptr;
  if (pool.head_dim == 128) return scores ? pick_rows<128, true>(G, v) : pick_rows<128, false>(G, v);
  return scores ? pick_rows<64, true>(G, v) : pick_rows<64, false>(G, v);
}

static bool opts_fine(const pa_decode_opts* opts) {
  return opts == nullptr || (opts->num_ctas >= 0 && opts->flags == 0);
}

}  // namespace fp4
}  // namespace pa

using namespace pa;
using namespace pa::fp4;
using namespace pa::thin;

extern "C" size_t pa_decode_fp4_workspace_bytes(int32_t num_seqs, int32_t num_q_heads,
                                                int32_t weights_max_blocks_per_seq, const pa_pool_desc* pool,
                                                const pa_decode_opts* opts) {
  int G = 0;
  if (num_seqs < 0 || weights_max_blocks_per_seq < 0 || !pool_ok(pool) || !opts_fine(opts) ||
      !group_of(*pool, num_q_heads, G))
    return 0;
  const bool scores = weights_max_blocks_per_seq > 0;
  if (static_cast<long long>(weights_max_blocks_per_seq) * pool->block_size > kMaxTokens) return 0;
  Variant v;
  int ctas = 0;
  if (select_fp4(*pool, G, scores, v) == nullptr || !query_ctas(v, opts, ctas)) return 0;
  const size_t base = workspace_bytes_for(0, pool->num_kv_heads, ctas, v.part_stride);
  return scores ? base + scores_bytes(num_seqs, num_q_heads, weights_max_blocks_per_seq, pool->block_size) : base;
}

extern "C" pa_status pa_decode_fp4(const void* q, const void* k_pool, const void* v_pool,
                                   const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                   int32_t num_seqs, int32_t num_q_heads, float scale, float k_scale, float v_scale,
                                   void* out, float* lse, const pa_token_weights* weights, void* workspace,
                                   size_t workspace_bytes, int32_t* dev_status, const pa_pool_desc* pool,
                                   const pa_decode_opts* opts, void* stream) {
  const pa_status st = check_decode_args(q, k_pool, v_pool, block_tables, max_blocks_per_seq, seq_lens, num_seqs,
                                         num_q_heads, scale, out, pool);
  if (st != PA_OK) return st;
  if (!scale_ok(k_scale) || !scale_ok(v_scale) || !std::isfinite(scale * k_scale) || !opts_fine(opts))
    return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * pool->block_size > kMaxTokens) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (weights != nullptr && !token_weights_ok(weights, max_blocks_per_seq, num_seqs, pool)) return PA_ERR_INVALID_ARG;
  int G = 0;
  if (!pool_ok(pool) || !group_of(*pool, num_q_heads, G)) return PA_ERR_UNSUPPORTED;
  Variant v;
  const ThinKernel kernel = select_fp4(*pool, G, weights != nullptr, v);
  if (kernel == nullptr) return PA_ERR_UNSUPPORTED;
  const int ctas = resolve_ctas(v, opts);
  if (ctas <= 0) return PA_ERR_CUDA;
  const size_t base = workspace_bytes_for(0, pool->num_kv_heads, ctas, v.part_stride);  // no counts behind the states
  const size_t need =
      weights == nullptr ? base : base + scores_bytes(num_seqs, num_q_heads, max_blocks_per_seq, pool->block_size);
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)) return PA_ERR_WORKSPACE;

  ThinParams p;
  p.d = make_params(q, nullptr, nullptr, block_tables, max_blocks_per_seq, seq_lens, num_seqs, num_q_heads, scale, out,
                    workspace, ctas, v.part_stride, dev_status, pool, 0);
  p.d.scale_log2 = scale * k_scale * 1.4426950408889634f;
  p.d.max_nb = max_blocks_per_seq * (pool->block_size / kUnit);
  p.d.unit_cost = v.unit_cost;
  p.d.lse = lse;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.score_tokens = score_tokens_of(max_blocks_per_seq, pool->block_size);
  p.norm2 = nullptr;
  p.scores = nullptr;
  if (weights != nullptr) split_scores(static_cast<char*>(workspace) + base, num_seqs, num_q_heads, &p.norm2, &p.scores);
  p.table_width = max_blocks_per_seq;
  p.log2_block = log2_of(pool->block_size);
  p.tile = tile_bytes(pool->block_size, pool->head_dim);
  p.block_bytes = pool->num_kv_heads * p.tile;
  p.G = G;
  p.bf16 = pool->dtype == PA_BF16;
  p.out_scale = v_scale;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_overlapped(kernel, dim3(ctas), dim3(kDecodeThreads), static_cast<size_t>(v.smem_bytes), s, p) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  if (weights == nullptr) return PA_OK;
  return accumulate_weights(p.scores, p.norm2, *weights, block_tables, seq_lens, num_seqs, num_q_heads,
                            max_blocks_per_seq, nullptr, dev_status, pool, s);
}
