// pa_decode_weights over 16-bit pools at head_dim 64: the thin decode
// (pa_thin_decode.cuh) with ldmatrix fragments, its scores and normalisers
// written for the second launch (pa_weights.cu).
//
// softmax(scale q K^T) V as pa_decode (study notes ch.05 §4).  A (token, kv
// head) pair is 256 bytes, and G products of each of its 128 elements: on CUDA
// cores the instructions outlast the copies, and the tensor-core kernel's tiles
// are of head_dim 128.  q and the pools enter as they are; p as a 16-bit value and its
// residual (22 bits) in fp16, and in bf16, where those two hold 16 bits, as
// three values (24): pa_decode takes p in fp32 at this head_dim.
//
// Rows are 128 bytes, a line each: their 16-byte pieces are placed by the
// exclusive-or with the row's number, so that ldmatrix reads 8 rows without a
// conflict.
//
// Bound by memory.  Measured (B200, decode and weights, both launches): 64
// sequences of 2000 tokens x 8 kv heads, G = 4, bf16: 56 us, 4.7 TB/s (0.71
// of the copy rate), 131 on CUDA cores; 5 sequences of at most 100 tokens x 4:
// 7.7 us, 14.5 on CUDA cores.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_host.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_thin_decode.cuh"

namespace pa {
namespace thin {

template <bool kBf16>
struct Wide {
  static constexpr int kD = 64, kCtasPerSm = 3;  // 3 x 70 KB of shared memory
  static constexpr bool kBf16P = kBf16;
  static constexpr int kCodeRow = kD * 2, kScaleRow = 0;
  static constexpr int kK = 0, kV = kStepTok * kCodeRow, kKs = 0, kVs = 0;
  static constexpr int kKXor = 16, kVXor = 16;
  static constexpr int kBytes = 2 * kStepTok * kCodeRow;

  // The 16-byte piece of a row of K or V (shared address of row 0).
  __device__ static __forceinline__ uint32_t piece_at(uint32_t base, int row, int piece) {
    return base + row * kCodeRow + ((piece ^ (row & 7)) << 4);
  }
  __device__ static __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16) {
      mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
    } else {
      mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
    }
  }

  // q's fragments of the unit's rows, two k steps of 16 a word of the unit.
  template <bool kEight, int kRows>
  __device__ static __forceinline__ void prepare(const ThinParams& p, int lane, Unit<kD, kRows>& unit) {
    const int g = lane >> 2, t = lane & 3;
    const int row = kEight ? g : (g & 3);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(unit.raw) + row * (kD / 2);
    unit.f[lane] = make_float2(p.d.scale_log2, p.d.scale_log2);
#pragma unroll
    for (int w = 0; w < kD / 32; ++w) {
      const uint32_t* x = words + 16 * w + t;
      unit.q[w][lane] = row < p.G ? make_uint4(x[0], x[4], x[8], x[12]) : make_uint4(0, 0, 0, 0);
    }
  }

  // S^T of a step's two halves: c[half] += K q^T.
  template <int kRows>
  __device__ static __forceinline__ void scores(const uint8_t* slot, int lane, const Unit<kD, kRows>& unit,
                                                float (&c)[2][4]) {
    const uint32_t k = smem_u32(slot) + kK;
#pragma unroll
    for (int w = 0; w < kD / 32; ++w) {
      const uint4 q = unit.q[w][lane];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = (lane & 15) + 16 * half, piece = 4 * w + (lane >> 4);
        uint32_t a[4], b[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                     : "r"(piece_at(k, row, piece))
                     : "memory");
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(piece_at(k, row, piece + 2))
                     : "memory");
        mma(c[half], a, q.x, q.y);
        mma(c[half], b, q.z, q.w);
      }
    }
  }

  // O^T += V^T p^T of 16 tokens, rows `at` of the slot: tile i is d's 16 i to
  // 16 i + 15.  b: p's values, a product each.
  template <int kParts>
  __device__ static __forceinline__ void values(const uint8_t* slot, int at, int lane, const uint32_t (&b)[kParts][2],
                                                float (&acc)[kD / 16][4]) {
    const uint32_t v = smem_u32(slot) + kV;
    const int tok = at + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      uint32_t a[4];
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                   : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                   : "r"(piece_at(v, tok, 2 * i + ((lane >> 3) & 1)))
                   : "memory");
#pragma unroll
      for (int j = 0; j < kParts; ++j) mma(acc[i], a, b[j][0], b[j][1]);
    }
  }

  // Column j of a thread's O^T.
  __device__ static __forceinline__ void put(float* row, int g, int j, const float (&acc)[kD / 16][4]) {
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      row[16 * i + g] = acc[i][j];
      row[16 * i + 8 + g] = acc[i][j + 2];
    }
  }
};

template <bool kBf16, bool kEight, int B>
static cudaError_t launch_wide(const Variant& v, const DecodeParams& prm, int ctas, cudaStream_t stream) {
  ThinParams p;
  p.d = prm;
  p.d.max_nb = prm.max_nb * (B / kUnit);
  p.d.lse = nullptr;
  p.k_pool = reinterpret_cast<const uint8_t*>(prm.k_pool);
  p.v_pool = reinterpret_cast<const uint8_t*>(prm.v_pool);
  p.scores = prm.scores;
  p.norm2 = prm.lse;
  p.score_tokens = prm.score_tokens;
  p.table_width = prm.max_nb;
  p.log2_block = B == 8 ? 3 : B == 16 ? 4 : 5;
  p.tile = B * Wide<kBf16>::kCodeRow;
  p.block_bytes = prm.num_kv_heads * p.tile;
  p.G = prm.num_q_heads / prm.num_kv_heads;
  p.bf16 = kBf16;
  p.out_scale = 1.f;
  return launch_overlapped(&decode_thin_kernel<Wide<kBf16>, kEight, true>, dim3(ctas), dim3(kDecodeThreads),
                           static_cast<size_t>(v.smem_bytes), stream, p);
}

template <bool kBf16, bool kEight>
static void pick_wide(int block_size, int G, Variant& v) {
  thin_kernel<Wide<kBf16>, kEight, true>(G, v);
  v.launch = block_size == 8    ? &launch_wide<kBf16, kEight, 8>
             : block_size == 16 ? &launch_wide<kBf16, kEight, 16>
                                : &launch_wide<kBf16, kEight, 32>;
}

}  // namespace thin

bool select_scores_d64(const pa_pool_desc& pool, int G, Variant& v) {
  if (pool.head_dim != 64 || (pool.block_size != 8 && pool.block_size != 16 && pool.block_size != 32)) return false;
  if (G != 1 && G != 2 && G != 4 && G != 8) return false;
  if (static_cast<long long>(pool.num_kv_heads) * pool.block_size * 128 > 0x7fffffffLL) return false;
  if (pool.dtype == PA_BF16) {
    G == 8 ? thin::pick_wide<true, true>(pool.block_size, G, v) : thin::pick_wide<true, false>(pool.block_size, G, v);
  } else {
    G == 8 ? thin::pick_wide<false, true>(pool.block_size, G, v) : thin::pick_wide<false, false>(pool.block_size, G, v);
  }
  return true;
}

}  // namespace pa
