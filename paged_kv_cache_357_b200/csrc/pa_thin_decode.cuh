// Decode attention with few query rows a kv head, on mma.sync: the kernel of
// the 4-bit cache (pa_fp4_decode.cu) and of 16-bit pools at head_dim 64 with
// accumulated weights (pa_weights_d64.cu).  A format class says how a step's
// rows lie in shared memory and become fragments:
//   kD, kBytes (a stage of 32 tokens), kCtasPerSm, kBf16P (p's type),
//   kCodeRow, kScaleRow (bytes of a row and of its scales in a pool tile),
//   kK, kV, kKs, kVs (where they go in a stage), kKXor, kVXor (the exclusive-or
//   of a 16-byte piece's place by its 128-byte line in a quarter of 8 tokens)
//   prepare  q's fragments; scores  S^T of 32 tokens; values  O^T of 16;
//   put      one column of a thread's O^T as elements of a row
//
//   S^T[token, row] = K[token, d] q^T[d, row]      16 x 8, D/16 steps
//   O^T[d, row]    += V^T[d, token] p^T[token, row]  D/16 tiles of 16 x 8
//
// Rows.  The 8 columns are the G query heads of the kv head.  p enters as a
// 16-bit value and the 16-bit value of its rounding residual: 22 significant
// bits in halves, of a p within 2^-8 of the largest, and 2^-32 of that below.
// In bf16 these are 16 bits (2^-17 of p), so a third value takes what is left:
// 24.  For G <= 4 columns 4..7 repeat the query rows, so their threads compute
// the same p and pass on the residual, and the two halves of O are added at the
// end; for G = 8 the residual is a second product.  The third value is one more.
//
// Work.  Ranges of equal cost per CTA (pa_decode_common.cuh) in granules of
// 128 tokens; the 4 warps of a CTA take 32-token steps in turn, each with
// its own two-stage ring of cp.async copies that runs ahead over segment
// borders, and its own running max and sum.  A segment's 4 states are merged
// in shared memory, and a unit split between CTAs by the last CTA to arrive
// (no CTA waits for another).  Where the walks over segments stand is kept
// in shared memory: it changes once a segment, and the registers are needed.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_host.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace thin {

constexpr int kWarps = 4;
constexpr int kDecodeThreads = kWarps * 32;
constexpr int kStepTok = 32;   // tokens of a warp's step: two halves of 16 (M of S^T, K of O^T)
constexpr int kStages = 2;     // steps in a warp's ring
constexpr int kUnit = 8;       // tokens of the partition's blocks (every block size is a multiple)
constexpr int kGranule = 16;   // of those: 128 tokens, a step for each warp
// A row's p = 2^(score - reference) with the reference kBelow under a running
// max that only moves when a score passes it by 8: p reaches 2^15, within
// half's range, and its smallest step, 2^-24, is 2^-31 of the largest p.
constexpr float kBelow = 7.f;
constexpr float kGap = kBelow + 8.f;
constexpr float kNoRef = -1e30f;  // reference of a row that has seen no score

struct ThinParams {
  DecodeParams d;          // q, out, tables, lengths, partials; max_nb in blocks of kUnit tokens
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  float* scores;           // [num_seqs][num_kv_heads][score_tokens][G] or null
  float* norm2;            // [num_seqs][num_q_heads] log2 normalisers, with scores
  long long score_tokens;
  int table_width;         // entries of a table row
  int log2_block;
  int tile;                // bytes of a pool tile
  int block_bytes;         // of a block: num_kv_heads tiles
  int G;
  int bf16;                // q and out
  float out_scale;         // the V pool's scale
};

// A walk over segments, in shared memory: where it stands, and the segment it
// found last.
struct Walk {
  Cursor c;
  Seg sg;
  int more;
};

// What a segment's arithmetic needs, prepared while the one before it runs:
// q's fragments by word of codes and lane, and per lane the factors that turn
// its two columns of S into log2-domain scores.
template <int D, int kRows>
struct Unit {
  uint4 q[D / 32][32];
  uint4 raw[kRows * D / 8];  // the unit's query rows as they are
  float2 f[32];
  Seg sg;
  int more;
};

struct Located {  // where a CTA's range starts
  Cursor c;
  int found;
};

template <class F, int kRows>
struct __align__(128) ThinSmem {
  static constexpr int D = F::kD;
  static_assert(kRows * D * 4 <= F::kBytes, "a state's output fits a stage");
  // a warp's stages; at a segment's end its free stage takes its state's
  // unnormalised output [kRows][D]
  uint8_t ring[kWarps][kStages][F::kBytes];
  uint32_t free_stage[kWarps];
  float m[kWarps][kRows];
  float l[kWarps][kRows];
  Unit<D, kRows> unit[2];     // the CTA's arithmetic: this segment and the next one
  Cursor now;          // where that walk stands
  Walk ahead[kWarps];  // each warp's copies
  RangeSmem range;
  Located from;
  int is_last;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// K and V: read once, the first to leave L2
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The cost line cut into the CTAs' ranges: of `each` or, in the first `more`
// CTAs, one longer.
struct Ranges {
  long long each;
  int more;
  int ctas;  // that own a range

  __device__ __forceinline__ Ranges(long long line, int grid) {
    const long long most = line / kGranuleCost;  // at least one granule of cost per range
    ctas = most < grid ? static_cast<int>(most) : grid;
    each = ctas > 0 ? divide(line, ctas) : 0;
    more = static_cast<int>(line - each * ctas);
  }
  __device__ __forceinline__ long long start(int c) const { return each * c + min(c, more); }
  // The CTA whose range holds position x.
  __device__ __forceinline__ int cta_of(long long x) const {
    const long long longer = (each + 1) * more;  // where the shorter ranges start
    return static_cast<int>(x < longer ? divide(x, each + 1) : more + divide(x - longer, each));
  }
  // In 32 bits where they hold both, as they do but for the largest batches.
  static __device__ __forceinline__ long long divide(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
  }
};

// Where a CTA's range starts on the line, found by all its threads: each sums
// the costs of neighbouring sequences, a scan over the threads gives what lies
// before them, and the one whose sequences hold the start walks them.  false:
// no work for this CTA.
__device__ __forceinline__ long long cost_of(const DecodeParams& p, int s) {
  const int blocks = (checked_len(p, s, kUnit) + kUnit - 1) / kUnit;
  return static_cast<long long>(p.num_kv_heads) * unit_cost_of(p, (blocks + kGranule - 1) / kGranule);
}
__device__ __forceinline__ bool locate(const ThinParams& p, RangeSmem& scan, Located& at, Ranges& ranges) {
  const int tid = threadIdx.x;
  const int each = (p.d.num_seqs + kDecodeThreads - 1) / kDecodeThreads;
  const int first = min(tid * each, p.d.num_seqs), end = min(first + each, p.d.num_seqs);
  long long mine = 0;
  for (int s = first; s < end; ++s) {
    if (blockIdx.x == 0) {
      const int raw = __ldg(p.d.seq_lens + s);
      if (raw < 0 || raw > p.d.max_nb * kUnit) record_status(p.d.status, PA_DEV_BAD_SEQ_LEN);
    }
    mine += cost_of(p.d, s);
  }
  if (tid == 0) at.found = 0;
  long long line;
  const long long upto = block_inclusive_scan<kDecodeThreads>(mine, scan, line);
  ranges = Ranges(line, static_cast<int>(gridDim.x));
  const int cta = static_cast<int>(blockIdx.x);
  if (cta >= ranges.ctas) return false;  // uniform across the CTA (also covers an empty line)
  const long long start = ranges.start(cta);
  if (mine > 0 && upto - mine <= start && start < upto) {
    long long before = upto - mine;
    int s = first;
    for (long long cost = cost_of(p.d, s); before + cost <= start; cost = cost_of(p.d, s)) {
      before += cost;
      ++s;
    }
    Cursor& c = at.c;
    c.s = s;
    load_seq<kUnit, kGranule>(c, p.d, WholeSequence());
    const long long ucost = unit_cost_of(p.d, c.ng);
    c.h = static_cast<int>(Ranges::divide(start - before, ucost));
    c.ucost = before + c.h * ucost;
    const long long rem = start - c.ucost - p.d.unit_cost;  // past the unit's fixed cost
    c.jg = rem <= 0 ? 0 : static_cast<int>((rem + kGranuleCost - 1) / kGranuleCost);
    c.end = ranges.start(cta + 1);
    c.done = false;
    if (c.jg >= c.ng) next_unit<kUnit, kGranule>(c, p.d, WholeSequence());  // the range starts after the unit's last granule
    at.found = 1;
  }
  __syncthreads();
  return at.found != 0;
}

// Steps of a segment.
__device__ __forceinline__ int steps_of(const Seg& sg) {
  const int end = min(sg.len, (sg.j0 + sg.n) * kUnit);
  return (end - sg.j0 * kUnit + kStepTok - 1) / kStepTok;
}

// A warp's producer side: its next step, and the table entries of that
// step's four 8-token quarters, loaded one step ahead of the copies that
// need them.  Eight lanes copy a quarter: of its codes 16 bytes of every
// 128-byte line, and its scales.  A step starts at a multiple of 32 tokens,
// so where a quarter's rows lie in their block is the same in every step.
template <class F>
struct Loader {
  static constexpr int kCodeRow = F::kCodeRow, kScaleRow = F::kScaleRow;
  static constexpr int kLines = 8 * kCodeRow / 128;   // of a quarter's codes
  static constexpr int kPieces = 8 * kScaleRow / 16;  // of its scales, for K and for V
  static constexpr int kStride = kWarps * kStepTok;   // tokens from a warp's step to its next

  const uint8_t *k, *v, *sc;  // this lane's codes and scales in block 0 of the segment's kv head
  const int32_t* at;          // the table entry of this lane's quarter in the next step
  int left;                   // tokens of the sequence from the next step on
  int steps;                  // of the segment from the next step on
  int block;                  // *at, not looked at before the copies
  uint32_t to, sc_to;         // this lane's places in a ring slot
  uint64_t policy;
  bool have;

  // The next segment that has a step for this warp.
  __device__ __forceinline__ void next_segment(const ThinParams& p, Walk& walk, int warp, int lane) {
    const int q = lane >> 3, sub = lane & 7;
    do {
      __syncwarp();
      if (lane == 0) walk.more = next_seg<kUnit, kGranule>(walk.c, walk.sg, p.d);
      __syncwarp();
      have = walk.more != 0;
      if (!have) return;
      steps = (steps_of(walk.sg) - warp + kWarps - 1) / kWarps;
    } while (steps <= 0);
    const Seg& sg = walk.sg;
    const int tok = sg.j0 * kUnit + warp * kStepTok;
    left = sg.len - tok;
    at = p.d.block_tables + static_cast<size_t>(sg.s) * p.table_width + ((tok + 8 * q) >> p.log2_block);
    const int row0 = (8 * q) & ((1 << p.log2_block) - 1);
    const size_t base = static_cast<size_t>(sg.h) * p.tile;
    const bool is_k = sub < kPieces;
    k = p.k_pool + (base + row0 * kCodeRow + sub * 16);
    v = p.v_pool + (base + row0 * kCodeRow + sub * 16);
    if constexpr (kPieces > 0) {
      sc = (is_k ? p.k_pool : p.v_pool) +
           (base + (kCodeRow << p.log2_block) + row0 * kScaleRow + (is_k ? sub : sub - kPieces) * 16);
    }
  }
  __device__ __forceinline__ void look_up(int lane) {
    block = (lane & 24) < left ? __ldg(at) : 0;  // a quarter past the end: nothing is copied
  }
  __device__ __forceinline__ void start(const ThinParams& p, Walk& walk, int warp, int lane) {
    const int q = lane >> 3, sub = lane & 7;
    const bool is_k = sub < kPieces;
    to = q * (8 * kCodeRow) + sub * 16;
    if constexpr (kPieces > 0) sc_to = (is_k ? F::kKs : F::kVs) + q * (8 * kScaleRow) + (is_k ? sub : sub - kPieces) * 16;
    policy = l2_policy_evict_first();
    next_segment(p, walk, warp, lane);
    if (have) look_up(lane);
  }
  // Copies of the step into a ring slot (shared address), rows past the
  // sequence's end as zeros; then on to the next step.
  __device__ __forceinline__ void issue(const ThinParams& p, Walk& walk, uint32_t slot, int warp, int lane) {
    if (have) {
      if (static_cast<uint32_t>(block) >= static_cast<uint32_t>(p.d.num_blocks)) {
        record_status(p.d.status, PA_DEV_BAD_BLOCK_ID);
        block = 0;
      }
      const size_t off = static_cast<size_t>(static_cast<uint32_t>(block)) * static_cast<uint32_t>(p.block_bytes);
      const uint32_t dst = slot + to;
      const int sub = lane & 7;
      if (left >= kStepTok) {
#pragma unroll
        for (int j = 0; j < kLines; ++j) {
          cp_async16((dst ^ (F::kKXor * j)) + F::kK + j * 128, k + off + j * 128, 16, policy);
          cp_async16((dst ^ (F::kVXor * j)) + F::kV + j * 128, v + off + j * 128, 16, policy);
        }
        if (kPieces > 0 && sub < 2 * kPieces) cp_async16(slot + sc_to, sc + off, 16, policy);
      } else {
        const int mine = left - (lane & 24);  // valid rows of the quarter
#pragma unroll
        for (int j = 0; j < kLines; ++j) {
          const int bytes = (j * 128 + sub * 16) / kCodeRow < mine ? 16 : 0;
          cp_async16((dst ^ (F::kKXor * j)) + F::kK + j * 128, k + off + j * 128, bytes, policy);
          cp_async16((dst ^ (F::kVXor * j)) + F::kV + j * 128, v + off + j * 128, bytes, policy);
        }
        if constexpr (kPieces > 0) {
          const int first = (sub % kPieces) * (16 / kScaleRow);
          const int rows = max(0, min(16 / kScaleRow, mine - first));
          if (sub < 2 * kPieces) cp_async16(slot + sc_to, sc + off, rows * kScaleRow, policy);
        }
      }
      left -= kStride;
      at += kStride >> p.log2_block;
      if (--steps == 0) next_segment(p, walk, warp, lane);
      if (have) look_up(lane);
    }
    cp_commit();
  }
};

// The CTA's next segment, and copies of its query rows.  One warp; the copies
// belong to the warp's next commit.
template <int D, int kRows>
__device__ __forceinline__ void fetch_unit(const ThinParams& p, Cursor& now, int lane, Unit<D, kRows>& unit) {
  if (lane == 0) unit.more = next_seg<kUnit, kGranule>(now, unit.sg, p.d);
  __syncwarp();
  if (!unit.more) return;
  const uint16_t* src =
      p.d.q + (static_cast<size_t>(unit.sg.s) * p.d.num_q_heads + static_cast<size_t>(unit.sg.h) * p.G) * D;
  for (int i = lane; i < p.G * D / 8; i += 32) cp_async16(smem_u32(&unit.raw[i]), src + i * 8, 16);
}

// A warp's softmax state: columns 2t and 2t + 1.
template <int D>
struct State {
  float m0, m1, l0, l1;
  float acc[D / 16][4];
  __device__ __forceinline__ void reset() {
    m0 = m1 = kNoRef;
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    }
  }
};

// One step of 32 tokens: scores, softmax, O^T.  `left`: valid tokens from its
// first one on.  In c, d and p: index 0, 1 the columns 2t, 2t + 1 of token g,
// 2, 3 those of token g + 8, of each half.
template <class F, bool kEight, bool kScores>
__device__ __forceinline__ void step(const ThinParams& p, const uint8_t* slot, int lane, int left,
                                     const Unit<F::kD, kEight ? 8 : 4>& unit, float f0, float f1, State<F::kD>& st,
                                     float* scores) {
  constexpr int D = F::kD;
  const int g = lane >> 2, t = lane & 3;
  float c[2][4] = {};
  F::scores(slot, lane, unit, c);
  if constexpr (kScores) {
    if (2 * t < p.G && (kEight || t < 2)) {
      const uint64_t keep_policy = l2_policy_evict_last();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = g + 8 * k;
        const float s0 = c[k >> 1][2 * (k & 1)] * f0, s1 = c[k >> 1][2 * (k & 1) + 1] * f1;
        float* to = scores + static_cast<size_t>(row) * p.G + 2 * t;
        if (row < left) {
          if (p.G == 1) {
            store_kept(to, s0, keep_policy);
          } else {
            store_kept(reinterpret_cast<float2*>(to), make_float2(s0, s1), keep_policy);
          }
        }
      }
    }
  }
  // ---- online softmax: the references m move when a score passes them by kGap
  float x[2][4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k][i] = fmaf(c[k][i], (i & 1) ? f1 : f0, (i & 1) ? -st.m1 : -st.m0);
  }
  if (left < kStepTok) {  // the sequence's last step: rows past its end
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (g + 8 * k >= left) x[k >> 1][2 * (k & 1)] = x[k >> 1][2 * (k & 1) + 1] = -INFINITY;
    }
  }
  const float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                          fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
  if (__any_sync(0xffffffffu, top > kGap)) {
    // the scores themselves: a first reference is too far off to add to
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[k][i] = x[k][i] == -INFINITY ? x[k][i] : c[k][i] * ((i & 1) ? f1 : f0);
    }
    float n0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
    float n1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
    }
    const float m0 = fmaxf(n0 - kBelow, st.m0), m1 = fmaxf(n1 - kBelow, st.m1);
    const float a0 = fast_exp2(st.m0 - m0), a1 = fast_exp2(st.m1 - m1);
    st.m0 = m0;
    st.m1 = m1;
    st.l0 *= a0;
    st.l1 *= a1;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      st.acc[i][0] *= a0;
      st.acc[i][1] *= a1;
      st.acc[i][2] *= a0;
      st.acc[i][3] *= a1;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (x[k][i] != -INFINITY) x[k][i] = fmaf(c[k][i], (i & 1) ? f1 : f0, (i & 1) ? -m1 : -m0);
      }
    }
  }
  // p as 16-bit values; columns 4..7 (kEight: a second product) take the
  // residuals, and one more product what bf16 leaves of those
  const float keep = t < 2 ? 0.f : 1.f;
  constexpr int kParts = (kEight ? 2 : 1) + (F::kBf16P ? 1 : 0);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t b[kParts][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p0 = fast_exp2(x[k][2 * i]), p1 = fast_exp2(x[k][2 * i + 1]);
      st.l0 += p0;
      st.l1 += p1;
      const uint32_t head = pack2<F::kBf16P>(p0, p1);
      float h0, h1;
      unpack2<F::kBf16P>(head, h0, h1);
      if constexpr (kEight || F::kBf16P) {
        const uint32_t rest = pack2<F::kBf16P>(p0 - h0, p1 - h1);
        b[0][i] = transpose8x8(kEight || t < 2 ? head : rest);
        if constexpr (kEight) b[1][i] = transpose8x8(rest);
        if constexpr (F::kBf16P) {
          float r0, r1;
          unpack2<true>(rest, r0, r1);
          const uint32_t last = pack2<true>(p0 - h0 - r0, p1 - h1 - r1);
          b[kParts - 1][i] = transpose8x8(kEight || t < 2 ? last : 0u);
        }
      } else {
        b[0][i] = transpose8x8(pack2<F::kBf16P>(fmaf(-keep, h0, p0), fmaf(-keep, h1, p1)));
      }
    }
    F::template values<kParts>(slot, 16 * k, lane, b, st.acc);
  }
}

// Writes four finished elements of a row: the output, and with the row's
// first ones its normalisers.
__device__ __forceinline__ void write_out(const ThinParams& p, int s, int h, int D, int r, int d, float M, float L,
                                          float4 a) {
  const size_t row = static_cast<size_t>(s) * p.d.num_q_heads + static_cast<size_t>(h) * p.G + r;
  const float inv = p.out_scale / L;
  uint2 w;
  if (p.bf16) {
    w = make_uint2(pack2<true>(a.x * inv, a.y * inv), pack2<true>(a.z * inv, a.w * inv));
  } else {
    w = make_uint2(pack2<false>(a.x * inv, a.y * inv), pack2<false>(a.z * inv, a.w * inv));
  }
  *reinterpret_cast<uint2*>(p.d.out + row * D + d) = w;
  if (d == 0) {
    const float n2 = M + log2f(L);
    if (p.d.lse != nullptr) p.d.lse[row] = n2 * 0.6931471805599453f;
    if (p.norm2 != nullptr) p.norm2[row] = n2;
  }
}

// out += x * a
__device__ __forceinline__ void axpy(float4& out, float x, const float4& a) {
  out.x = fmaf(x, a.x, out.x);
  out.y = fmaf(x, a.y, out.y);
  out.z = fmaf(x, a.z, out.z);
  out.w = fmaf(x, a.w, out.w);
}

// A partial state's place: m[G], l[G], acc[G][D] on a 16-byte boundary, and
// two arrival counts, which are zero between launches: of the unit whose first
// piece this is, and of the group of pieces whose first it is.  Counts that lie
// in the pieces' places stay where they are whatever the batch, so that a
// workspace serves batches of any size one after another.
constexpr int kFan = 8;  // pieces whose loads are on the way together, and pieces of a group
__host__ __device__ constexpr int state_outputs(int G) { return G < 2 ? 4 : 2 * G; }
__host__ __device__ constexpr int state_counts(int G, int D) { return state_outputs(G) + G * D; }
__host__ __device__ constexpr int state_floats(int G, int D) { return state_counts(G, D) + 4; }
__host__ __device__ constexpr int merged_quads(int rows, int D) {
  return (rows * D / 4 + kDecodeThreads - 1) / kDecodeThreads;
}

__device__ __forceinline__ float4 load_quad(const float* at) { return __ldcg(reinterpret_cast<const float4*>(at)); }

// Arrival of one of n, by one thread behind a barrier after its CTA's stores:
// true for the last, which leaves the count at zero.
__device__ __forceinline__ int arrive(int32_t* count, int n) {
  __threadfence();
  const bool is_last = atomicAdd(count, 1) == n - 1;
  if (is_last) *count = 0;
  __threadfence();
  return is_last;
}

// The merge of the states of a unit's pieces, piece(0), piece(1), ...: the
// online-softmax rule with the largest m as the common reference.  More than
// 2 kFan pieces are merged in two levels, kFan neighbours by the last of them
// to arrive and the groups by the last group.  Over the 444 CTAs of a default
// launch, two sequences of 38k tokens, G = 4 to 8: 8 units of 55 pieces 23.7 us
// in two levels and 28.6 where one CTA merges them all, 16 units of 28 pieces
// 28.4 and 28.7, 26 units of 17 pieces 38.7 and 38.0.
//
// A few pieces, by one warp: a lane's elements 4 (lane + 32 j), two j at a
// time with all their loads on the way together.
constexpr int kFew = 4;
template <int D, int kRows, typename Piece>
__device__ __forceinline__ void merge_few(const ThinParams& p, int s, int h, int pieces, Piece piece, int lane) {
  const int G = p.G;
#pragma unroll 1
  for (int j0 = 0; 4 * 32 * j0 < G * D; j0 += 2) {
    float m[2][kFew], l[2][kFew];
    float4 x[2][kFew];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int f = min(lane + 32 * (j0 + j), G * D / 4 - 1), r = 4 * f / D;
#pragma unroll
      for (int c = 0; c < kFew; ++c) {
        const float* at = piece(min(c, pieces - 1));
        m[j][c] = __ldcg(at + r);
        l[j][c] = __ldcg(at + G + r);
        x[j][c] = load_quad(at + state_outputs(G) + 4 * f);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int f = lane + 32 * (j0 + j), r = 4 * f / D;
      const float M = fmaxf(fmaxf(m[j][0], m[j][1]), fmaxf(m[j][2], m[j][3]));
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kFew; ++c) {
        if (c < pieces) {
          const float w = fast_exp2(m[j][c] - M);
          L = fmaf(l[j][c], w, L);
          axpy(acc, w, x[j][c]);
        }
      }
      if (r < G) write_out(p, s, h, D, r, 4 * f % D, M, L, acc);
    }
  }
}

// Any number, by the whole CTA: a thread's elements 4 (tid + 128 j) of the
// merged state.  kFan pieces at a time, all their loads but half of the
// outputs' on the way together; later ones rescale what came before.
struct Merged {
  float M, L;
  float4 a;
};
template <int D, int kRows, typename Piece>
__device__ __forceinline__ void merge_many(int G, int pieces, Piece piece, int tid,
                                           Merged (&merged)[merged_quads(kRows, D)]) {
#pragma unroll
  for (int j = 0; j < merged_quads(kRows, D); ++j) {
    const int f = tid + kDecodeThreads * j, r = 4 * f / D;
    Merged s{kNoRef, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int c0 = 0; r < G && c0 < pieces; c0 += kFan) {
      constexpr int kHalf = kFan / 2;
      float m[kFan], l[kHalf];
      float4 x[kHalf];
#pragma unroll
      for (int i = 0; i < kFan; ++i) m[i] = __ldcg(piece(min(c0 + i, pieces - 1)) + r);
      float top = s.M;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int first = c0 + half * kHalf;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          const float* at = piece(min(first + i, pieces - 1));
          l[i] = __ldcg(at + G + r);
          x[i] = load_quad(at + state_outputs(G) + 4 * f);
        }
        if (half == 0) {
#pragma unroll
          for (int i = 0; i < kFan; ++i) top = fmaxf(top, m[i]);
          const float was = fast_exp2(s.M - top);
          s.M = top;
          s.L *= was;
          s.a = make_float4(s.a.x * was, s.a.y * was, s.a.z * was, s.a.w * was);
        }
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          if (first + i < pieces) {
            const float w = fast_exp2(m[half * kHalf + i] - top);
            s.L = fmaf(l[i], w, s.L);
            axpy(s.a, w, x[i]);
          }
        }
      }
    }
    merged[j] = s;
  }
}

// The first of a unit's pieces ends its CTA's range, the others start theirs.
struct Pieces {
  float* first;
  int stride;
  __device__ __forceinline__ Pieces(const ThinParams& p, int cta, int stride_)
      : first(p.d.partials + static_cast<size_t>(cta) * 2 * stride_), stride(stride_) {}
  __device__ __forceinline__ float* operator()(int c) const {
    return first + (static_cast<size_t>(c) * 2 + (c == 0 ? 1 : 0)) * stride;
  }
};

// A piece of a split unit is written: count it, and merge the pieces if it
// was the last.
template <int D, int kRows>
__device__ __forceinline__ void finish_few(const ThinParams& p, int s, int h, int first, int pieces) {
  const Pieces piece(p, first, state_floats(p.G, D));
  const int lane = threadIdx.x & 31;
  int is_last = 0;
  if (lane == 0) is_last = arrive(reinterpret_cast<int32_t*>(piece(0) + state_counts(p.G, D)), pieces);
  if (__shfl_sync(0xffffffffu, is_last, 0)) merge_few<D, kRows>(p, s, h, pieces, piece, lane);
}
template <int D, int kRows>
__device__ __forceinline__ void finish_split(const ThinParams& p, int s, int h, int first, int pieces, int* is_last) {
  const int G = p.G, tid = threadIdx.x;
  const Pieces piece(p, first, state_floats(G, D));
  const int groups = pieces > 2 * kFan ? (pieces + kFan - 1) / kFan : 1;
  Merged merged[merged_quads(kRows, D)];
  if (groups > 1) {
    const int lead = (static_cast<int>(blockIdx.x) - first) / kFan * kFan;  // the group's first piece
    const int n = min(kFan, pieces - lead);
    float* to = piece(lead);
    if (tid == 0) *is_last = arrive(reinterpret_cast<int32_t*>(to + state_counts(G, D)) + 1, n);
    __syncthreads();
    const bool go = *is_last != 0;
    if (go) merge_many<D, kRows>(G, n, [&](int c) { return piece(lead + c); }, tid, merged);
    __syncthreads();  // the first piece has been read, and is_last
    if (!go) return;
#pragma unroll
    for (int j = 0; j < merged_quads(kRows, D); ++j) {
      const int f = tid + kDecodeThreads * j, r = 4 * f / D;
      if (r >= G) continue;
      if (4 * f % D == 0) {
        to[r] = merged[j].M;
        to[G + r] = merged[j].L;
      }
      *reinterpret_cast<float4*>(to + state_outputs(G) + 4 * f) = merged[j].a;
    }
    __syncthreads();
  }
  const int left = groups > 1 ? groups : pieces, apart = groups > 1 ? kFan : 1;
  if (tid == 0) *is_last = arrive(reinterpret_cast<int32_t*>(piece(0) + state_counts(G, D)), left);
  __syncthreads();
  if (*is_last) {
    merge_many<D, kRows>(G, left, [&](int c) { return piece(c * apart); }, tid, merged);
#pragma unroll
    for (int j = 0; j < merged_quads(kRows, D); ++j) {
      const int f = tid + kDecodeThreads * j, r = 4 * f / D;
      if (r < G) write_out(p, s, h, D, r, 4 * f % D, merged[j].M, merged[j].L, merged[j].a);
    }
  }
  __syncthreads();  // is_last has been read
}

// The rows of sequences without a token: outputs of 0, normalisers of 0 (log: -inf).
template <int D>
__device__ __forceinline__ void empty_rows(const ThinParams& p) {
  zero_empty_outputs<kDecodeThreads, kUnit>(p.d, D);
  if (p.d.lse == nullptr) return;
  const long long rows = static_cast<long long>(p.d.num_seqs) * p.d.num_q_heads;
  for (long long i = static_cast<long long>(blockIdx.x) * kDecodeThreads + threadIdx.x; i < rows;
       i += static_cast<long long>(gridDim.x) * kDecodeThreads) {
    if (checked_len(p.d, static_cast<int>(i / p.d.num_q_heads), kUnit) == 0) p.d.lse[i] = -INFINITY;
  }
}

template <class F, bool kEight, bool kScores>
__global__ void __launch_bounds__(kDecodeThreads, F::kCtasPerSm) decode_thin_kernel(const ThinParams p) {
  constexpr int kRows = kEight ? 8 : 4;
  constexpr int D = F::kD;
  using Smem = ThinSmem<F, kRows>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.G;
  const long long cta = blockIdx.x;

  grid_dependency_wait();
  grid_launch_dependents();
  Ranges ranges(0, 1);
  if (!locate(p, sm.range, sm.from, ranges)) {
    empty_rows<D>(p);
    return;
  }
  if (lane == 0) sm.ahead[warp].c = sm.from.c;
  if (tid == 0) sm.now = sm.from.c;

  const uint8_t* ring = sm.ring[warp][0];
  const uint32_t ring_at = smem_u32(ring);
  Loader<F> ld;
  ld.start(p, sm.ahead[warp], warp, lane);
  if (warp == 0) fetch_unit(p, sm.now, lane, sm.unit[0]);  // thread 0 has set its walk
  ld.issue(p, sm.ahead[warp], ring_at, warp, lane);
  empty_rows<D>(p);  // while the first copies are on their way
  if (warp == 0) {
    cp_wait<0>();
    __syncwarp();
    F::template prepare<kEight>(p, lane, sm.unit[0]);
  }
  __syncthreads();
  int slot = 0;
  for (int u = 0; sm.unit[u].more; u ^= 1) {
    const Unit<D, kRows>& unit = sm.unit[u];
    // the last warp has the fewest steps: it looks a segment ahead
    if (warp == kWarps - 1) fetch_unit(p, sm.now, lane, sm.unit[u ^ 1]);
    const Seg& sg = unit.sg;
    const float2 f = unit.f[lane];
    State<D> st;
    st.reset();
    const int n = steps_of(sg), tok0 = sg.j0 * kUnit, len = sg.len;
    float* scores = nullptr;
    if constexpr (kScores) {
      scores = p.scores + ((static_cast<size_t>(sg.s) * p.d.num_kv_heads + sg.h) * p.score_tokens + tok0) *
                              static_cast<size_t>(G);
    }
    for (int i = warp; i < n; i += kWarps) {
      __syncwarp();  // the other slot was read a step ago
      ld.issue(p, sm.ahead[warp], ring_at + (slot ^ 1) * F::kBytes, warp, lane);
      cp_wait<1>();
      __syncwarp();
      step<F, kEight, kScores>(p, ring + slot * F::kBytes, lane, len - (tok0 + i * kStepTok), unit,
                                          f.x, f.y, st,
                                          kScores ? scores + static_cast<size_t>(i) * kStepTok * G : nullptr);
      slot ^= 1;
    }
    if (warp == kWarps - 1) {
      cp_wait_all();
      __syncwarp();
      if (sm.unit[u ^ 1].more) F::template prepare<kEight>(p, lane, sm.unit[u ^ 1]);
    }
    // ---- the segment's states into shared memory
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
      st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
    }
    if constexpr (!kEight) {  // the residuals' half of O
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) st.acc[i][j] += __shfl_xor_sync(0xffffffffu, st.acc[i][j], 2);
      }
    }
    if (lane == 0) sm.free_stage[warp] = slot ^ 1;  // read for the last time; the other one is being filled
    __syncwarp();
    if (2 * t < kRows) {
      if (g == 0) {
        sm.m[warp][2 * t] = st.m0;
        sm.m[warp][2 * t + 1] = st.m1;
        sm.l[warp][2 * t] = st.l0;
        sm.l[warp][2 * t + 1] = st.l1;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        F::put(reinterpret_cast<float*>(sm.ring[warp][slot ^ 1]) + (2 * t + j) * D, g, j, st.acc);
      }
    }
    __syncthreads();
    const Seg last = sg;  // its place may be taken by the segment after the next one
    const bool whole = sg.j0 == sg.first && sg.j0 + sg.n == sg.nb;
    const int stride = state_floats(G, D);
    // a CTA's two places for partial states: the unit its range starts in, and the unit where it ends
    float* mine = whole ? nullptr
                        : p.d.partials + (static_cast<size_t>(cta) * 2 + (sg.j0 == sg.first ? 1 : 0)) * stride;
    float* stage[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) stage[w] = reinterpret_cast<float*>(sm.ring[w][sm.free_stage[w]]);
    for (int f = tid; f < G * D / 4; f += kDecodeThreads) {
      const int r = 4 * f / D, d = 4 * f % D;
      float M = sm.m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm.m[w][r]);
      float L = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float x = fast_exp2(sm.m[w][r] - M);
        L = fmaf(sm.l[w][r], x, L);
        axpy(a, x, reinterpret_cast<const float4*>(stage[w])[f]);
      }
      if (whole) {
        write_out(p, sg.s, sg.h, D, r, d, M, L, a);
      } else {
        if (d == 0) {
          mine[r] = M;
          mine[G + r] = L;
        }
        *reinterpret_cast<float4*>(&mine[state_outputs(G) + r * D + d]) = a;
      }
    }
    __syncthreads();  // the merge buffers and the segment have been read, a partial state is written
    if (!whole) {
      // Count this piece; the last CTA to arrive merges the unit's pieces.  A
      // few of them the first warp merges alone, while the others go on.
      const int first = ranges.cta_of(last.unit_first);
      const int pieces = ranges.cta_of(last.unit_last) - first + 1;
      if (pieces > kFew || sm.unit[u ^ 1].more == 0) {
        finish_split<D, kRows>(p, last.s, last.h, first, pieces, &sm.is_last);
      } else if (warp == 0) {
        finish_few<D, kRows>(p, last.s, last.h, first, pieces);
      }
    }
  }
  cp_wait<0>();
}

// The instance's launch values, and its kernel.
using ThinKernel = void (*)(const ThinParams);
template <class F, bool kEight, bool kScores>
ThinKernel thin_kernel(int G, Variant& v) {
  ThinKernel kernel = &decode_thin_kernel<F, kEight, kScores>;
  v.kernel = reinterpret_cast<const void*>(kernel);
  v.threads = kDecodeThreads;
  v.smem_bytes = static_cast<int>(sizeof(ThinSmem<F, kEight ? 8 : 4>));
  v.part_stride = state_floats(G, F::kD);
  // The same count whatever registers an instance takes: the states' places, and
  // the scores behind them, lie alike for either type and with weights or without
  v.ctas_per_sm = F::kCtasPerSm;
  v.launch = nullptr;  // launched with its own parameters
  // what finishing a unit adds, in 1/8 granules (B200, ragged 4-bit batch: 94.3
  // us at 6, 91.4 at 10, 89.5 at 14, 91.0 at 20)
  v.unit_cost = 14;
  return kernel;
}

}  // namespace thin
}  // namespace pa
