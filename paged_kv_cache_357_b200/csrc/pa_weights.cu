// Accumulated attention weights: what pa_decode_weights and pa_decode_fp4 add
// to each cached token's entry,
//   w[h][t] += sum over the query heads g of kv head h of softmax_t(scale q_g K^T),
// set instead of added for a sequence's newest tokens.  The pages' method
// keeps every token; keeping those that attention uses is what the entries
// are for (pa_evict).
//
// A weight needs its row's normaliser, which is known once the row's last
// token is done.  The decode therefore writes its scores (4 G bytes a token
// and kv head, against 4 D or 9/8 D that it reads) and its rows' log2
// normalisers, and this kernel, the same call's second launch, adds
// 2^(score - normaliser).  Reading K again instead would cost 2 D bytes.
//
// HBM-bound: 4 G bytes of scores (stored to stay in L2, and dropped from it
// once read) and 8 of weights a (token, kv head), one thread each, in the
// order of memory.
//
// Measured (B200, in a captured graph): decode and weights of 256 sequences
// (log-normal lengths, median 1024, 8 kv heads, G = 4, D = 128, 16-bit pools) 237
// us, 5.9 TB/s of what the two must move (0.90 of the copy rate), 245 through the
// entry point; 8 more with scores that go to memory and come back.  128 sequences
// of 2304 tokens, G = 8, 4-bit pools: 113 us (120), of which this launch is about
// 12.  The look at the table's entries (see accumulate_kernel) is 2 us of each.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_host.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kWeightThreads = 256;

struct WeightParams {
  const float* scores;
  const float* norm2;
  float* weights;
  const int32_t* rows;
  const int32_t* seq_lens;
  const int32_t* tables;
  const int32_t* failed;  // of the decode, or null
  int32_t* status;
  long long score_tokens, row_tokens;
  int num_rows, num_new, num_heads, num_q_heads, max_tokens;
  int table_width, block_size, num_blocks;
};

template <int G>
__global__ void __launch_bounds__(kWeightThreads) accumulate_kernel(const WeightParams p) {
  const int s = blockIdx.x / p.num_heads, h = blockIdx.x - s * p.num_heads;
  // The lengths, rows and tables are inputs that the decode before this kernel
  // does not write, and it lets this one start only once what came before it
  // is complete: they are read while it runs.
  const int n = __ldg(p.seq_lens + s);
  const int row = p.rows != nullptr ? __ldg(p.rows + s) : s;
  const bool fine = n > 0 && n <= p.max_tokens;
  const int entries = fine ? (n - 1) / p.block_size + 1 : 0;
  bool bad = false;
  for (int i = threadIdx.x; i < entries; i += kWeightThreads) {
    const int b = __ldg(p.tables + static_cast<size_t>(s) * p.table_width + i);
    bad |= static_cast<uint32_t>(b) >= static_cast<uint32_t>(p.num_blocks);
  }
  bad = __syncthreads_or(bad) != 0;
  grid_dependency_wait();
  grid_launch_dependents();
  if (!fine || bad) return;  // recorded by the decode
  // The entries outlast this call: scores that a decode left unfinished are not
  // added to them.
  const bool failed = p.failed != nullptr && __ldcg(p.failed) != 0;
  if (failed || row < 0 || row >= p.num_rows) {
    if (threadIdx.x == 0) record_status(p.status, failed ? PA_DEV_TIMEOUT : PA_DEV_BAD_ROW);
    return;
  }
  float norm[G];
#pragma unroll
  for (int g = 0; g < G; ++g) norm[g] = p.norm2[static_cast<size_t>(s) * p.num_q_heads + h * G + g];
  const float* src = p.scores + (static_cast<size_t>(s) * p.num_heads + h) * p.score_tokens * G;
  float* dst = p.weights + (static_cast<size_t>(row) * p.num_heads + h) * p.row_tokens;
  const int stride = gridDim.y * kWeightThreads;
  const int lane = threadIdx.x & 31;
  for (long long t0 = blockIdx.y * kWeightThreads + (threadIdx.x & ~31); t0 < n; t0 += stride) {
    const long long t = t0 + lane;
    const bool in = t < n;
    float x[G];
    float w = 0.f;
    if (in) {
      if constexpr (G % 4 == 0) {
#pragma unroll
        for (int g = 0; g < G; g += 4) {
          *reinterpret_cast<float4*>(x + g) = *reinterpret_cast<const float4*>(src + t * G + g);
        }
      } else {
#pragma unroll
        for (int g = 0; g < G; ++g) x[g] = src[t * G + g];
      }
      if (t < static_cast<long long>(n) - p.num_new) w = dst[t];
    } else {
#pragma unroll
      for (int g = 0; g < G; ++g) x[g] = 0.f;
    }
    float add = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) add += fast_exp2(x[g] - norm[g]);
    if (in) dst[t] = w + add;
    // the warp's scores, G whole lines, have been read for the last time: they
    // need not be written to memory
    __syncwarp();
    if (lane < G) discard_line(src + t0 * G + lane * 32);
  }
}

// Tokens of a unit's scores: whole lines of 128 bytes, whatever the group.
long long score_tokens_of(int max_blocks_per_seq, int block_size) {
  return (static_cast<long long>(max_blocks_per_seq) * block_size + 31) / 32 * 32;
}

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t scores_bytes(int num_seqs, int num_q_heads, int max_blocks_per_seq, int block_size) {
  const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
  const size_t most = (size_t{1} << 60) / static_cast<size_t>(score_tokens_of(max_blocks_per_seq, block_size) + 1);
  if (rows > most) return size_t{1} << 62;  // more than any workspace
  return 256 + align256(rows * sizeof(float)) +  // 256: the workspace itself is 16-byte aligned
         align256(rows * static_cast<size_t>(score_tokens_of(max_blocks_per_seq, block_size)) * sizeof(float));
}

void split_scores(char* base, int num_seqs, int num_q_heads, float** norm2, float** scores) {
  base = reinterpret_cast<char*>(align256(reinterpret_cast<uintptr_t>(base)));  // lines are dropped whole
  *norm2 = reinterpret_cast<float*>(base);
  *scores = reinterpret_cast<float*>(base + align256(static_cast<size_t>(num_seqs) * num_q_heads * sizeof(float)));
}

bool token_weights_ok(const pa_token_weights* w, int max_blocks_per_seq, int num_seqs, const pa_pool_desc* pool) {
  if (w == nullptr || w->weights == nullptr || (reinterpret_cast<uintptr_t>(w->weights) & 3u) != 0) return false;
  if ((reinterpret_cast<uintptr_t>(w->rows) & 3u) != 0 || w->num_rows <= 0 || w->num_new < 0) return false;
  if (w->rows == nullptr && w->num_rows < num_seqs) return false;
  return w->row_tokens >= static_cast<int64_t>(max_blocks_per_seq) * pool->block_size;
}

pa_status accumulate_weights(const float* scores, const float* norm2, const pa_token_weights& w,
                             const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_q_heads,
                             int max_blocks_per_seq, const int32_t* failed, int32_t* dev_status,
                             const pa_pool_desc* pool, cudaStream_t stream) {
  WeightParams p;
  p.scores = scores;
  p.norm2 = norm2;
  p.weights = w.weights;
  p.rows = w.rows;
  p.seq_lens = seq_lens;
  p.tables = block_tables;
  p.failed = failed;
  p.status = dev_status;
  p.table_width = max_blocks_per_seq;
  p.block_size = pool->block_size;
  p.num_blocks = pool->num_blocks;
  p.max_tokens = max_blocks_per_seq * pool->block_size;
  p.score_tokens = score_tokens_of(max_blocks_per_seq, pool->block_size);
  p.row_tokens = w.row_tokens;
  p.num_rows = w.num_rows;
  p.num_new = w.num_new;
  p.num_heads = pool->num_kv_heads;
  p.num_q_heads = num_q_heads;
  const long long units = static_cast<long long>(num_seqs) * pool->num_kv_heads;
  if (units > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  // enough blocks for the card (16 a SM) where there are few units, and no
  // more than the longest sequence can use
  const long long want = (148LL * 16 + units - 1) / units;
  const long long most = (static_cast<long long>(p.max_tokens) + kWeightThreads - 1) / kWeightThreads;
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(want < most ? want : most));
  cudaError_t e;
  switch (num_q_heads / pool->num_kv_heads) {
    case 1: e = launch_overlapped(accumulate_kernel<1>, grid, dim3(kWeightThreads), 0, stream, p); break;
    case 2: e = launch_overlapped(accumulate_kernel<2>, grid, dim3(kWeightThreads), 0, stream, p); break;
    case 4: e = launch_overlapped(accumulate_kernel<4>, grid, dim3(kWeightThreads), 0, stream, p); break;
    case 8: e = launch_overlapped(accumulate_kernel<8>, grid, dim3(kWeightThreads), 0, stream, p); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
