// pa_cache_write_fp4, pa_cache_read_fp4 and pa_copy_blocks_fp4 — the 4-bit
// cache's storage (format and rounding: pa_fp4.cuh): new tokens' K/V stored
// in their slots, the stored values read back, and whole blocks copied for
// copy on write (study notes ch.05 §5 item 2, §6.1; the 4-bit form has no
// counterpart on the pages).
//
// Data movement with a little arithmetic.  A thread takes 8 elements of K and
// the same 8 of V, so that every load and store of 16-bit values is 16 bytes
// and neighbouring threads touch neighbouring bytes; the two threads of a
// group exchange their maxima.  Each thread has kUnroll such pieces on the way.
//
// Measured (B200, D = 128, 8 kv heads, bf16; in a captured graph): a store of
// 16384 tokens 19.8 us, 4.4 TB/s (0.66 of the copy rate), whether their slots
// are scattered or whole blocks in order; their read-back 17.3 us, 5.0 TB/s
// (0.76); the two in turn 35.7, and 35.9 through the Python entry points.  What
// bounds them is instructions: 0.73 and 0.79 issued a cycle, DRAM a third busy.
// 44 us with 8 bytes a thread and load, 37 with divisions instead of a
// reciprocal rounded to where midpoints are exact.  A decode step's 256 tokens:
// 2.4 us on the GPU, 5.9 through the entry point.  Block copies: 4096 pairs 24.8
// us, 6.1 TB/s (0.93), 96 pairs 2.2.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace fp4 {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

// n / d for n below 2^31 as a multiplication: with 2^(s-1) < d <= 2^s and
// m = ceil(2^(31+s) / d), n / d = (n * m) >> (31 + s).
struct Divisor {
  uint32_t d, m, s;
  explicit Divisor(uint32_t d_) : d(d_), m(0), s(0) {
    while ((uint64_t(1) << s) < d) ++s;
    m = static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t divide(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
  }
};

struct StoreParams {
  const int64_t* slots;
  int32_t* status;
  uint8_t* k_pool;
  uint8_t* v_pool;
  long long pieces;        // tokens * kv heads * D / 8
  long long num_slots;
  Divisor per_token;       // pieces of a token
  int heads;
  int log2_block;
  int tile;                // bytes of a tile
  float k_scale, v_scale;  // the pools' scales (write: their inverses)
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The codes of a thread's 8 values (four 16-bit pairs), and its group's scale
// byte.  All lanes of the warp call.
//
// Quotients are taken with an approximate reciprocal and rounded to a
// multiple of 2^-15 (adding 384 does it, whose last place that is).  The
// midpoints between codes are multiples of it, a quotient that is one comes
// out within 2^-19 and so exactly, and one that is not is 2^-13 away or more.
template <bool kBf16>
__device__ __forceinline__ uint32_t encode_piece(const uint4& w, float inv_g, uint32_t& scale) {
  float x[8];
  unpack2<kBf16>(w.x, x[0], x[1]);
  unpack2<kBf16>(w.y, x[2], x[3]);
  unpack2<kBf16>(w.z, x[4], x[5]);
  unpack2<kBf16>(w.w, x[6], x[7]);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1)) * inv_g;
  // top / 6, corrected by its own remainder: exact wherever the quotient is
  constexpr float kSixth = 1.f / 6.f;
  const float t0 = top * kSixth;
  const float t = top <= 3.0e38f ? fmaf(fmaf(-t0, 6.f, top), kSixth, t0) : top;
  scale = t == t ? e4m3_of(t) : 0x7fu;
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(halves_of_e4m3(scale) & 0xffffu)));
  if (!(s > 0.f)) return 0u;  // nothing above half the smallest scale, or a NaN
  const float inv = __fdividef(inv_g, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = fmaf(fabsf(x[i]), inv, 384.f) - 384.f;
    x[i] = copysignf(r, x[i]);
  }
  return e2m1_of(x);
}

// The 8 values of a piece as 16-bit floats.
template <bool kBf16>
__device__ __forceinline__ uint4 decode_piece(uint32_t codes, uint32_t scale, float g) {
  const uint32_t s2 = halves_of_e4m3(scale | (scale << 8));
  uint32_t h[4], out[4];
  halves_of_e2m1(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    unpack2<false>(hmul2(h[i], s2), x, y);
    out[i] = pack2<kBf16>(x * g, y * g);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Where piece i of the token list lies.
struct Place {
  size_t codes, scale;
  bool pad, bad;  // a padding token; a slot beyond the pool
};
template <int D>
__device__ __forceinline__ Place locate(const StoreParams& p, long long i) {
  constexpr int kRow = D / 8;  // pieces of a row
  const unsigned long long t = p.pieces <= 0x7fffffffLL ? p.per_token.divide(static_cast<uint32_t>(i))
                                                        : static_cast<unsigned long long>(i) / p.per_token.d;
  const int rest = static_cast<int>(i - static_cast<long long>(t) * p.per_token.d);
  const int h = rest / kRow, c = rest % kRow;
  const long long slot = __ldg(p.slots + t);
  Place at;
  at.pad = slot < 0;
  at.bad = slot >= p.num_slots;
  if (at.bad && rest == 0) record_status(p.status, PA_DEV_BAD_SLOT);
  const int row = static_cast<int>(slot & ((1 << p.log2_block) - 1));
  const size_t base = (static_cast<size_t>(slot >> p.log2_block) * p.heads + h) * p.tile;
  at.codes = base + row * code_row_bytes(D) + c * 4;
  at.scale = base + (code_row_bytes(D) << p.log2_block) + row * scale_row_bytes(D) + (c >> 1);
  return at;
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads)
    cache_write_fp4_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, const StoreParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  // a whole warp's pieces lie in the list or none (its length is a multiple
  // of 8, and the group exchange takes all lanes): lanes past it repeat the last
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 kw[kUnroll], vw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = min(first + u * kThreads, p.pieces - 1);
    kw[u] = __ldcs(k + i);  // read once
    vw[u] = __ldcs(v + i);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = first + u * kThreads;
    uint32_t ks, vs;
    const uint32_t kc = encode_piece<kBf16>(kw[u], p.k_scale, ks);
    const uint32_t vc = encode_piece<kBf16>(vw[u], p.v_scale, vs);
    if (i >= p.pieces) continue;
    const Place at = locate<D>(p, i);
    if (at.pad || at.bad) continue;
    *reinterpret_cast<uint32_t*>(p.k_pool + at.codes) = kc;
    *reinterpret_cast<uint32_t*>(p.v_pool + at.codes) = vc;
    if ((i & 1) == 0) {
      p.k_pool[at.scale] = static_cast<uint8_t>(ks);
      p.v_pool[at.scale] = static_cast<uint8_t>(vs);
    }
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads)
    cache_read_fp4_kernel(uint4* __restrict__ k, uint4* __restrict__ v, const StoreParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint32_t kc[kUnroll], vc[kUnroll], ks[kUnroll], vs[kUnroll];
  bool write[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = first + u * kThreads;
    kc[u] = vc[u] = ks[u] = vs[u] = 0u;
    write[u] = false;
    if (i < p.pieces) {
      const Place at = locate<D>(p, i);
      write[u] = !at.bad;
      if (!at.pad && !at.bad) {
        kc[u] = *reinterpret_cast<const uint32_t*>(p.k_pool + at.codes);
        vc[u] = *reinterpret_cast<const uint32_t*>(p.v_pool + at.codes);
        ks[u] = p.k_pool[at.scale];
        vs[u] = p.v_pool[at.scale];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = first + u * kThreads;
    if (write[u]) {
      k[i] = decode_piece<kBf16>(kc[u], ks[u], p.k_scale);
      v[i] = decode_piece<kBf16>(vc[u], vs[u], p.v_scale);
    }
  }
}

static int grid_for(long long items) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long want = (items + kThreads - 1) / kThreads;
  const long long cap = static_cast<long long>(sms) * 8;
  return static_cast<int>(want < cap ? want : cap);
}

// CTAs for the pieces of a write or a read; 0: more than a grid holds.
static unsigned store_grid(const StoreParams& p) {
  const long long n = (p.pieces + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  return n <= 0x7fffffffLL ? static_cast<unsigned>(n) : 0u;
}

static pa_status check_store(const void* k, const void* v, const int64_t* slots, int32_t num_tokens, float k_scale,
                             float v_scale, const void* k_pool, const void* v_pool, const pa_pool_desc* pool) {
  if (!pool_ok(pool) || num_tokens < 0 || !scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (k == nullptr || v == nullptr || slots == nullptr || k_pool == nullptr || v_pool == nullptr)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pool) || !aligned16(v_pool) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

static StoreParams store_params(const int64_t* slots, int32_t num_tokens, const void* k_pool, const void* v_pool,
                                int32_t* status, const pa_pool_desc* pool) {
  const uint32_t per_token = static_cast<uint32_t>(pool->num_kv_heads) * (pool->head_dim / 8);
  StoreParams p{slots, nullptr, nullptr, nullptr, 0, 0, Divisor(per_token), 0, 0, 0, 1.f, 1.f};
  p.status = status;
  p.k_pool = static_cast<uint8_t*>(const_cast<void*>(k_pool));
  p.v_pool = static_cast<uint8_t*>(const_cast<void*>(v_pool));
  p.pieces = static_cast<long long>(num_tokens) * per_token;
  p.num_slots = static_cast<long long>(pool->num_blocks) * pool->block_size;
  p.heads = pool->num_kv_heads;
  p.log2_block = log2_of(pool->block_size);
  p.tile = tile_bytes(pool->block_size, pool->head_dim);
  return p;
}

// Bit copies of whole blocks, in 16-byte chunks; work item
// ((pair * 2 + pool) * chunks_per_block + chunk).
__global__ void __launch_bounds__(kThreads)
    copy_blocks_fp4_kernel(const int64_t* __restrict__ pairs, long long total, long long chunks_per_block,
                           long long num_blocks, uint4* k_pool, uint4* v_pool, int32_t* status) {
  grid_dependency_wait();
  grid_launch_dependents();
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += stride) {
    const long long chunk = i % chunks_per_block, pw = i / chunks_per_block, pair = pw >> 1;
    const long long src = __ldg(pairs + 2 * pair), dst = __ldg(pairs + 2 * pair + 1);
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
      if (chunk == 0 && (pw & 1) == 0) record_status(status, PA_DEV_BAD_PAIR);
      continue;
    }
    if (src == dst) continue;
    uint4* pool = (pw & 1) ? v_pool : k_pool;
    pool[dst * chunks_per_block + chunk] = pool[src * chunks_per_block + chunk];
  }
}

}  // namespace fp4
}  // namespace pa

using namespace pa;
using namespace pa::fp4;

extern "C" pa_status pa_cache_write_fp4(const void* k, const void* v, const int64_t* slot_mapping,
                                        int32_t num_tokens, float k_scale, float v_scale, void* k_pool, void* v_pool,
                                        int32_t* dev_status, const pa_pool_desc* pool, void* stream) {
  const pa_status st = check_store(k, v, slot_mapping, num_tokens, k_scale, v_scale, k_pool, v_pool, pool);
  if (st != PA_OK || num_tokens == 0) return st;
  StoreParams p = store_params(slot_mapping, num_tokens, k_pool, v_pool, dev_status, pool);
  p.k_scale = 1.f / k_scale;
  p.v_scale = 1.f / v_scale;
  const bool bf16 = pool->dtype == PA_BF16;
  auto* kernel = pool->head_dim == 128 ? (bf16 ? &cache_write_fp4_kernel<true, 128> : &cache_write_fp4_kernel<false, 128>)
                                       : (bf16 ? &cache_write_fp4_kernel<true, 64> : &cache_write_fp4_kernel<false, 64>);
  if (store_grid(p) == 0) return PA_ERR_INVALID_ARG;
  const cudaError_t e = launch_overlapped(kernel, dim3(store_grid(p)), dim3(fp4::kThreads), 0,
                                          static_cast<cudaStream_t>(stream), static_cast<const uint4*>(k),
                                          static_cast<const uint4*>(v), p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_cache_read_fp4(const int64_t* slot_mapping, int32_t num_tokens, const void* k_pool,
                                       const void* v_pool, float k_scale, float v_scale, void* k, void* v,
                                       int32_t* dev_status, const pa_pool_desc* pool, void* stream) {
  const pa_status st = check_store(k, v, slot_mapping, num_tokens, k_scale, v_scale, k_pool, v_pool, pool);
  if (st != PA_OK || num_tokens == 0) return st;
  StoreParams p = store_params(slot_mapping, num_tokens, k_pool, v_pool, dev_status, pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const bool bf16 = pool->dtype == PA_BF16;
  auto* kernel = pool->head_dim == 128 ? (bf16 ? &cache_read_fp4_kernel<true, 128> : &cache_read_fp4_kernel<false, 128>)
                                       : (bf16 ? &cache_read_fp4_kernel<true, 64> : &cache_read_fp4_kernel<false, 64>);
  if (store_grid(p) == 0) return PA_ERR_INVALID_ARG;
  const cudaError_t e = launch_overlapped(kernel, dim3(store_grid(p)), dim3(fp4::kThreads), 0,
                                          static_cast<cudaStream_t>(stream), static_cast<uint4*>(k),
                                          static_cast<uint4*>(v), p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_copy_blocks_fp4(const int64_t* src_dst_pairs, int32_t num_pairs, void* k_pool, void* v_pool,
                                        int32_t* dev_status, const pa_pool_desc* pool, void* stream) {
  if (!pool_ok(pool) || num_pairs < 0) return PA_ERR_INVALID_ARG;
  if (num_pairs == 0) return PA_OK;
  if (src_dst_pairs == nullptr || k_pool == nullptr || v_pool == nullptr) return PA_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool) || (reinterpret_cast<uintptr_t>(src_dst_pairs) & 7u) != 0)
    return PA_ERR_INVALID_ARG;
  const long long cpb = static_cast<long long>(pool->num_kv_heads) * tile_bytes(pool->block_size, pool->head_dim) / 16;
  const long long total = static_cast<long long>(num_pairs) * 2 * cpb;
  const cudaError_t e = launch_overlapped(copy_blocks_fp4_kernel, dim3(grid_for(total)), dim3(fp4::kThreads), 0,
                                          static_cast<cudaStream_t>(stream), src_dst_pairs, total, cpb,
                                          static_cast<long long>(pool->num_blocks), static_cast<uint4*>(k_pool),
                                          static_cast<uint4*>(v_pool), dev_status);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
