// pa_evict — keep the tokens that attention uses most, and move them together
// (the pages' method keeps every token of a sequence; this drops some, for
// callers whose pool or context is too small for all of them).
//
// For each sequence s with a budget and each kv head h on its own, of the n
// cached tokens m = min(n, budget) stay: the last `recent`, the first
// `sinks`, and of those between the ones with the largest accumulated
// weights (pa_weights.cu), ties to the lower position.  Kept tokens keep
// their order: kept[j], ascending, becomes token j.  Attention does not
// depend on the order of a sequence's rows (positions are in the keys
// already), and in order the newest tokens stay the last ones, so `recent`
// means the same at the next eviction.
//
// Two launches.
//   select  a CTA, or up to eight (a cluster), for each (sequence, kv head).  The
//           weights are mapped to unsigned keys of the same order and, up to
//           16 a thread, kept in registers.  The key of the last token kept
//           is found 11 bits at a time from histograms in shared memory, the
//           CTAs' histograms added up over the cluster; then every token
//           knows whether it stays, and counts by warp and CTA tell where it
//           goes.
//   move    a CTA for each chunk of kept rows of K and V (and of a 4-bit
//           pool's scale rows) and their weights: 32 KB, all on the way at
//           once, six CTAs on an SM.  In place a row moves down or stays
//           (kept[j] >= j), so a chunk's places are sources of its own rows
//           and of earlier chunks' only: a CTA loads its rows, says so, and
//           stores them once the earlier chunks that read its places have
//           said so too.  They say it in `kept`: select writes the
//           complement of each position, and a CTA whose loads are done
//           writes the positions.  A CTA waits for none with a higher index,
//           and loads before it waits; the wait is bounded all the same.
//
// Bounded by memory: 4 bytes a token for the weights, then every moved row
// read and written once.
//
// Measured (B200, 8 kv heads, D = 128, 16-bit pools): 64 sequences of 1040
// tokens cut to 1024 in place 96 us, 5.6 TB/s (0.86 of the copy rate); 16 of
// about 5000 cut to 1024 into fresh blocks 37 us, 3.5 TB/s; two of 65536 cut to
// 16384 in place 84 us, 3.3 TB/s (4-bit pools: 40, 30 and 51 us).  The last two
// pay for the selection first (about 11 and 22 us of dependent passes over a
// cluster's histograms; 1 and 4 more when all three were always made), then for
// rows of 256 bytes that lie apart.  Clusters that moved 64 KB batches behind barriers took 128, 50 and
// 130 us; a persistent, pipelined form of them 148 where they took 106.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_decode_host.h"
#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace evict {

namespace cg = cooperative_groups;

constexpr int kKeys = 16;       // keys a thread holds: a CTA of NT threads holds 16 NT tokens
constexpr int kBinsAll = 2048;  // of a pass: 11 bits of the key (11, 11 and the last 10)
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kRounds = 8;      // 512-byte copies a warp has in flight
constexpr int kChunkBytes = kMoveWarps * kRounds * 512;
constexpr int kMaxCluster = 8;  // the largest portable one

struct EvictParams {
  const int32_t* tables;
  const int32_t* dst_tables;
  const int32_t* seq_lens;
  const int32_t* budgets;
  const int32_t* rows;       // weight rows or null
  const float* weights;
  float* new_weights;
  int32_t* kept;
  int32_t* new_lens;
  int32_t* status;
  uint8_t* k_pool;
  uint8_t* v_pool;
  long long row_tokens;
  long long max_kept;
  int num_rows, num_seqs, num_heads, num_blocks, table_width, max_tokens;
  int sinks, recent;
  int log2_block;
  int tile;                  // bytes of a (block, kv head)
  int withhold;              // PA_EVICT_TEST_WITHHOLD
  unsigned long long wait_limit_ns;
};

// What happens to sequence s: its tokens, how many stay, its row of weights;
// move false: it is left as it is.
struct Plan {
  int n, m, row;
  bool move;
};

__device__ __forceinline__ Plan plan_of(const EvictParams& p, int s, bool report) {
  Plan q;
  q.n = __ldg(p.seq_lens + s);
  q.m = q.n;
  q.row = p.rows != nullptr ? __ldg(p.rows + s) : s;
  q.move = false;
  const int budget = __ldg(p.budgets + s);
  int32_t bad = PA_DEV_OK;
  if (q.n < 0 || q.n > p.max_tokens) {
    bad = PA_DEV_BAD_SEQ_LEN;
    q.n = q.m = 0;
  } else if (budget >= 0) {
    const int m = min(q.n, budget);
    if (m > p.max_kept) {
      bad = PA_DEV_BAD_BUDGET;
    } else if (q.row < 0 || q.row >= p.num_rows) {
      bad = PA_DEV_BAD_ROW;
    } else {
      q.m = m;
      q.move = true;
    }
  }
  if (report && bad != PA_DEV_OK) record_status(p.status, bad);
  return q;
}

// Unsigned keys in the order of the floats, both zeros alike, NaN below all.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return w != w ? 0u : k;
}

// Two counts that are summed together.
struct Pair {
  uint32_t x, y;
};

template <int NT>
struct SelectSmem {
  static constexpr int kWarps = NT / 32;
  static constexpr int kSlots = kKeys * kWarps;  // a tile's (key slot, warp) pairs
  uint4 hist[2][kBinsAll / 4];  // by the parity of the pass
  Pair slot[kSlots];      // keys above the last kept one and equal to it, by slot; then the sums before
  Pair part;              // of a tile
  Pair warp_sum[kWarps];
  uint32_t digit;
  Pair before;            // keys above the digit: of all CTAs, of those before this one
  uint32_t equal_before;  // keys with the digit in the CTAs before this one
  int all;                // every key with the digit stays
};

// Sums of `v` over the threads before this one (all threads call).
template <int NT>
__device__ __forceinline__ Pair sums_before(Pair v, SelectSmem<NT>& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Pair u = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, u.x, o), y = __shfl_up_sync(0xffffffffu, u.y, o);
    if (lane >= o) {
      u.x += x;
      u.y += y;
    }
  }
  if (lane == 31) sm.warp_sum[warp] = u;
  __syncthreads();
  u.x -= v.x;
  u.y -= v.y;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const Pair w = sm.warp_sum[i];
    if (i < warp) {
      u.x += w.x;
      u.y += w.y;
    }
  }
  return u;
}

// The keys of a tile, token t0 + i * NT + thread in slot i.
template <int NT>
__device__ __forceinline__ void load_keys(const float* w, int t0, int end, uint32_t (&keys)[kKeys]) {
  float x[kKeys];  // all loads on their way before the first is looked at
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int t = t0 + i * NT + static_cast<int>(threadIdx.x);
    x[i] = __ldg(w + min(t, end - 1));
  }
#pragma unroll
  for (int i = 0; i < kKeys; ++i) keys[i] = key_of(x[i]);
}

template <int NT>
__global__ void __launch_bounds__(NT) select_kernel(const EvictParams p) {
  constexpr int kTile = kKeys * NT;
  __shared__ SelectSmem<NT> sm;
  grid_dependency_wait();
  grid_launch_dependents();
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank_in = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / ctas;
  const int s = unit / p.num_heads, h = unit - s * p.num_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool first = h == 0 && rank_in == 0 && tid == 0;
  const Plan q = plan_of(p, s, first);  // the same in the whole cluster
  if (first) p.new_lens[s] = q.m;
  if (!q.move) return;
  int32_t* kept = p.kept + (static_cast<size_t>(s) * p.num_heads + h) * p.max_kept;
  const int step = ctas * NT, mine = rank_in * NT + tid;
  if (q.m == q.n) {
    for (int j = mine; j < q.m; j += step) kept[j] = ~j;
    return;
  }
  const int recent = min(p.recent, q.m), sinks = min(p.sinks, q.m - recent);
  const int lo = sinks, hi = q.n - recent;        // the tokens that compete
  const uint32_t want = static_cast<uint32_t>(q.m - recent - sinks);  // places for them, fewer than hi - lo
  for (int j = mine; j < sinks; j += step) kept[j] = ~j;
  for (int j = mine; j < recent; j += step) kept[q.m - recent + j] = ~(hi + j);
  if (want == 0) return;

  // this CTA's tokens, and their keys while one tile holds them
  const float* w = p.weights + (static_cast<size_t>(q.row) * p.num_heads + h) * p.row_tokens;
  const int part = (hi - lo + ctas - 1) / ctas;
  const int begin = min(lo + rank_in * part, hi), end = min(begin + part, hi);
  uint32_t keys[kKeys];
  const bool held = end - begin <= kTile;
  if (held && begin < end) load_keys<NT>(w, begin, end, keys);

  // the want-th largest key, from its highest bits down: `prefix` holds the
  // bits found, `rank` its rank among the keys that share them; `above` counts
  // the larger keys of the CTAs before this one, `equal` in the end their
  // equal ones
  uint32_t prefix = 0, known = 0, rank = want, above = 0, equal = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    // read by the whole cluster; zeroed again two passes, and so one cluster
    // barrier after every reader, later
    uint32_t* hist = reinterpret_cast<uint32_t*>(sm.hist[pass & 1]);
    for (int i = tid; i < kBinsAll / 4; i += NT) sm.hist[pass & 1][i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int t0 = begin; t0 < end; t0 += kTile) {
      if (!held) load_keys<NT>(w, t0, end, keys);
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        if (t0 + i * NT >= end) break;  // slots that hold nothing
        if (t0 + i * NT + tid < end && (keys[i] & known) == prefix) atomicAdd(&hist[(keys[i] >> shift) & mask], 1u);
      }
    }
    if (ctas > 1) {
      cluster.sync();
    } else {
      __syncthreads();
    }
    // the bins from the top one down, kBins neighbours a thread, by fours
    constexpr int kBins = kBinsAll / NT;
    static_assert(kBins % 4 == 0, "whole vectors");
    const int top4 = (kBinsAll - kBins * (tid + 1)) / 4;  // this thread's lowest vector
    Pair count[kBins];  // descending bins: of all CTAs, of those before this one
#pragma unroll
    for (int b = 0; b < kBins / 4; ++b) {
      uint4 u = make_uint4(0, 0, 0, 0), v = u;
      if (ctas > 1) {
        uint4 of[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          of[c] = c < ctas ? cluster.map_shared_rank(sm.hist[pass & 1], c)[top4 + b] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          u.x += of[c].x;
          u.y += of[c].y;
          u.z += of[c].z;
          u.w += of[c].w;
          if (c < rank_in) {
            v.x += of[c].x;
            v.y += of[c].y;
            v.z += of[c].z;
            v.w += of[c].w;
          }
        }
      } else {
        u = sm.hist[pass & 1][top4 + b];
      }
      count[kBins - 1 - 4 * b] = Pair{u.x, v.x};
      count[kBins - 2 - 4 * b] = Pair{u.y, v.y};
      count[kBins - 3 - 4 * b] = Pair{u.z, v.z};
      count[kBins - 4 - 4 * b] = Pair{u.w, v.w};
    }
    Pair sum{0, 0};
#pragma unroll
    for (int b = 0; b < kBins; ++b) {
      sum.x += count[b].x;
      sum.y += count[b].y;
    }
    Pair before = sums_before<NT>(sum, sm);
#pragma unroll
    for (int b = 0; b < kBins; ++b) {
      if (before.x < rank && before.x + count[b].x >= rank) {
        sm.digit = kBinsAll - 1 - (tid * kBins + b);
        sm.before = before;
        sm.equal_before = count[b].y;
        sm.all = before.x + count[b].x == rank;
      }
      before.x += count[b].x;
      before.y += count[b].y;
    }
    __syncthreads();
    prefix |= sm.digit << shift;
    known |= mask << shift;
    rank -= sm.before.x;
    above += sm.before.y;
    equal = sm.equal_before;
    // all keys with these bits stay: the bits below do not matter.  Nearly
    // always so after two passes, where few tokens share 22 bits
    if (sm.all) break;
  }
  // nobody reads another CTA's memory after this; the others' leave to go is
  // awaited at the end
  if (ctas > 1) cluster.barrier_arrive();

  // In the bits known, keys above `prefix` all stay, and of the equal ones the
  // first `rank`.
  const uint32_t below = (1u << lane) - 1u;
  for (int t0 = begin; t0 < end; t0 += kTile) {
    if (!held) load_keys<NT>(w, t0, end, keys);
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      if (t0 + i * NT >= end) {
        if (lane == 0) sm.slot[i * (NT / 32) + warp] = Pair{0, 0};
        continue;
      }
      const bool in = t0 + i * NT + tid < end;
      const uint32_t a = __ballot_sync(0xffffffffu, in && (keys[i] & known) > prefix);
      const uint32_t e = __ballot_sync(0xffffffffu, in && (keys[i] & known) == prefix);
      if (lane == 0) sm.slot[i * (NT / 32) + warp] = Pair{static_cast<uint32_t>(__popc(a)), static_cast<uint32_t>(__popc(e))};
    }
    __syncthreads();
    // slots a thread sums: neighbours, all of them below NT threads
    constexpr int kSlots = SelectSmem<NT>::kSlots;
    static_assert(kSlots <= NT, "a thread for each slot");
    const Pair own = tid < kSlots ? sm.slot[tid] : Pair{0, 0};
    const Pair pre = sums_before<NT>(own, sm);
    if (tid < kSlots) sm.slot[tid] = pre;
    if (tid == NT - 1) sm.part = Pair{pre.x + own.x, pre.y + own.y};  // of this tile, for the next one
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      if (t0 + i * NT >= end) break;
      const int t = t0 + i * NT + tid;
      const bool in = t < end;
      const uint32_t ab = __ballot_sync(0xffffffffu, in && (keys[i] & known) > prefix);
      const uint32_t eb = __ballot_sync(0xffffffffu, in && (keys[i] & known) == prefix);
      const Pair at = sm.slot[i * (NT / 32) + warp];
      const uint32_t na = above + at.x + __popc(ab & below), ne = equal + at.y + __popc(eb & below);
      const uint32_t key = keys[i] & known;
      if (in && (key > prefix || (key == prefix && ne < rank))) kept[sinks + na + min(ne, rank)] = ~t;
    }
    above += sm.part.x;
    equal += sm.part.y;
    __syncthreads();
  }
  if (ctas > 1) cluster.barrier_wait();
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A position in `kept`, whether its chunk's loads are done or not.
__device__ __forceinline__ int position(int k) { return k < 0 ? ~k : k; }

__device__ __forceinline__ int load_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int load_relaxed(const int32_t* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(int32_t* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void store_relaxed(int32_t* p, int v) {
  asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Waits until every earlier chunk of the unit that reads positions [first,
// end) has loaded its rows.  false: the limit passed.
__device__ __forceinline__ bool wait_for_readers(const int32_t* kept, int chunk, int rows, int first, int end,
                                                 unsigned long long limit_ns) {
  bool ok = true;
  for (int c = threadIdx.x; ok && c < chunk; c += kMoveThreads) {
    const int32_t* at = kept + static_cast<size_t>(c) * rows;
    const int low = load_acquire(at), high = load_relaxed(at + rows - 1);  // earlier chunks are full
    if (low >= 0 || position(low) >= end || position(high) < first) continue;
    const uint64_t t0 = global_timer_ns();
    while (load_acquire(at) < 0) {
      if (global_timer_ns() - t0 > limit_ns) {
        ok = false;
        break;
      }
    }
  }
  return __syncthreads_and(ok) != 0;
}

// kPieces: 16-byte pieces of a row of both pools (4-bit pools: of its codes);
// a warp's round copies 32 / kPieces rows.  kScale: a scale row's words (0 for
// 16-bit pools).
template <int kPieces, int kScale>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  constexpr int kRowsRound = 32 / kPieces;
  constexpr int kRowsWarp = kRounds * kRowsRound;
  constexpr int kRows = kMoveWarps * kRowsWarp;     // of a chunk
  constexpr int kRowBytes = kPieces / 2 * 16;       // in one pool
  constexpr int kLooks = (kRowsWarp + 31) / 32;     // rows a lane looks up
  __shared__ __align__(128) uint8_t stage[kChunkBytes];
  const int units = p.num_seqs * p.num_heads;
  const int chunk = blockIdx.x / units, unit = blockIdx.x - chunk * units;  // a unit's earlier chunks start earlier
  const int s = unit / p.num_heads, h = unit - s * p.num_heads;
  // what the plan is read from select does not write, and it lets this kernel
  // start only once what came before it is complete
  const Plan q = plan_of(p, s, false);
  const int j0 = chunk * kRows;
  const bool idle = !q.move || j0 >= q.m;
  // chunks past a sequence's kept tokens leave at once (where `kept` is wider
  // than the budgets they are most of the grid); the first CTA stays, so that
  // this launch does not end before select
  if (idle && blockIdx.x != 0) return;
  grid_dependency_wait();
  grid_launch_dependents();
  if (idle) return;
  int32_t* kept = p.kept + static_cast<size_t>(unit) * p.max_kept;
  const int32_t* from_table = p.tables + static_cast<size_t>(s) * p.table_width;
  const int32_t* to_table = p.dst_tables + static_cast<size_t>(s) * p.table_width;
  const size_t weights = (static_cast<size_t>(q.row) * p.num_heads + h) * p.row_tokens;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t scales = static_cast<size_t>(kRowBytes) << p.log2_block;  // in a 4-bit tile, behind the codes
  const int mask = (1 << p.log2_block) - 1;

  // ---- every lane looks up some of the warp's rows, and loads their words
  long long from[kLooks], to[kLooks];  // byte offsets in a pool; -1: the row is not moved
  int token[kLooks];
  float w[kLooks];
  uint32_t sk[kLooks][kScale > 0 ? kScale : 1], sv[kLooks][kScale > 0 ? kScale : 1];
  long long scale_to[kScale > 0 ? kLooks : 1];
  bool in_place = p.new_weights == p.weights;  // something is stored where rows may still be read
#pragma unroll
  for (int g = 0; g < kLooks; ++g) {
    const int r = lane + 32 * g, j = j0 + warp * kRowsWarp + r;
    token[g] = r < kRowsWarp && j < q.m ? position(__ldcg(kept + j)) : -1;
  }
#pragma unroll
  for (int g = 0; g < kLooks; ++g) {
    from[g] = to[g] = -1;
    if constexpr (kScale > 0) scale_to[g] = -1;
    if (token[g] >= 0) {
      const int j = j0 + warp * kRowsWarp + lane + 32 * g;
      const int a = __ldg(from_table + (token[g] >> p.log2_block)), b = __ldg(to_table + (j >> p.log2_block));
      const int c = __ldg(from_table + (j >> p.log2_block));
      w[g] = p.weights[weights + token[g]];
      in_place |= b == c;
      if (static_cast<unsigned>(a) >= static_cast<unsigned>(p.num_blocks) ||
          static_cast<unsigned>(b) >= static_cast<unsigned>(p.num_blocks)) {
        record_status(p.status, PA_DEV_BAD_BLOCK_ID);
      } else if (a != b || token[g] != j) {  // a row that keeps its place is not touched
        const size_t x = (static_cast<size_t>(a) * p.num_heads + h) * p.tile;
        const size_t y = (static_cast<size_t>(b) * p.num_heads + h) * p.tile;
        const int rx = token[g] & mask, ry = j & mask;
        from[g] = static_cast<long long>(x + rx * kRowBytes);
        to[g] = static_cast<long long>(y + ry * kRowBytes);
        if constexpr (kScale > 0) {
          const size_t sx = x + scales + rx * (kScale * 4);
          scale_to[g] = static_cast<long long>(y + scales + ry * (kScale * 4));
#pragma unroll
          for (int i = 0; i < kScale; ++i) {
            sk[g][i] = reinterpret_cast<const uint32_t*>(p.k_pool + sx)[i];
            sv[g][i] = reinterpret_cast<const uint32_t*>(p.v_pool + sx)[i];
          }
        }
      }
    }
  }
  // ---- the rows themselves: a round's lanes are the pieces of kRowsRound rows
  const int piece = lane % kPieces, in_round = lane / kPieces;
  uint8_t* pool = (piece < kPieces / 2 ? p.k_pool : p.v_pool) + piece % (kPieces / 2) * 16;
  uint8_t* mine = stage + warp * (kRounds * 512) + lane * 16;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const long long at = __shfl_sync(0xffffffffu, from[i * kRowsRound / 32], (i * kRowsRound + in_round) & 31);
    if (at >= 0) copy16(smem_u32(mine + i * 512), pool + at);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  const bool wait = __syncthreads_or(in_place) != 0;  // every load of the chunk is done
  if (p.withhold && blockIdx.x == 0) return;
  // Say so: the chunk's word is its first position, the first thread's.  The
  // barrier orders the other threads' loads before its release, which a waiting
  // CTA acquires before it stores; the other words are only looked at.
#pragma unroll
  for (int g = 0; g < kLooks; ++g) {
    if (token[g] < 0) continue;
    int32_t* at = kept + j0 + warp * kRowsWarp + lane + 32 * g;
    if (g == 0 && threadIdx.x == 0) {
      store_release(at, token[g]);
    } else {
      store_relaxed(at, token[g]);
    }
  }
  if (wait && !wait_for_readers(kept, chunk, kRows, j0, j0 + kRows, p.wait_limit_ns)) {
    if (threadIdx.x == 0) record_status(p.status, PA_DEV_TIMEOUT);
    return;
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const long long at = __shfl_sync(0xffffffffu, to[i * kRowsRound / 32], (i * kRowsRound + in_round) & 31);
    if (at >= 0) *reinterpret_cast<uint4*>(pool + at) = *reinterpret_cast<const uint4*>(mine + i * 512);
  }
#pragma unroll
  for (int g = 0; g < kLooks; ++g) {
    if (token[g] < 0) continue;
    p.new_weights[weights + j0 + warp * kRowsWarp + lane + 32 * g] = w[g];
    if constexpr (kScale > 0) {
      if (scale_to[g] >= 0) {
#pragma unroll
        for (int i = 0; i < kScale; ++i) {
          reinterpret_cast<uint32_t*>(p.k_pool + scale_to[g])[i] = sk[g][i];
          reinterpret_cast<uint32_t*>(p.v_pool + scale_to[g])[i] = sv[g][i];
        }
      }
    }
  }
}

// Launch on clusters of `ctas`, overlapping the kernel before (as
// launch_overlapped).
static cudaError_t launch_clusters(void (*kernel)(EvictParams), long long units, int ctas, int threads,
                                   cudaStream_t stream, const EvictParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * ctas));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// CTAs of a cluster for `items` at `each` a CTA: a power of two.
static int cluster_for(long long items, int each) {
  int c = 1;
  while (c < kMaxCluster && static_cast<long long>(c) * each < items) c *= 2;
  return c;
}

// The move launch of a kind of pool: a CTA for each chunk of `rows` rows of
// every unit.
struct Move {
  void (*kernel)(EvictParams);
  long long grid;
};
template <int kPieces, int kScale>
static Move move_of(long long units, long long rows) {
  constexpr int kRows = kMoveWarps * kRounds * (32 / kPieces);
  return Move{&move_kernel<kPieces, kScale>, units * ((rows + kRows - 1) / kRows)};
}

struct Span {
  const void* at;
  size_t bytes;
};
static bool overlap(const Span& a, const Span& b) {
  const auto x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at != nullptr && b.at != nullptr && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace evict
}  // namespace pa

using namespace pa;
using namespace pa::evict;

extern "C" pa_status pa_evict(const int32_t* block_tables, const int32_t* dst_tables, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t num_seqs, const int32_t* budgets, int32_t sinks,
                              int32_t recent, const pa_token_weights* weights, float* new_weights, int32_t* kept,
                              int32_t max_kept, int32_t* new_lens, int32_t fp4, void* k_pool, void* v_pool,
                              int32_t* dev_status, const pa_pool_desc* pool, void* stream) {
  if (pool == nullptr || pool->num_blocks <= 0 || pool->num_kv_heads <= 0 || num_seqs < 0 || max_blocks_per_seq <= 0 ||
      sinks < 0 || recent < 0 || max_kept < 0 || (fp4 & ~(1 | PA_EVICT_TEST_WITHHOLD)) != 0)
    return PA_ERR_INVALID_ARG;
  const bool fp4_pools = (fp4 & 1) != 0, withhold = (fp4 & PA_EVICT_TEST_WITHHOLD) != 0;
  if (!pa::fp4::pool_ok(pool)) return PA_ERR_UNSUPPORTED;  // the same block sizes and head_dims in both kinds of pool
  if (static_cast<long long>(max_blocks_per_seq) * pool->block_size > pa::fp4::kMaxTokens) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  auto aligned4 = [](const void* x) { return x != nullptr && (reinterpret_cast<uintptr_t>(x) & 3u) == 0; };
  if (!aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(budgets) || !aligned4(new_lens) ||
      (max_kept > 0 && !aligned4(kept)) || k_pool == nullptr || v_pool == nullptr || !aligned16(k_pool) ||
      !aligned16(v_pool) || (reinterpret_cast<uintptr_t>(dst_tables) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(new_weights) & 3u) != 0)
    return PA_ERR_INVALID_ARG;
  if (!token_weights_ok(weights, max_blocks_per_seq, num_seqs, pool)) return PA_ERR_INVALID_ARG;
  const size_t seqs = static_cast<size_t>(num_seqs), heads = static_cast<size_t>(pool->num_kv_heads);
  {  // what is written while the inputs may still be read
    const size_t table = seqs * max_blocks_per_seq * 4;
    const Span all{weights->weights,
                   static_cast<size_t>(weights->num_rows) * heads * static_cast<size_t>(weights->row_tokens) * 4};
    const Span in[] = {{seq_lens, seqs * 4}, {budgets, seqs * 4}, {weights->rows, seqs * 4}, {block_tables, table},
                       {dst_tables, table}, all};
    const Span moved{new_weights != weights->weights ? new_weights : nullptr, all.bytes};
    const Span out[] = {{new_lens, seqs * 4}, {kept, seqs * heads * max_kept * 4}, moved};
    for (const Span& o : out) {
      for (const Span& i : in) {
        if (overlap(o, i)) return PA_ERR_INVALID_ARG;
      }
    }
    if (overlap(out[0], out[1]) || overlap(out[0], moved) || overlap(out[1], moved)) return PA_ERR_INVALID_ARG;
  }
  EvictParams p;
  p.tables = block_tables;
  p.dst_tables = dst_tables != nullptr ? dst_tables : block_tables;
  p.seq_lens = seq_lens;
  p.budgets = budgets;
  p.rows = weights->rows;
  p.weights = weights->weights;
  p.new_weights = new_weights != nullptr ? new_weights : weights->weights;
  p.kept = kept;
  p.new_lens = new_lens;
  p.status = dev_status;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.row_tokens = weights->row_tokens;
  p.max_kept = max_kept;
  p.num_rows = weights->num_rows;
  p.num_seqs = num_seqs;
  p.num_heads = pool->num_kv_heads;
  p.num_blocks = pool->num_blocks;
  p.table_width = max_blocks_per_seq;
  p.max_tokens = max_blocks_per_seq * pool->block_size;
  p.sinks = sinks;
  p.recent = recent;
  p.log2_block = pa::fp4::log2_of(pool->block_size);
  p.tile = fp4_pools ? pa::fp4::tile_bytes(pool->block_size, pool->head_dim) : pool->block_size * pool->head_dim * 2;
  p.withhold = withhold;
  p.wait_limit_ns = withhold ? 20ull * 1000 * 1000 : 2ull * 1000 * 1000 * 1000;
  const long long units = static_cast<long long>(num_seqs) * pool->num_kv_heads;
  const long long rows = max_kept < p.max_tokens ? max_kept : p.max_tokens;  // at most, of a sequence
  if (units * kMaxCluster > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  const Move move = fp4_pools ? (pool->head_dim == 128 ? move_of<8, 2>(units, rows) : move_of<4, 1>(units, rows))
                              : (pool->head_dim == 128 ? move_of<32, 0>(units, rows) : move_of<16, 0>(units, rows));
  if (move.grid > 0x7fffffffLL) return PA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // The smallest CTA that holds the longest sequence in its registers, else
  // clusters of the largest.  512 units (sequence, kv head): 96.7 us with 128
  // threads and 99.7 with 256 at 1040 tokens, 32.2 with 256 and 36.1 with 512
  // at 3000 (32 units: 11.8 and 11.4).  8 keys a thread and twice the CTAs
  // instead of 16: 38.7 us for 36.8 at 8192 tokens, 30.6 for 21.0 at 32768.
  const cudaError_t selected =
      p.max_tokens <= kKeys * 128   ? launch_clusters(&select_kernel<128>, units, 1, 128, st, p)
      : p.max_tokens <= kKeys * 256 ? launch_clusters(&select_kernel<256>, units, 1, 256, st, p)
                                    : launch_clusters(&select_kernel<512>, units, cluster_for(p.max_tokens, kKeys * 512),
                                                      512, st, p);
  if (selected != cudaSuccess) return PA_ERR_CUDA;
  if (rows == 0) return PA_OK;
  const cudaError_t e =
      launch_overlapped(move.kernel, dim3(static_cast<unsigned>(move.grid)), dim3(kMoveThreads), 0, st, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
