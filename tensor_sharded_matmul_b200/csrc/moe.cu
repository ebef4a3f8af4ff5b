// The router of a mixture-of-experts MLP (softmax top-k, rows sorted by expert) and the combine of the
// experts' rows, with their gradients; and the same sort for adapters.
//
// Router: a warp takes one token, its E logits spread over the lanes (lane l holds experts l, l + 32,
// ...). The largest is found k times with two warp reductions each: the order-preserving integer key,
// then the lowest index among the lanes that hold it. Everything is binary32.
//
// Sort by expert: tokens of a block of 64 set one bit each in a bitmap per expert, so a token's place
// among its expert's rows of the block is a population count: no atomic's order enters. Per-block
// counts are scanned per expert (one warp each), and every block places its own tokens. A batch of at
// most 64 tokens is one block and one launch.
//
// Adapters: the same sort, with the tokens that have none behind all others; and for the pair kernel, which takes
// tokens in their own order, the adapters of every tile of 256 tokens. x A of few tokens has a kernel of its own
// here: it is what the second product waits for.
//
// Combine: y_n = sum_j weight_nj u[slot_nj], bound by reading u: one thread per eight columns, the k
// rows' loads issued together. Its gradient reads dy and the k rows once, a warp per token.
#include <cfloat>
#include <cstring>

#include "ragged.cuh"

namespace tpx {
namespace {

constexpr int TB = 64;                // tokens per block of the router and the sort
constexpr int WORDS = TB / 32;
template <int VPL>
constexpr int ROUTE_THREADS = VPL <= 8 ? 1024 : 512;      // registers of a long list

// See launch_beside.
__device__ __forceinline__ void begin_beside() {
  wait_prerequisites();
  launch_dependents();
}

// Order-preserving integer of a float (no NaN): a < b <=> key(a) < key(b). key(-inf) = 0x007fffff.
constexpr uint32_t KEY_MASKED = 0x007fffffu;
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);      // -0 orders like +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t at) {
  const float x = BF16 ? bf(ld_u16(static_cast<const uint16_t*>(logits) + at)) : ld_f32(static_cast<const float*>(logits) + at);
  // NaN masks like -inf; +inf counts as the largest finite number
  return x != x ? -INFINITY : fminf(x, FLT_MAX);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

struct SortParams {
  int64_t N;
  int E, k;                  // buckets, entries per token
  int rest;                  // 1: entries outside 0..E-1 form a last bucket (rows behind offsets[E])
  int blocks;
  int32_t* expert;           // [N][k]
  int32_t* slot;             // [N][k] or nullptr
  int32_t* offsets;          // [E + 1]
  int32_t* row_token;        // [N * k]
  int32_t* counts;           // [E + rest][blocks], then the buckets' totals [E + rest]
  int32_t* rank;             // [N][k]: places inside the block (slot itself where there is one)
};

__device__ __forceinline__ void clear_bits(uint32_t* bits, int buckets) {
  for (int i = threadIdx.x; i < buckets * WORDS; i += blockDim.x) bits[i] = 0u;
}
__device__ __forceinline__ int bucket_count(const uint32_t* bits, int e) {
  int c = 0;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) c += __popc(bits[e * WORDS + w]);
  return c;
}

// Exclusive scan of `n` values in shared memory in place, the total behind them. One warp.
__device__ __forceinline__ void scan_in_place(int* v, int n, int lane) {
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int x = i < n ? v[i] : 0;
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += up;
    }
    if (i < n) v[i] = base + inc - x;
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) v[n] = base;
  __syncwarp();
}

// The place of entry (t, e) among the block's entries of bucket e.
__device__ __forceinline__ int rank_in_block(const uint32_t* bits, int e, int t) {
  int r = __popc(bits[e * WORDS + t / 32] & ((1u << (t % 32)) - 1u));
  for (int w = 0; w < t / 32; ++w) r += __popc(bits[e * WORDS + w]);
  return r;
}

// This block's entries: `pick` [tokens][k] their buckets (-1: none), `bits` set, `start` room for the buckets
// and one more. A batch of one block is finished; otherwise the counts go to p.counts and the ranks to
// p.rank, for sort_scan_kernel and sort_place_kernel.
__device__ __forceinline__ void place_block(const SortParams& p, const uint32_t* bits, int* start, const int* pick, int64_t n0) {
  const int buckets = p.E + p.rest;
  const int entries = static_cast<int>(p.N - n0 < TB ? p.N - n0 : TB) * p.k;
  if (p.blocks == 1) {
    for (int e = threadIdx.x; e < buckets; e += blockDim.x) start[e] = bucket_count(bits, e);
    __syncthreads();
    if (threadIdx.x < 32) scan_in_place(start, buckets, threadIdx.x);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = start[e];
  } else {
    for (int e = threadIdx.x; e < buckets; e += blockDim.x)
      p.counts[static_cast<int64_t>(e) * p.blocks + blockIdx.x] = bucket_count(bits, e);
  }
  for (int i = threadIdx.x; i < entries; i += blockDim.x) {
    const int e = pick[i], t = i / p.k;
    int row = e >= 0 ? rank_in_block(bits, e, t) : -1;
    if (p.blocks == 1) {
      if (e >= 0) {
        row += start[e];
        p.row_token[row] = static_cast<int32_t>(n0 + t);
      }
      if (p.slot != nullptr) p.slot[n0 * p.k + i] = row;
    } else {
      p.rank[n0 * p.k + i] = row;
    }
  }
}

// A lane's keys in descending order, equal keys by ascending expert (an odd-even network; the lane's
// experts ascend with i, so equal neighbours need no exchange).
template <int VPL>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[VPL], int (&at)[VPL]) {
#pragma unroll
  for (int r = 0; r < VPL; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < VPL; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const uint32_t k = key[i];
      const int a = at[i];
      key[i] = swap ? key[i + 1] : k;
      key[i + 1] = swap ? k : key[i + 1];
      at[i] = swap ? at[i + 1] : a;
      at[i + 1] = swap ? a : at[i + 1];
    }
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(ROUTE_THREADS<VPL>) route_kernel(const void* logits, int gate,
                                                              float* weight, SortParams p) {
  extern __shared__ int s_dyn[];
  uint32_t* bits = reinterpret_cast<uint32_t*>(s_dyn);         // [E][WORDS]
  int* start = s_dyn + p.E * WORDS;                            // [E + 1]
  int* s_pick = start + p.E + 1;                               // [TB][k]: the block's choices
  constexpr bool SORTED = VPL <= 8;                            // a longer list is searched each time
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TB;
  clear_bits(bits, p.E);
  begin_beside();
  __syncthreads();
  for (int t = warp; t < TB && n0 + t < p.N; t += blockDim.x / 32) {
    const int64_t n = n0 + t;
    uint32_t key[VPL];
    int at[VPL];                                               // the expert of each key
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < p.E ? load_logit<BF16>(logits, n * p.E + e) : -INFINITY;
      key[i] = key_of(v[i]);
      at[i] = e;
    }
    if constexpr (SORTED) sort_lane(key, at);
    int my_e = -1;
    uint32_t my_key = KEY_MASKED, first = KEY_MASKED;          // lane j: the j-th choice; all: the first
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = key[0];
      int best_e = at[0];
      if constexpr (!SORTED) {
#pragma unroll
        for (int i = 1; i < VPL; ++i)
          if (key[i] > best) { best = key[i]; best_e = at[i]; }
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      if (top <= KEY_MASKED) break;                            // no expert left
      const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(best_e) : 0xffffffffu));
      const bool mine = best_e == e;                           // this lane's is taken
      if constexpr (SORTED) {
#pragma unroll
        for (int i = 0; i + 1 < VPL; ++i) {
          key[i] = mine ? key[i + 1] : key[i];
          at[i] = mine ? at[i + 1] : at[i];
        }
        key[VPL - 1] = mine ? 0u : key[VPL - 1];
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (mine && at[i] == best_e) key[i] = 0;
      }
      if (j == 0) first = top;
      if (lane == j) {
        my_e = e;
        my_key = top;
      }
    }
    const float m = of_key(first);
    const float my_w = my_e >= 0 ? expf(of_key(my_key) - m) : 0.0f;
    float total = my_w;
    if (gate == TP_GATE_SOFTMAX) {
      total = 0.0f;
      if (first > KEY_MASKED) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) total += expf(v[i] - m);
      }
    }
    total = warp_sum(total);
    if (lane < p.k) {
      p.expert[n * p.k + lane] = my_e;
      weight[n * p.k + lane] = my_e >= 0 ? my_w / total : 0.0f;
      s_pick[t * p.k + lane] = my_e;
      if (my_e >= 0) atomicOr(bits + my_e * WORDS + t / 32, 1u << (t % 32));
    }
  }
  __syncthreads();
  place_block(p, bits, start, s_pick, n0);
}

__global__ void __launch_bounds__(256) sort_count_kernel(SortParams p) {
  extern __shared__ int s_dyn[];
  const int buckets = p.E + p.rest;
  uint32_t* bits = reinterpret_cast<uint32_t*>(s_dyn);
  int* start = s_dyn + buckets * WORDS;
  int* s_pick = start + buckets + 1;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TB;
  clear_bits(bits, buckets);
  begin_beside();
  __syncthreads();
  for (int i = threadIdx.x; i < TB * p.k && n0 + i / p.k < p.N; i += blockDim.x) {
    int e = p.expert[n0 * p.k + i];
    if (e < 0 || e >= p.E) e = p.rest ? p.E : -1;
    s_pick[i] = e;
    if (e >= 0) atomicOr(bits + e * WORDS + i / p.k / 32, 1u << (i / p.k % 32));
  }
  __syncthreads();
  place_block(p, bits, start, s_pick, n0);
}

// One warp per bucket: its blocks' counts become the rows before each block; the total goes behind all.
__global__ void __launch_bounds__(256) sort_scan_kernel(SortParams p) {
  const int lane = threadIdx.x % 32;
  const int e = blockIdx.x * 8 + threadIdx.x / 32;
  const int buckets = p.E + p.rest;
  begin_beside();
  if (e >= buckets) return;
  constexpr int GROUP = 8;
  int32_t* c = p.counts + static_cast<int64_t>(e) * p.blocks;
  int base = 0;
  for (int b0 = 0; b0 < p.blocks; b0 += 32 * GROUP) {          // loads of a group together: one wait for memory
    int x[GROUP];
#pragma unroll
    for (int g = 0; g < GROUP; ++g) x[g] = b0 + 32 * g + lane < p.blocks ? c[b0 + 32 * g + lane] : 0;
#pragma unroll
    for (int g = 0; g < GROUP; ++g) {
      const int b = b0 + 32 * g + lane;
      int inc = x[g];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += up;
      }
      if (b < p.blocks) c[b] = base + inc - x[g];
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (lane == 0) p.counts[static_cast<int64_t>(buckets) * p.blocks + e] = base;
}

__global__ void __launch_bounds__(256) sort_place_kernel(SortParams p) {
  extern __shared__ int start[];                    // [buckets + 1], then this block's rows before it [buckets]
  constexpr int MINE = TB * TP_MAX_TOPK / 256;
  const int buckets = p.E + p.rest;
  int* before = start + buckets + 1;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TB;
  const int entries = static_cast<int>(p.N - n0 < TB ? p.N - n0 : TB) * p.k;
  begin_beside();
  int bucket[MINE], row[MINE];                      // loaded beside the counts
#pragma unroll
  for (int m = 0; m < MINE; ++m) {
    const int i = threadIdx.x + 256 * m;
    bucket[m] = i < entries ? p.expert[n0 * p.k + i] : 0;
    row[m] = i < entries ? p.rank[n0 * p.k + i] : -1;
  }
  for (int e = threadIdx.x; e < buckets; e += blockDim.x) {
    start[e] = p.counts[static_cast<int64_t>(buckets) * p.blocks + e];
    before[e] = p.counts[static_cast<int64_t>(e) * p.blocks + blockIdx.x];
  }
  __syncthreads();
  if (threadIdx.x < 32) scan_in_place(start, buckets, threadIdx.x);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = start[e];
#pragma unroll
  for (int m = 0; m < MINE; ++m) {
    const int i = threadIdx.x + 256 * m;
    if (i >= entries) break;
    if (row[m] >= 0) {
      const int e = bucket[m] < 0 || bucket[m] >= p.E ? p.E : bucket[m];     // the rest, behind all
      row[m] += start[e] + before[e];
      p.row_token[row[m]] = static_cast<int32_t>(n0 + i / p.k);
    }
    if (p.slot != nullptr) p.slot[n0 * p.k + i] = row[m];
  }
}

// dlogits of one token per warp. With q the weights' softmax (over all experts, or over the chosen):
// dl_i = q_i (dw_i - inner), inner = sum_j q_j dw_j, dw zero where not chosen. Every lane writes -q_i inner
// (TOPK: zero) for its experts; then lane j writes the j-th choice's, from its own copy of that logit. A
// choice that is named twice has the sum of its dw.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(256) route_bwd_kernel(const void* logits, int64_t N, int E, int k, int gate,
                                                        const int32_t* expert,
                                                        const float* dweight, void* dlogits) {
  const int lane = threadIdx.x % 32;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  begin_beside();
  if (n >= N) return;
  float v[VPL];
  if (gate == TP_GATE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < E ? load_logit<BF16>(logits, n * E + e) : -INFINITY;
    }
  }
  int my_e = lane < k ? ld_s32(expert + n * k + lane) : -1;
  if (my_e >= E) my_e = -1;
  float my_d = my_e >= 0 ? ld_f32(dweight + n * k + lane) : 0.0f;
  const float my_v = my_e >= 0 ? load_logit<BF16>(logits, n * E + my_e) : -INFINITY;
  bool first = my_e >= 0, again = false;           // the lowest lane of equal choices takes the sum of their dw
  for (int j = 0; j < k; ++j) {
    const bool same = __shfl_sync(0xffffffffu, my_e, j) == my_e && my_e >= 0;
    if (j < lane && same) first = false;
    if (j != lane && same) again = true;
  }
  if (__any_sync(0xffffffffu, again)) {
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) {
      const float d = __shfl_sync(0xffffffffu, my_d, j);
      if (__shfl_sync(0xffffffffu, my_e, j) == my_e) sum += d;
    }
    my_d = sum;
  }
  float m = first ? my_v : -INFINITY;
  if (gate == TP_GATE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
  }
  m = warp_max(m);
  const bool any = m > -INFINITY;
  const float my_p = first && any ? expf(my_v - m) : 0.0f;
  float total = my_p;
  if (gate == TP_GATE_SOFTMAX) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = any ? expf(v[i] - m) : 0.0f;
      total += v[i];
    }
  }
  float inner = my_p > 0.0f ? my_p * my_d : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, d);
    inner += __shfl_xor_sync(0xffffffffu, inner, d);
  }
  const float r = total > 0.0f ? 1.0f / total : 0.0f;
  inner *= r;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    if (e >= E) continue;
    const float g = gate == TP_GATE_SOFTMAX && v[i] > 0.0f ? -v[i] * r * inner : 0.0f;
    if constexpr (BF16)
      static_cast<uint16_t*>(dlogits)[n * E + e] = to_bf(g);
    else
      static_cast<float*>(dlogits)[n * E + e] = g;
  }
  __syncwarp();
  if (first && my_p > 0.0f) {
    const float g = my_p * r * (my_d - inner);
    if constexpr (BF16)
      static_cast<uint16_t*>(dlogits)[n * E + my_e] = to_bf(g);
    else
      static_cast<float*>(dlogits)[n * E + my_e] = g;
  }
}

// ------------------------------------------------------------------ adapters
// The segment of sorted row i among L with clamped bounds `off`, -1 if it lies in none: by halving where the bounds ascend,
// as a plan's do, or else by trying each (a segment that ends before it begins is empty, wherever the next one begins).
__device__ __forceinline__ int segment_of(const int* off, int L, int i, bool ascending) {
  int lo = 0, hi = ascending ? L : 0;
  while (lo + 1 < hi) {
    const int mid = (lo + hi) / 2;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  while (!ascending && lo + 1 < L && !(off[lo] <= i && i < off[lo + 1])) ++lo;
  return off[lo] <= i && i < off[lo + 1] ? lo : -1;
}
// Where row_token names a token; entries of tokens that it does not name stay whatever they were. (A launch of its own:
// 300 tokens take 0.3 us more than with every tile's block looking through all of row_token, 4000 tokens 8 us less, and
// 1.5 million 3.5 ms where that took 11.3.)
__global__ void __launch_bounds__(256) lora_places_kernel(const int32_t* row_token, int N, int32_t* pos) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  begin_beside();
  if (i >= N) return;
  const int t = ld_s32(row_token + i);
  if (t >= 0 && t < N) pos[t] = static_cast<int>(i);
}

// For every tile of `tile` tokens (one block of LORA_TILE threads): where each token lies in the sorted order (-1: without an
// adapter, -2: not named), and the adapters that the tile has, ascending, behind their number. An entry that
// lora_places_kernel did not write is told by row_token, which names another token there.
__global__ void __launch_bounds__(LORA_TILE) lora_tiles_kernel(const int32_t* offsets, const int32_t* row_token, int N, int L,
                                                               int tile, int32_t* pos, int32_t* lists) {
  __shared__ unsigned s_has[(TP_MAX_EXPERTS + 31) / 32];
  __shared__ int s_off[TP_MAX_EXPERTS + 1];
  const int tid = threadIdx.x, token = blockIdx.x * tile + tid;
  const bool mine = tid < tile && token < N;
  begin_beside();
  const int i = mine ? ld_s32(pos + token) : -1;
  const bool named = i >= 0 && i < N && ld_s32(row_token + i) == token;
  for (int a = tid; a <= L; a += LORA_TILE) s_off[a] = seg_bound(offsets, a, N);
  for (int w = tid; w < (L + 31) / 32; w += LORA_TILE) s_has[w] = 0u;
  __syncthreads();
  bool up = true;
  for (int a = tid; a < L; a += LORA_TILE) up = up && s_off[a] <= s_off[a + 1];
  const bool ascending = __syncthreads_and(up);
  const int a = named ? segment_of(s_off, L, i, ascending) : -1;
  if (a >= 0) atomicOr(s_has + a / 32, 1u << (a % 32));
  if (mine) pos[token] = a >= 0 ? i : named ? -1 : -2;
  __syncthreads();
  if (tid < 32) {
    int32_t* list = lists + static_cast<int64_t>(blockIdx.x) * LORA_LIST;
    int n = 0;
    for (int a0 = 0; a0 < L; a0 += 32) {
      const bool in = a0 + tid < L && (s_has[a0 / 32] >> tid & 1u);
      const unsigned m = __ballot_sync(0xffffffffu, in);
      const int at = n + __popc(m & ((1u << tid) - 1u));
      if (in && at < LORA_TILE) list[1 + at] = a0 + tid;
      n += __popc(m);
    }
    if (tid == 0) list[0] = min(n, LORA_TILE);
  }
}

// v = scale_a x A_a of few tokens, a block for each token and sixteen ranks: a thread takes eight ranks of every
// 512th k, the threads' sums meet in shared memory, and a warp adds those of one rank (always in the same order). Bound by
// latency: one round of loads, one meeting.
constexpr int V_THREADS = 1024, V_RANKS = 16;
constexpr int V_SMEM = V_THREADS * 8 + V_RANKS;              // floats: [ranks][lanes + 1] of either 16 or 8 ranks
__global__ void __launch_bounds__(V_THREADS, 1) lora_v_kernel(const uint16_t* x, const int32_t* offsets, const int32_t* row_token, int N,
                                                           int L, int K, int rank, const uint16_t* a, const float* scale, float* v) {
  __shared__ float s_part[V_SMEM];                           // [ranks][lanes + 1]
  __shared__ int s_adapter;
  const int i = blockIdx.x, tid = threadIdx.x;
  const int first = blockIdx.y * V_RANKS, ranks = min(V_RANKS, rank - first);
  const int groups = ranks / 8, lanes = V_THREADS / groups, stride = lanes + 1;
  if (tid == 0) s_adapter = -1;
  begin_beside();
  const int token = ld_s32(row_token + i);
  __syncthreads();
  for (int e = tid; e < L; e += V_THREADS)
    if (seg_bound(offsets, e, N) <= i && i < seg_bound(offsets, e + 1, N)) s_adapter = e;
  __syncthreads();
  const int adapter = s_adapter;
  if (adapter < 0) return;
  const bool in = token >= 0 && token < N;                   // others read as zeros
  const int j = tid / groups, r0 = (tid - j * groups) * 8;
  {
    float sum[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = 0.0f;
    const uint16_t* at = a + static_cast<int64_t>(adapter) * K * rank + first + r0;
    const uint16_t* xt = x + static_cast<int64_t>(in ? token : 0) * K;
    for (int k0 = j; in && k0 < K; k0 += 8 * lanes) {
      uint4 w[8];
      uint32_t xv[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k0 + u * lanes;
        w[u] = k < K ? ld_stream_v4(at + static_cast<int64_t>(k) * rank) : make_uint4(0, 0, 0, 0);
        xv[u] = k < K ? ld_u16(xt + k) : 0u;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float f[8];
        unpack_bf8(w[u], f);
        const float xf = bf(static_cast<uint16_t>(xv[u]));
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] = fmaf(xf, f[q], sum[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s_part[(r0 + q) * stride + j] = sum[q];
  }
  __syncthreads();
  const float sc = scale != nullptr ? ld_f32(scale + adapter) : 1.0f;
  for (int r = tid / 32; r < ranks; r += V_THREADS / 32) {
    float t = 0.0f;
    for (int l = tid % 32; l < lanes; l += 32) t += s_part[r * stride + l];
    t = warp_sum(t);
    if (tid % 32 == 0) v[static_cast<int64_t>(i) * rank + first + r] = in ? sc * t : 0.0f;
  }
}

// ------------------------------------------------------------------ combine
// Eight values as loaded, converted when they are used.
template <bool BF16>
struct Raw8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (BF16) {
      a = ld_stream_v4(static_cast<const uint16_t*>(base) + at);
    } else {
      a = ld_stream_v4(static_cast<const float*>(base) + at);
      b = ld_stream_v4(static_cast<const float*>(base) + at + 4);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (BF16) {
      unpack_bf8(a, f);
    } else {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
};

template <int KMAX, bool U_BF16, bool Y_BF16>
__global__ void __launch_bounds__(256) combine_kernel(const void* u, int64_t R, const float* weight,
                                                      const int32_t* slot, int64_t N, int h, int k,
                                                      void* y) {
  const int per_row = h / 8;
  const int64_t items = N * per_row;
  begin_beside();
  for (int64_t it = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; it < items;
       it += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t n = it / per_row;
    const int col = static_cast<int>(it - n * per_row) * 8;
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += KMAX) {
      Raw8<U_BF16> raw[KMAX];
      float w[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const int s = j0 + j < k ? ld_s32(slot + n * k + j0 + j) : -1;
        const bool in = s >= 0 && s < R;
        w[j] = !in ? 0.0f : weight != nullptr ? ld_f32(weight + n * k + j0 + j) : 1.0f;
        raw[j].a = raw[j].b = make_uint4(0, 0, 0, 0);
        if (in) raw[j].load(u, static_cast<int64_t>(s) * h + col);
      }
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        float f[8];
        raw[j].get(f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[j], f[q], acc[q]);
      }
    }
    if constexpr (Y_BF16) {
      st_v4(static_cast<uint16_t*>(y) + n * h + col, pack_bf8(acc));
    } else {
      float* o = static_cast<float*>(y) + n * h + col;
      st_v4(o, make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3])));
      st_v4(o + 4, make_uint4(__float_as_uint(acc[4]), __float_as_uint(acc[5]), __float_as_uint(acc[6]), __float_as_uint(acc[7])));
    }
  }
}

template <int KMAX, bool DY_BF16, bool U_BF16>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const void* dy, const void* u, int64_t R,
                                                          const float* weight, const int32_t* slot,
                                                          int64_t N, int h, int k, uint16_t* du,
                                                          float* dweight) {
  const int lane = threadIdx.x % 32;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  begin_beside();
  if (n >= N) return;
  int s[KMAX];
  float w[KMAX], dot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    s[j] = j < k ? ld_s32(slot + n * k + j) : -1;
    if (s[j] >= R) s[j] = -1;
    w[j] = s[j] >= 0 ? ld_f32(weight + n * k + j) : 0.0f;
    dot[j] = 0.0f;
  }
  for (int col = lane * 8; col < h; col += 256) {
    float g[8];
    Raw8<DY_BF16> dyv;
    dyv.load(dy, n * h + col);
    dyv.get(g);
    Raw8<U_BF16> raw[KMAX];                    // all rows' loads in flight before the first is used
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (s[j] >= 0) raw[j].load(u, static_cast<int64_t>(s[j]) * h + col);
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (s[j] < 0) continue;
      float f[8], o[8];
      raw[j].get(f);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        dot[j] = fmaf(g[q], f[q], dot[j]);
        o[q] = w[j] * g[q];
      }
      st_v4(du + static_cast<int64_t>(s[j]) * h + col, pack_bf8(o));
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const float t = warp_sum(dot[j]);
    if (lane == 0 && j < k) dweight[n * k + j] = t;
  }
}

// ------------------------------------------------------------------ launches
template <bool BF16>
tp_status launch_route(const void* logits, int gate, float* weight, const SortParams& p, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(p.E) * WORDS + p.E + 1 + TB * p.k) * 4;
  const int vpl = (p.E + 31) / 32;
  // a warp for each token, and four at least to place them
  auto threads = [&](int most) { return p.N >= most / 32 ? most : p.N > 4 ? 32 * static_cast<int>(p.N) : 128; };
  if (vpl <= 2) return launch_beside("route_kernel", route_kernel<2, BF16>, p.blocks, threads(ROUTE_THREADS<2>), smem, s, logits, gate, weight, p);
  if (vpl <= 4) return launch_beside("route_kernel", route_kernel<4, BF16>, p.blocks, threads(ROUTE_THREADS<4>), smem, s, logits, gate, weight, p);
  if (vpl <= 8) return launch_beside("route_kernel", route_kernel<8, BF16>, p.blocks, threads(ROUTE_THREADS<8>), smem, s, logits, gate, weight, p);
  return launch_beside("route_kernel", route_kernel<32, BF16>, p.blocks, threads(ROUTE_THREADS<32>), smem, s, logits, gate, weight, p);
}

template <bool BF16>
tp_status launch_route_bwd(const void* logits, int64_t N, int E, int k, int gate, const int32_t* expert,
                           const float* dweight, void* dlogits, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((N + 7) / 8);
  const int vpl = (E + 31) / 32;
  if (vpl <= 2) return launch_beside("route_bwd_kernel", route_bwd_kernel<2, BF16>, grid, 256, 0, s, logits, N, E, k, gate, expert, dweight, dlogits);
  if (vpl <= 4) return launch_beside("route_bwd_kernel", route_bwd_kernel<4, BF16>, grid, 256, 0, s, logits, N, E, k, gate, expert, dweight, dlogits);
  if (vpl <= 8) return launch_beside("route_bwd_kernel", route_bwd_kernel<8, BF16>, grid, 256, 0, s, logits, N, E, k, gate, expert, dweight, dlogits);
  return launch_beside("route_bwd_kernel", route_bwd_kernel<32, BF16>, grid, 256, 0, s, logits, N, E, k, gate, expert, dweight, dlogits);
}

// Offsets and places of a batch of more than one block, from the counts of its blocks.
tp_status scan_and_place(const SortParams& p, cudaStream_t s) {
  const int buckets = p.E + p.rest;
  if (tp_status st = launch_beside("sort_scan_kernel", sort_scan_kernel, (buckets + 7) / 8, 256, 0, s, p)) return st;
  return launch_beside("sort_place_kernel", sort_place_kernel, p.blocks, 256, static_cast<size_t>(2 * buckets + 1) * 4, s, p);
}

int64_t sort_blocks(int64_t N) { return (N + TB - 1) / TB; }
size_t sort_ws_bytes(int64_t N, int64_t buckets) {
  const int64_t b = sort_blocks(N);
  return b > 1 ? static_cast<size_t>(buckets) * (b + 1) * 4 : 0;
}

template <int KMAX, bool U_BF16>
tp_status launch_combine(const void* u, int64_t R, const float* weight, const int32_t* slot, int64_t N, int h, int k,
                         void* y, bool y_bf16, cudaStream_t s) {
  const int64_t blocks = (N * (h / 8) + 255) / 256;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 16;
  if (cap <= 0) return fail(TP_ECUDA, "cannot query the SM count");
  const unsigned grid = static_cast<unsigned>(blocks < cap ? blocks : cap);
  if (y_bf16) return launch_beside("combine_kernel", combine_kernel<KMAX, U_BF16, true>, grid, 256, 0, s, u, R, weight, slot, N, h, k, y);
  return launch_beside("combine_kernel", combine_kernel<KMAX, U_BF16, false>, grid, 256, 0, s, u, R, weight, slot, N, h, k, y);
}

template <int KMAX>
tp_status launch_combine_bwd(const void* dy, bool dy_bf16, const void* u, bool u_bf16, int64_t R, const float* weight,
                             const int32_t* slot, int64_t N, int h, int k, uint16_t* du, float* dweight, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((N + 7) / 8);
  if (dy_bf16 && u_bf16)
    return launch_beside("combine_bwd_kernel", combine_bwd_kernel<KMAX, true, true>, grid, 256, 0, s, dy, u, R, weight, slot, N, h, k, du, dweight);
  if (dy_bf16)
    return launch_beside("combine_bwd_kernel", combine_bwd_kernel<KMAX, true, false>, grid, 256, 0, s, dy, u, R, weight, slot, N, h, k, du, dweight);
  if (u_bf16)
    return launch_beside("combine_bwd_kernel", combine_bwd_kernel<KMAX, false, true>, grid, 256, 0, s, dy, u, R, weight, slot, N, h, k, du, dweight);
  return launch_beside("combine_bwd_kernel", combine_bwd_kernel<KMAX, false, false>, grid, 256, 0, s, dy, u, R, weight, slot, N, h, k, du, dweight);
}

// x A of few tokens by lora_v_kernel: its blocks run at once, and each token reads its own A. Whole calls, K = 4096, n = 6144 over
// 8 shards, rank 16: one token 15.0 us against 18.6 with the product kernel, 64 tokens of 32 adapters 26.7 against 31.3; rank 64,
// one token 15.9 against 19.2. Beyond: 16 tokens of rank 128 (17 MB of A) 34.9 and 32.2, 64 of rank 64 (256 blocks) 57 and 46.
bool lora_v_by_token(int64_t N, int64_t k, int rank) {
  return N <= 64 && N * ((rank + V_RANKS - 1) / V_RANKS) <= sm_count() && N * k * rank <= 6 << 20;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool valid_dtype(tp_dtype d) { return d == TP_F32 || d == TP_BF16; }
bool valid_act(tp_act a) { return a == TP_ACT_NONE || a == TP_ACT_GELU || a == TP_ACT_GELU_TANH || a == TP_ACT_SWIGLU; }
constexpr int64_t MAX_SIZE = INT32_MAX / 4;        // rows and columns: tile coordinates stay in 32 bits

tp_status check_route(int64_t N, int E, int k, tp_gate gate, tp_dtype dtype) {
  if (N < 0 || E <= 0 || k <= 0) return fail(TP_EINVAL, "negative size, or no experts");
  if (!valid_dtype(dtype)) return fail(TP_EINVAL, "bad dtype");
  if (gate != TP_GATE_SOFTMAX && gate != TP_GATE_TOPK) return fail(TP_EINVAL, "bad gate %d", static_cast<int>(gate));
  if (E > TP_MAX_EXPERTS) return fail(TP_EUNSUPPORTED, "%d experts: at most %d", E, TP_MAX_EXPERTS);
  if (k > TP_MAX_TOPK) return fail(TP_EUNSUPPORTED, "k=%d: at most %d experts for a token", k, TP_MAX_TOPK);
  if (k > E) return fail(TP_ESHAPE, "k=%d exceeds the %d experts", k, E);
  if (N > MAX_SIZE / k) return fail(TP_ESHAPE, "too many tokens");
  return TP_OK;
}

// Sizes and pointers that the three ragged products share. y/dy rows: R; x rows: x_rows.
tp_status check_ragged(int64_t x_rows, const int32_t* row_index, int64_t R, int E, int64_t k, int64_t n) {
  if (x_rows < 0 || R < 0 || E <= 0 || k <= 0 || n <= 0) return fail(TP_EINVAL, "negative size or empty contraction");
  if (E > TP_MAX_EXPERTS) return fail(TP_EUNSUPPORTED, "%d segments: at most %d", E, TP_MAX_EXPERTS);
  if (x_rows > MAX_SIZE || R > MAX_SIZE || k > MAX_SIZE || n > MAX_SIZE) return fail(TP_ESHAPE, "size too large");
  if (row_index == nullptr && x_rows < R) return fail(TP_ESHAPE, "x has %lld rows for %lld", (long long)x_rows, (long long)R);
  if (k % 8 || n % 8) return fail(TP_EALIGN, "k and n must be multiples of 8");
  return TP_OK;
}

}  // namespace
}  // namespace tpx

using namespace tpx;

extern "C" {

size_t tp_moe_route_ws_bytes(int64_t N, int E, int k) {
  if (N <= 0 || E <= 0 || E > TP_MAX_EXPERTS || k <= 0 || N > MAX_SIZE) return 0;
  return sort_ws_bytes(N, E);
}

tp_status tp_moe_route(const void* logits, tp_dtype dtype, int64_t N, int E, int k, tp_gate gate, int32_t* expert,
                       float* weight, int32_t* slot, int32_t* offsets, int32_t* row_token, void* ws, size_t ws_bytes,
                       void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tp_status st = check_route(N, E, k, gate, dtype)) return st;
  if (N == 0) return TP_OK;
  if (!logits || !expert || !weight || !slot || !offsets || !row_token) return fail(TP_EINVAL, "null pointer");
  if (!aligned4(expert) || !aligned4(weight) || !aligned4(slot) || !aligned4(offsets) || !aligned4(row_token) || !aligned4(ws) ||
      (dtype == TP_F32 && !aligned4(logits)) || (reinterpret_cast<uintptr_t>(logits) & 1u))
    return fail(TP_EALIGN, "pointer not aligned to its elements");
  const size_t need = tp_moe_route_ws_bytes(N, E, k);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return fail(TP_ENOSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  SortParams p = {N, E, k, 0, static_cast<int>(sort_blocks(N)), expert, slot, offsets, row_token, static_cast<int32_t*>(ws), slot};
  if (tp_status st = dtype == TP_BF16 ? launch_route<true>(logits, gate, weight, p, s) : launch_route<false>(logits, gate, weight, p, s))
    return st;
  return p.blocks == 1 ? TP_OK : scan_and_place(p, s);
}

tp_status tp_moe_route_bwd(const void* logits, tp_dtype dtype, int64_t N, int E, int k, tp_gate gate, const int32_t* expert,
                           const float* dweight, void* dlogits, void* stream) {
  if (tp_status st = check_route(N, E, k, gate, dtype)) return st;
  if (N == 0) return TP_OK;
  if (!logits || !expert || !dweight || !dlogits) return fail(TP_EINVAL, "null pointer");
  const uintptr_t mask = dtype == TP_F32 ? 3u : 1u;
  if (!aligned4(expert) || !aligned4(dweight) || (reinterpret_cast<uintptr_t>(logits) & mask) ||
      (reinterpret_cast<uintptr_t>(dlogits) & mask))
    return fail(TP_EALIGN, "pointer not aligned to its elements");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == TP_BF16 ? launch_route_bwd<true>(logits, N, E, k, gate, expert, dweight, dlogits, s)
                          : launch_route_bwd<false>(logits, N, E, k, gate, expert, dweight, dlogits, s);
}

tp_status tp_ragged_linear(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const int32_t* offsets, int64_t R,
                           int E, int64_t k, int64_t n, tp_act act, const uint16_t* w, void* y, tp_dtype y_dtype,
                           uint16_t* pre, void* stream) {
  if (tp_status st = check_ragged(x_rows, row_index, R, E, k, n)) return st;
  if (!valid_act(act) || !valid_dtype(y_dtype)) return fail(TP_EINVAL, "bad activation or dtype");
  if (act == TP_ACT_NONE && pre != nullptr) return fail(TP_EINVAL, "pre is the activation's input: there is no activation");
  if (R == 0) return TP_OK;
  if (!x || !offsets || !w || !y) return fail(TP_EINVAL, "null pointer");
  if (x_rows == 0) return fail(TP_ESHAPE, "x has no rows");
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(pre)) return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (!aligned4(offsets) || !aligned4(row_index)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  RaggedArgs g;
  std::memset(&g, 0, sizeof(g));
  g.x = x; g.x_rows = x_rows; g.row_index = row_index; g.offsets = offsets; g.R = R; g.E = E; g.K = k; g.n = n;
  g.w = w; g.act = act; g.y = y; g.out_f32 = y_dtype == TP_F32; g.pre = pre;
  return ragged_product(g, static_cast<cudaStream_t>(stream));
}

tp_status tp_ragged_linear_dx(const uint16_t* dy, const int32_t* offsets, int64_t R, int E, int64_t k, int64_t n,
                              const uint16_t* w, tp_act act, const uint16_t* h_pre, uint16_t* dx, void* stream) {
  if (tp_status st = check_ragged(R, nullptr, R, E, k, n)) return st;
  if (!valid_act(act)) return fail(TP_EINVAL, "bad activation");
  if (R == 0) return TP_OK;
  if (!dy || !offsets || !w || !dx) return fail(TP_EINVAL, "null pointer");
  if ((act != TP_ACT_NONE) != (h_pre != nullptr)) return fail(TP_EINVAL, "h_pre is given exactly with an activation");
  if (!aligned16(dy) || !aligned16(w) || !aligned16(dx) || !aligned16(h_pre)) return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (!aligned4(offsets)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  RaggedArgs g;
  std::memset(&g, 0, sizeof(g));
  g.x = dy; g.x_rows = R; g.offsets = offsets; g.R = R; g.E = E; g.K = n; g.n = k;
  g.w = w; g.w_km = true; g.act = act; g.backward = true; g.h_pre = h_pre; g.y = dx;
  return ragged_product(g, static_cast<cudaStream_t>(stream));
}

tp_status tp_ragged_linear_dw(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const uint16_t* dy,
                              const int32_t* offsets, int64_t R, int E, int64_t k, int64_t n, void* dw, tp_dtype dw_dtype,
                              void* stream) {
  if (tp_status st = check_ragged(x_rows, row_index, R, E, k, n)) return st;
  if (!valid_dtype(dw_dtype)) return fail(TP_EINVAL, "bad dtype");
  if (!offsets || !dw) return fail(TP_EINVAL, "null pointer");
  if (R > 0 && (!x || !dy)) return fail(TP_EINVAL, "null pointer");
  if (R > 0 && x_rows == 0) return fail(TP_ESHAPE, "x has no rows");
  if (!aligned16(x) || !aligned16(dy) || !aligned16(dw)) return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (!aligned4(offsets) || !aligned4(row_index)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (R == 0) {                                   // no rows: every gradient is zero
    if (cudaMemsetAsync(dw, 0, static_cast<size_t>(E) * k * n * (dw_dtype == TP_F32 ? 4 : 2), s) != cudaSuccess)
      return fail(TP_ECUDA, "cannot clear the weight gradients");
    return TP_OK;
  }
  const RaggedDwArgs g = {x, x_rows, row_index, dy, offsets, R, E, k, n, dw, dw_dtype == TP_F32};
  return ragged_dw(g, s);
}

tp_status tp_moe_combine(const void* u, tp_dtype u_dtype, int64_t R, const float* weight, const int32_t* slot, int64_t N,
                         int64_t h, int k, void* y, tp_dtype y_dtype, void* stream) {
  if (N < 0 || R < 0 || h <= 0 || k <= 0) return fail(TP_EINVAL, "negative size");
  if (!valid_dtype(u_dtype) || !valid_dtype(y_dtype)) return fail(TP_EINVAL, "bad dtype");
  if (k > TP_MAX_TOPK) return fail(TP_EUNSUPPORTED, "k=%d: at most %d experts for a token", k, TP_MAX_TOPK);
  if (N > MAX_SIZE / k || R > MAX_SIZE || h > MAX_SIZE) return fail(TP_ESHAPE, "size too large");
  if (h % 8) return fail(TP_EALIGN, "h must be a multiple of 8");
  if (N == 0) return TP_OK;
  if (!slot || !y || (R > 0 && !u)) return fail(TP_EINVAL, "null pointer");
  if (!aligned16(u) || !aligned16(y)) return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (!aligned4(weight) || !aligned4(slot)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool yb = y_dtype == TP_BF16;
  const int hh = static_cast<int>(h);
  if (u_dtype == TP_BF16) {
    if (k <= 2) return launch_combine<2, true>(u, R, weight, slot, N, hh, k, y, yb, s);
    if (k <= 4) return launch_combine<4, true>(u, R, weight, slot, N, hh, k, y, yb, s);
    return launch_combine<8, true>(u, R, weight, slot, N, hh, k, y, yb, s);
  }
  if (k <= 2) return launch_combine<2, false>(u, R, weight, slot, N, hh, k, y, yb, s);
  return launch_combine<4, false>(u, R, weight, slot, N, hh, k, y, yb, s);
}

tp_status tp_moe_combine_bwd(const void* dy, tp_dtype dy_dtype, const void* u, tp_dtype u_dtype, int64_t R,
                             const float* weight, const int32_t* slot, int64_t N, int64_t h, int k, uint16_t* du,
                             float* dweight, void* stream) {
  if (N < 0 || R < 0 || h <= 0 || k <= 0) return fail(TP_EINVAL, "negative size");
  if (!valid_dtype(u_dtype) || !valid_dtype(dy_dtype)) return fail(TP_EINVAL, "bad dtype");
  if (k > TP_MAX_TOPK) return fail(TP_EUNSUPPORTED, "k=%d: at most %d experts for a token", k, TP_MAX_TOPK);
  if (N > MAX_SIZE / k || R > MAX_SIZE || h > MAX_SIZE) return fail(TP_ESHAPE, "size too large");
  if (h % 8) return fail(TP_EALIGN, "h must be a multiple of 8");
  if (N == 0) return TP_OK;
  if (!dy || !weight || !slot || !dweight || (R > 0 && (!u || !du))) return fail(TP_EINVAL, "null pointer");
  if (!aligned16(dy) || !aligned16(u) || !aligned16(du)) return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (!aligned4(weight) || !aligned4(slot) || !aligned4(dweight)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool db = dy_dtype == TP_BF16, ub = u_dtype == TP_BF16;
  const int hh = static_cast<int>(h);
  if (k <= 2) return launch_combine_bwd<2>(dy, db, u, ub, R, weight, slot, N, hh, k, du, dweight, s);
  if (k <= 8) return launch_combine_bwd<8>(dy, db, u, ub, R, weight, slot, N, hh, k, du, dweight, s);
  return launch_combine_bwd<TP_MAX_TOPK>(dy, db, u, ub, R, weight, slot, N, hh, k, du, dweight, s);
}

size_t tp_moe_mlp_ws_bytes(int64_t N, int E, int k) { return tp_moe_route_ws_bytes(N, E, k); }

tp_status tp_moe_mlp_fwd(const uint16_t* x, int64_t N, int64_t h, int64_t F, int E, int k, tp_gate gate, tp_act act,
                         const void* logits, tp_dtype logits_dtype, const uint16_t* w_in, const uint16_t* w_down,
                         int32_t* expert, float* weight, int32_t* slot, int32_t* offsets, int32_t* row_token,
                         uint16_t* h_pre, uint16_t* z, uint16_t* u, void* y, tp_dtype y_dtype, void* ws, size_t ws_bytes,
                         void* stream) {
  if (tp_status st = check_route(N, E, k, gate, logits_dtype)) return st;
  if (tp_status st = check_ragged(N, nullptr, N, E, h, F)) return st;
  if (!valid_act(act) || !valid_dtype(y_dtype)) return fail(TP_EINVAL, "bad activation or dtype");
  if (N == 0) return TP_OK;
  if (!x || !logits || !w_in || !w_down || !expert || !weight || !slot || !offsets || !row_token || !z || !u || !y)
    return fail(TP_EINVAL, "null pointer");
  if (!aligned16(x) || !aligned16(w_in) || !aligned16(w_down) || !aligned16(h_pre) || !aligned16(z) || !aligned16(u) || !aligned16(y))
    return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (act == TP_ACT_NONE && h_pre != nullptr) return fail(TP_EINVAL, "h_pre is the activation's input: there is no activation");
  const int64_t R = N * k;
  if (tp_status st = tp_moe_route(logits, logits_dtype, N, E, k, gate, expert, weight, slot, offsets, row_token, ws, ws_bytes, stream))
    return st;
  RaggedArgs g;                                    // (u is not needed yet: it takes the gathered rows)
  std::memset(&g, 0, sizeof(g));
  g.x = x; g.x_rows = N; g.row_index = row_token; g.x_copy = u; g.offsets = offsets; g.R = R; g.E = E; g.K = h; g.n = F;
  g.w = w_in; g.act = act; g.y = z; g.pre = h_pre;
  if (tp_status st = ragged_product(g, static_cast<cudaStream_t>(stream))) return st;
  if (tp_status st = tp_ragged_linear(z, R, nullptr, offsets, R, E, F, h, TP_ACT_NONE, w_down, u, TP_BF16, nullptr, stream)) return st;
  return tp_moe_combine(u, TP_BF16, R, weight, slot, N, h, k, y, y_dtype, stream);
}

tp_status tp_moe_mlp_bwd(const uint16_t* x, const uint16_t* dy, int64_t N, int64_t h, int64_t F, int E, int k, tp_gate gate,
                         tp_act act, const void* logits, tp_dtype logits_dtype, const uint16_t* w_in,
                         const uint16_t* w_down, const int32_t* expert, const float* weight, const int32_t* slot,
                         const int32_t* offsets, const int32_t* row_token, const uint16_t* h_pre, const uint16_t* z,
                         const uint16_t* u, uint16_t* du_ws, uint16_t* dh_ws, float* dweight_ws, float* dw_in,
                         float* dw_down, void* dx, tp_dtype dx_dtype, void* dlogits, void* stream) {
  if (tp_status st = check_route(N, E, k, gate, logits_dtype)) return st;
  if (tp_status st = check_ragged(N, nullptr, N, E, h, F)) return st;
  if (!valid_act(act) || !valid_dtype(dx_dtype)) return fail(TP_EINVAL, "bad activation or dtype");
  const int64_t R = N * k, wn = act == TP_ACT_SWIGLU ? 2 * F : F;
  if (wn > MAX_SIZE) return fail(TP_ESHAPE, "size too large");
  if (N > 0 && (!x || !dy || !logits || !w_in || !w_down || !expert || !weight || !slot || !row_token || !z || !u || !du_ws ||
                !dh_ws || !dweight_ws || !dx || !dlogits))
    return fail(TP_EINVAL, "null pointer");
  if (!offsets || !dw_in || !dw_down) return fail(TP_EINVAL, "null pointer");
  if (N > 0 && (act != TP_ACT_NONE) != (h_pre != nullptr)) return fail(TP_EINVAL, "h_pre is given exactly with an activation");
  if (!aligned16(x) || !aligned16(dy) || !aligned16(w_in) || !aligned16(w_down) || !aligned16(h_pre) || !aligned16(z) ||
      !aligned16(u) || !aligned16(du_ws) || !aligned16(dh_ws) || !aligned16(dw_in) || !aligned16(dw_down) || !aligned16(dx))
    return fail(TP_EALIGN, "pointer not 16-byte aligned");
  const uintptr_t logit_mask = logits_dtype == TP_F32 ? 3u : 1u;
  if (!aligned4(expert) || !aligned4(weight) || !aligned4(slot) || !aligned4(offsets) || !aligned4(row_token) || !aligned4(dweight_ws) ||
      (reinterpret_cast<uintptr_t>(logits) & logit_mask) || (reinterpret_cast<uintptr_t>(dlogits) & logit_mask))
    return fail(TP_EALIGN, "pointer not aligned to its elements");
  // combine -> down (both gradients) -> activation (in the down product's epilogue) -> up (both) -> tokens
  if (tp_status st = tp_moe_combine_bwd(dy, TP_BF16, u, TP_BF16, R, weight, slot, N, h, k, du_ws, dweight_ws, stream)) return st;
  if (tp_status st = tp_moe_route_bwd(logits, logits_dtype, N, E, k, gate, expert, dweight_ws, dlogits, stream)) return st;
  if (tp_status st = tp_ragged_linear_dw(z, R, nullptr, du_ws, offsets, R, E, F, h, dw_down, TP_F32, stream)) return st;
  if (tp_status st = tp_ragged_linear_dx(du_ws, offsets, R, E, F, h, w_down, act, h_pre, dh_ws, stream)) return st;
  // du is not needed any more: where experts have many rows, x's gathered ones are put side by side there (8192 rows, 8
  // experts, 4096 x 14336: 970..1120 us gathered, 850 side by side, 26 the copy; 384 rows an expert: 184 and 193)
  const bool copy = R >= 512 * static_cast<int64_t>(E);
  if (copy) {
    if (tp_status st = gather_rows(x, N, row_token, offsets, E, R, h, du_ws, h, static_cast<cudaStream_t>(stream))) return st;
  }
  if (tp_status st = tp_ragged_linear_dw(copy ? du_ws : x, copy ? R : N, copy ? nullptr : row_token, dh_ws, offsets, R, E, h, wn, dw_in,
                                         TP_F32, stream))
    return st;
  if (N == 0) return TP_OK;
  // every row's gradient of x takes the place of du
  if (tp_status st = tp_ragged_linear_dx(dh_ws, offsets, R, E, h, wn, w_in, TP_ACT_NONE, nullptr, du_ws, stream)) return st;
  return tp_moe_combine(du_ws, TP_BF16, R, nullptr, slot, N, h, k, dx, dx_dtype, stream);
}

size_t tp_lora_plan_ws_bytes(int64_t N, int L) {
  if (N <= 0 || L <= 0 || L > TP_MAX_EXPERTS || N > MAX_SIZE) return 0;
  const size_t counts = sort_ws_bytes(N, L + 1);
  return counts > 0 ? counts + static_cast<size_t>(N) * 4 : 0;     // and every token's place in its block
}

tp_status tp_lora_plan(const int32_t* id, int64_t N, int L, int32_t* offsets, int32_t* row_token, void* ws, size_t ws_bytes,
                       void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N < 0 || L <= 0) return fail(TP_EINVAL, "negative size, or no adapters");
  if (L > TP_MAX_EXPERTS) return fail(TP_EUNSUPPORTED, "%d adapters: at most %d", L, TP_MAX_EXPERTS);
  if (N > MAX_SIZE) return fail(TP_ESHAPE, "too many tokens");
  if (N == 0) return TP_OK;
  if (!id || !offsets || !row_token) return fail(TP_EINVAL, "null pointer");
  if (!aligned4(id) || !aligned4(offsets) || !aligned4(row_token) || !aligned4(ws)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  const size_t need = tp_lora_plan_ws_bytes(N, L);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return fail(TP_ENOSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  SortParams p = {N, L, 1, 1, static_cast<int>(sort_blocks(N)), const_cast<int32_t*>(id), nullptr, offsets, row_token,
                  static_cast<int32_t*>(ws), static_cast<int32_t*>(ws) + (L + 1) * (sort_blocks(N) + 1)};
  if (tp_status st = launch_beside("sort_count_kernel", sort_count_kernel, p.blocks, 256,
                                   (static_cast<size_t>(L + 1) * WORDS + L + 2 + TB) * 4, s, p))
    return st;
  return p.blocks == 1 ? TP_OK : scan_and_place(p, s);
}

size_t tp_lora_ws_bytes(int64_t N, int rank) {
  if (N <= 0 || rank <= 0 || N > MAX_SIZE) return 0;
  const size_t tiles = (static_cast<size_t>(N) + LORA_TILE_MIN - 1) / LORA_TILE_MIN;
  // v; beyond one tile of few tokens, every token's place and every tile's adapters
  return static_cast<size_t>(N) * rank * 4 + (N > 64 ? static_cast<size_t>(N) * 4 + tiles * LORA_LIST * 4 : 0);
}

tp_status tp_lora_linear(const uint16_t* x, int64_t N, int64_t k, int64_t n, int t, const uint16_t* w, int L, int rank,
                         const uint16_t* a, const uint16_t* b, const float* scale, const int32_t* offsets,
                         const int32_t* row_token, uint16_t* y, void* ws, size_t ws_bytes, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!valid_t(t)) return fail(TP_EINVAL, "t=%d outside 1..%d", t, TP_MAX_SHARDS);
  if (N < 0 || k <= 0 || n <= 0 || L <= 0 || rank <= 0) return fail(TP_EINVAL, "negative size, empty contraction or no adapters");
  if (L > TP_MAX_EXPERTS) return fail(TP_EUNSUPPORTED, "%d adapters: at most %d", L, TP_MAX_EXPERTS);
  if (n % t) return fail(TP_EDIVIS, "t=%d does not divide n=%lld", t, (long long)n);
  if (N > MAX_SIZE || k > MAX_SIZE || n > MAX_SIZE || rank > MAX_SIZE) return fail(TP_ESHAPE, "size too large");
  if (k % 8 || (n / t) % 8 || rank % 8) return fail(TP_EALIGN, "k, n/t and rank must be multiples of 8");
  if (N == 0) return TP_OK;
  if (!x || !w || !a || !b || !offsets || !row_token || !y) return fail(TP_EINVAL, "null pointer");
  if (!aligned16(x) || !aligned16(w) || !aligned16(a) || !aligned16(b) || !aligned16(y) || !aligned16(ws))
    return fail(TP_EALIGN, "pointer not 16-byte aligned");
  if (!aligned4(scale) || !aligned4(offsets) || !aligned4(row_token)) return fail(TP_EALIGN, "pointer not aligned to its elements");
  const size_t need = tp_lora_ws_bytes(N, rank);
  if (ws == nullptr || ws_bytes < need) return fail(TP_ENOSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, need);
  int32_t* pos = nullptr;
  int32_t* lists = nullptr;
  if (lora_takes_pairs(N, n / t, t)) {
    pos = reinterpret_cast<int32_t*>(static_cast<float*>(ws) + N * rank);
    lists = pos + N;
    const int tile = lora_tile(N, n / t, t);
    if (tp_status st = launch_beside("lora_places_kernel", lora_places_kernel, static_cast<unsigned>((N + 255) / 256), 256, 0, s, row_token,
                                     static_cast<int>(N), pos))
      return st;
    if (tp_status st = launch_beside("lora_tiles_kernel", lora_tiles_kernel, static_cast<unsigned>((N + tile - 1) / tile), LORA_TILE, 0, s,
                                     offsets, row_token, static_cast<int>(N), L, tile, pos, lists))
      return st;
  }
  RaggedArgs g;                                    // v = scale * x A over the adapters' segments, binary32
  std::memset(&g, 0, sizeof(g));
  if (lora_v_by_token(N, k, rank)) {
    if (tp_status st = launch_beside("lora_v_kernel", lora_v_kernel, dim3(static_cast<unsigned>(N), (rank + V_RANKS - 1) / V_RANKS), V_THREADS, 0, s, x, offsets, row_token,
                                static_cast<int>(N), L, static_cast<int>(k), rank, a, scale, static_cast<float*>(ws)))
      return st;
  } else {
    g.x = x; g.x_rows = N; g.row_index = row_token; g.offsets = offsets; g.R = N; g.E = L; g.K = k; g.n = rank;
    g.w = a; g.act = TP_ACT_NONE; g.y = ws; g.out_f32 = true; g.seg_scale = scale;
    if (tp_status st = ragged_product(g, s)) return st;
  }
  std::memset(&g, 0, sizeof(g));                   // y[r] = x W[r] + v B[r]
  g.x = x; g.x_rows = N; g.row_index = row_token; g.offsets = offsets; g.R = N; g.E = t; g.K = k; g.n = n / t;
  g.w = w; g.act = TP_ACT_NONE; g.y = y; g.v = static_cast<const float*>(ws); g.lora_b = b; g.L = L; g.rank = rank;
  g.lora_pos = pos; g.lora_lists = lists;
  return ragged_product(g, s);
}

}  // extern "C"
