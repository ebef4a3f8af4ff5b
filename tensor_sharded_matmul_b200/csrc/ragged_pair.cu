// The ragged products of ragged.cu for segments of many rows: CTA pairs, persistent.
//
// The same transposed product, D^T = W_e^T x^T, on tcgen05 cta_group::2: 256 columns of W are the M
// of a pair (128 per CTA; SwiGLU: 64 gate and 64 up columns per CTA), and up to 256 rows of a segment
// its N, in steps of 32, each CTA holding half of them. A segment of r rows is cut into ceil(r / 256)
// tiles of nearly equal height, so that its last tile is not a sliver that streams all of W for a few rows.
//
// Per CTA: warp 0 loads W, and x where its rows lie side by side, by TMA; warps 10..17 copy gathered rows with
// cp.async (adapters: they put the values of v into shared memory) and warps 18, 19 hand them over; one thread
// of the leader's warp 1 issues the MMAs; warps 2..9 turn the accumulator's rows around through shared memory and
// write whole row pieces while the next tile is multiplied into the other accumulator. A stage holds two 64-deep
// k-blocks, three stages fit.
//
// What bounds it: with rows side by side, the MMAs (their thread waits 90 cycles a stage, of 940); 8 experts of
// 1024 rows, K = 4096, n = 14336, SwiGLU: 1270..1330 us over the GPUs measured, 1450..1520 TFLOP/s in a burst of calls (with
// `pre` written besides 1360 beside 1320); under the power cap the clock falls to 1.2..1.6 GHz. Before the loading thread had a loop with little else than its loads, its 1500 cycles a stage were the bound
// (1600 us). (Stages of one k-block, six of them: 1480 us.)
// Gathered rows (1820 us there if all are fetched by index, 1430 put side by side first): TMA's tile::gather4 took about 75 cycles for four 128-byte rows, 221 TFLOP/s; loads into
// registers two stages ahead, 897; cp.async by four warps, 922, by eight, 1089, by sixteen, 1076. What remains is the way
// through a stage: 500 cycles to issue the copies, as many for them to land, and 1430 for the other CTA's release
// at cluster scope to reach the leader, of 4100 for three stages. Wide products therefore put many gathered rows side
// by side first (ragged_product).
//
// A stage's barrier lives in the leader, which alone announces the bytes of both CTAs' TMA loads (they are
// equal): a second announcement from the other CTA cost a fifth of the rate (1058 against 1351 TFLOP/s).
//
// A wait that runs out is agreed on by the eight epilogue warps before any of them leaves, since they meet
// at named barriers.
#include <cstring>

#include "ragged.cuh"
#include "tmap.cuh"

namespace tpx {
namespace {

constexpr int BK = 64;
constexpr int KB = 2;                               // k-blocks per stage
constexpr int STAGES = 3;
constexpr int NT = 256;                             // rows of a tile, at most
constexpr uint32_t HALF = 128 * BK * 2;             // one k-block of one operand of this CTA: 16 KiB
constexpr uint32_t BOX = 64 * BK * 2;               // 64 columns x 64 k: 8 KiB
constexpr uint32_t OP_STAGE = KB * HALF;
constexpr uint32_t TMEM_COLS = 512;
constexpr int LOADERS = 8, RELAYS = 2;              // warps that fetch gathered rows, and that pass them on
constexpr int EPI = 8;                              // epilogue warps: two groups of four
constexpr int LOAD0 = 2 + EPI, RELAY0 = LOAD0 + LOADERS;   // first warps; before them TMA, MMA, epilogue
constexpr int THREADS = 32 * (RELAY0 + RELAYS);
static_assert(32 * LOADERS == 2 * 128, "two threads build one row of adapter values");
constexpr int STG_LD = 128 + 4;                     // floats between staged rows
constexpr int CHUNK = 16;                           // rows that a group turns around at a time
constexpr uint32_t STAGING = 2 * CHUNK * STG_LD * 4;
constexpr size_t SMEM = 1024 + STAGES * 2 * OP_STAGE + STAGING + 256 + 2 * (TP_MAX_EXPERTS + 4) * 4;
constexpr unsigned long long DRAIN = 400000000ull;

struct Pair {
  uint8_t *sW, *sX;
  uint32_t full0, empty0, rows0, go0, accf0, acce0, drain, full0_leader, acce0_leader;
  volatile uint32_t* abort_flag;
  uint32_t rank;
};

__device__ __forceinline__ bool pair_fail(const RaggedParams& p, const Pair& c, uint32_t site) {
  if (!*c.abort_flag) record_timeout(p.status, site);
  *c.abort_flag = 1u;
  return false;
}

// Bounded waits of one thread, on a barrier that this CTA's threads and copies arrive on, and on one
// that the other CTA's do too.
__device__ __forceinline__ bool lane_wait(const RaggedParams& p, const Pair& c, uint32_t bar, uint32_t parity, uint32_t site) {
  return mbar_wait_bounded(bar, parity, p.budget, c.abort_flag) ? true : pair_fail(p, c, site);
}
__device__ __forceinline__ bool lane_wait_cluster(const RaggedParams& p, const Pair& c, uint32_t bar, uint32_t parity,
                                                  uint32_t site) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  while (!*c.abort_flag && static_cast<unsigned long long>(clock64() - t0) <= p.budget)
    if (mbar_try_wait_cluster(bar, parity)) return true;
  return pair_fail(p, c, site);
}
// The same of a whole warp: all lanes agree.
__device__ __forceinline__ bool warp_wait(const RaggedParams& p, const Pair& c, uint32_t bar, uint32_t parity, uint32_t site) {
  const bool got = mbar_wait_bounded(bar, parity, p.budget, c.abort_flag);
  return __all_sync(0xffffffffu, got) ? true : pair_fail(p, c, site);
}

struct Tile {
  int e, i0, valid, n_mma, n0;
  int rt;                                             // adapters: which tile of tokens
  bool live;
};

// first[e]: the units before segment e, for e = 0 .. E, in ascending order whatever the offsets are (a sum beyond
// what units are counted in is cut off, and what lies behind it has none). One warp.
__device__ __forceinline__ void count_units(const RaggedParams& p, const int* off, int* first, int lane) {
  long long base = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    const int rows = e < p.E ? max(off[e + 1] - off[e], 0) : 0;
    long long inc = static_cast<long long>((rows + NT - 1) / NT) * p.tiles_n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += up;
    }
    if (e < p.E) first[e + 1] = static_cast<int>(min(base + inc, static_cast<long long>(INT32_MAX / 2)));
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) first[0] = 0;
}

// Tile u. Token tiles of a segment are neighbours, so that the running pairs share W's columns. Whole warp.
template <bool SWIGLU, bool LORA>
__device__ __forceinline__ Tile find_tile(const RaggedParams& p, const int* off, const int* first, int u, int lane) {
  Tile t;
  unsigned ct;
  if (LORA) {
    const unsigned count = static_cast<unsigned>(p.R + p.lora_tile - 1) / static_cast<unsigned>(p.lora_tile);
    ct = u / count;
    t.rt = u - ct * count;
    t.i0 = t.rt * p.lora_tile;
    t.valid = min(p.lora_tile, p.R - t.i0);
    t.e = ct / static_cast<unsigned>(p.tiles_n);
    ct -= t.e * p.tiles_n;
    t.live = t.e < p.E;
  } else {
    t.e = 0;
    t.live = false;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const unsigned hit = __ballot_sync(0xffffffffu, e0 + lane < p.E && first[e0 + lane + 1] > u);
      if (hit != 0) {
        t.e = e0 + __ffs(hit) - 1;
        t.live = true;
        break;
      }
    }
    if (!t.live) return t;
    const int begin = off[t.e], rows = off[t.e + 1] - begin;
    const unsigned count = (rows + NT - 1) / NT, local = u - first[t.e];
    ct = local / count;
    const int rt = local - ct * count;
    const int steps = (rows + 31) / 32, each = static_cast<unsigned>(steps) / count, more = steps - each * count;
    const int from = 32 * (rt * each + min(rt, more));
    t.i0 = begin + from;
    t.valid = min(32 * (each + (rt < more ? 1 : 0)), rows - from);
  }
  t.n_mma = (t.valid + 31) & ~31;
  t.n0 = (p.tile0 + ct) * (SWIGLU ? 128 : 256);
  return t;
}

// Which groups of 32 rows of one CTA's half (rows first .. first + mine - 1 of the sorted order) lie side by
// side in x: bit g of the result, and the row of x that group g begins at. Whole warp.
__device__ __forceinline__ uint32_t runs_of_half(const RaggedParams& p, int first, int mine, int lane, int (&begin)[4]) {
  int r[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) r[g] = 32 * g + lane < mine ? ld_s32(p.row_index + first + 32 * g + lane) : 0;
  uint32_t runs = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    begin[g] = __shfl_sync(0xffffffffu, r[g], 0);
    const bool fits = 32 * g + lane >= mine || (r[g] == begin[g] + lane && r[g] >= 0 && r[g] < p.x_rows);
    if (__all_sync(0xffffffffu, fits) && 32 * g < mine) runs |= 1u << g;
  }
  return runs;
}

// Whether the stage that begins at k-block kb holds values of v.
__device__ __forceinline__ bool has_v(const RaggedParams& p, int kb, int total_kb) {
  return kb + KB > p.num_kb && total_kb > p.num_kb;
}

// Adapters: a tile's list as lora_tiles_kernel leaves it, [count, adapters ...] of LIST ints.
__device__ __forceinline__ const int32_t* tile_list(const RaggedParams& p, const Tile& t) {
  return p.lora_lists + static_cast<int64_t>(t.rt) * LORA_LIST;
}

template <bool SWIGLU, bool LORA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    ragged_pair_kernel(const __grid_constant__ RaggedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  Pair c;
  c.sW = smem;
  c.sX = smem + STAGES * OP_STAGE;
  float* staging = reinterpret_cast<float*>(smem + STAGES * 2 * OP_STAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * 2 * OP_STAGE + STAGING);
  c.full0 = smem_u32(bars);
  c.empty0 = c.full0 + 8 * STAGES;
  c.rows0 = c.empty0 + 8 * STAGES;
  c.go0 = c.rows0 + 8 * STAGES;
  c.accf0 = c.go0 + 8 * STAGES;
  c.acce0 = c.accf0 + 16;
  c.drain = c.acce0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 5);
  static_assert(4 * STAGES + 6 <= 32, "barriers and the TMEM slot");
  c.abort_flag = tmem_slot + 1;
  int* s_off = reinterpret_cast<int*>(bars + 32);
  int* s_first = s_off + TP_MAX_EXPERTS + 4;
  c.rank = cluster_ctarank();
  const bool gather = !LORA && p.row_index != nullptr;     // adapters: the tokens' own order
  if (threadIdx.x == 0) {
    prefetch_tmap(&p.tw);
    if (SWIGLU) prefetch_tmap(&p.tw2);
    if (LORA) prefetch_tmap(&p.tb);
    if (!gather) prefetch_tmap(&p.tx_box);
    prefetch_tmap(&p.tx_box32);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(c.full0 + 8 * s, gather || LORA ? 3 : 1);   // the leader's TMA thread, and a relay of each CTA
      mbar_init(c.rows0 + 8 * s, 32 * LOADERS);
      mbar_init(c.go0 + 8 * s, 1);
      mbar_init(c.empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(c.accf0 + 8 * a, 1);
      mbar_init(c.acce0 + 8 * a, 2 * EPI);           // epilogue warps of both CTAs
    }
    mbar_init(c.drain, 1);
    *c.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  // Up to here beside the kernel before, from here the next one beside this. Adapters: x, W and offsets are read without
  // that wait, from L2, which the call's own kernel before this one has made safe (see ragged.cu); all else, the writes above
  // all, comes behind it. (200 tokens, 4096 x 28672, rank 16: 70 us, waiting first 80; 4000 tokens, 4096 x 6144, rank 64: 274 and 279.)
  if (!LORA) wait_prerequisites();
  launch_dependents();
  const int segs = LORA ? p.L : p.E;
  for (int e = threadIdx.x; e <= segs; e += THREADS) {
    if constexpr (LORA) s_off[e] = min(max(ld_gpu_s32(p.offsets + e), 0), p.R);
    else s_off[e] = seg_bound(p.offsets, e, p.R);
  }
  if (!LORA) {
    __syncthreads();
    if (warp == 2) count_units(p, s_off, s_first, lane);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  c.full0_leader = mapa_shared(c.full0, 0);
  c.acce0_leader = mapa_shared(c.acce0, 0);
  const uint32_t tmem_base = *tmem_slot;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int per_adapter = LORA ? (p.rank + 15) / 16 : 1;
  bool mma_issued = false;
  int loaded = 0;                                    // warp 0: stages begun

  if (warp == 0) {
    // What a thread executes for one stage is on the critical path (some 5 cycles an instruction), so a
    // stage of whole k-blocks, which nearly all are, has a loop of its own with little else than its loads.
    const bool km = p.w_km;
    const int num_kb = p.num_kb;
    const uint32_t sw = smem_u32(c.sW), sx = smem_u32(c.sX);
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; ok; u += pairs) {
      const Tile t = find_tile<SWIGLU, LORA>(p, s_off, s_first, u, lane);
      if (!t.live) break;
      const int col = t.n0 + static_cast<int>(c.rank) * (SWIGLU ? 64 : 128), col2 = SWIGLU ? col : col + 64, e = t.e;
      const int nh = t.n_mma / 2, row0 = t.i0 + static_cast<int>(c.rank) * nh;
      // rows side by side: one box of 128 rows, or (a low tile) as many of 32 as it takes
      const bool whole = !gather && nh > 96;
      const int low = gather || whole ? 0 : (nh + 31) / 32;
      // gathered rows: groups that happen to lie side by side come by TMA all the same
      uint32_t runs = 0;
      int begin[4] = {0, 0, 0, 0};
      uint32_t x_both = whole ? 2 * HALF : 8192u * low;   // bytes of both CTAs
      if (gather) {
        const int other = t.i0 + static_cast<int>(c.rank ^ 1u) * nh;
        x_both = 4096u * __popc(runs_of_half(p, other, min(nh, t.i0 + t.valid - other), lane, begin));
        runs = runs_of_half(p, row0, min(nh, t.i0 + t.valid - row0), lane, begin);
        x_both += 4096u * __popc(runs);
      }
      if (lane == 0) {
        int chunks = LORA && u != pair ? ld_s32(tile_list(p, t)) * per_adapter : 0;
        auto load_kb = [&](int kb, uint32_t w, uint32_t x, uint32_t fb) {
          const int k0 = kb * BK;
          if (km) {
            tma_load_3d_pair(w, &p.tw, k0, col, e, fb);
          } else {
            tma_load_3d_pair(w, &p.tw, col, k0, e, fb);
            tma_load_3d_pair(w + BOX, SWIGLU ? &p.tw2 : &p.tw, col2, k0, e, fb);
          }
          if (whole) {
            tma_load_2d_pair(x, &p.tx_box, k0, row0, fb);
          } else {
            for (int b = 0; b < low; ++b) tma_load_2d_pair(x + 4096u * b, &p.tx_box32, k0, row0 + 32 * b, fb);
            if (runs != 0) {
#pragma unroll
              for (int g = 0; g < 4; ++g)
                if (runs >> g & 1) tma_load_2d_pair(x + 4096u * g, &p.tx_box32, k0, begin[g], fb);
            }
          }
        };
        const uint32_t stage_bytes = KB * (2 * HALF + x_both);
        int kb = 0;
        for (; kb + KB <= num_kb; kb += KB) {
          ok = lane_wait(p, c, c.empty0 + 8 * st, phase ^ 1u, WAIT_PRODUCER_EMPTY);
          if (!ok) break;
          if (c.rank == 0) {
            mbar_arrive_expect_tx(c.full0 + 8 * st, stage_bytes);     // of both CTAs
            if (LORA) mbar_arrive_n(c.full0 + 8 * st, 2);             // nothing for the relays
          }
#pragma unroll
          for (int h = 0; h < KB; ++h)
            load_kb(kb + h, sw + st * OP_STAGE + h * HALF, sx + st * OP_STAGE + h * HALF, c.full0_leader + 8 * st);
          ++loaded;
          if (++st == STAGES) { st = 0; phase ^= 1u; }
        }
        if (LORA && u == pair) {                                      // the first tile's adapters, behind its x and W
          wait_prerequisites();
          chunks = ld_s32(tile_list(p, t)) * per_adapter;
        }
        const int total_kb = num_kb + (chunks + 1) / 2;
        int chunk = 0;
        for (; ok && kb < total_kb; kb += KB) {                       // a last odd k-block, and adapters
          ok = lane_wait(p, c, c.empty0 + 8 * st, phase ^ 1u, WAIT_PRODUCER_EMPTY);
          if (!ok) break;
          const bool v = LORA && has_v(p, kb, total_kb);
          if (v) mbar_arrive(c.go0 + 8 * st);                         // the loaders may fill their part
          const uint32_t fb = c.full0_leader + 8 * st;
          uint32_t bytes = 0;
          for (int h = 0; h < KB; ++h) {
            if (kb + h < num_kb) bytes += 2 * HALF + x_both;
            else if (LORA && kb + h < total_kb) bytes += min(2, chunks - 2 * (kb + h - num_kb)) * 8192u;
          }
          if (c.rank == 0) {
            mbar_arrive_expect_tx(c.full0 + 8 * st, bytes);
            if (LORA && !v) mbar_arrive_n(c.full0 + 8 * st, 2);
          }
          for (int h = 0; h < KB; ++h) {
            const uint32_t w = sw + st * OP_STAGE + h * HALF, x = sx + st * OP_STAGE + h * HALF;
            if (kb + h < num_kb) {
              load_kb(kb + h, w, x, fb);
            } else if (LORA && kb + h < total_kb) {
              const int nch = min(2, chunks - 2 * (kb + h - num_kb));
              for (int ch = 0; ch < nch; ++ch, ++chunk) {
                const int a = ld_s32(tile_list(p, t) + 1 + chunk / per_adapter), r0 = chunk % per_adapter * 16;
                tma_load_3d_pair(w + ch * 2048u, &p.tb, col, r0, e * p.L + a, fb);
                tma_load_3d_pair(w + ch * 2048u + BOX, &p.tb, col + 64, r0, e * p.L + a, fb);
              }
            }
          }
          ++loaded;
          if (++st == STAGES) { st = 0; phase ^= 1u; }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
  } else if (warp == 1) {
    if (c.rank == 0) {
      // Descriptors (addresses in units of 16 bytes) of stage 0; a 16-deep step of W is 32 bytes or 16 rows further on.
      const bool km = p.w_km;
      const int num_kb = p.num_kb;
      const uint64_t w0 = smem_desc_sw128(smem_u32(c.sW), km ? 16u : BOX, 1024u), x0 = smem_desc_sw128(smem_u32(c.sX), 16u, 1024u);
      const uint32_t w_step = km ? 2u : 128u;
      int st = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = pair; ok; u += pairs) {
        const Tile t = find_tile<SWIGLU, LORA>(p, s_off, s_first, u, lane);
        if (!t.live) break;
        const uint32_t idesc = idesc_bf16_f32(256, t.n_mma, !km, false);
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc) * 256u;
        if (lane == 0) {
          int chunks = LORA && u != pair ? ld_s32(tile_list(p, t)) * per_adapter : 0;
          ok = lane_wait_cluster(p, c, c.acce0 + 8 * acc, acc_phase ^ 1u, WAIT_MMA_ACC_EMPTY);
          tc_fence_after();
          int kb = 0;
          for (; ok && kb + KB <= num_kb; kb += KB) {                 // whole stages, as in warp 0
            ok = lane_wait_cluster(p, c, c.full0 + 8 * st, phase, WAIT_MMA_FULL);
            if (!ok) break;
            tc_fence_after();
            const uint64_t w = w0 + st * (OP_STAGE >> 4), x = x0 + st * (OP_STAGE >> 4);
#pragma unroll
            for (int h = 0; h < KB; ++h)
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                umma_bf16_pair(d, w + h * (HALF >> 4) + k * w_step, x + h * (HALF >> 4) + k * 2, idesc, h != 0 || k != 0 || kb != 0 ? 1u : 0u);
            mma_issued = true;
            umma_commit_pair_mc(c.empty0 + 8 * st, 0x3);
            if (++st == STAGES) { st = 0; phase ^= 1u; }
          }
          if (LORA && u == pair) {                                    // as in warp 0
            wait_prerequisites();
            chunks = ld_s32(tile_list(p, t)) * per_adapter;
          }
          const int total_kb = num_kb + (chunks + 1) / 2;
          for (; ok && kb < total_kb; kb += KB) {                     // a last odd k-block, and adapters
            ok = lane_wait_cluster(p, c, c.full0 + 8 * st, phase, WAIT_MMA_FULL);
            if (!ok) break;
            tc_fence_after();
            for (int h = 0; h < KB; ++h) {
              const uint64_t w = w0 + ((st * OP_STAGE + h * HALF) >> 4), x = x0 + ((st * OP_STAGE + h * HALF) >> 4);
              if (kb + h < num_kb) {
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) umma_bf16_pair(d, w + k * w_step, x + k * 2, idesc, (kb + h) != 0 || k != 0 ? 1u : 0u);
              } else if (LORA && kb + h < total_kb) {
                const int nch = min(2, chunks - 2 * (kb + h - num_kb));
                for (int ch = 0; ch < nch; ++ch)      // hi and lo of each step against the same rows of B
                  for (int half = 0; half < 2; ++half) umma_bf16_pair(d, w + ch * 128, x + (ch + 2 * half) * 2, idesc, 1u);
              }
            }
            mma_issued = true;
            umma_commit_pair_mc(c.empty0 + 8 * st, 0x3);
            if (++st == STAGES) { st = 0; phase ^= 1u; }
          }
          if (ok) umma_commit_pair_mc(c.accf0 + 8 * acc, 0x3);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
    }
  } else if (warp < LOAD0) {
    // Two groups of four warps, one TMEM lane quadrant each, take the tile's rows 16 at a time in turn.
    const int quad = warp & 3, group = (warp - 2) >> 2;
    const int tid = (threadIdx.x - 64) & 127;
    float* stg = staging + group * CHUNK * STG_LD;
    constexpr int GROUPS = SWIGLU ? 8 : 16;           // eight columns each
    constexpr int ITEMS = CHUNK * GROUPS / 128;       // of a chunk, for each thread
    int acc = 0;
    uint32_t acc_phase = 0;
    if (LORA) wait_prerequisites();
    for (int u = pair;; u += pairs) {
      const Tile t = find_tile<SWIGLU, LORA>(p, s_off, s_first, u, lane);
      if (!t.live) break;
      const int col0 = t.n0 + static_cast<int>(c.rank) * (SWIGLU ? 64 : 128);
      const bool adapters = LORA && ld_s32(tile_list(p, t)) > 0;
      // h_pre of the group's next chunk is on its way while this one is finished (it comes from DRAM)
      uint4 h0[ITEMS], h1[ITEMS];
      auto fetch_h = [&](int j0) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
          const int it = tid + 128 * k, j = j0 + it / GROUPS, col = col0 + (it % GROUPS) * 8;
          if (j < t.valid && col < p.n) load_h_pre(p, t.i0 + j, col, h0[k], h1[k]);
        }
      };
      if (!SWIGLU && !LORA && p.backward) fetch_h(group * CHUNK);
      int got = warp_wait(p, c, c.accf0 + 8 * acc, acc_phase, WAIT_EPI_ACC_FULL) ? 1 : 0;
      // all warps go on, or none
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.s32 p, %0, 0;\n\t"
          "barrier.cta.red.and.pred q, 3, 256, p;\n\t"
          "selp.s32 %0, 1, 0, q;\n\t}\n"
          : "+r"(got)::"memory");
      if (!got) break;
      tc_fence_after();
      const uint32_t tm = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * 256);
      bool held = true;
      for (int j0 = group * CHUNK; j0 < t.valid; j0 += 2 * CHUNK) {
        int sorted[ITEMS];                            // adapters: on their way before they are needed
        if constexpr (LORA) {
#pragma unroll
          for (int k = 0; k < ITEMS; ++k) {
            const int j = j0 + (tid + 128 * k) / GROUPS;
            sorted[k] = j < t.valid ? ld_s32(p.lora_pos + t.i0 + j) : -2;
          }
        }
        uint32_t v[CHUNK];
        tmem_ld16(tm + j0, v);
        tmem_ld_wait();
        if (j0 + 2 * CHUNK >= t.valid) {              // this warp's part is read: the next tile may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(c.acce0_leader + 8 * acc);
          held = false;
        }
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) stg[j * STG_LD + quad * 32 + lane] = __uint_as_float(v[j]);
        asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
        float4 f4[ITEMS][2], u4[ITEMS][2];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
          const int it = tid + 128 * k;
          const float4* src = reinterpret_cast<const float4*>(stg + (it / GROUPS) * STG_LD + (it % GROUPS) * 8);
          f4[k][0] = src[0];
          f4[k][1] = src[1];
          u4[k][0] = SWIGLU ? src[16] : src[0];
          u4[k][1] = SWIGLU ? src[17] : src[1];
        }
        asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
        uint4 g0[ITEMS], g1[ITEMS];
        if (!SWIGLU && !LORA && p.backward) {
#pragma unroll
          for (int k = 0; k < ITEMS; ++k) {
            g0[k] = h0[k];
            g1[k] = h1[k];
          }
          fetch_h(j0 + 2 * CHUNK);
        }
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
          const int it = tid + 128 * k;
          const int j = j0 + it / GROUPS, col = col0 + (it % GROUPS) * 8;
          if (j >= t.valid || col >= p.n) continue;
          float f[8] = {f4[k][0].x, f4[k][0].y, f4[k][0].z, f4[k][0].w, f4[k][1].x, f4[k][1].y, f4[k][1].z, f4[k][1].w};
          float up[8] = {u4[k][0].x, u4[k][0].y, u4[k][0].z, u4[k][0].w, u4[k][1].x, u4[k][1].y, u4[k][1].z, u4[k][1].w};
          const int i = t.i0 + j;
          if (!SWIGLU && !LORA && p.backward) {
            store_backward8(p, i, col, f, g0[k], g1[k]);
            continue;
          }
          if (!LORA && p.seg_scale != nullptr) {
            const float sc = ld_f32(p.seg_scale + t.e);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] *= sc;
          }
          if constexpr (LORA) {
            if (sorted[k] < -1) continue;
            if (adapters) lora_settle8(p, s_off, t.e, i, sorted[k], col, f);
            store_row8(p, static_cast<int64_t>(t.e) * p.R + i, col, f, up);
          } else {
            store_row8(p, i, col, f, up);
          }
        }
      }
      if (held) {                                     // a low tile: the other group had all of it
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(c.acce0_leader + 8 * acc);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  } else if ((gather || LORA) && warp < RELAY0) {
    // Row loaders: eight lanes copy one row's 128 bytes of a k-block. The copies arrive on this CTA's
    // barrier when they have landed.
    const int tid = threadIdx.x - 32 * LOAD0;
    constexpr int STEP = LOADERS * 4;                  // rows of one pass
    const int piece = tid & 7, r0 = tid >> 3;
    const uint32_t line0 = smem_u32(c.sX) + r0 * 128 + ((piece ^ (r0 & 7)) << 4);   // (STEP is a multiple of 8)
    const int v_row = tid >> 1;                        // adapters: two threads build one row of 32 values
    if (LORA) wait_prerequisites();
    int st = 0;
    uint32_t phase = 0, go_phase = 0;                  // go_phase: one bit per stage
    bool ok = true;
    for (int u = pair; ok; u += pairs) {
      const Tile t = find_tile<SWIGLU, LORA>(p, s_off, s_first, u, lane);
      if (!t.live) break;
      const int nh = t.n_mma / 2, half0 = static_cast<int>(c.rank) * nh;
      const int mine = min(nh, t.valid - half0);       // rows that this CTA fetches (may be <= 0)
      const uint16_t* src[128 / STEP];                 // this thread's piece of its rows, at k = 0
      uint32_t mine_bits = 0, in_bits = 0;             // rows that it fetches, and those of them that lie in x (others: zeros)
      if (!LORA) {
        int begin[4];
        const uint32_t runs = runs_of_half(p, t.i0 + half0, mine, lane, begin);   // come by TMA
#pragma unroll
        for (int i = 0; i < 128 / STEP; ++i) {
          const int row = r0 + STEP * i;               // (no row: left as it is, its column is not read)
          src[i] = p.x;
          if (row < mine && !(runs >> (row >> 5) & 1)) {
            const int r = ld_s32(p.row_index + t.i0 + half0 + row);
            mine_bits |= 1u << i;
            if (r >= 0 && r < p.x_rows) {
              in_bits |= 1u << i;
              src[i] = p.x + static_cast<int64_t>(r) * p.K + piece * 8;
            }
          }
        }
      }
      if constexpr (LORA) {
        // Only the stages that hold values of v are theirs. They may be far ahead of the others or behind them,
        // so that a parity of the stages' own barriers would say nothing: the TMA thread lets them go.
        const int pos = v_row < mine ? ld_s32(p.lora_pos + t.i0 + half0 + v_row) : -1;   // the token's v, or -1
        const int chunks = ld_s32(tile_list(p, t)) * per_adapter;
        const int total_kb = p.num_kb + (chunks + 1) / 2;
        int chunk = 0;
        for (int kb = 0; kb < total_kb; kb += KB) {
          if (has_v(p, kb, total_kb)) {
            uint4 hi[2 * KB], lo[2 * KB];              // loaded before the slot is waited for
#pragma unroll
            for (int i = 0; i < 2 * KB; ++i) {
              hi[i] = lo[i] = make_uint4(0, 0, 0, 0);
              if (kb + i / 2 < p.num_kb || chunk >= chunks) continue;
              const int a = ld_s32(tile_list(p, t) + 1 + chunk / per_adapter), k0 = chunk % per_adapter * 16 + (tid & 1) * 8;
              if (pos >= 0 && pos >= s_off[a] && pos < s_off[a + 1] && k0 < p.rank)
                split_bf8(p.v + static_cast<int64_t>(pos) * p.rank + k0, hi[i], lo[i]);
              ++chunk;
            }
            ok = warp_wait(p, c, c.go0 + 8 * st, (go_phase >> st) & 1u, WAIT_PRODUCER_EMPTY);
            if (!ok) break;
            go_phase ^= 1u << st;
#pragma unroll
            for (int h = 0; h < KB; ++h) {
              if (kb + h < p.num_kb || v_row >= nh) continue;
              uint8_t* line = c.sX + st * OP_STAGE + h * HALF + v_row * 128;
#pragma unroll
              for (int ch = 0; ch < 2; ++ch) {
                const int pc = 2 * ch + (tid & 1);
                *reinterpret_cast<uint4*>(line + ((pc ^ (v_row & 7)) << 4)) = hi[2 * h + ch];
                *reinterpret_cast<uint4*>(line + (((pc + 4) ^ (v_row & 7)) << 4)) = lo[2 * h + ch];
              }
            }
            mbar_arrive(c.rows0 + 8 * st);
          }
          if (++st == STAGES) st = 0;
        }
      } else {
        for (int kb = 0; kb < p.num_kb; kb += KB) {
          ok = warp_wait(p, c, c.empty0 + 8 * st, phase ^ 1u, WAIT_PRODUCER_EMPTY);
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < KB; ++h) {
            if (kb + h >= p.num_kb) break;
            const uint32_t x = line0 + st * OP_STAGE + h * HALF;
            const int k0 = (kb + h) * BK;
            const uint32_t in = k0 + piece * 8 < p.K ? in_bits : 0u;
#pragma unroll
            for (int i = 0; i < 128 / STEP; ++i)
              if (mine_bits >> i & 1) cp_async16(x + i * STEP * 128, in >> i & 1 ? src[i] + k0 : p.x, in >> i & 1 ? 16u : 0u);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(c.rows0 + 8 * st) : "memory");
          if (++st == STAGES) { st = 0; phase ^= 1u; }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (gather || LORA) {
    // Relays: what the loaders wrote is ordered before the tensor cores' reads and passed on to the leader's
    // barrier. A slot has one relay, which waits for each of its uses: one that skipped some could take a
    // phase's parity for the next one's. (The loaders cannot do it themselves: a release to the other CTA
    // waits for every copy that its thread has in flight.)
    const int mine = warp - RELAY0;
    if (LORA) wait_prerequisites();
    int st = 0;
    uint32_t used_phase = 0;                           // one bit per stage
    bool ok = true;
    for (int u = pair; ok; u += pairs) {
      const Tile t = find_tile<SWIGLU, LORA>(p, s_off, s_first, u, lane);
      if (!t.live) break;
      const int chunks = LORA ? ld_s32(tile_list(p, t)) * per_adapter : 0;
      const int total_kb = p.num_kb + (chunks + 1) / 2;
      if (lane == 0) {
        for (int kb = 0; kb < total_kb; kb += KB) {
          const bool used = !LORA || has_v(p, kb, total_kb);     // a stage without values of v is not passed on
          if (used && st % RELAYS == mine) {
            ok = lane_wait(p, c, c.rows0 + 8 * st, (used_phase >> st) & 1u, WAIT_MMA_FULL);
            if (!ok) break;
            fence_proxy_async();
            if (c.rank == 0) mbar_arrive(c.full0 + 8 * st);
            else mbar_arrive_cluster(c.full0_leader + 8 * st);
          }
          if (used) used_phase ^= 1u << st;
          if (++st == STAGES) st = 0;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
  }
  // all pair MMAs done, then both CTAs meet before either frees TMEM or exits. After a wait that ran
  // out, the copies still in flight land first (they count on the leader's barriers).
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*c.abort_flag != 0u && warp == 0 && lane == 0 && c.rank == 0) {
    for (int s = 0; s < STAGES; ++s) {
      const int uses = (loaded - s + STAGES - 1) / STAGES;
      if (uses > 0 && !mbar_wait_bounded(c.full0 + 8 * s, (uses - 1) & 1, DRAIN, nullptr)) record_timeout(p.status, WAIT_TEARDOWN);
    }
  }
  if (warp == 1 && lane == 0 && c.rank == 0 && mma_issued) {
    umma_commit_pair(c.drain);
    if (!mbar_wait_bounded(c.drain, 0, 4000000000ull, nullptr)) record_timeout(p.status, WAIT_TEARDOWN);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// A warp copies one row, four 16-byte pieces a lane in flight.
__global__ void __launch_bounds__(256) gather_rows_kernel(const uint16_t* x, int x_rows, const int32_t* row_index, const int32_t* offsets,
                                                          int E, int R, int K, uint16_t* dst, int64_t ld) {
  const int lane = threadIdx.x % 32;
  const int i = blockIdx.x * 8 + threadIdx.x / 32;
  wait_prerequisites();
  launch_dependents();
  if (i >= R) return;
  bool in_segment = false;                             // other rows are left as they were
  for (int e0 = 0; e0 < E && !in_segment; e0 += 32) {
    const int e = e0 + lane;
    in_segment = __any_sync(0xffffffffu, e < E && seg_bound(offsets, e, R) <= i && i < seg_bound(offsets, e + 1, R));
  }
  if (!in_segment) return;
  const int r = ld_s32(row_index + i);
  const bool in = r >= 0 && r < x_rows;
  const uint16_t* src = x + static_cast<int64_t>(in ? r : 0) * K;
  uint16_t* to = dst + i * ld;
  for (int k0 = lane * 8; k0 < K; k0 += 4 * 256) {
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = in && k0 + 256 * q < K ? ld_stream_v4(src + k0 + 256 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (k0 + 256 * q < K) st_v4(to + k0 + 256 * q, v[q]);
  }
}

template <bool SWIGLU, bool LORA>
tp_status launch_pair(const RaggedParams& p, int64_t units, cudaStream_t s) {
  static int configured_for[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(TP_ECUDA, "cudaGetDevice failed");
  if (dev < 0 || dev >= 64 || !configured_for[dev]) {
    if (cudaFuncSetAttribute(ragged_pair_kernel<SWIGLU, LORA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(SMEM)) != cudaSuccess)
      return fail(TP_ECUDA, "cannot reserve %zu bytes of shared memory", SMEM);
    if (dev >= 0 && dev < 64) configured_for[dev] = 1;
  }
  const int sms = sm_count();
  int grid = 2 * units < sms ? static_cast<int>(2 * units) : (sms & ~1);
  if (grid < 2) grid = 2;
  return launch_beside("ragged_pair_kernel", ragged_pair_kernel<SWIGLU, LORA>, grid, THREADS, SMEM, s, p);
}

}  // namespace

tp_status gather_rows(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const int32_t* offsets, int E, int64_t R, int64_t K,
                      uint16_t* dst, int64_t ld, cudaStream_t s) {
  return launch_beside("gather_rows_kernel", gather_rows_kernel, static_cast<unsigned>((R + 7) / 8), 256, 0, s, x, static_cast<int>(x_rows),
                       row_index, offsets, E, static_cast<int>(R), static_cast<int>(K), dst, ld);
}

tp_status ragged_pairs(RaggedParams& p, bool swiglu, bool lora, int64_t row_tiles, cudaStream_t s) {
  const int64_t units = row_tiles * p.tiles_n * (lora ? p.E : 1);
  if (units > INT32_MAX / 2) return fail(TP_ESHAPE, "too many tiles");
  if (lora) return launch_pair<false, true>(p, units, s);
  return swiglu ? launch_pair<true, false>(p, units, s) : launch_pair<false, false>(p, units, s);
}

}  // namespace tpx
