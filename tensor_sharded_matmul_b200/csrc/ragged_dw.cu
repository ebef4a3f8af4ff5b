// Weight gradients over ragged segments: dW_e = sum over the rows i of segment e of x[row_i]^T dy_i.
//
// Here the ragged dimension is the contraction. CTA pairs (tcgen05 cta_group::2) compute 256 x 256 tiles
// of dW_e, each CTA holding 128 of x's columns and 128 of dy's per 64-row k-block; both operands are
// M-major as they lie in memory. Whole k-blocks come by TMA; gathered rows of x by cp.async (see
// ragged_pair.cu). A segment's last, partial k-block is put together from boxes of 32, 16, .. 1 rows, and the
// rest of the tile from boxes past the end of the matrix, which TMA reads as zeros (cp.async: its zero
// fill): in both operands, so that a neighbour's rows (whatever they hold) never enter. (Single rows
// alone, 256 loads of about 75 cycles, cost more than the product of a small segment.)
//
// Tensor cores add each K=16 step to the accumulator with truncation: over a long contraction the
// sum is short by about K / 32 times 2^-24 of itself (measured 4.4e-6 at K = 4096, 1.9e-5 at 16384).
// A tile is therefore accumulated in spans of at most 512 rows, alternating between the two TMEM
// accumulators; the epilogue warps add the spans in binary32, round-to-nearest, in registers (span
// order, so results do not depend on timing). An empty segment writes zeros.
#include <cstring>

#include "ragged.cuh"
#include "tmap.cuh"

namespace tpx {
namespace {

constexpr int BK = 64;
constexpr int KB = 2;                                // k-blocks per stage
constexpr int STAGES = 3;
constexpr uint32_t HALF = 128 * BK * 2;              // one k-block of one operand of this CTA: 16 KiB
constexpr uint32_t BOX = 64 * BK * 2;                // 64 columns x 64 rows: 8 KiB
constexpr uint32_t OP_STAGE = KB * HALF;             // 32 KiB
constexpr uint32_t TMEM_COLS = 512;
constexpr int SPAN_KB = 8;                           // k-blocks per accumulator span (512 rows)
constexpr int LOADERS = 4;                           // warps that copy gathered rows
// TMA and MMA warps, two relays (gathered rows), eight epilogue warps, the loaders.
template <bool GATHER>
constexpr int EPI0 = GATHER ? 4 : 2;
template <bool GATHER>
constexpr int THREADS = 32 * (EPI0<GATHER> + 8 + (GATHER ? LOADERS : 0));
constexpr uint32_t STG_WARP = 32 * 128;
constexpr size_t SMEM = 1024 + STAGES * 2 * OP_STAGE + 8 * STG_WARP + 256;

struct DwParams {
  CUtensorMap tx[7];           // x [x_rows][k]: boxes of 64 columns, 64 >> i rows high
  CUtensorMap td[7];           // dy [R][n]
  CUtensorMap tdw;             // dw [E][k][n], 32 x 32 boxes
  const int32_t* offsets;
  const int32_t* row_index;
  const uint16_t* x;
  int R, x_rows, E, k, n, tiles_k, tiles_n, units;
  bool out_f32;
  uint32_t* status;
  unsigned long long budget;
};

struct Dw {
  uint8_t *sA, *sB;
  uint32_t full0, empty0, rows0, accf0, acce0, drain, full0_leader, acce0_leader;
  volatile uint32_t* abort_flag;
  uint32_t rank;
};

__device__ __forceinline__ bool dw_fail(const DwParams& p, const Dw& c, uint32_t site) {
  if (!*c.abort_flag) record_timeout(p.status, site);
  *c.abort_flag = 1u;
  return false;
}

// One 64-row k-block of one operand by TMA (this CTA's 128 columns from x0): rows r0 .. r0 + v - 1, and
// zeros for the other rows of the tile (a box past the matrix, from row `limit` on, reads as zeros). Two
// lanes, 64 columns each; always counts 16 KiB. A partial block is put together from boxes of falling
// height, at most seven a lane.
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* maps, int limit, int x0, int r0, int v,
                                             uint32_t fb, int lane) {
  if (lane >= 2) return;
  const int x = x0 + 64 * lane;
  dst += lane * BOX;
  if (v == BK) {
    tma_load_2d_pair(dst, maps, x, r0, fb);
    return;
  }
  for (int part = 0, at = 0; part < 2; ++part) {
    const int rows = part == 0 ? v : BK - v;
    for (int i = 1; i < 7; ++i) {
      const int high = BK >> i;
      if (rows & high) {
        tma_load_2d_pair(dst + at * 128u, maps + i, x, part == 0 ? r0 + at : limit, fb);
        at += high;
      }
    }
  }
}

template <bool GATHER>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS<GATHER>, 1)
    ragged_dw_kernel(const __grid_constant__ DwParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  Dw c;
  c.sA = smem;
  c.sB = smem + STAGES * OP_STAGE;
  const uint32_t staging0 = smem_u32(smem + STAGES * 2 * OP_STAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * 2 * OP_STAGE + 8 * STG_WARP);
  c.full0 = smem_u32(bars);
  c.empty0 = c.full0 + 8 * STAGES;
  c.rows0 = c.empty0 + 8 * STAGES;
  c.accf0 = c.rows0 + 8 * STAGES;
  c.acce0 = c.accf0 + 16;
  c.drain = c.acce0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * STAGES + 5);
  c.abort_flag = tmem_slot + 1;
  c.rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    if (!GATHER) prefetch_tmap(&p.tx[0]);
    prefetch_tmap(&p.td[0]);
    prefetch_tmap(&p.tdw);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(c.full0 + 8 * s, GATHER ? 3 : 1);   // the leader's TMA warp, and a relay of each CTA
      mbar_init(c.rows0 + 8 * s, 32 * LOADERS);
      mbar_init(c.empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(c.accf0 + 8 * a, 1);
      mbar_init(c.acce0 + 8 * a, 16);           // epilogue warps of both CTAs
    }
    mbar_init(c.drain, 1);
    *c.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  wait_prerequisites();
  launch_dependents();
  c.full0_leader = mapa_shared(c.full0, 0);
  c.acce0_leader = mapa_shared(c.acce0, 0);
  const uint32_t tmem_base = *tmem_slot;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int per_seg = p.tiles_k * p.tiles_n;
  bool mma_issued = false;
  int loaded = 0;                               // warp 0: stages filled

  auto produce = [&]() {
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; ok && u < p.units; u += pairs) {
      const int e = u / per_seg, local = u - e * per_seg;
      const int a0 = (local % p.tiles_k) * 256 + static_cast<int>(c.rank) * 128;
      const int b0 = (local / p.tiles_k) * 256 + static_cast<int>(c.rank) * 128;
      const int begin = seg_bound(p.offsets, e, p.R), end = seg_bound(p.offsets, e + 1, p.R);
      for (int r = begin; r < end; r += KB * BK) {
        ok = mbar_wait_bounded(c.empty0 + 8 * st, phase ^ 1u, p.budget, c.abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          dw_fail(p, c, WAIT_PRODUCER_EMPTY);
          break;
        }
        const uint32_t fb = c.full0_leader + 8 * st;
        if (lane == 0 && c.rank == 0) mbar_arrive_expect_tx(c.full0 + 8 * st, (end - r > BK ? 4 : 2) * (GATHER ? 1 : 2) * HALF);   // of both CTAs
        __syncwarp();
#pragma unroll
        for (int h = 0; h < KB; ++h) {
          const int r0 = r + h * BK, v = min(BK, end - r0);
          if (v <= 0) break;                    // not multiplied either
          const uint32_t off = st * OP_STAGE + h * HALF;
          if (!GATHER) load_operand(smem_u32(c.sA + off), p.tx, p.x_rows, a0, r0, v, fb, lane);
          load_operand(smem_u32(c.sB + off), p.td, p.R, b0, r0, v, fb, lane);
        }
        ++loaded;
        if (++st == STAGES) { st = 0; phase ^= 1u; }
      }
    }
  };
  auto multiply = [&]() {
    if (lane == 0 && c.rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(256, 256, true, true);
      int st = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < p.units; u += pairs) {
        const int e = u / per_seg;
        const int rows = seg_bound(p.offsets, e + 1, p.R) - seg_bound(p.offsets, e, p.R);
        const int num_kb = rows > 0 ? (rows + BK - 1) / BK : 0;
        for (int kb = 0; ok && kb < num_kb; kb += KB) {
          const int in_span = kb % SPAN_KB;
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc) * 256u;
          if (in_span == 0) {
            bool got = mbar_try_wait_cluster(c.acce0 + 8 * acc, acc_phase ^ 1u);
            const long long t0 = clock64();
            while (!got && !*c.abort_flag && static_cast<unsigned long long>(clock64() - t0) <= p.budget)
              got = mbar_try_wait_cluster(c.acce0 + 8 * acc, acc_phase ^ 1u);
            if (!got) { ok = dw_fail(p, c, WAIT_MMA_ACC_EMPTY); break; }
            tc_fence_after();
          }
          {
            bool got = mbar_try_wait_cluster(c.full0 + 8 * st, phase);
            const long long t0 = clock64();
            while (!got && !*c.abort_flag && static_cast<unsigned long long>(clock64() - t0) <= p.budget)
              got = mbar_try_wait_cluster(c.full0 + 8 * st, phase);
            if (!got) { ok = dw_fail(p, c, WAIT_MMA_FULL); break; }
          }
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < KB; ++h) {
            if (kb + h < num_kb) {
              const uint32_t a = smem_u32(c.sA + st * OP_STAGE + h * HALF);
              const uint32_t b = smem_u32(c.sB + st * OP_STAGE + h * HALF);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                umma_bf16_pair(d, smem_desc_sw128(a + 2048u * k, BOX, 1024u), smem_desc_sw128(b + 2048u * k, BOX, 1024u),
                               idesc, (in_span + h) != 0 || k != 0 ? 1u : 0u);
            }
          }
          mma_issued = true;
          umma_commit_pair_mc(c.empty0 + 8 * st, 0x3);
          if (++st == STAGES) { st = 0; phase ^= 1u; }
          if (in_span + KB >= SPAN_KB || kb + KB >= num_kb) {
            umma_commit_pair_mc(c.accf0 + 8 * acc, 0x3);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
          }
        }
      }
    }
  };
  auto relay = [&]() {
    // Relays, each with slots of its own (see ragged_pair.cu): the loaders' copies are ordered before the tensor cores' reads and passed
    // on to the leader's barrier.
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < p.units; u += pairs) {
        const int e = u / per_seg;
        const int begin = seg_bound(p.offsets, e, p.R), end = seg_bound(p.offsets, e + 1, p.R);
        for (int r = begin; r < end; r += KB * BK) {
          if (2 + st % 2 == warp) {
            if (!mbar_wait_bounded(c.rows0 + 8 * st, phase, p.budget, c.abort_flag)) {
              ok = dw_fail(p, c, WAIT_MMA_FULL);
              break;
            }
            fence_proxy_async();
            if (c.rank == 0) mbar_arrive(c.full0 + 8 * st);
            else mbar_arrive_cluster(c.full0_leader + 8 * st);
          }
          if (++st == STAGES) { st = 0; phase ^= 1u; }
        }
      }
    }
  };
  auto load_rows = [&]() {
    // Row loaders: sixteen lanes copy one row's 256 bytes of this CTA's columns, zeros for rows past the
    // segment and for indices outside x. The copies arrive on this CTA's barrier when they have landed.
    const int tid = threadIdx.x - 32 * (EPI0<GATHER> + 8);
    constexpr int STEP = 2 * LOADERS;                 // rows of one pass
    const int piece = tid & 15, row0 = tid >> 4;
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; ok && u < p.units; u += pairs) {
      const int e = u / per_seg, local = u - e * per_seg;
      const int col = (local % p.tiles_k) * 256 + static_cast<int>(c.rank) * 128 + piece * 8;
      const int begin = seg_bound(p.offsets, e, p.R), end = seg_bound(p.offsets, e + 1, p.R);
      for (int r = begin; r < end; r += KB * BK) {
        int idx[KB][BK / STEP];
#pragma unroll
        for (int h = 0; h < KB; ++h)
#pragma unroll
          for (int i = 0; i < BK / STEP; ++i) {
            const int at = r + h * BK + row0 + STEP * i;
            idx[h][i] = at < end ? ld_s32(p.row_index + at) : -1;
          }
        ok = mbar_wait_bounded(c.empty0 + 8 * st, phase ^ 1u, p.budget, c.abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          dw_fail(p, c, WAIT_PRODUCER_EMPTY);
          break;
        }
        const uint32_t dst = smem_u32(c.sA + st * OP_STAGE) + (piece >> 3) * BOX;
#pragma unroll
        for (int h = 0; h < KB; ++h) {
          if (r + h * BK >= end) break;               // not multiplied either
#pragma unroll
          for (int i = 0; i < BK / STEP; ++i) {
            const int row = row0 + STEP * i;
            const bool in = idx[h][i] >= 0 && idx[h][i] < p.x_rows && col < p.k;
            const uint16_t* src = in ? p.x + static_cast<int64_t>(idx[h][i]) * p.k + col : p.x;
            cp_async16(dst + h * HALF + row * 128 + (((piece & 7) ^ (row & 7)) << 4), src, in ? 16u : 0u);
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(c.rows0 + 8 * st) : "memory");
        if (++st == STAGES) { st = 0; phase ^= 1u; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  };
  auto epilogue = [&]() {
    // Epilogue: TMEM lane quadrant = warp % 4 (rows of dW); the first four warps the left 128 columns, the
    // others the right. Each thread holds the running sums of one row's 128 columns.
    const int quad = warp & 3, half = (warp - EPI0<GATHER>) >> 2;
    const uint32_t stg = staging0 + static_cast<uint32_t>(warp - EPI0<GATHER>) * STG_WARP;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    float sum[4][32];
    for (int u = pair; ok && u < p.units; u += pairs) {
      const int e = u / per_seg, local = u - e * per_seg;
      const int row0 = (local % p.tiles_k) * 256 + static_cast<int>(c.rank) * 128 + quad * 32;
      const int col0 = (local / p.tiles_k) * 256 + half * 128;
      const int rows = seg_bound(p.offsets, e + 1, p.R) - seg_bound(p.offsets, e, p.R);
      const int spans = rows > 0 ? (rows + SPAN_KB * BK - 1) / (SPAN_KB * BK) : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[q][i] = 0.0f;
      for (int s = 0; s < spans; ++s) {
        if (!mbar_wait_bounded(c.accf0 + 8 * acc, acc_phase, p.budget, c.abort_flag)) {
          ok = dw_fail(p, c, WAIT_EPI_ACC_FULL);
          break;
        }
        tc_fence_after();
        const uint32_t t = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * 256 + half * 128);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t v[16];
          tmem_ld16(t + q * 16, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sum[q / 2][(q % 2) * 16 + i] = __fadd_rn(sum[q / 2][(q % 2) * 16 + i], __uint_as_float(v[i]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(c.acce0_leader + 8 * acc);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (!ok) break;
      // 32 x 32 blocks, one row a lane, swizzled into this warp's staging buffer and stored by TMA, which
      // leaves out what lies outside dW_e. (16-byte stores from the threads held the kernel at 446
      // TFLOP/s where it runs at 1032 without any, at 64 experts of 384 rows, 1024 x 2048.)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bulk_wait_read();                          // lane 0: the last block has left the buffer
        __syncwarp();
        if (p.out_f32) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(stg + lane * 128 + ((j ^ (lane & 7)) << 4)),
                         "f"(sum[q][4 * j]), "f"(sum[q][4 * j + 1]), "f"(sum[q][4 * j + 2]), "f"(sum[q][4 * j + 3])
                         : "memory");
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)),
                         "r"(pack_bf2(sum[q][8 * j], sum[q][8 * j + 1])), "r"(pack_bf2(sum[q][8 * j + 2], sum[q][8 * j + 3])),
                         "r"(pack_bf2(sum[q][8 * j + 4], sum[q][8 * j + 5])), "r"(pack_bf2(sum[q][8 * j + 6], sum[q][8 * j + 7]))
                         : "memory");
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && row0 < p.k && col0 + q * 32 < p.n) {
          tma_store_3d(&p.tdw, stg, col0 + q * 32, row0, e);
          bulk_commit();
        }
      }
    }
    bulk_wait();
  };
  if constexpr (GATHER) {
    // The running sums take 128 registers a thread; these 512 threads start at 128 each, and
    // 256 * 168 + 256 * 56 = 57344 of the 65536 are asked for.
    if (warp >= 4 && warp < 12) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      epilogue();
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp == 0) produce();
      else if (warp == 1) multiply();
      else if (warp < 4) relay();
      else load_rows();
    }
  } else {
    if (warp == 0) produce();
    else if (warp == 1) multiply();
    else epilogue();
  }
  // all pair MMAs done, then both CTAs meet before either frees TMEM or exits. After a wait that ran
  // out, the copies still in flight land first (they count on the leader's barriers).
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*c.abort_flag != 0u && warp == 0 && lane == 0 && c.rank == 0) {
    for (int s = 0; s < STAGES; ++s) {
      const int uses = (loaded - s + STAGES - 1) / STAGES;
      if (uses > 0 && !mbar_wait_bounded(c.full0 + 8 * s, (uses - 1) & 1, 400000000ull, nullptr))
        record_timeout(p.status, WAIT_TEARDOWN);
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

template <bool GATHER>
tp_status launch_dw(const DwParams& p, cudaStream_t s) {
  static int configured_for[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(TP_ECUDA, "cudaGetDevice failed");
  if (dev < 0 || dev >= 64 || !configured_for[dev]) {
    if (cudaFuncSetAttribute(ragged_dw_kernel<GATHER>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM)) !=
        cudaSuccess)
      return fail(TP_ECUDA, "cannot reserve %zu bytes of shared memory", SMEM);
    if (dev >= 0 && dev < 64) configured_for[dev] = 1;
  }
  const int sms = sm_count();
  int grid = 2 * static_cast<int64_t>(p.units) < sms ? 2 * p.units : (sms & ~1);
  if (grid < 2) grid = 2;
  return launch_beside("ragged_dw_kernel", ragged_dw_kernel<GATHER>, grid, THREADS<GATHER>, SMEM, s, p);
}

}  // namespace

tp_status ragged_dw(const RaggedDwArgs& g, cudaStream_t s) {
  DwParams p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = g.offsets; p.row_index = g.row_index; p.x = g.x;
  p.R = static_cast<int>(g.R); p.x_rows = static_cast<int>(g.x_rows);
  p.E = g.E; p.k = static_cast<int>(g.k); p.n = static_cast<int>(g.n);
  p.tiles_k = (p.k + 255) / 256;
  p.tiles_n = (p.n + 255) / 256;
  const int64_t units = static_cast<int64_t>(g.E) * p.tiles_k * p.tiles_n;
  if (units > INT32_MAX / 2) return fail(TP_ESHAPE, "too many tiles");
  p.units = static_cast<int>(units);
  p.out_f32 = g.out_f32;
  for (int i = 0; i < 7; ++i)
    if ((g.row_index == nullptr && !encode_bf16_2d(&p.tx[i], g.x, g.k, g.x_rows, g.k, 64, 64 >> i)) ||
        !encode_bf16_2d(&p.td[i], g.dy, g.n, g.R, g.n, 64, 64 >> i))
      return fail(TP_ECUDA, "cannot encode the TMA descriptors");
  if (!encode_out_3d(&p.tdw, g.dw, g.out_f32, g.n, g.k, g.E)) return fail(TP_ECUDA, "cannot encode the TMA descriptor of dW");
  p.status = status_word();
  p.budget = wait_budget();
  if (p.status == nullptr) return fail(TP_ECUDA, "cannot resolve the device status word");
  return g.row_index != nullptr ? launch_dw<true>(p, s) : launch_dw<false>(p, s);
}

}  // namespace tpx
