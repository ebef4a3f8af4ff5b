// Matrix products over ragged segments of rows: y_i = epilogue(x[row_i] W_e) for the rows i of every
// segment e, the segments known on the device alone (an expert's tokens, an adapter's tokens).
//
// The product is computed transposed, D^T = W_e^T x^T: 128 columns of W are the M of
// tcgen05.mma and the segment's rows are its N, which is chosen for each tile in steps of 16. A
// segment's last tile so costs what its rows cost, and a decode step's few rows need no padding to
// 128. W as stored ([K][n], n contiguous) is the M-major operand, the rows of x the K-major one; both
// come by TMA: x's rows in boxes where they lie side by side, up to 16 gathered rows four at a time by index
// (tile::gather4); of more, four warps copy them with cp.async. One CTA computes one tile: warp 0 loads, one
// thread of warp 1 issues the MMAs, all warps write the output rows. What bounds it: the bytes of W (8 experts of
// four rows, 4096 x 14336: 0.94 GB in 140 us; two experts of one token, SwiGLU, 0.47 GB in 80 us, where a plain
// copy's rate would take 72).
//
// With few tiles the contraction is split over the CTAs of a cluster. Each leaves its partial tile in
// its shared memory; the cluster then sums the partials in rank order (no atomics: results do not
// depend on timing) and writes the rows, each CTA a share of them.
//
// Adapters (y = x W + s_a (x A_a) B_a): the rows are the tokens sorted by adapter (up to one tile of tokens: in their
// own order, with zeros where a token has another adapter), v = s_a x A_a comes
// from a first product over the adapters' segments, and v B_a is accumulated into the same TMEM tile
// as further k-blocks: 16 ranks of one adapter are one MMA step over the (sixteens of) rows that it owns, with
// zeros for other rows among them. The second product is launched as a dependent of the first: it
// multiplies x by W while v is still being made (see the wait below). v is held in binary32 and enters as two bf16
// numbers (v = hi + lo, |v - hi - lo| <= 2^-16 |v|), so that nothing is rounded to bf16 between the two
// products.
#include <cstring>

#include "ragged.cuh"
#include "tmap.cuh"

namespace tpx {
namespace {

constexpr int BM = 128;                       // columns of W per tile (the MMA's M)
constexpr int BK = 64;                        // one 128-byte swizzle atom of bf16
constexpr int STAGES = 4;
constexpr uint32_t W_STAGE = BM * BK * 2;     // 16 KiB
constexpr uint32_t W_BOX = 64 * BK * 2;       // 64 columns x 64 k: 8 KiB
constexpr int THREADS = 192;                  // loads, MMA, 4 warps that read TMEM
constexpr int COPY_FROM = 17;                 // rows of a tile from which cp.async fetches x
constexpr int STG_LD = BM + 4;                // floats between rows of the staged output tile
constexpr int MAX_SEGS = TP_MAX_EXPERTS;

constexpr size_t TWO_PER_SM = 80 * 1024;      // more than a third of an SM's shared memory
// A tile has 64 rows at most, or 16: then a CTA's stages take 72 KiB instead of 96, and three of them fit an SM.
template <int NT>
constexpr uint32_t X_STAGE = NT * BK * 2;
template <int NT>
constexpr int BOX_ROWS = NT < 32 ? NT : 32;   // rows of x that one load brings when they lie side by side
// Dynamic shared memory: stages, barriers, the segments' bounds, the tile's rows and adapters.
template <int NT>
size_t smem_bytes(int segs) {
  return 1024 + STAGES * (W_STAGE + X_STAGE<NT>) + (4 * STAGES + 4) * 8 + 16 + ((segs + 4) & ~3) * 4 + 2 * NT * 4;
}

template <int NT, bool SWIGLU, bool LORA>
__global__ void __launch_bounds__(THREADS) ragged_kernel(const __grid_constant__ RaggedParams p) {
  constexpr uint32_t X_STAGE = tpx::X_STAGE<NT>;
  constexpr uint32_t X_BOX = BOX_ROWS<NT> * BK * 2;
  constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
  static_assert(NT % 16 == 0 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "TMEM is allocated in powers of two from 32 columns");
  static_assert(STAGES % 2 == 0, "the bounds behind the 4 * STAGES + 4 barriers start on 16 bytes");
  static_assert(NT * STG_LD * 4 <= STAGES * (W_STAGE + NT * BK * 2), "the staged output tile reuses the operand stages");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_w = smem;
  uint8_t* s_x = smem + STAGES * W_STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_x + STAGES * X_STAGE);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, rows0 = empty0 + 8 * STAGES;
  const uint32_t go0 = rows0 + 8 * STAGES, accf = go0 + 8 * STAGES, drain = accf + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int* s_count = reinterpret_cast<int*>(tmem_slot + 2);            // adapters of this tile
  int* s_off = reinterpret_cast<int*>(bars + 4 * STAGES + 4) + 4;  // 16-byte aligned
  const int segs = LORA ? p.L : p.E;
  int* s_idx = s_off + ((segs + 4) & ~3);
  int* s_list = s_idx + NT;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.tw);
    prefetch_tmap(p.row_index != nullptr ? &p.tx : &p.tx_box32);
    if (SWIGLU) prefetch_tmap(&p.tw2);
    if (LORA) prefetch_tmap(&p.tb);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(rows0 + 8 * s, 128);
      mbar_init(go0 + 8 * s, 1);
    }
    mbar_init(accf, 1);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  // Up to here beside the kernel before this one, and from here the next one beside this.
  // A product with v waits before it reads v or writes anything, and reads x, W, offsets and row_index without that wait.
  // The kernel before it is always the same call's own, which makes v from them. Every thread of that one has waited
  // before it let this kernel begin, so whatever wrote x, W, offsets and row_index has completed and its results lie in
  // global memory; and they are read from L2 (TMA, cp.async.cg, ld_gpu_s32), since this SM's L1 may hold what was there
  // before. (Waiting first, with W fetched into L2 meanwhile: one token 20.9 us against 14.7, 64 tokens of 32 adapters
  // 31.5 against 26.6.)
  if (!LORA) wait_prerequisites();
  launch_dependents();
  for (int e = threadIdx.x; e <= segs; e += THREADS) {
    if constexpr (LORA) s_off[e] = min(max(ld_gpu_s32(p.offsets + e), 0), p.R);
    else s_off[e] = seg_bound(p.offsets, e, p.R);
  }
  // Rows side by side in x: no index, or adapters whose tokens fit one tile, which then takes them in their
  // own order and looks up where each lies in the sorted one (s_idx; -1: a token that is not named).
  const bool own_order = LORA && p.R <= NT;
  const bool box = own_order || p.row_index == nullptr;
  if (own_order && threadIdx.x < NT) s_idx[threadIdx.x] = -1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // This cluster's tile: segment (adapters: shard) e, rows i0 .. i0 + valid - 1, columns n0 ...
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / p.split;
  int e, i0, valid, ct;
  bool live;
  if (LORA) {
    const int row_tiles = (p.R + NT - 1) / NT;
    const int rt = unit % row_tiles;
    ct = unit / row_tiles;
    e = ct / p.tiles_n;
    ct -= e * p.tiles_n;
    i0 = rt * NT;
    valid = min(NT, p.R - i0);
    live = e < p.E;
  } else {
    const SegTile t = find_seg_tile<NT>(s_off, p.E, unit / p.tiles_n, lane);
    live = t.live;
    e = t.e;
    const int local = unit - t.before * p.tiles_n;
    const int rt = live ? local % t.count : 0;
    ct = live ? local / t.count : 0;
    i0 = s_off[e] + rt * NT;
    valid = min(NT, s_off[e + 1] - i0);
  }
  constexpr int TILE_N = SWIGLU ? BM / 2 : BM;       // output columns per tile
  const int n0 = ct * TILE_N;
  // this CTA's share of the contraction: k-blocks of x (k-blocks of adapters follow)
  const int kb0 = live ? static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / p.split) : 0;
  const int base = live ? static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / p.split) - kb0 : 0;
  // Rows side by side come by TMA in boxes of 32 (16); few others four a load, from 17 on warps 2..5 copy them.
  const bool copy = live && !box && valid >= COPY_FROM;
  const int groups = copy || box || !live ? 0 : (valid + 3) / 4;
  const int boxes = box && live ? (valid + BOX_ROWS<NT> - 1) / BOX_ROWS<NT> : 0;
  auto load_w = [&](int step) {
    const uint32_t fb = full0 + 8 * (step % STAGES), dst = smem_u32(s_w + (step % STAGES) * W_STAGE);
    const int k0 = (kb0 + step) * BK;
    mbar_arrive_expect_tx(fb, W_STAGE + groups * 512u + boxes * X_BOX);
    if (p.w_km) {
      tma_load_3d(dst, &p.tw, k0, n0, e, fb);
    } else {
      tma_load_3d(dst, &p.tw, n0, k0, e, fb);
      tma_load_3d(dst + W_BOX, SWIGLU ? &p.tw2 : &p.tw, SWIGLU ? n0 : n0 + 64, k0, e, fb);
    }
    for (int b = 0; b < boxes; ++b)
      tma_load_2d(smem_u32(s_x + (step % STAGES) * X_STAGE) + b * X_BOX, &p.tx_box32, k0, i0 + BOX_ROWS<NT> * b, fb);
  };
  const int ahead = min(base, STAGES);               // W of the first stages is on its way before the rows are known
  if (warp == 0 && lane == 0)
    for (int step = 0; step < ahead; ++step) load_w(step);
  if (live && warp != 0) {
    if (own_order) {
      for (int i = threadIdx.x - 32; i < p.R; i += THREADS - 32) {
        const int r = ld_gpu_s32(p.row_index + i);
        if (r >= 0 && r < p.R) s_idx[r] = i;
      }
    } else {
      // x's row of every row of the tile; -1: the index lies outside x (the row reads as zeros)
      for (int j = threadIdx.x - 32; j < ((valid + 3) & ~3); j += THREADS - 32) {
        const int i = i0 + min(j, valid - 1);
        const int r = p.row_index == nullptr ? i : LORA ? ld_gpu_s32(p.row_index + i) : ld_s32(p.row_index + i);
        s_idx[j] = r >= 0 && r < p.x_rows ? r : -1;
      }
    }
    if (LORA && warp == 2) {                         // the adapters that own rows of this tile, ascending
      int n_list = 0;
      for (int a0 = 0; a0 < p.L; a0 += 32) {
        const int a = a0 + lane;
        const bool in = a < p.L && max(s_off[a], i0) < min(s_off[a + 1], i0 + valid);
        const unsigned m = __ballot_sync(0xffffffffu, in);
        const int at = n_list + __popc(m & ((1u << lane) - 1));
        if (in && at < NT) s_list[at] = a;
        n_list += __popc(m);
      }
      if (lane == 0) *s_count = min(n_list, NT);
    }
  }
  __syncthreads();

  const int per_adapter = LORA ? (p.rank + 15) / 16 : 1;            // 16-rank steps of one adapter
  const int chunks = LORA && live ? *s_count * per_adapter : 0;
  const int extra = (chunks + 1) / 2;                               // k-blocks of two adapter steps
  const int x0 = extra * rank / p.split;
  const int steps = live ? base + extra * (rank + 1) / p.split - x0 : 0;
  const int n_mma = live ? (valid + 15) & ~15 : 16;
  int loaded = 0;                                                   // warp 0: k-blocks loaded
  bool mma_issued = false;

  if (warp == 0 && live) {
    for (int step = 0; step < steps; ++step) {
      const int st = loaded % STAGES;
      // (a stage that was filled ahead may have been used and freed by now: its wait would be for the next round)
      bool ok = step < ahead || mbar_wait_bounded(empty0 + 8 * st, ((loaded / STAGES) & 1) ^ 1, p.budget, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (!*abort_flag) record_timeout(p.status, WAIT_PRODUCER_EMPTY);
        *abort_flag = 1u;
        break;
      }
      const uint32_t fb = full0 + 8 * st;
      const uint32_t w_dst = smem_u32(s_w + st * W_STAGE), x_dst = smem_u32(s_x + st * X_STAGE);
      if (!LORA || step < base) {
        const int k0 = (kb0 + step) * BK;
        if (lane == 0 && step >= ahead) load_w(step);
        __syncwarp();
        for (int g = lane; g < groups; g += 32) {
          const int4 r = *reinterpret_cast<const int4*>(s_idx + 4 * g);
          if ((r.x | r.y | r.z | r.w) >= 0) {
            tma_gather4(x_dst + 512u * g, &p.tx, k0, r.x, r.y, r.z, r.w, fb);
          } else {                                         // rows outside x by themselves, from behind x: TMA's zeros
            for (int q = 0; q < 4; ++q) {
              const int row = s_idx[4 * g + q];
              tma_load_2d(x_dst + 512u * g + 128u * q, &p.tx, k0, row >= 0 ? row : p.x_rows, fb);
            }
          }
        }
      } else {
        // two 16-rank steps: B's rows (v of the tokens comes from warps 2..5, which may fill the slot now)
        if (lane == 0) {
          mbar_arrive(go0 + 8 * st);
          const int c0 = 2 * (x0 + step - base), nch = min(2, chunks - c0);
          mbar_arrive_expect_tx(fb, nch * 4096u);
          for (int ch = 0; ch < nch; ++ch) {
            const int a = s_list[(c0 + ch) / per_adapter];
            const int r0 = ((c0 + ch) % per_adapter) * 16;
            tma_load_3d(w_dst + ch * 2048u, &p.tb, n0, r0, e * p.L + a, fb);
            tma_load_3d(w_dst + ch * 2048u + W_BOX, &p.tb, n0 + 64, r0, e * p.L + a, fb);
          }
        }
        __syncwarp();
      }
      ++loaded;
    }
  } else if (warp == 1 && lane == 0 && live) {
    const uint32_t idesc = idesc_bf16_f32(BM, n_mma, !p.w_km, false);
    int done = 0;
    uint32_t rows_phase = 0;                               // one bit per stage
    for (int step = 0; step < steps; ++step, ++done) {
      const int st = done % STAGES;
      if (!mbar_wait_bounded(full0 + 8 * st, (done / STAGES) & 1, p.budget, abort_flag)) {
        if (!*abort_flag) record_timeout(p.status, WAIT_MMA_FULL);
        *abort_flag = 1u;
        break;
      }
      if (copy || (LORA && step >= base)) {                // the rows that warps 2..5 brought
        if (!mbar_wait_bounded(rows0 + 8 * st, (rows_phase >> st) & 1, p.budget, abort_flag)) {
          if (!*abort_flag) record_timeout(p.status, WAIT_MMA_FULL);
          *abort_flag = 1u;
          break;
        }
        rows_phase ^= 1u << st;
        fence_proxy_async();
      }
      tc_fence_after();
      const uint32_t w_base = smem_u32(s_w + st * W_STAGE), x_base = smem_u32(s_x + st * X_STAGE);
      if (!LORA || step < base) {
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) {
          const uint64_t ad = p.w_km ? smem_desc_sw128(w_base + 32u * k, 16u, 1024u)
                                     : smem_desc_sw128(w_base + 2048u * k, W_BOX, 1024u);
          umma_bf16(tmem_base, ad, smem_desc_sw128(x_base + 32u * k, 16u, 1024u), idesc, (step | k) != 0 ? 1u : 0u);
        }
      } else {
        // hi and lo of each step against the same rows of B, for the adapter's rows alone (in sixteens)
        const int c0 = 2 * (x0 + step - base);
        for (int ch = 0; ch < min(2, chunks - c0); ++ch) {
          const int a = s_list[(c0 + ch) / per_adapter];
          const int first = own_order ? 0 : (max(s_off[a], i0) - i0) & ~15;
          const int last = own_order ? n_mma : (min(s_off[a + 1], i0 + valid) - i0 + 15) & ~15;
          const uint32_t id = idesc_bf16_f32(BM, last - first, true, false);
          const uint64_t ad = smem_desc_sw128(w_base + 2048u * ch, W_BOX, 1024u);
          for (int half = 0; half < 2; ++half)
            umma_bf16(tmem_base + first, ad, smem_desc_sw128(x_base + first * 128u + 32u * (ch + 2 * half), 16u, 1024u), id, 1u);
        }
      }
      mma_issued = true;
      umma_commit(empty0 + 8 * st);
    }
    umma_commit(accf);
  } else if (warp >= 2 && live) {
    const int tid = threadIdx.x - 64;
    const int piece = tid & 7, r0 = tid >> 3;
    if (copy || (LORA && steps > base)) {
      int idx[NT / 16];
#pragma unroll
      for (int i = 0; i < NT / 16; ++i) idx[i] = r0 + 16 * i < valid ? s_idx[r0 + 16 * i] : -2;
      uint32_t go_phase = 0;                               // one bit per stage
      uint4 hi[2], lo[2];                                  // the next step's v, on its way while slots are waited for
      auto fetch_v = [&](int step) {
        const int c0 = 2 * (x0 + step - base);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          hi[ch] = lo[ch] = make_uint4(0, 0, 0, 0);
          if (c0 + ch >= chunks) continue;
          const int a = s_list[(c0 + ch) / per_adapter];
          const int j = tid >> 1, k = ((c0 + ch) % per_adapter) * 16 + (tid & 1) * 8;
          const int i = j >= valid ? -1 : own_order ? s_idx[j] : i0 + j;
          if (i >= 0 && i >= s_off[a] && i < s_off[a + 1] && k < p.rank)
            split_bf8(p.v + static_cast<int64_t>(i) * p.rank + k, hi[ch], lo[ch]);
        }
      };
      for (int step = copy ? 0 : base; step < steps; ++step) {
        const int st = step % STAGES;
        if (LORA && step == base) {
          wait_prerequisites();                            // v is the kernel before's
          fetch_v(step);
        }
        // Rows of x: they follow every use of every slot. v: they may not have, and the parity of `empty` would
        // say nothing to them; warp 0, which has waited for the slot, lets them go.
        const bool v_step = LORA && step >= base;
        bool ok = v_step ? mbar_wait_bounded(go0 + 8 * st, (go_phase >> st) & 1u, p.budget, abort_flag)
                         : mbar_wait_bounded(empty0 + 8 * st, ((step / STAGES) & 1) ^ 1, p.budget, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (!*abort_flag) record_timeout(p.status, WAIT_PRODUCER_EMPTY);
          *abort_flag = 1u;
          break;
        }
        if (v_step) go_phase ^= 1u << st;
        const uint32_t x_dst = smem_u32(s_x + st * X_STAGE);
        if (!LORA || step < base) {
          const int k = (kb0 + step) * BK + piece * 8;
#pragma unroll
          for (int i = 0; i < NT / 16; ++i) {
            const int row = r0 + 16 * i;
            if (idx[i] != -2) {
              const bool in = idx[i] >= 0 && k < p.K;
              cp_async16(x_dst + row * 128 + ((piece ^ (row & 7)) << 4),
                         in ? p.x + static_cast<int64_t>(idx[i]) * p.K + k : p.x, in ? 16u : 0u);
            }
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(rows0 + 8 * st) : "memory");
        } else {
          const int row = tid >> 1;
          uint8_t* line = s_x + st * X_STAGE + row * 128;
          for (int ch = 0; ch < 2 && row < NT; ++ch) {     // hi in pieces 0..3, lo in 4..7
            const int at = 2 * ch + (tid & 1);
            *reinterpret_cast<uint4*>(line + ((at ^ (row & 7)) << 4)) = hi[ch];
            *reinterpret_cast<uint4*>(line + (((at + 4) ^ (row & 7)) << 4)) = lo[ch];
          }
          mbar_arrive(rows0 + 8 * st);
          if (step + 1 < steps) fetch_v(step + 1);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (LORA) wait_prerequisites();                        // completes after the kernel before, always
    // TMEM lane = column of W, TMEM column = row of the tile -> staged [row][column] in shared memory
    // (the operand stages are free: the commit says that every MMA, and so every load, is done)
    if (!mbar_wait_bounded(accf, 0, p.budget, abort_flag)) {
      if (!*abort_flag) record_timeout(p.status, WAIT_EPI_ACC_FULL);
      *abort_flag = 1u;
    } else if (!*abort_flag) {
      tc_fence_after();
      const int quad = warp & 3;
      float* stg = reinterpret_cast<float*>(smem) + quad * 32 + lane;
      for (int j0 = 0; j0 < n_mma; j0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + j0, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j0 + j < valid) stg[(j0 + j) * STG_LD] = __uint_as_float(v[j]);
      }
      tc_fence_before();
    }
  }
  __syncwarp();

  // Partial tiles staged: the cluster's (or this CTA's) threads sum them and write the rows.
  if (p.split > 1) cluster_sync(); else __syncthreads();
  if (live && !*abort_flag) {
    constexpr int GROUPS = TILE_N / 8;
    const uint32_t stg = smem_u32(smem);
    for (int it = rank * THREADS + threadIdx.x; it < valid * GROUPS; it += p.split * THREADS) {
      const int j = it / GROUPS, c8 = (it % GROUPS) * 8;
      const int col = n0 + c8;
      if (col >= p.n) continue;
      float f[8], u[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = u[q] = 0.0f;
      for (int s = 0; s < p.split; ++s) {
        const uint32_t at = stg + (j * STG_LD + c8) * 4;
        const uint32_t src = p.split > 1 ? mapa_shared(at, s) : at;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 x = ld_cluster_v4(src + 16 * q);
          f[4 * q] += x.x; f[4 * q + 1] += x.y; f[4 * q + 2] += x.z; f[4 * q + 3] += x.w;
          if constexpr (SWIGLU) {
            const float4 z = ld_cluster_v4(src + 256 + 16 * q);
            u[4 * q] += z.x; u[4 * q + 1] += z.y; u[4 * q + 2] += z.z; u[4 * q + 3] += z.w;
          }
        }
      }
      if (p.seg_scale != nullptr) {
        const float sc = ld_f32(p.seg_scale + e);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] *= sc;
      }
      if constexpr (LORA) {
        const int r = s_idx[j];
        if (r < 0) continue;                           // no token
        const int token = own_order ? j : r;
        if (*s_count > 0) lora_settle8(p, s_off, e, token, own_order ? r : i0 + j, col, f);
        store_row8(p, static_cast<int64_t>(e) * p.R + token, col, f, u);
      } else {
        store_row8(p, i0 + j, col, f, u);
      }
    }
  }
  if (p.split > 1) cluster_sync();     // a CTA's shared memory outlives its peers' reads
  tc_fence_before();
  __syncthreads();
  if (*abort_flag != 0u) {             // a wait ran out: let copies and MMAs in flight land first
    const unsigned long long drain_budget = 4000000000ull;
    if (warp == 0 && lane == 0) {
      for (int s = 0; s < STAGES; ++s) {
        const int uses = (loaded - s + STAGES - 1) / STAGES;
        if (uses > 0 && !mbar_wait_bounded(full0 + 8 * s, (uses - 1) & 1, drain_budget, nullptr))
          record_timeout(p.status, WAIT_TEARDOWN);
      }
    }
    if (warp == 1 && lane == 0 && mma_issued) {
      umma_commit(drain);
      if (!mbar_wait_bounded(drain, 0, drain_budget, nullptr)) record_timeout(p.status, WAIT_TEARDOWN);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

template <int NT, bool SWIGLU, bool LORA>
tp_status launch_ragged(const RaggedParams& p, int64_t units, cudaStream_t s) {
  static int configured_for[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(TP_ECUDA, "cudaGetDevice failed");
  if (dev < 0 || dev >= 64 || !configured_for[dev]) {
    if (cudaFuncSetAttribute(ragged_kernel<NT, SWIGLU, LORA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes<NT>(MAX_SEGS) > TWO_PER_SM ? smem_bytes<NT>(MAX_SEGS) : TWO_PER_SM)) != cudaSuccess)
      return fail(TP_ECUDA, "cannot reserve %zu bytes of shared memory", smem_bytes<NT>(MAX_SEGS));
    if (dev >= 0 && dev < 64) configured_for[dev] = 1;
  }
  if (units * p.split > INT32_MAX) return fail(TP_ESHAPE, "too many tiles");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * p.split));
  cfg.blockDim = dim3(THREADS);
  // Low tiles: three CTAs on an SM, but two (by asking for more shared memory) where the grid is neither
  // well below one round of three nor several: 1104 CTAs 86 us by threes, 96 by twos; 448 CTAs 91 and 80
  // (444 fit at once), 256 CTAs 163 and 130 (some SMs get three, others one).
  size_t smem = smem_bytes<NT>(LORA ? p.L : p.E);
  const int64_t ctas = units * p.split, sms = sm_count();
  if (NT < 64 && 2 * ctas > 3 * sms && ctas < 6 * sms && smem < TWO_PER_SM) smem = TWO_PER_SM;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(p.split);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;    // starts beside the kernel before
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, ragged_kernel<NT, SWIGLU, LORA>, p);
  if (err != cudaSuccess) return fail(TP_ECUDA, "ragged_kernel: %s", cudaGetErrorString(err));
  return check_launch("ragged_kernel");
}

}  // namespace

bool lora_takes_pairs(int64_t N, int64_t n, int t) {
  return N > 64 && 4 * ((N + LORA_TILE - 1) / LORA_TILE) * ((n + 255) / 256) * t >= sm_count();
}

// The height whose tiles take the least time in whole rounds of the pairs, an eighth of the largest added for what a tile
// costs whatever its height. 4000 tokens, 6144 columns in 8 shards: 384 tiles of 256 are six rounds of 74, 432 of 224 are six
// as well, 193 -> 181 us. (From four rounds on. Lower tiles load more of W for what they multiply, which counts where not all pairs
// work all the time: 1000 tokens in two rounds of 192 instead of two of 256, 82 -> 92 us, in three of 160, 100.)
int lora_tile(int64_t N, int64_t n, int t) {
  const int64_t cols = (n + 255) / 256 * t, pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
  auto rounds = [&](int tile) { return ((N + tile - 1) / tile * cols + pairs - 1) / pairs; };
  int best = LORA_TILE;
  for (int tile = LORA_TILE - 32; tile >= LORA_TILE_MIN && rounds(LORA_TILE) >= 4; tile -= 32)
    if (rounds(tile) * (tile + LORA_TILE / 8) < rounds(best) * (best + LORA_TILE / 8)) best = tile;
  return best;
}

tp_status ragged_product(const RaggedArgs& g, cudaStream_t s) {
  RaggedParams p;
  std::memset(&p, 0, sizeof(p));
  const bool lora = g.v != nullptr;
  const bool swiglu = g.act == TP_ACT_SWIGLU && !g.backward;
  const int64_t segs = lora ? 1 : (g.E < g.R ? g.E : g.R);       // segments that can hold rows
  // Pairs for segments of more than 64 rows on average, if their tiles (256 rows x 256 columns) keep at
  // least half of the pairs busy. x A of 4000 tokens, 8 adapters of rank 64, K = 4096: 23 tiles of pairs,
  // 52 us; 284 CTAs here, 14 us.
  const int tokens = lora ? lora_tile(g.R, g.n, g.E) : 0;
  const int64_t wide_rows = lora ? (g.R + tokens - 1) / tokens : g.R / 256 + segs;
  const int64_t wide_units = wide_rows * ((g.n + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256));
  const bool pairs = lora ? g.lora_pos != nullptr : g.R > 64 * segs && 4 * wide_units >= sm_count();
  const int pair_tile = swiglu ? 128 : 256;                         // output columns
  const int64_t pair_tiles = (g.n + pair_tile - 1) / pair_tile;
  // Rows that lie side by side are multiplied faster than gathered ones (8192 rows of uneven segments, K = 4096, n =
  // 14336, SwiGLU: 1540 against 2030 us), and copying them takes 4 K bytes a row (26 us). So where W has many columns they
  // are copied first: to x_copy, or else to the end of y's own rows, as long as at least half of y lies before that (1600
  // us); the columns that take the copy's place are then multiplied last, from x itself. That takes two launches
  // with their last rounds, and pays from K = 2048 on (16384 rows, n = 4096, SwiGLU: 480 against 501 us; K = 1024, n = 4096:
  // 171 against 163).
  if (pairs && !lora && g.row_index != nullptr && g.tiles == 0 && g.n * (swiglu ? 2 : 1) >= 4096) {
    RaggedArgs a = g;
    a.row_index = nullptr;
    a.x_rows = g.R;
    a.x_copy = nullptr;
    if (g.x_copy != nullptr) {
      a.x = g.x_copy;
      if (tp_status st = gather_rows(g.x, g.x_rows, g.row_index, g.offsets, g.E, g.R, g.K, g.x_copy, g.K, s)) return st;
      return ragged_product(a, s);
    }
    const int64_t taken = g.out_f32 ? g.K / 2 : g.K, before = g.n > taken ? (g.n - taken) / pair_tile : 0;
    if (g.K >= 2048 && 2 * before >= pair_tiles && wide_rows * (pair_tiles - before) >= 2 * sm_count()) {
      a.x_ld = g.out_f32 ? 2 * g.n : g.n;
      uint16_t* copy = static_cast<uint16_t*>(g.y) + a.x_ld - g.K;
      a.x = copy;
      a.tiles = static_cast<int>(before);
      if (tp_status st = gather_rows(g.x, g.x_rows, g.row_index, g.offsets, g.E, g.R, g.K, copy, a.x_ld, s)) return st;
      if (tp_status st = ragged_product(a, s)) return st;
      RaggedArgs b = g;
      b.tile0 = a.tiles;
      b.tiles = static_cast<int>(pair_tiles - before);
      return ragged_product(b, s);
    }
  }
  const int64_t x_ld = g.x_ld != 0 ? g.x_ld : g.K;
  // Low tiles where segments have eight rows or fewer on average (most then fit one).
  const bool low = !pairs && g.R <= 8 * segs;
  const int nt = low ? 16 : 64;
  if (g.w_km ? !encode_bf16_3d(&p.tw, g.w, g.K, g.n, g.E, g.K, BK, BM)
             : !encode_bf16_3d(&p.tw, g.w, g.n, g.K, g.E, swiglu ? 2 * g.n : g.n, 64, BK))
    return fail(TP_ECUDA, "cannot encode the TMA descriptor of the weights");
  if (swiglu && !encode_bf16_3d(&p.tw2, g.w + g.n, g.n, g.K, g.E, 2 * g.n, 64, BK))
    return fail(TP_ECUDA, "cannot encode the TMA descriptor of the up half of the weights");
  if (g.row_index != nullptr && !encode_bf16_2d(&p.tx, g.x, g.K, g.x_rows, g.K, BK, 1))
    return fail(TP_ECUDA, "cannot encode the TMA descriptor of the rows");
  if (((g.row_index == nullptr || lora) && !encode_bf16_2d(&p.tx_box, g.x, g.K, g.x_rows, x_ld, BK, 128)) ||
      !encode_bf16_2d(&p.tx_box32, g.x, g.K, g.x_rows, x_ld, BK, low ? BOX_ROWS<16> : BOX_ROWS<64>))
    return fail(TP_ECUDA, "cannot encode the TMA descriptor of the rows");
  if (lora && !encode_bf16_3d(&p.tb, g.lora_b, g.n, g.rank, static_cast<uint64_t>(g.E) * g.L, g.n, 64, 16))
    return fail(TP_ECUDA, "cannot encode the TMA descriptor of the adapters");
  p.x = g.x; p.offsets = g.offsets; p.row_index = g.row_index; p.seg_scale = g.seg_scale;
  p.y = g.y; p.pre = g.pre; p.h_pre = g.h_pre; p.v = g.v; p.lora_pos = g.lora_pos; p.lora_lists = g.lora_lists;
  p.w = g.w; p.lora_b = g.lora_b;
  p.R = static_cast<int>(g.R); p.x_rows = static_cast<int>(g.x_rows);
  p.E = g.E; p.n = static_cast<int>(g.n); p.K = static_cast<int>(g.K);
  p.num_kb = static_cast<int>((g.K + BK - 1) / BK);
  p.L = g.L; p.rank = g.rank; p.lora_tile = tokens;
  p.act = g.act; p.w_km = g.w_km; p.out_f32 = g.out_f32; p.backward = g.backward;
  p.status = status_word();
  p.budget = wait_budget();
  if (p.status == nullptr) return fail(TP_ECUDA, "cannot resolve the device status word");
  const int tile_n = swiglu ? BM / 2 : BM;
  p.tiles_n = static_cast<int>((g.n + tile_n - 1) / tile_n);
  if (pairs) {
    p.tile0 = g.tile0;
    p.tiles_n = g.tiles != 0 ? g.tiles : static_cast<int>(pair_tiles);
    return ragged_pairs(p, swiglu, lora, wide_rows, s);
  }
  const int64_t units = (lora ? (g.R + nt - 1) / nt : g.R / nt + segs) * p.tiles_n * (lora ? g.E : 1);
  // Two CTAs fit an SM (three of low tiles): split the contraction (in shares of four k-blocks at least) by
  // powers of two while all CTAs find room at once. 50 MB of W for one token: 35 us unsplit, 23 by two, 20
  // by four, 27 by eight (more than fit), 29 by six (clusters of six pack badly).
  const int64_t room = 2ll * sm_count();
  p.split = 1;
  while (p.split < 8 && units * p.split * 2 <= room && p.num_kb >= 8 * p.split) p.split *= 2;
  if (low) {
    if (lora) return launch_ragged<16, false, true>(p, units, s);
    return swiglu ? launch_ragged<16, true, false>(p, units, s) : launch_ragged<16, false, false>(p, units, s);
  }
  if (lora) return launch_ragged<64, false, true>(p, units, s);
  return swiglu ? launch_ragged<64, true, false>(p, units, s) : launch_ragged<64, false, false>(p, units, s);
}

}  // namespace tpx
