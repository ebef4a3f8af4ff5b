// What the kernels over ragged segments of rows share: the launch parameters, the place of a tile
// among the segments, and the form of the output rows.
//
// Rows sorted by segment (expert, adapter) are given by offsets[S + 1] in device memory: segment e
// holds rows offsets[e] .. offsets[e + 1] - 1. The host never reads them. Every offset is taken as
// clamped to 0 .. R and a segment that ends before it begins is empty, so that no offsets whatever
// lead outside a buffer of R rows.
#pragma once

#include <cuda.h>

#include <utility>

#include "act.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace tpx {

// Product y_i = epilogue(x[row_i] W_e) over the rows i of every segment e.
struct RaggedParams {
  CUtensorMap tw;             // W: [E][K][n], or [E][n][K] (w_km); the gate half for SwiGLU
  CUtensorMap tw2;            // SwiGLU: the up half
  CUtensorMap tx;             // x: [x_rows][K], boxes one row high (gathered rows)
  CUtensorMap tx_box;         // x: boxes of 128 rows (rows side by side)
  CUtensorMap tx_box32;       // x: boxes of 32 rows
  CUtensorMap tb;             // adapters: B [t * L][rank][n]
  const int32_t* offsets;     // [E + 1]; adapters: [L + 1], the segments of the adapters
  const int32_t* row_index;   // x's row of sorted row i; nullptr: i
  const uint16_t* x;
  const float* seg_scale;     // optional factor of every row of segment e
  void* y;                    // output rows, stride n
  uint16_t* pre;              // optional: the products before the activation (SwiGLU: [gate | up], stride 2n)
  const uint16_t* h_pre;      // backward: what the activation was applied to (stride n, SwiGLU 2n)
  const float* v;             // adapters: scale * x A of sorted row i, [N][rank]
  const uint16_t* w;          // adapters: what tw and tb describe
  const uint16_t* lora_b;
  const int32_t* lora_pos;    // pairs: a token's sorted row if it has an adapter, -1 if not, -2 if it is not named
  const int32_t* lora_lists;  // pairs: the adapters of every tile of tokens
  int R, x_rows;              // sorted rows, rows of x
  int E, n, K, num_kb, tiles_n;
  int tile0;                  // pairs: first of the tiles_n column tiles
  int L, rank;                // adapters: their number and rank
  int lora_tile;              // pairs: tokens of a tile
  int split;                  // CTAs along the contraction
  int act;                    // tp_act of the epilogue
  bool w_km;                  // W stored [E][n][K]
  bool out_f32;
  bool backward;              // multiply by the activation's derivative at h_pre
  uint32_t* status;
  unsigned long long budget;
};

// Launches a kernel that may begin while the one before it on the stream still runs: every thread of it waits
// (wait_prerequisites) before it touches global memory, and then lets the next one begin. (The adapters' second product
// reads some of its inputs before its wait: see ragged_kernel.) Back to back
// such launches hide about 2 us each: the launch and, for the products, barriers and TMEM.
template <typename... P, typename... A>
tp_status launch_beside(const char* what, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
  if (err != cudaSuccess) return fail(TP_ECUDA, "%s: %s", what, cudaGetErrorString(err));
  return check_launch(what);
}

// Host-side arguments of ragged_product (checked by the entry points).
struct RaggedArgs {
  const uint16_t* x;          // [x_rows][K]
  int64_t x_rows;
  int64_t x_ld;               // pairs, rows side by side: elements between rows (0: K)
  const int32_t* row_index;   // see RaggedParams
  uint16_t* x_copy;           // room for [R][K], to put gathered rows side by side; or nullptr
  const int32_t* offsets;
  int64_t R;                  // rows of y (adapters: tokens)
  int E;                      // segments (adapters: shards, each over all R rows)
  int64_t K, n;
  const uint16_t* w;
  bool w_km;
  int act;
  bool backward;
  const uint16_t* h_pre;
  void* y;
  bool out_f32;
  uint16_t* pre;
  const float* seg_scale;
  const float* v;             // adapters, or nullptr
  const int32_t* lora_pos;    // see RaggedParams; nullptr: the pair kernel is not used
  const int32_t* lora_lists;
  const uint16_t* lora_b;     // [E][L][rank][n]
  int L, rank;
  int tile0, tiles;           // pairs: some of the column tiles (0, 0: all)
};
tp_status ragged_product(const RaggedArgs& g, cudaStream_t s);

// Adapters on pairs: tiles of up to LORA_TILE tokens in their own order, each with a list of LORA_LIST ints (its
// adapters, ascending, behind their number).
constexpr int LORA_TILE = 256, LORA_TILE_MIN = 192, LORA_LIST = LORA_TILE + 1;
// Tokens of a tile for N tokens and t shards of n columns.
int lora_tile(int64_t N, int64_t n, int t);
// Whether a product with adapters takes the pair kernel (which needs lora_pos and lora_lists).
bool lora_takes_pairs(int64_t N, int64_t n, int t);
// x[row_index[i]] for every row i of a segment, zeros for an index outside x, to dst + i * ld.
tp_status gather_rows(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const int32_t* offsets, int E, int64_t R, int64_t K,
                      uint16_t* dst, int64_t ld, cudaStream_t s);
// The same on CTA pairs (row_tiles: how many tiles of 256 rows there can be; p.tile0 and p.tiles_n are set).
tp_status ragged_pairs(RaggedParams& p, bool swiglu, bool lora, int64_t row_tiles, cudaStream_t s);

// Host-side arguments of ragged_dw: dw[e] = x_e^T dy_e for every segment.
struct RaggedDwArgs {
  const uint16_t* x;          // [x_rows][k]
  int64_t x_rows;
  const int32_t* row_index;   // nullptr: row i of x
  const uint16_t* dy;         // [R][n]
  const int32_t* offsets;
  int64_t R;
  int E;
  int64_t k, n;
  void* dw;                   // [E][k][n]
  bool out_f32;
};
tp_status ragged_dw(const RaggedDwArgs& g, cudaStream_t s);

// offsets[e], clamped to the rows that exist.
__device__ __forceinline__ int seg_bound(const int32_t* offsets, int e, int R) {
  return min(max(ld_s32(offsets + e), 0), R);
}

// Tile number g among all segments' row tiles of NT rows (segment ascending): its segment, and the
// number of tiles before and in that segment. `off`: clamped offsets in shared memory. Whole warp.
struct SegTile {
  int e, before, count;
  bool live;
};
template <int NT>
__device__ __forceinline__ SegTile find_seg_tile(const int* off, int E, int g, int lane) {
  SegTile s{0, 0, 0, false};
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const int rows = e < E ? max(off[e + 1] - off[e], 0) : 0;
    const int cnt = (rows + NT - 1) / NT;
    int inc = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + inc > g);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s.e = e0 + src;
      s.count = __shfl_sync(0xffffffffu, cnt, src);
      s.before = base + __shfl_sync(0xffffffffu, inc, src) - s.count;
      s.live = true;
      return s;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return s;
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  return static_cast<uint32_t>(to_bf(lo)) | (static_cast<uint32_t>(to_bf(hi)) << 16);
}
__device__ __forceinline__ uint4 pack_bf8(const float (&f)[8]) {
  return make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
}
__device__ __forceinline__ void unpack_bf8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight binary32 numbers as bf16 pairs, v = hi + lo with |v - hi - lo| <= 2^-16 |v|. An infinite or NaN
// v is carried by hi alone.
__device__ __forceinline__ void split_bf8(const float* v, uint4& hi, uint4& lo) {
  const float4 a = *reinterpret_cast<const float4*>(v), b = *reinterpret_cast<const float4*>(v + 4);
  const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float h[8], l[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    h[q] = bf(to_bf(f[q]));
    l[q] = f[q] - h[q];
    if (!(fabsf(l[q]) < 1e38f)) l[q] = 0.0f;
  }
  hi = pack_bf8(h);
  lo = pack_bf8(l);
}

__device__ __forceinline__ float apply_act(float x, int act) {
  return act == TP_ACT_GELU ? gelu_erf(x) : act == TP_ACT_GELU_TANH ? gelu_tanh(x) : x;
}

// Backward: what the activation was applied to at eight columns of one row (h1: SwiGLU's up half), and the
// gradient there.
__device__ __forceinline__ void load_h_pre(const RaggedParams& p, int64_t row, int col, uint4& h0, uint4& h1) {
  if (p.act == TP_ACT_SWIGLU) {
    h0 = ld_stream_v4(p.h_pre + row * 2 * p.n + col);
    h1 = ld_stream_v4(p.h_pre + row * 2 * p.n + p.n + col);
  } else if (p.act != TP_ACT_NONE) {
    h0 = ld_stream_v4(p.h_pre + row * p.n + col);
  }
}
__device__ __forceinline__ void store_backward8(const RaggedParams& p, int64_t row, int col, float (&f)[8], uint4 h0, uint4 h1) {
  uint16_t* y = static_cast<uint16_t*>(p.y);
  float h[8];
  unpack_bf8(h0, h);
  if (p.act == TP_ACT_SWIGLU) {
    float up[8], dg[8], du[8];
    unpack_bf8(h1, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // The sigmoid: __expf's argument is rounded, so that for negative h it is off by up to about (4 + 1.2 |h|) * 2^-23 of
      // itself (2^-18 of itself at -24), for positive h by a few units; 0 where __expf overflows. The gradient's rounding to
      // bf16 is 2^-9 on average; a division in place of the reciprocal would save 2 of those units (and took 159 us where
      // this takes 137: 64 experts, 24558 rows, 1024 x 2048).
      const float s = __fdividef(1.0f, 1.0f + __expf(-h[i]));
      dg[i] = f[i] * up[i] * (s * (1.0f + h[i] * (1.0f - s)));
      du[i] = f[i] * (h[i] * s);
    }
    st_v4(y + row * 2 * p.n + col, pack_bf8(dg));
    st_v4(y + row * 2 * p.n + p.n + col, pack_bf8(du));
    return;
  }
  if (p.act != TP_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= p.act == TP_ACT_GELU ? gelu_grad(h[i]) : gelu_tanh_grad(h[i]);
  }
  st_v4(y + row * p.n + col, pack_bf8(f));
}

// Eight neighbouring columns of one output row: f the products (SwiGLU: the gate's, u the up's), in
// binary32 until the one rounding at the store.
__device__ __forceinline__ void store_row8(const RaggedParams& p, int64_t row, int col, float (&f)[8], float (&u)[8]) {
  if (p.backward) {
    uint4 h0 = make_uint4(0, 0, 0, 0), h1 = h0;
    load_h_pre(p, row, col, h0, h1);
    store_backward8(p, row, col, f, h0, h1);
    return;
  }
  if (p.act == TP_ACT_SWIGLU) {
    if (p.pre != nullptr) {
      st_v4(p.pre + row * 2 * p.n + col, pack_bf8(f));
      st_v4(p.pre + row * 2 * p.n + p.n + col, pack_bf8(u));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = silu(f[i]) * u[i];
  } else if (p.act != TP_ACT_NONE) {
    if (p.pre != nullptr) st_v4(p.pre + row * p.n + col, pack_bf8(f));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = apply_act(f[i], p.act);
  }
  if (p.out_f32) {
    float* y = static_cast<float*>(p.y) + row * p.n + col;
    st_v4(y, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    st_v4(y + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
  } else {
    st_v4(static_cast<uint16_t*>(p.y) + row * p.n + col, pack_bf8(f));
  }
}

// Adapters: the matrix instructions multiply the B of every adapter of a tile with all of the tile's tokens, by
// zeros where it is not theirs, and 0 * inf is NaN. So where a tile with adapters comes out as something that is
// not finite, its eight columns are summed again from this token's own adapter alone (`sorted` its row of v, or
// negative). That costs nothing where all is finite; a token whose x holds a NaN is NaN without the sum.
__device__ __forceinline__ bool not_finite8(const float (&f)[8]) {
  bool odd = false;
#pragma unroll
  for (int q = 0; q < 8; ++q) odd |= !(fabsf(f[q]) < INFINITY);
  return odd;
}
inline __device__ __noinline__ void lora_again8(const RaggedParams& p, const int* off, int e, int64_t token, int sorted, int col, float* f) {
  const uint16_t* x = p.x + token * p.K;
  bool nan = false;
  for (int k = 0; k < p.K; k += 8) {
    float a[8];
    unpack_bf8(ld_stream_v4(x + k), a);
#pragma unroll
    for (int q = 0; q < 8; ++q) nan |= a[q] != a[q];
  }
  float sum[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) sum[q] = nan ? NAN : 0.0f;
  auto add = [&](float a, const uint16_t* row) {
    float b[8];
    unpack_bf8(ld_stream_v4(row), b);
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = fmaf(a, b[q], sum[q]);
  };
  for (int k = 0; !nan && k < p.K; ++k) add(bf(ld_u16(x + k)), p.w + (static_cast<int64_t>(e) * p.K + k) * p.n + col);
  for (int a = 0; !nan && sorted >= 0 && a < p.L; ++a) {
    if (sorted < off[a] || sorted >= off[a + 1]) continue;
    const uint16_t* b = p.lora_b + (static_cast<int64_t>(e) * p.L + a) * p.rank * p.n + col;
    for (int k = 0; k < p.rank; ++k) add(ld_f32(p.v + static_cast<int64_t>(sorted) * p.rank + k), b + static_cast<int64_t>(k) * p.n);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = sum[q];
}
__device__ __forceinline__ void lora_settle8(const RaggedParams& p, const int* off, int e, int64_t token, int sorted, int col, float (&f)[8]) {
  if (!not_finite8(f)) return;
  float again[8];
  lora_again8(p, off, e, token, sorted, col, again);
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = again[q];
}

}  // namespace tpx
