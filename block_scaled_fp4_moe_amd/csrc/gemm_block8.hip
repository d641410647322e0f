// fp8_block_linear and fp8_block_grouped_gemm: E4M3 x E4M3 with one scale per
// 1x128 block of the activations and per 128x128 block of the weights.
//
//   out[m,n] = sum_b sa[m,b] * sw[n/128,b] * sum_{k in b} A[m,k] W[n,k]
//
// The scales are arbitrary floats, so they cannot enter the MFMA (its scale
// operands are powers of two).  Each 128-wide block is multiplied into a fresh
// accumulator (C = 0) and joined with one fma per result element.  Weights are
// the first MFMA operand and activations the second: a lane's results then
// belong to one activation row, and both scales of a result tile are one
// number per lane.
#include "fp8_block.h"

#include <algorithm>
#include <type_traits>

namespace fp4moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct Block8Params {
  int M, N, K, a_rows;
  const uint8_t* a;
  int64_t lda;
  const float* a_scale;
  int64_t as_row, as_blk;
  const uint8_t* w;
  int64_t ldw, w_expert;
  const float* w_scale;
  int64_t ld_ws, ws_expert;
  void* out;
  int64_t ldo;
  int n_experts, block_m, gather_div, max_tiles;   // n_experts 0: dense
  uint32_t tile_run, col_split;
  const int32_t *gather, *offsets, *tiles, *n_tiles;
};

// Output types: one value, and two packed (the conversion instructions round to
// nearest even).
struct OutBf16 {
  using type = uint16_t;
  __device__ static __forceinline__ uint16_t of(float f) { return TBf16::down(f); }
  __device__ static __forceinline__ uint32_t of2(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
  }
};
struct OutF16 {
  using type = uint16_t;
  __device__ static __forceinline__ uint16_t of(float f) { return TF16::down(f); }
  __device__ static __forceinline__ uint32_t of2(float a, float b) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
  }
};
// Rows [row0, row_end) of the output that a row tile covers, its expert's
// weights, and the activation row behind an output row.  Index tensors are
// data: whatever they hold, rows stay inside [0, M) and [0, a_rows).
struct RowTile {
  int row0, row_end;
  const uint8_t* w;
  const float* ws;
};

__device__ __forceinline__ bool find_tile(const Block8Params& p, int t, int rows_per_tile,
                                          RowTile& rt) {
  if (p.n_experts == 0) {
    rt.row0 = t * rows_per_tile;
    rt.row_end = rt.row0 + min(p.M - rt.row0, rows_per_tile);
    rt.w = p.w;
    rt.ws = p.w_scale;
    return rt.row0 < p.M;
  }
  const int sub = max(p.block_m / rows_per_tile, 1), entry = t / sub;
  if (entry >= p.max_tiles) return false;
  const int n = *p.n_tiles, e = p.tiles[2 * entry], m = p.tiles[2 * entry + 1];   // one latency
  if (entry >= n || e < 0 || e >= p.n_experts || m < 0) return false;
  const int64_t lo = max(p.offsets[e], 0), hi = min(p.offsets[e + 1], p.M);
  // entries of the list cover block_m rows: smaller tiles share one, and of larger
  // ones the segment has no more than entries, so entry m stands for tile m
  const int64_t r0 = lo + ((int64_t)m * sub + t % sub) * rows_per_tile;
  if (r0 >= hi) return false;
  rt.row0 = (int)r0;
  rt.row_end = (int)min(hi, r0 + rows_per_tile);
  rt.w = p.w + e * p.w_expert;
  rt.ws = p.w_scale + e * p.ws_expert;
  return true;
}

__device__ __forceinline__ int a_row_of(const Block8Params& p, int r) {
  if (p.gather) r = (int)((uint32_t)max(p.gather[r], 0) / (uint32_t)p.gather_div);
  return min(r, p.a_rows - 1);
}

// ---------------------------------------------------------------------------
// Few rows: weights stream from memory once and set the time (1 x 4096 x 7168: 7.6 us,
// 3.9 TB/s; of it a launch, one memory latency and the join).
//
// A workgroup owns 16 weight rows x 16 activation rows; its NW waves take the
// 128-wide K blocks in turn, U of them in flight each, and their sums are joined
// through LDS in wave order.  v_mfma_f32_16x16x128_f8f6f4 multiplies exactly one
// scale block.  Operands go from memory straight to registers: lane l holds the
// 16-byte pieces l/16 and l/16 + 4 of row l%16 (the same K order on both sides, so
// the products pair up whatever order the instruction takes), which makes each
// load instruction read 64 contiguous bytes a row.  TAIL: the last block is short;
// pieces past the row's end are zero.
template <int NW, int U, bool TAIL, class Out>
__global__ __launch_bounds__(NW * 64) void skinny_kernel(Block8Params p, int64_t tiles) {
  __shared__ float red[NW][16][20];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  // work items: row tile outer, weight rows inner
  const int n_blocks = (p.N - 1) / 16 + 1;      // N may be the largest int
  for (int64_t item = blockIdx.x; item < tiles * n_blocks; item += gridDim.x) {
    RowTile rt;
    if (!find_tile(p, (int)(item / n_blocks), 16, rt)) continue;
    const int n0 = (int)(item % n_blocks) * 16;
    const uint8_t* wrow = rt.w + (int64_t)min(n0 + r16, p.N - 1) * p.ldw + g * 16;
    const float* wsc = rt.ws + (int64_t)(n0 >> 7) * p.ld_ws;   // 16 rows lie in one 128-row block
    const int r = a_row_of(p, min(rt.row0 + r16, rt.row_end - 1));
    const uint8_t* arow = p.a + (int64_t)r * p.lda + g * 16;
    const float* asc = p.a_scale + (int64_t)r * p.as_row;
    v4f acc = {0.f, 0.f, 0.f, 0.f};

    // NB K blocks from block c on, NW apart
    auto step = [&](auto n_of, int c) {
      constexpr int NB = decltype(n_of)::value;
      u4v wv[NB][2], av[NB][2];
      float sa[NB], sw[NB];
      auto load = [&](const uint8_t* q, int b, int h) -> u4v {
        const int k = b * 128 + h * 64;
        if constexpr (TAIL) {
          const bool in = k + g * 16 < p.K;
          const u4v v = *reinterpret_cast<const u4v*>(q + (in ? k : -g * 16));
          return in ? v : u4v{0, 0, 0, 0};
        }
        return *reinterpret_cast<const u4v*>(q + k);
      };
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int b = c + u * NW;
        wv[u][0] = load(wrow, b, 0);
        wv[u][1] = load(wrow, b, 1);
        sw[u] = wsc[b];
        av[u][0] = load(arow, b, 0);
        av[u][1] = load(arow, b, 1);
        sa[u] = asc[b * p.as_blk];
      }
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        v8i af, bf;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          af[d] = (int)wv[u][0][d], af[4 + d] = (int)wv[u][1][d];
          bf[d] = (int)av[u][0][d], bf[4 + d] = (int)av[u][1][d];
        }
        const v4f zero = {0.f, 0.f, 0.f, 0.f};
        v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af, bf, zero, 0, 0, 0, 0, 0, 0);
        // the operands stay live past the MFMA: its result never takes their registers
        asm volatile("" : "+v"(part) : "v"(af), "v"(bf));
        const float s = sa[u] * sw[u];
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[d] = fmaf(part[d], s, acc[d]);
      }
    };
    using std::integral_constant;
    const int blocks = (p.K + 127) >> 7;
    int c = wave;
    for (; c + (U - 1) * NW < blocks; c += U * NW) step(integral_constant<int, U>{}, c);
    const int left = c < blocks ? (blocks - 1 - c) / NW + 1 : 0;
    static_assert(U == 4, "what is left: 0 to 3 blocks");
    if (left == 3) step(integral_constant<int, 3>{}, c);
    else if (left == 2) step(integral_constant<int, 2>{}, c);
    else if (left == 1) step(integral_constant<int, 1>{}, c);

    // lane l holds results (n = 4*(l/16) + d, m = l%16)
    *reinterpret_cast<v4f*>(&red[wave][r16][g * 4]) = acc;
    __syncthreads();
#pragma unroll
    for (int o = threadIdx.x; o < 256; o += NW * 64) {
      const int m = o >> 4, n = o & 15;
      if (rt.row0 + m < rt.row_end && n0 + n < p.N) {
        float sum = red[0][m][n];
#pragma unroll
        for (int w = 1; w < NW; ++w) sum += red[w][m][n];
        static_cast<typename Out::type*>(p.out)[(int64_t)(rt.row0 + m) * p.ldo + n0 + n] = Out::of(sum);
      }
    }
    __syncthreads();   // the next item writes red again
  }
}

// ---------------------------------------------------------------------------
// Many rows: tiles of WM*MT*32 activation rows x WN*NT*32 weight rows through
// LDS, v_mfma_f32_32x32x64_f8f6f4 twice per 128-wide block.
//
// Measured: 16384 x 7168 x 7168 0.71 to 0.73 ms = 2.3 to 2.4 PFLOP/s, the matrix units busy 64% of the
// cycles at 1.8 GHz (power sets the clock); 8192 tokens over 384 + 1 experts of 4096 x 7168
// 3.45 ms, bound by weights (19.5 GB leave L2, 5.7 TB/s); 8 tokens over the same 0.31 ms =
// 5.8 TB/s; 64 x 7168 x 2048 7.0 us, latencies.
//
// A K block of a row is 128 bytes, one cache line: rows are copied to LDS as they
// are (global_load_lds_dwordx4, eight rows an instruction), two buffers deep.
// The 16-byte piece p of row r sits at slot p ^ (r/2 % 8) of its 128 bytes: sixteen
// lanes that read the same piece of sixteen rows then touch every one of the 64
// banks once (r % 8 instead, two rows to a bank, showed half of the LDS cycles as
// conflicts).  The permutation is applied to the copies' source addresses,
// within the line.
// Lane l of K step ks takes pieces 4*ks + 2*(l/32) and the next of row l % 32, on
// both sides alike.
//
// Wave (mi, ni) owns weight rows [ni*NT*32, +NT*32) of the tile, inside one
// 128-row scale block, and the 32-row activation tiles mi, mi + WM, ...: where
// a segment ends inside the tile the dead ones are spread over the waves, and
// the two waves of a SIMD (w and w + 4) own different mi.
typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void copy4(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("global_load_lds_dword %0, %1"
               :: "v"(voff), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}
__device__ __forceinline__ void copy16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("global_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// The row tile and column block of a workgroup (workgroups go to the XCDs in
// turn).  Dense: XCD x takes a contiguous eighth of the items, in groups of eight
// row tiles, weight columns outside, so that its 32 workgroups share both operands
// in L2.  Experts: col_split XCDs take tile_run consecutive tiles of the list at a
// time and deal out their column blocks (whose workgroups share activation rows), or,
// with few tiles, the column blocks of a tile go round the XCDs; nothing here
// waits for the tile count.
// (At most kMaxGrid items: 32-bit arithmetic.)
__device__ __forceinline__ bool pick_item(const Block8Params& p, int bm, uint32_t n_blocks,
                                          uint32_t slot_id, int& t, int& nb) {
  const uint32_t xcd = slot_id & 7, slot = slot_id >> 3;
  if (p.n_experts) {
    const uint32_t run = p.tile_run;
    if (run == 0) {
      t = (int)(slot_id / n_blocks);
      nb = (int)(slot_id - t * n_blocks);
      return true;
    }
    const uint32_t per = n_blocks / p.col_split, idx = slot / per;   // column blocks of a tile here
    t = (int)((idx / run * (8 / p.col_split) + xcd / p.col_split) * run + idx % run);
    nb = (int)((slot - idx * per) * p.col_split + xcd % p.col_split);
    return true;
  }
  const uint32_t n_t = (uint32_t)(p.M + bm - 1) / (uint32_t)bm;
  const uint32_t total = n_t * n_blocks, per = (total + 7) / 8, it = xcd * per + slot;
  if (slot >= per || it >= total) return false;
  const uint32_t g = it / (8 * n_blocks), r = it - g * 8 * n_blocks;
  const uint32_t gm = min(8u, n_t - g * 8);
  t = (int)(g * 8 + r % gm);
  nb = (int)(r / gm);
  return true;
}

//
// KG > 1: KG groups of WM*WN waves with buffers of their own take the K blocks
// in turn (group g blocks g, g + KG, ...) and their sums are added in group order
// through LDS.  A block in flight takes a memory latency whatever its size, so
// few tiles with many blocks need several under way (one group of the 64x64 tile
// takes about 0.8 us a block).
//
// WS: buffers of the weight blocks (2, or 3: their copies then have two turns to land;
// experts' weights come from memory, activations from L2).
template <int WM, int WN, int MT, int NT, int KG, int WS, int OCC, bool GROUPED, class Out>
__global__ __launch_bounds__(KG * WM * WN * 64, OCC) void tile_kernel(Block8Params p) {
  constexpr int NW = WM * WN, BM = WM * MT * 32, BN = WN * NT * 32;
  constexpr int AJ = BM / 8 / NW, WJ = BN / 8 / NW;      // copies a wave makes per K block
  constexpr int A_BUF = BM * 128, W_BUF = BN * 128, OFF_W = 2 * A_BUF;
  constexpr int PITCH = NT * 64 + 16;                    // epilogue row of a wave, bytes
  constexpr int EPI = NW * MT * 32 * PITCH;
  constexpr int SW_AT = (BM + 63) / 64 * 256, S_STAGE = SW_AT + 256;   // scales of a block: rows, weight blocks
  constexpr int OFF_S = OFF_W + WS * W_BUF, RING = OFF_S + 2 * S_STAGE;
  constexpr int SUMS = NT * MT * 4096;                   // a wave's sums, bytes
  constexpr int LDS = KG * RING > EPI ? KG * RING : EPI;
  static_assert(LDS <= 160 * 1024 && (KG - 1) * NW * SUMS <= LDS, "LDS");
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
  const int lane = threadIdx.x & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG > 1 ? wave_id / NW : 0, wave = wave_id - kg * NW;   // K group, wave in it
  uint8_t* const smem = lds + kg * RING;
  const int ni = wave / WM, mi = (wave + (NW == 8 ? WM / 2 * (wave >> 2) : 0)) % WM;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + kg * RING;

  int t, nb;
  if (!pick_item(p, BM, (p.N + BN - 1) / BN, blockIdx.x, t, nb)) return;
  RowTile rt;
  if (!find_tile(p, t, BM, rt)) return;
  const int n0 = nb * BN;
  const int live_tiles = (rt.row_end - rt.row0 + 31) / 32;
  const int live = __builtin_amdgcn_readfirstlane(
      live_tiles > mi ? (live_tiles - mi + WM - 1) / WM : 0);   // this wave's 32-row tiles

  // copy sources: lane i brings slot i%8 of row i/8 of its eight rows, which
  // holds piece (i%8) ^ (i/16), with bit 2 flipped in every other group of rows
  static_assert(AJ >= 1 && WJ >= 1 && AJ * NW * 8 == BM && WJ * NW * 8 == BN, "copies");
  // (pieces past the end of rows shorter than a block: their first piece instead)
  const uint32_t piece = (lane & 7) ^ (lane >> 4);
  auto piece_at = [&](int group) -> uint32_t {
    const uint32_t at = (piece ^ (4 * (group & 1))) * 16;
    return at < (uint32_t)p.K ? at : 0;
  };
  uint32_t a_off[AJ], w_off[WJ];
#pragma unroll
  for (int j = 0; j < AJ; ++j) {
    const int r = min(rt.row0 + (wave * AJ + j) * 8 + (lane >> 3), rt.row_end - 1);
    a_off[j] = (uint32_t)a_row_of(p, r) * (uint32_t)p.lda + piece_at(wave * AJ + j);
  }
#pragma unroll
  for (int j = 0; j < WJ; ++j)
    w_off[j] = (uint32_t)min(n0 + (wave * WJ + j) * 8 + (lane >> 3), p.N - 1) * (uint32_t)p.ldw +
               piece_at(wave * WJ + j);
  // one register each, not the pairs that the 64-bit products left
#pragma unroll
  for (int j = 0; j < AJ; ++j) asm volatile("" : "+v"(a_off[j]));
#pragma unroll
  for (int j = 0; j < WJ; ++j) asm volatile("" : "+v"(w_off[j]));
  // Whole K blocks and the bytes of a short last one, which comes first: it is the first
  // turn of group 0.  Turns past a group's blocks take the last whole one again.
  const int full = p.K >> 7, tail = p.K & 127, total = full + (tail ? 1 : 0);
  const int turns = (total + KG - 1) / KG;
  const bool short_first = tail && kg == 0;
  auto block_of = [&](int turn) { return max(min(kg + turn * KG - (tail ? 1 : 0), full - 1), 0); };
  // This wave's copies of K block c (of all) into buffer buf; back[group%2] is taken off
  // the lane's source.
  auto copy_a = [&](int c, int buf, const uint32_t* back) {
#pragma unroll
    for (int j = 0; j < AJ; ++j)
      copy16(p.a + (int64_t)c * 128, a_off[j] - back[(wave * AJ + j) & 1],
             lds0 + buf * A_BUF + (wave * AJ + j) * 1024);
  };
  auto copy_w = [&](int c, int buf, const uint32_t* back) {
#pragma unroll
    for (int j = 0; j < WJ; ++j)
      copy16(rt.w + (int64_t)c * 128, w_off[j] - back[(wave * WJ + j) & 1],
             lds0 + OFF_W + buf * W_BUF + (wave * WJ + j) * 1024);
  };
  const uint32_t none[2] = {0, 0};

  // Scales of a block: one number per activation row (64 rows a wave) and one per
  // NT*32 weight rows (the waves left, all the same ones; a lone wave copies both).
  // Loads into registers would make the compiler wait for every copy in flight.
  constexpr int SWAVES = (BM + 63) / 64;
  static_assert(SWAVES < NW || (SWAVES == 1 && NW == 1), "a wave is left for the weight scales");
  const bool row_scales = wave < SWAVES;
  const uint32_t sw_off =
      (uint32_t)(min(n0 + (lane % WN) * NT * 32, p.N - 1) >> 7) * (uint32_t)(p.ld_ws * 4);
  uint32_t s_off = row_scales
      ? (uint32_t)a_row_of(p, min(rt.row0 + wave * 64 + lane, rt.row_end - 1)) * (uint32_t)(p.as_row * 4)
      : sw_off;
  asm volatile("" : "+v"(s_off));
  const float* s_base = row_scales ? p.a_scale : rt.ws;
  const int64_t s_step = row_scales ? p.as_blk : 1;
  const uint32_t s_to = lds0 + OFF_S + (row_scales ? wave * 256 : SW_AT);
  auto copy_scales = [&](int c, int buf) {
    copy4(s_base + c * s_step, s_off, s_to + buf * S_STAGE);
    if constexpr (NW == 1) copy4(rt.ws + c, sw_off, lds0 + OFF_S + SW_AT + buf * S_STAGE);
  };
  v16f acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int d = 0; d < 16; ++d) acc[j][i][d] = 0.f;

  // LDS reads: lane l's piece 2*(l/32) of row l % 32; pieces of the other half and
  // K step differ in two bits of the slot.
  const uint32_t lane_slot =
      (lane & 31) * 128 + ((((lane >> 5) * 2) ^ ((lane >> 1) & 7)) * 16);
  auto frag = [&](uint32_t base, int tile, int ks) -> v8i {
    const uint8_t* lo = smem + ((lane_slot ^ (64 * ks)) + base);
    const uint8_t* hi = smem + ((lane_slot ^ (64 * ks + 16)) + base);
    const u4v l = *reinterpret_cast<const u4v*>(lo + tile * 4096);
    const u4v h = *reinterpret_cast<const u4v*>(hi + tile * 4096);
    return v8i{(int)l[0], (int)l[1], (int)l[2], (int)l[3], (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
  };
  // The group's reads are done and its copies have landed, but for the newest
  // weight block's with three buffers.  (A barrier takes in all groups; a group of one
  // wave has no one to wait for.)
  static_assert(WS == 2 || WS == 3, "weight buffers");
  auto sync = [&]() {
    constexpr int NEWEST = (WS - 2) * WJ;
    if constexpr (NW == 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(NEWEST) : "memory");
    else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(NEWEST) : "memory");
  };
  auto sync_all = [&]() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  // Pieces past the end of a short block would lie outside the operand for its last
  // row: they are copied from the block's first piece and cleared in LDS.
  auto clear_tail = [&]() {
    for (int e = wave * 64 + lane; e < (BM + BN) * 8; e += NW * 64) {
      const int r = e >> 3, pc = e & 7;
      if (pc >= (tail >> 4))
        *reinterpret_cast<uint4*>(smem + (r < BM ? r * 128 : OFF_W + (r - BM) * 128) +
                                  ((pc ^ ((r >> 1) & 7)) * 16)) = make_uint4(0, 0, 0, 0);
    }
  };

  // The K loop of a wave that has L live 32-row tiles.  Every wave passes the
  // same barriers, whatever its L.
  //
  // One step multiplies a 32x32 result tile over the block (two MFMAs) while the
  // previous step's sums are scaled and added: `part` alternates, and the last
  // step of a block is added during the first of the next.  Operands are read
  // one step or more ahead.  The one barrier of a block sits behind the MFMAs of
  // its last step but one: by then every operand of block c has been read
  // (its buffer takes block c+2 from here on) and block c+1 has landed, whose first
  // operands are read under the last MFMAs.  The fences keep the compiler
  // from hoisting operand reads until the registers spill.
  auto k_loop = [&](auto live_n) {
    constexpr int L = decltype(live_n)::value;
    constexpr int STEPS = NT * L;
    static_assert(STEPS != 1 && STEPS % 2 == 0, "part alternates over blocks too");
    constexpr int L1 = L ? L : 1;
    v16f part[2];
    v8i af[L1][2], wf[2][2];
    float s_last = 0.f, s[L1];
    const uint32_t a_base = mi * 4096, w_base = OFF_W + ni * NT * 4096;
    // of the block in buffer buf; a turn that a group has no block for multiplies
    // the last block again, and adds it with scale 0
    auto scales = [&](int buf, int turn) {
      const float* q = reinterpret_cast<const float*>(smem + OFF_S + buf * S_STAGE);
#pragma unroll
      for (int i = 0; i < L; ++i) {
        s[i] = q[(mi + i * WM) * 32 + (lane & 31)] * q[SW_AT / 4 + ni];
        if (KG > 1 && kg + turn * KG >= total) s[i] = 0.f;
      }
    };
#pragma unroll
    for (int d = 0; d < 16; ++d) part[0][d] = part[1][d] = 0.f;
    uint32_t back[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = (piece ^ (4 * h)) * 16;
      back[h] = short_first && full > 0 && at >= (uint32_t)tail ? at : 0;
    }
    const int c0 = short_first ? full : block_of(0);
    copy_a(c0, 0, back);
    copy_scales(c0, 0);
    copy_w(c0, 0, back);
    if (WS == 3) copy_w(block_of(1), 1, none);
    sync();
    if (tail) {
      if (kg == 0) clear_tail();
      sync();
    }
    copy_a(block_of(1), 1, none);
    copy_scales(block_of(1), 1);
    copy_w(block_of(WS - 1), WS - 1, none);
    if constexpr (L > 0) {
      scales(0, 0);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        wf[0][ks] = frag(w_base, 0, ks);
#pragma unroll
        for (int i = 0; i < L; ++i) af[i][ks] = frag(a_base, i * WM, ks);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    int w_buf = 0;
    for (int c = 0; c < turns; ++c) {
      // The block two turns on; past the last whole block that one is copied
      // again, into the buffer that is free (no branch in the steps).
      const int a_next = block_of(c + 2), w_next = block_of(c + WS), buf = c & 1;
      const int w_after = w_buf + 1 == WS ? 0 : w_buf + 1;
      if constexpr (L == 0) {
        sync();
        copy_a(a_next, buf, none);
        copy_scales(a_next, buf);
        copy_w(w_next, w_buf, none);
      } else {
        const uint32_t wst = w_base + w_buf * W_BUF, w_follows = w_base + w_after * W_BUF;
        const uint32_t a_follows = a_base + (buf ^ 1) * A_BUF;
        float s_now[L];
#pragma unroll
        for (int i = 0; i < L; ++i) s_now[i] = s[i];
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
          const int j = q / L, i = q % L;
          if (i == 0 && j + 1 < NT) {
            wf[(j + 1) & 1][0] = frag(wst, j + 1, 0);
            wf[(j + 1) & 1][1] = frag(wst, j + 1, 1);
          }
          v16f z;
#pragma unroll
          for (int d = 0; d < 16; ++d) z[d] = 0.f;
          z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[j & 1][0], af[i][0], z, 0, 0, 0, 0, 0, 0);
          z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[j & 1][1], af[i][1], z, 0, 0, 0, 0, 0, 0);
          // the operands stay live past the MFMAs: no result takes their registers
          asm volatile("" : "+v"(z) : "v"(wf[j & 1][0]), "v"(wf[j & 1][1]), "v"(af[i][0]), "v"(af[i][1]));
          part[q & 1] = z;
          __builtin_amdgcn_sched_barrier(0);
          if (q == STEPS - 2) {
            sync();
            scales(buf ^ 1, c + 1);
          }
          // first operands of the next block, into registers whose last use is past
          if (q == STEPS - 1) {
            wf[0][0] = frag(w_follows, 0, 0);
            wf[0][1] = frag(w_follows, 0, 1);
          }
#pragma unroll
          for (int r = 0; r < L; ++r)
            if ((q == STEPS - 2 && j == NT - 1 && r <= i) || (q == STEPS - 1 && r == i)) {
              af[r][0] = frag(a_follows, r * WM, 0);
              af[r][1] = frag(a_follows, r * WM, 1);
            }
          if (q == STEPS - 2) {
            copy_a(a_next, buf, none);
            copy_scales(a_next, buf);
          }
          if (q == STEPS - 1) copy_w(w_next, w_buf, none);
          // the step before: of this block, or the last of the block before
          const int pq = (q + STEPS - 1) % STEPS, pj = pq / L, pi = pq % L;
          const float ps = q == 0 ? s_last : s_now[pi];
#pragma unroll
          for (int d = 0; d < 16; ++d) acc[pj][pi][d] = fmaf(part[(q + 1) & 1][d], ps, acc[pj][pi][d]);
          __builtin_amdgcn_sched_barrier(0);
        }
        s_last = s_now[L - 1];
      }
      w_buf = w_after;
    }
    if constexpr (L > 0)
#pragma unroll
      for (int d = 0; d < 16; ++d)
        acc[NT - 1][L - 1][d] = fmaf(part[1][d], s_last, acc[NT - 1][L - 1][d]);
  };
  if (!GROUPED || live == MT) k_loop(std::integral_constant<int, MT>{});
  else if (MT > 2 && live == 2) k_loop(std::integral_constant<int, (MT > 2 ? 2 : MT)>{});
  else if (MT > 1 && live > 0) k_loop(std::integral_constant<int, NT % 2 ? MT : 1>{});
  else k_loop(std::integral_constant<int, 0>{});
  static_assert(MT <= 3, "live counts handled");

  // Results of a lane: activation row l % 32, weight rows 8q + 4*(l/32) + d.
  // Through LDS into rows of the output, 16 bytes a lane (the copies that the
  // last block issued have to land first).
  sync_all();
  if constexpr (KG > 1) {
    float4* sums = reinterpret_cast<float4*>(lds);
    if (kg > 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int d = 0; d < 4; ++d)
            sums[((((kg - 1) * NW + wave) * NT * MT + j * MT + i) * 4 + d) * 64 + lane] =
                make_float4(acc[j][i][4 * d], acc[j][i][4 * d + 1], acc[j][i][4 * d + 2],
                            acc[j][i][4 * d + 3]);
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll 1
      for (int g = 0; g < KG - 1; ++g)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const float4 v = sums[(((g * NW + wave) * NT * MT + j * MT + i) * 4 + d) * 64 + lane];
              acc[j][i][4 * d] += v.x, acc[j][i][4 * d + 1] += v.y;
              acc[j][i][4 * d + 2] += v.z, acc[j][i][4 * d + 3] += v.w;
            }
    }
    __syncthreads();
    if (kg > 0) return;                // no barrier of the whole workgroup follows
  }
  uint8_t* ep = lds + wave * (MT * 32 * PITCH);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        *reinterpret_cast<uint2*>(ep + (i * 32 + (lane & 31)) * PITCH + j * 64 + q * 16 +
                                  (lane >> 5) * 8) =
            make_uint2(Out::of2(acc[j][i][4 * q], acc[j][i][4 * q + 1]),
                       Out::of2(acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]));
      }
  // a wave reads what it wrote itself
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  wait_lds();
  uint16_t* out = static_cast<uint16_t*>(p.out);
  constexpr int LPR = NT * 4, ROWS = 64 / LPR;           // lanes per row of NT*32 values, rows at a time
  const int lr0 = lane / LPR, col = (lane % LPR) * 8, n = n0 + ni * NT * 32 + col;
  auto row_of = [&](int lr) { return rt.row0 + (mi + (lr >> 5) * WM) * 32 + (lr & 31); };
  // Stores of 16 bytes at any address of an element (the hardware takes them; odd N:
  // 16000 x 700 x 400 33.5 us element by element, 17.6 so).
  if (n0 + BN <= p.N && rt.row0 + BM <= rt.row_end) {
#pragma unroll 4
    for (int lr = lr0; lr < MT * 32; lr += ROWS) {
      const uint4 v = *reinterpret_cast<const uint4*>(ep + lr * PITCH + col * 2);
      __builtin_memcpy(out + (int64_t)row_of(lr) * p.ldo + n, &v, 16);
    }
    return;
  }
  if (n >= p.N) return;
#pragma unroll 4
  for (int lr = lr0; lr < MT * 32; lr += ROWS) {
    const uint4 v = *reinterpret_cast<const uint4*>(ep + lr * PITCH + col * 2);
    const int row = row_of(lr);
    if (row >= rt.row_end) continue;
    uint16_t* o = out + (int64_t)row * p.ldo + n;
    if (n + 8 <= p.N) {
      __builtin_memcpy(o, &v, 16);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      for (int d = 0; d < 8; ++d)
        if (n + d < p.N) o[d] = (uint16_t)(w[d >> 1] >> (16 * (d & 1)));
    }
  }
}

// Workgroups of one launch at most (a HIP grid holds fewer than 2^32 threads).  A
// workgroup of the tile kernel takes one item, so products of more items go to the 16x16
// kernel, which steps over the rest of its own.
constexpr int64_t kMaxGrid = 1 << 20;

// Which kernel takes a product.  Measured on MI355X (us a launch; bfloat16 out, weights
// from memory; "x3" K groups, "w3" three weight buffers):
//
// dense 4096 x 7168   M=16    64   128   256   512  1024  2048  4096
//   16x16                11    29    66
//   64x32 x6             14    17    17    30    55
//   64x64 x4                   24    23    23    43    81
//   64x128 x3                  35    34    33    34    63   124
//   128x128 x2                             43    44    45    84
//   128x256 w3                                         53    61   122
//   192x256 w3                                         67    75   141
//   256x256                                            90    92   107
// A tile shape is best up to one workgroup on each of the 256 CUs, then the next one;
// the same held at 7168 x 2048, 1000 x 2000 and 576 x 7168.  With few K blocks there is
// nothing for K groups to take in parallel: 64x128 alone (2048 x 512: M=256 4.9 against
// 5.1, M=1024 6.1 against 7.2).  Of the large shapes a round of workgroups takes about
// 1, 0.79 and 0.57 (7168 x 7168: M=3000 181, 152, 165; M=8192 395, 388, 405; M=16384 720,
// 791, 819).
//
// experts, 384 + 1 of 4096 x 7168, unevenly routed:
//   tokens               64   256  1024  2048  4096  8192   (average rows 1.5 .. 191)
//   64x128              952  1595  2179  3421  4444  6485
//   128x256 w3          997  1664  2190  2199  2679  3747
//   192x256 w3         1013  1689  2240  2161  2643  3643
//   256x256            1182  1971  2634  2480  2902  3869
// (Averages above these were not timed and take the last row's shape.)
// Few tiles: 16x16 (9 tiles x 32 column blocks of 128: 56 against 63 for 64x128), K groups
// (15 x 32: 49 against 63).
template <class Out>
void launch(const Block8Params& p, hipStream_t s) {
  const bool dense = p.n_experts == 0;
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  auto workgroups = [&](int bm, int bn) { return ceil_div(p.M, bm) * ceil_div(p.N, bn); };
  auto tiled = [&](auto kernel, int bm, int bn, int threads) {
    const int64_t tiles = dense ? ceil_div(p.M, bm) : p.max_tiles * ceil_div(p.block_m, bm);
    // Small tiles are dealt out singly, few of them by column block.  Large ones: the
    // tiles of an expert should meet in one L2 (they read the same weights), its XCDs
    // should have tiles of the same sizes at a time (workgroups start on them strictly in
    // turn), and an activation row should not go to too many: eight tiles at
    // a time to four XCDs.  8192 tokens, 384 + 1 experts of 4096 x 7168, unevenly routed:
    // 3400 us, to one XCD 3700 (four tiles: 3640), to eight 3515.  Column blocks that do not
    // divide by four would leave some of the XCDs idle (N = 1600, 48 + 1 experts: 123 us,
    // 114 as four tiles to one).
    Block8Params q = p;
    const bool split = bm > 64 && ceil_div(p.N, bn) % 4 == 0;
    q.col_split = split ? 4 : 1;
    q.tile_run = tiles <= 128 ? 0 : split ? 8 : bm > 64 ? 4 : 1;
    // grids in multiples of what pick_item deals out
    const int64_t run = dense || q.tile_run == 0 ? 1 : 8 / q.col_split * q.tile_run;
    const int64_t items = ceil_div(tiles, run) * run * ceil_div(p.N, bn);
    if (items > kMaxGrid) return false;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(ceil_div(items, 8) * 8)), dim3(threads), 0, s, q);
    return true;
  };
  auto go = [&](auto dense_kernel, auto expert_kernel, int bm, int bn, int threads) {
    return dense ? tiled(dense_kernel, bm, bn, threads) : tiled(expert_kernel, bm, bn, threads);
  };
#define FP8BLOCK_TILE(WM, WN, MT, NT, KG, WS, OCC)                                          \
  go(tile_kernel<WM, WN, MT, NT, KG, WS, OCC, false, Out>,                                  \
     tile_kernel<WM, WN, MT, NT, KG, WS, OCC, true, Out>, WM * MT * 32, WN * NT * 32,       \
     KG * WM * WN * 64)
  // the tile kernel has 32-bit byte offsets
  const bool tiles = (int64_t)p.a_rows * p.lda <= UINT32_MAX &&
                     (int64_t)p.N * p.ldw <= UINT32_MAX &&
                     (int64_t)p.a_rows * p.as_row <= UINT32_MAX / 4 &&
                     ceil_div(p.N, 128) * p.ld_ws <= UINT32_MAX / 4;
  bool done = false;
  if (tiles && dense) {
    // the 16x16 kernel reads both operands once a tile through L2: good while that is little
    const double skinny_bytes = ceil_div(p.M, 16) * ceil_div(p.N, 16) * 32.0 * p.K;
    if (p.M <= 16 || (p.M <= 128 && skinny_bytes <= 48e6)) done = false;
    else if (p.K <= 1024 && workgroups(64, 128) <= 768) done = FP8BLOCK_TILE(1, 4, 2, 1, 1, 2, 3);
    else if (workgroups(64, 32) <= 256) done = tiled(tile_kernel<1, 1, 2, 1, 6, 2, 2, false, Out>, 64, 32, 384);
    else if (workgroups(64, 64) <= 256) done = tiled(tile_kernel<1, 2, 2, 1, 4, 2, 2, false, Out>, 64, 64, 512);
    else if (workgroups(64, 128) <= 256) done = FP8BLOCK_TILE(1, 4, 2, 1, 3, 2, 3);
    else if (workgroups(128, 128) <= 256) done = tiled(tile_kernel<2, 2, 2, 2, 2, 2, 2, false, Out>, 128, 128, 512);
    else {
      const double t256 = (double)ceil_div(workgroups(256, 256), 256);
      const double t192 = 0.79 * ceil_div(workgroups(192, 256), 256);
      const double t128 = 0.57 * ceil_div(workgroups(128, 256), 256);
      if (t128 < t192 && t128 < t256) done = FP8BLOCK_TILE(2, 4, 2, 2, 1, 3, 2);
      else if (t192 < t256) done = FP8BLOCK_TILE(2, 4, 3, 2, 1, 3, 2);
      else done = tiled(tile_kernel<4, 2, 2, 4, 1, 2, 2, false, Out>, 256, 256, 512);
    }
  } else if (tiles) {
    const int64_t average = p.M / p.n_experts;
    const int64_t wgs = std::min<int64_t>(p.max_tiles, p.n_experts + p.M / 64) * ceil_div(p.N, 128);
    if (average > 128) done = FP8BLOCK_TILE(2, 4, 3, 2, 1, 3, 2);
    else if (average > 32) done = FP8BLOCK_TILE(2, 4, 2, 2, 1, 3, 2);
    else if (wgs >= 400) done = FP8BLOCK_TILE(1, 4, 2, 1, 1, 2, 3);
    else if (p.M > 32) done = FP8BLOCK_TILE(1, 4, 2, 1, 3, 2, 3);
  }
#undef FP8BLOCK_TILE
  if (done) return;
  const int64_t tiles16 = dense ? ceil_div(p.M, 16) : p.max_tiles * ceil_div(p.block_m, 16);
  const int64_t items = tiles16 * ceil_div(p.N, 16);
  const dim3 grid((unsigned)(items < kMaxGrid ? items : kMaxGrid));
  // Up to two items a CU each has eight waves; of more items eight waves would hold a
  // CU's slots with a block or two each, and two waves keep four in flight: 6 rows over
  // experts of 7168 x 1024 14.6 against 10.7 us (eight, two), 12288 x 2048 M=1 9.1, 7.5; 256 items
  // of 4096 x 7168 M=1 9.2, 11.3; 384 and 512 items within 5% either way.
#define FP8BLOCK_SKINNY(NW, TAIL) \
  hipLaunchKernelGGL((skinny_kernel<NW, 4, TAIL, Out>), grid, dim3(NW * 64), 0, s, p, tiles16)
  if (items > 512) {
    if (p.K & 127) FP8BLOCK_SKINNY(2, true);
    else FP8BLOCK_SKINNY(2, false);
  } else {
    if (p.K & 127) FP8BLOCK_SKINNY(8, true);
    else FP8BLOCK_SKINNY(8, false);
  }
#undef FP8BLOCK_SKINNY
}

int run(const char* name, const fp8block_gemm_args* a, bool grouped, void* stream) {
  FP4MOE_REQUIRE(a, "%s: null args", name);
  FP4MOE_REQUIRE(a->M >= 0 && a->N >= 1 && a->K >= 16 && a->K % 16 == 0,
                 "%s: M=%d N=%d K=%d (K %% 16 != 0)", name, a->M, a->N, a->K);
  FP4MOE_REQUIRE(a->out_dtype == FP8BLOCK_BF16 || a->out_dtype == FP8BLOCK_F16,
                 "%s: out_dtype=%d (bfloat16 or float16)", name, a->out_dtype);
  FP4MOE_REQUIRE(a->lda >= a->K && a->lda % 16 == 0 && a->ldw >= a->K && a->ldw % 16 == 0,
                 "%s: lda=%lld ldw=%lld (multiples of 16, at least K=%d)", name, (long long)a->lda,
                 (long long)a->ldw, a->K);
  FP4MOE_REQUIRE(a->ldo >= a->N, "%s: ldo=%lld for N=%d", name, (long long)a->ldo, a->N);
  FP4MOE_REQUIRE(a->as_row >= 0 && a->as_blk >= 0 && a->ld_ws >= 0, "%s: negative scale stride",
                 name);
  if (grouped) {
    FP4MOE_REQUIRE(a->block_m == 16 || a->block_m == 32 || a->block_m == 64 || a->block_m == 128,
                   "%s: block_m=%d (16, 32, 64 or 128)", name, a->block_m);
    FP4MOE_REQUIRE(a->n_experts >= 1 && a->max_tiles >= 0 && a->gather_div >= 1,
                   "%s: n_experts=%d max_tiles=%d gather_div=%d", name, a->n_experts, a->max_tiles,
                   a->gather_div);
    FP4MOE_REQUIRE((int64_t)a->max_tiles * (a->block_m / 16) <= INT32_MAX,
                   "%s: max_tiles=%d of block_m=%d", name, a->max_tiles, a->block_m);
    FP4MOE_REQUIRE(a->w_expert >= 0 && a->w_expert % 16 == 0 && a->ws_expert >= 0,
                   "%s: w_expert=%lld ws_expert=%lld", name, (long long)a->w_expert,
                   (long long)a->ws_expert);
  }
  if (a->M == 0 || (grouped && a->max_tiles == 0)) return FP4MOE_OK;
  FP4MOE_REQUIRE(a->a_rows >= 1 && (a->a_rows >= a->M || (grouped && a->a_row_gather)),
                 "%s: a_rows=%d for M=%d", name, a->a_rows, a->M);
  FP4MOE_REQUIRE(a->a && a->a_scale && a->w && a->w_scale && a->out, "%s: null pointer", name);
  FP4MOE_REQUIRE((((uintptr_t)a->a | (uintptr_t)a->w) & 15) == 0,
                 "%s: a and w must be 16-byte aligned", name);
  FP4MOE_REQUIRE((((uintptr_t)a->a_scale | (uintptr_t)a->w_scale) & 3) == 0 &&
                     ((uintptr_t)a->out & 1) == 0,
                 "%s: a pointer is not aligned to its element", name);
  FP4MOE_REQUIRE(!grouped || (a->expert_offsets && a->tiles && a->n_tiles), "%s: null pointer",
                 name);
  Block8Params p;
  p.M = a->M, p.N = a->N, p.K = a->K, p.a_rows = a->a_rows;
  p.a = a->a, p.lda = a->lda, p.a_scale = a->a_scale, p.as_row = a->as_row, p.as_blk = a->as_blk;
  p.w = a->w, p.ldw = a->ldw, p.w_expert = grouped ? a->w_expert : 0;
  p.w_scale = a->w_scale, p.ld_ws = a->ld_ws, p.ws_expert = grouped ? a->ws_expert : 0;
  p.out = a->out, p.ldo = a->ldo;
  p.n_experts = grouped ? a->n_experts : 0;
  p.block_m = a->block_m, p.gather_div = a->gather_div, p.max_tiles = a->max_tiles;
  p.gather = grouped ? a->a_row_gather : nullptr;
  p.offsets = a->expert_offsets, p.tiles = a->tiles, p.n_tiles = a->n_tiles;
  FP4MOE_CHECK_DEVICE();
  hipStream_t s = as_stream(stream);
  if (a->out_dtype == FP8BLOCK_BF16) launch<OutBf16>(p, s);
  else launch<OutF16>(p, s);
  return check_launch(name);
}

}  // namespace
}  // namespace fp4moe

using namespace fp4moe;

extern "C" int fp8_block_linear(const fp8block_gemm_args* args, void* stream) {
  return run("fp8_block_linear", args, false, stream);
}

extern "C" int fp8_block_grouped_gemm(const fp8block_gemm_args* args, void* stream) {
  return run("fp8_block_grouped_gemm", args, true, stream);
}
