// Products of microscaled 4-bit operands (mx4.h), both along their rows: y = act(x W^T + b), one weight or one an
// expert. A tile body of its own on the pieces of gemm_dma.hpp: operands go HBM -> LDS by DMA through a ring of K-steps of
// 128 bytes (256 values) a row, 16-byte chunks (one block of 32 values each) XOR-swizzled by row, and come out as the
// fragments of v_mfma_scale_f32_32x32x64_f8f6f4: a lane's 16 bytes are a whole block, so its scale is one byte. The scales of a
// K-step are 8 bytes a row, one run of memory for a tile's rows (mx4.h's planes): one more DMA a wave. In
// substep s of four the lane half h takes block 4 h + s, so a lane's four scales of a step are the four bytes of one word, which
// the instruction picks from by number.
//
// Four waves, 2 x 2, one a SIMD. A 256 x 256 tile's step, one on every CU, takes 1.8 us with random operands (4.8 PFLOP/s; 2.0
// beyond 64 steps) and 1.4 with constant ones; the 4-bit MFMA alone runs at 6 PFLOP/s with random operands (power: 8.4 with constant
// ones), with its LDS reads at 4.9. Beside its steps a tile takes 10 us to start and end, in which its CU multiplies nothing, and a
// launch 4: 4096 x 4096 outputs, one round of 256 tiles, take 28 us at K = 2048, 42 at 4096, 72 at 8192, 129 at 16384 (2.5, 3.2,
// 3.8 and 4.3 PFLOP/s). At K = 2048 constant operands take 26.5: what short K loses there is not power. Half steps of 64 bytes in a
// ring of four were no faster (a DMA of half lines takes 1.28 us a step by itself, of whole ones 1.05).
#pragma once

#include "gemm_dma.hpp"
#include "gemm_experts.hpp"
#include "launch.hpp"
#include "mx4.hpp"

namespace gmlp {

template <int BM, int BN> constexpr int mx_stage_bytes() { return (BM + BN) * (128 + 8); }
template <int BM, int BN> constexpr int mx_ring_bytes() { return ring_stages(mx_stage_bytes<BM, BN>(), BM * BN) * mx_stage_bytes<BM, BN>(); }

// One 32 x 32 x 64 product: A's and B's scales are byte S of sa and sb.
template <int S>
__device__ __forceinline__ void mx_mma(const u32x4& a, const u32x4& b, uint32_t sa, uint32_t sb, f32x16& acc) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc, 4, 4, S, (int)sa, S, (int)sb);   // 4: e2m1
}

// A tile: rows row0 .. row0 + rows - 1 of expert e (e = the number of experts: rows of none) by the columns from n0 on.
struct MxPlace {
  int e, rows, n0, split;
  int64_t row0;
};

// Tile b of the product; false: there is none.
template <int BM, int BNC>
__device__ __forceinline__ bool mx_place(const Mx4Gemm& a, int b, MxPlace& at) {
  const int tiles_n = a.g.tiles_n;
  int tile = 0, split = 0;
  RowPiece t;
  const bool found = find_row_piece(a.offsets, a.experts, a.rows, BM, [&](int total) {
    const int tiles = (int)min((int64_t)total * tiles_n, (int64_t)(a.tiles / a.splits));
    if (b >= tiles * a.splits) return -1;
    tile = xcd_remap(b, tiles * a.splits);
    split = tile / tiles;
    tile -= split * tiles;
    return tile / tiles_n;
  }, t);
  if (!found) return false;
  int tm, tn;
  grouped_tile(tile - t.first * tiles_n, (t.rows + BM - 1) / BM, tiles_n, a.g.group_m, tm, tn);
  at = {t.e, min(t.rows - tm * BM, BM), tn * BNC, split, t.row0 + (int64_t)tm * BM};
  return true;
}

// A tile of rows of no expert: zeros (plus the residual).
template <typename IoT, int BNC, bool GATED>
__device__ __forceinline__ void mx_zero_rows(const GemmArgs& p, const MxPlace& t) {
  constexpr int V = 16 / ElemTraits<IoT>::bytes, W = BNC / V;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int i = threadIdx.x; i < t.rows * W; i += blockDim.x) {
    const int64_t m = t.row0 + i / W;
    const int n = t.n0 + i % W * V;
    if (n >= p.N) continue;
    if (p.flags & 1) {
      *reinterpret_cast<u32x4*>(elem_ptr<IoT>(p.aux, m, p.ld_aux, n)) = zero;
      if (GATED) *reinterpret_cast<u32x4*>(elem_ptr<IoT>(p.aux, m, p.ld_aux, p.half + n)) = zero;
    }
    *reinterpret_cast<u32x4*>(elem_ptr<IoT>(p.C0, m, p.ldc0, n)) =
        p.res ? *reinterpret_cast<const u32x4*>(elem_ptr<IoT>(p.res, m, p.ld_res, n)) : zero;
  }
}

// The K loop of a BM x BN tile of four waves, and its ring. GATED: half of the columns are rows of B0, half of B1.
template <int BM, int BN, bool GATED> struct MxPipe {
  static constexpr int WAVES = 4, WM = BM / 2, WN = BN / 2, MI = WM / 32, NI = WN / 32, BNC = GATED ? BN / 2 : BN;
  static constexpr int BK = 128;   // bytes of a row in a step
  static constexpr int A_BYTES = BM * BK, S_AT = (BM + BN) * BK, STAGE = mx_stage_bytes<BM, BN>();
  static constexpr int NS = ring_stages(STAGE, BM * BN), SCH = (BM + BN) / 2 / WAVES;   // SCH: lanes of a wave's scale DMA
  using DA = KTileDma<e4m3, BM, WAVES>;   // (a byte is its element)
  using DB = KTileDma<e4m3, BN, WAVES>;
  static constexpr int N_DMA = DA::kInst + DB::kInst + 1, N_MMA = MI * NI, N_RD = MI + NI;
  static_assert(NS >= 2 && (NS - 1) * N_DMA < 64, "ring and vmcnt range");

  char* smem;
  int lane, wave, wm, wn, frow, fhalf;
  DA ka;
  DB kb;
  const char* sc;        // per lane: its 16 bytes (two rows') of the first step's scales
  int64_t sc_plane;
  int rows, n0, N, b_split, k_left, planes;
  bool stacked;
  int a_base[MI], b_base[NI];   // first tile row of each block
  u32x4 fa[2][MI], fb[2][NI];
  uint32_t sa[MI], sb[NI], na[MI], nb[NI];
  f32x16 acc[MI][NI];

  __device__ __forceinline__ void init(char* lds) {
    smem = lds;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / 2;
    wn = wave % 2;
    frow = lane & 31;
    fhalf = lane >> 5;
#pragma unroll
    for (int i = 0; i < MI; ++i) a_base[i] = wm * WM + i * 32;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      constexpr int NH = NI / 2;
      b_base[j] = !GATED ? wn * WN + j * 32 : j < NH ? wn * (WN / 2) + j * 32 : BN / 2 + wn * (WN / 2) + (j - NH) * 32;
    }
  }

  // Tile t's operands: bytes [kbeg, kend) of the rows. Rows past the matrix are given an existing row, and pairs of scales past the
  // padded rows the last one (their products are never stored).
  __device__ __forceinline__ void place(const Mx4Gemm& a, const MxPlace& t, int kbeg, int kend) {
    const GemmArgs& p = a.g;
    constexpr int b_half = BN / 2;
    rows = t.rows;
    n0 = t.n0;
    N = p.N;
    b_split = p.b_split;
    stacked = p.B1 != nullptr;
    k_left = kend - kbeg;
    planes = (p.K + BK - 1) / BK - kbeg / BK;
    const char* a0 = static_cast<const char*>(p.A) + t.row0 * p.lda;
    ka.init(lane, kbeg, a0, a0, p.lda, BM, rows == BM);
    const char* w0 = static_cast<const char*>(p.B0) + t.e * a.w_stride;
    const char* w1 = stacked ? static_cast<const char*>(p.B1) + t.e * a.w_stride : nullptr;
    const char* b0 = w0 + (int64_t)n0 * p.ldb;
    const bool inner = n0 + BNC <= N;
    auto before = [&](int64_t rel) { return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(w1) + rel * p.ldb); };
    if constexpr (GATED) kb.init(lane, kbeg, b0, before(n0 - b_half), p.ldb, b_half, inner);
    else if (stacked) kb.init(lane, kbeg, b0, before(n0 - b_split), p.ldb, b_split - n0, inner);
    else kb.init(lane, kbeg, b0, b0, p.ldb, BN, inner);
    const int q = 2 * (wave * SCH + lane);   // the first of the lane's two tile rows: A's, then B's
    const char* base;
    int64_t row;
    if (q < BM) {
      base = a.sa;
      row = t.row0 + q;
      sc_plane = a.sa_plane;
    } else {
      const int r = q - BM;
      sc_plane = a.sb_plane;
      const bool second = GATED ? r >= b_half : stacked && n0 + r >= b_split;
      base = (second ? a.sb1 : a.sb0) + t.e * a.ws_stride;
      row = GATED ? n0 + (r >= b_half ? r - b_half : r) : second ? n0 + r - b_split : n0 + r;
    }
    const int64_t last = sc_plane / 8 - 2;
    sc = base + (row < last ? row : last) * 8 + (int64_t)(kbeg / BK) * sc_plane;
  }
  __device__ __forceinline__ int2 loc_a(int r) const { return make_int2(0, min(r, rows - 1)); }
  __device__ __forceinline__ int2 loc_b(int r) const {
    constexpr int b_half = BN / 2;
    if constexpr (GATED) {
      return r < b_half ? make_int2(0, min(n0 + r, N - 1) - n0) : make_int2(1, min(n0 + r - b_half, N - 1) - (n0 - b_half));
    } else {
      const int n = min(n0 + r, N - 1);
      return make_int2(stacked && n >= b_split ? 1 : 0, n - n0);
    }
  }
  // Steps below this are wholly in range, and no row is clamped: their DMAs need no work per lane.
  __device__ __forceinline__ int fast_steps() const { return ka.interior && kb.interior ? k_left / BK : 0; }

  // DMA d of step kt into ring stage st; steps past the end load zeros, and scales that are not used. (Without a branch:
  // products sink below one.)
  template <bool FAST> __device__ __forceinline__ void issue_one(int kt, int st, int d) const {
    char* stage = smem + st * STAGE;
    if (d < DA::kInst) {
      if constexpr (FAST) ka.issue_fast_i(stage, wave, d, kt * BK);
      else ka.issue_i(stage, wave, lane, d, kt * BK, k_left, [&](int r) { return loc_a(r); });
    } else if (d < DA::kInst + DB::kInst) {
      if constexpr (FAST) kb.issue_fast_i(stage + A_BYTES, wave, d - DA::kInst, kt * BK);
      else kb.issue_i(stage + A_BYTES, wave, lane, d - DA::kInst, kt * BK, k_left, [&](int r) { return loc_b(r); });
    } else if (SCH == 64 || lane < SCH) {
      dma16(sc + (int64_t)min(kt, planes - 1) * sc_plane, stage + S_AT + wave * SCH * 16);
    }
  }
  __device__ __forceinline__ void issue(int kt, int st) const {
    if (kt < fast_steps()) {
#pragma unroll
      for (int d = 0; d < N_DMA; ++d) issue_one<true>(kt, st, d);
    } else {
#pragma unroll
      for (int d = 0; d < N_DMA; ++d) issue_one<false>(kt, st, d);
    }
  }

  __device__ __forceinline__ void read_frags(int st, int s, int slot) {
    const char* stage = smem + st * STAGE;
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[slot][i] = DA::read_block(stage, a_base[i], frow, 4 * fhalf + s);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[slot][j] = DB::read_block(stage + A_BYTES, b_base[j], frow, 4 * fhalf + s);
  }
  __device__ __forceinline__ void read_scales(int st) {   // of the lane's row: the half's four bytes
    const char* stage = smem + st * STAGE + S_AT;
#pragma unroll
    for (int i = 0; i < MI; ++i) na[i] = *reinterpret_cast<const uint32_t*>(stage + (a_base[i] + frow) * 8 + 4 * fhalf);
#pragma unroll
    for (int j = 0; j < NI; ++j) nb[j] = *reinterpret_cast<const uint32_t*>(stage + (BM + b_base[j] + frow) * 8 + 4 * fhalf);
  }
  __device__ __forceinline__ void take_scales() {
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = na[i];
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = nb[j];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  }
  template <int S> __device__ __forceinline__ void mma() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) mx_mma<S>(fb[S & 1][j], fa[S & 1][i], sb[j], sa[i], acc[i][j]);
  }
  // The first fragments of ring stage 0, whose step must have landed for every wave.
  __device__ __forceinline__ void begin() {
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    read_frags(0, 0, 0);
    read_scales(0);
    take_scales();
    wait_lgkmcnt0();
  }
  // The step in stage cur, whose first fragments are there; then the DMAs of step kt into that stage, and the next stage's
  // first fragments.
  template <bool FAST> __device__ __forceinline__ void step(int kt, int& cur) {
    const int nxt = cur + 1 == NS ? 0 : cur + 1;
    read_frags(cur, 1, 1);
    mma<0>();
    interleave<N_MMA, N_RD, 0>();
    read_frags(cur, 2, 0);
    mma<1>();
    interleave<N_MMA, N_RD, 0>();
    read_frags(cur, 3, 1);
    mma<2>();
    interleave<N_MMA, N_RD, 0>();
    // the next step must have landed; after the barrier every wave is done reading this stage
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<(NS - 2) * N_DMA>();
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int d = 0; d < N_DMA; ++d) issue_one<FAST>(kt, cur, d);
    read_frags(nxt, 0, 0);
    read_scales(nxt);
    mma<3>();
    interleave<N_MMA, 2 * N_RD, N_DMA>();
    take_scales();
    cur = nxt;
  }
};

// The epilogue of a tile: the accumulators go to LDS (two block rows of 32 at a time, a wave its own), and come back as 8 consecutive
// columns of a row a lane, U rows at a time: the loop is rolled and its activation's switch taken once for all U, as a wave
// that is alone on its SIMD waits out every branch and a cold line of code (4096 x 4096 x 1024 with a row at a time
// 26.6 us, unrolled over every row 33).
constexpr int mx_staged_blocks(int MI) { return MI > 2 ? 2 : MI; }
template <int BM, int BN> constexpr int mx_epilogue_bytes() { return 4 * mx_staged_blocks(BM / 64) * 32 * (BN / 2 * 4 + 16); }
template <int EPI, typename IoT, int BM, int BN, int MI, int NI>
__device__ __forceinline__ void mx_epilogue(const GemmArgs& p, f32x16 (&acc)[MI][NI], int n0, int wm, int wn, int lane, int wave, char* lds) {
  constexpr bool GATED = epi_gated(EPI);
  constexpr int WM = BM / 2, WN = BN / 2, IB = mx_staged_blocks(MI);   // block rows staged at once
  constexpr int STRIDE = WN * 4 + 16, UNITS = GATED ? WN / 2 : WN, LPR = UNITS / 8, RPI = 64 / LPR;
  constexpr int U = IB * 32 / RPI < 4 ? IB * 32 / RPI : 4;
  const int frow = lane & 31, fhalf = lane >> 5;
  char* wbuf = lds + wave * IB * 32 * STRIDE;
  const int nbase = GATED ? n0 + wn * (WN / 2) : n0 + wn * WN;
  const int rl = lane / LPR, cl = (lane % LPR) * 8, n = nbase + cl;
  const bool col = n < p.N;
  const int nin = col ? n : 0;
  const bool full = p.M >= BM && n0 + (GATED ? BN / 2 : BN) <= p.N;   // (uniform)
  float bias0[8] = {}, bias1[8] = {};
  if constexpr (epi_linear(EPI)) {
    if (p.bias0) Vec8<IoT>::load(elem_ptr<IoT>(p.bias0, 0, 0, nin), bias0);
    if constexpr (GATED) if (p.bias1) Vec8<IoT>::load(elem_ptr<IoT>(p.bias1, 0, 0, nin), bias1);
  }
#pragma unroll
  for (int i0 = 0; i0 < MI; i0 += IB) {
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4*>(wbuf + (i * 32 + frow) * STRIDE + (j * 32 + 8 * g + 4 * fhalf) * 4) =
              f32x4{acc[i0 + i][j][4 * g], acc[i0 + i][j][4 * g + 1], acc[i0 + i][j][4 * g + 2], acc[i0 + i][j][4 * g + 3]};
    wait_lgkmcnt0();   // this wave's rows are written
    __builtin_amdgcn_wave_barrier();
    const int m1 = wm * WM + i0 * 32 + rl;
#pragma unroll 1
    for (int r0 = 0; r0 < IB * 32; r0 += U * RPI) {
      float v[8 * U], u[GATED ? 8 * U : 1], y[8 * U], o[8 * U];
      auto each = [&](auto f) {
#pragma unroll
        for (int k = 0; k < U; ++k) f(k, m1 + r0 + k * RPI, reinterpret_cast<float(&)[8]>(v[8 * k]));
      };
      auto store = [&](auto where, float* z) {   // 8 columns of row m to where(m)
        each([&](int k, int m, float(&)[8]) {
          if (full || (col && m < p.M)) Vec8<typename std::conditional<EPI == EPI_PARTIAL, float, IoT>::type>::store(where(m), z + 8 * k);
        });
      };
      if (EPI != EPI_PARTIAL && p.res) {
        each([&](int k, int m, float(&)[8]) { Vec8<IoT>::load(elem_ptr<IoT>(p.res, min(m, p.M - 1), p.ld_res, nin), o + 8 * k); });
      } else {
#pragma unroll
        for (int q = 0; q < 8 * U; ++q) o[q] = 0.0f;
      }
      each([&](int k, int, float(&z)[8]) {
        const char* src = wbuf + (rl + r0 + k * RPI) * STRIDE + cl * 4;
        const f32x4 a0 = *reinterpret_cast<const f32x4*>(src), a1 = *reinterpret_cast<const f32x4*>(src + 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) { z[q] = a0[q] + bias0[q]; z[4 + q] = a1[q] + bias0[4 + q]; }
        if constexpr (GATED) {
          const f32x4 b0 = *reinterpret_cast<const f32x4*>(src + UNITS * 4), b1 = *reinterpret_cast<const f32x4*>(src + UNITS * 4 + 16);
#pragma unroll
          for (int q = 0; q < 4; ++q) { u[8 * k + q] = b0[q] + bias1[q]; u[8 * k + 4 + q] = b1[q] + bias1[4 + q]; }
        }
      });
      if constexpr (EPI == EPI_PARTIAL) {
        store([&](int m) { return elem_ptr<float>(p.partial, m, p.N, n); }, v);
      } else {
        if (p.flags & 1) {
          store([&](int m) { return elem_ptr<IoT>(p.aux, m, p.ld_aux, n); }, v);
          if constexpr (GATED) store([&](int m) { return elem_ptr<IoT>(p.aux, m, p.ld_aux, p.half + n); }, u);
        }
        if constexpr (GATED) linear_act<8 * U, true>(p.act, v, u, y);
        else linear_act<8 * U, false>(p.act, v, v, y);
#pragma unroll
        for (int q = 0; q < 8 * U; ++q) y[q] += o[q];
        store([&](int m) { return elem_ptr<IoT>(p.C0, m, p.ldc0, n); }, y);
      }
    }
    wait_lgkmcnt0();   // read before the next rows are written
    __builtin_amdgcn_wave_barrier();
  }
}

// The activation on a wave's accumulators and its rows to memory straight from registers, for 16-bit outputs without residual and
// pre-activation. Lane l has row l % 32 of a block and, in register 4 g + r, column 8 g + 4 (l / 32) + r; swapping halves
// between two g's registers leaves 8 consecutive columns a lane. Rows and columns past the tile are stored at an offset past
// the buffer's end, which stores nothing and needs no branch. Against the way through LDS (us): 4096 x 4096 x 11008 132 and 119,
// 32768 rows of 32 experts of 2048 x 1376 gate and up 163 and 148.
template <typename IoT, int FN, bool GATED, int MI, int NI>
__device__ __forceinline__ void mx_store_tile(const f32x16 (&acc)[MI][NI], __amdgpu_buffer_rsrc_t out, int ldc_bytes, int rows,
                                              int cols, int m0, int c0, int frow, int fhalf) {
  constexpr int NO = GATED ? NI / 2 : NI;
  constexpr uint32_t kNowhere = 0x80000000u;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = m0 + i * 32 + frow;
    const uint32_t row = m < rows ? (uint32_t)m * (uint32_t)ldc_bytes : kNowhere;
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      float v[16], u[16], y[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[r] = acc[i][j][r];
        u[r] = acc[i][GATED ? NO + j : j][r];
      }
      linear_act<16, GATED>(FN, v, u, y);
#pragma unroll
      for (int g = 0; g < 4; g += 2) {
        u32x4 w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto s = __builtin_amdgcn_permlane32_swap(pack16x2<IoT>(y[4 * g + 2 * h], y[4 * g + 2 * h + 1]),
                                                          pack16x2<IoT>(y[4 * g + 4 + 2 * h], y[4 * g + 5 + 2 * h]), false, false);
          w[h] = s[0];
          w[2 + h] = s[1];
        }
        const int c = c0 + j * 32 + 8 * g + 8 * fhalf;
        __builtin_amdgcn_raw_buffer_store_b128(w, out, (int)(c < cols ? row + 2u * (uint32_t)c : kNowhere), 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);   // (else every block's accumulators are fetched at once)
    }
  }
}

// Workgroup b's tile, any epilogue.
template <typename IoT, int BM, int BN, int EPI, bool DIRECT>
__device__ __forceinline__ void mx_tile(const Mx4Gemm& a, int b, char* smem) {
  using Pipe = MxPipe<BM, BN, epi_gated(EPI)>;
  constexpr int NS = Pipe::NS;
  MxPlace t;
  if (!mx_place<BM, Pipe::BNC>(a, b, t)) return;
  if (t.e == a.experts) {
    mx_zero_rows<IoT, Pipe::BNC, epi_gated(EPI)>(a.g, t);
    return;
  }
  GemmArgs p = a.g;
  p.M = t.rows;
  p.C0 = shift<IoT>(p.C0, t.row0 * p.ldc0);
  p.aux = shift<IoT>(p.aux, t.row0 * p.ld_aux);
  p.res = shift<IoT>(p.res, t.row0 * p.ld_res);
  p.bias0 = shift<IoT>(p.bias0, t.e * a.bias_stride);
  p.bias1 = shift<IoT>(p.bias1, t.e * a.bias_stride);
  if (EPI == EPI_PARTIAL) p.partial += ((int64_t)t.split * a.rows + t.row0) * p.N;
  const int kbeg = t.split * p.k_per_split, kend = min(p.K, kbeg + p.k_per_split);
  const int nk = (kend - kbeg + Pipe::BK - 1) / Pipe::BK;
  Pipe k;
  k.init(smem);
  k.place(a, t, kbeg, kend);
  if constexpr (DIRECT) {   // the sums start from the bias: a lane's columns of block j are 8 g + 4 (l / 32) + r
    constexpr int NI = Pipe::NI, NO = epi_gated(EPI) ? NI / 2 : NI;
    u32x2 b[NI][4];   // (beside the first stage: behind the others the sums would wait for those, too)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = t.n0 + k.wn * (Pipe::BNC / 2) + (j % NO) * 32 + 8 * g + 4 * k.fhalf;
        const void* bias = j < NO ? p.bias0 : p.bias1;
        b[j][g] = bias != nullptr ? *reinterpret_cast<const u32x2*>(elem_ptr<IoT>(bias, 0, 0, n < p.N ? n : 0)) : u32x2{0u, 0u};
      }
    __builtin_amdgcn_sched_barrier(0);
    k.issue(0, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float f = Bits16<IoT>::to_f32(r & 1 ? b[j][g][r / 2] >> 16 : b[j][g][r / 2] & 0xffffu);
#pragma unroll
          for (int i = 0; i < Pipe::MI; ++i) k.acc[i][j][4 * g + r] = f;
        }
    __builtin_amdgcn_sched_barrier(0);
  } else {
    k.issue(0, 0);
    k.clear();
  }
#pragma unroll
  for (int s = 1; s < NS; ++s) k.issue(s, s);
  wait_vmcnt<(NS - 1) * Pipe::N_DMA>();   // step 0 landed
  k.begin();
  const int fast = k.fast_steps() - NS;
  int cur = 0, kt = 0;
  for (; kt < min(nk, fast); ++kt) k.template step<true>(kt + NS, cur);
  for (; kt < nk; ++kt) k.template step<false>(kt + NS, cur);
  if constexpr (DIRECT) {
    const auto out = __builtin_amdgcn_make_buffer_rsrc(elem_ptr<IoT>(p.C0, 0, 0, t.n0), 0, 0x7fffffff, 0x00020000);
    // The trailing DMAs have landed: what is in flight when the workgroup ends are stores, which the next one need not wait for.
    wait_vmcnt<0>();
    auto store = [&](auto fn) {
      mx_store_tile<IoT, decltype(fn)::value, epi_gated(EPI)>(k.acc, out, (int)p.ldc0 * 2, t.rows, p.N - t.n0, k.wm * Pipe::WM,
                                                              k.wn * (Pipe::BNC / 2), k.frow, k.fhalf);
    };
    switch (p.act) {   // (once a tile: a switch inside would be one a block)
      case FN_SILU: store(std::integral_constant<int, FN_SILU>{}); break;
      case FN_GELU_TANH: store(std::integral_constant<int, FN_GELU_TANH>{}); break;
      case FN_RELU: store(std::integral_constant<int, FN_RELU>{}); break;
      case FN_SIGMOID: store(std::integral_constant<int, FN_SIGMOID>{}); break;
      case FN_RELU_SQ: store(std::integral_constant<int, FN_RELU_SQ>{}); break;
      default: store(std::integral_constant<int, FN_NONE>{});
    }
    return;
  }
  // the trailing DMAs have landed and no wave reads the ring any more: its LDS becomes the epilogue's staging area
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  __builtin_amdgcn_s_barrier();
  static_assert(mx_epilogue_bytes<BM, BN>() <= NS * Pipe::STAGE, "epilogue staging must fit the ring");
  mx_epilogue<EPI, IoT, BM, BN, Pipe::MI, Pipe::NI>(p, k.acc, t.n0, k.wm, k.wn, k.lane, k.wave, smem);
}

template <typename IoT, int BM, int BN, int EPI, bool DIRECT>
__global__ __launch_bounds__(256, 1) void mx_kernel(const Mx4Gemm a) {
  __shared__ __attribute__((aligned(1024))) char smem[mx_ring_bytes<BM, BN>()];
  mx_tile<IoT, BM, BN, EPI, DIRECT>(a, blockIdx.x, smem);
}

template <typename IoT, int BM, int BN, int EPI> hipError_t launch_mx(const Mx4Gemm& a, hipStream_t s) {
  if constexpr (ElemTraits<IoT>::bytes == 2 && EPI != EPI_PARTIAL && BM == 256) {
    // (offsets inside a tile's rows are 31 bits; tiles of 128 x 128, two on a CU, are no faster so: 1024 x 4096 x 4096 17.9 us through
    // LDS and 18.5, 512 x 4096 x 11008 22.5 and 22.5)
    if (a.g.res == nullptr && !(a.g.flags & 1) && a.g.ldc0 <= (1 << 21)) {
      hipLaunchKernelGGL((mx_kernel<IoT, BM, BN, EPI, true>), dim3(a.tiles), dim3(256), 0, s, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_kernel<IoT, BM, BN, EPI, false>), dim3(a.tiles), dim3(256), 0, s, a);
  return hipGetLastError();
}

// The linear epilogues in one output type.
template <typename IoT> hipError_t mx_linear(int epi, TileShape tile, const Mx4Gemm& a, hipStream_t s) {
  const bool gated = epi == EPI_LIN_GATED;
  switch (tile) {
    case TILE_256x256: return gated ? launch_mx<IoT, 256, 256, EPI_LIN_GATED>(a, s) : launch_mx<IoT, 256, 256, EPI_LIN>(a, s);
    case TILE_128x128: return gated ? launch_mx<IoT, 128, 128, EPI_LIN_GATED>(a, s) : launch_mx<IoT, 128, 128, EPI_LIN>(a, s);
    case TILE_64x64: return gated ? launch_mx<IoT, 64, 128, EPI_LIN_GATED>(a, s) : launch_mx<IoT, 64, 64, EPI_LIN>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace gmlp
