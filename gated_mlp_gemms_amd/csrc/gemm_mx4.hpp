// Products of microscaled 4-bit operands (mx4.h), both along their rows: y = act(x W^T + b), one weight or one an
// expert. A tile body of its own on the pieces of gemm_dma.hpp: operands go HBM -> LDS by DMA through a ring of K-steps of
// 128 bytes (256 values) a row, 16-byte chunks (one block of 32 values each) XOR-swizzled by row, and come out as the
// fragments of v_mfma_scale_f32_32x32x64_f8f6f4: a lane's 16 bytes are a whole block, so its scale is one byte. The scales of a
// K-step are 8 bytes a row, one run of memory for a tile's rows (mx4.h's planes): one more DMA a wave. In
// substep s of four the lane half h takes block 4 h + s, so a lane's four scales of a step are the four bytes of one word, which
// the instruction picks from by number.
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

// Workgroup b's tile.
template <typename IoT, int BM, int BN, int EPI>
__device__ __forceinline__ void mx_tile(const Mx4Gemm& a, int b, char* smem) {
  constexpr int WAVES = 4, WM = BM / 2, WN = BN / 2, MI = WM / 32, NI = WN / 32;
  constexpr bool GATED = epi_gated(EPI);
  constexpr int BNC = GATED ? BN / 2 : BN;
  constexpr int BK = 128, NSUB = 4;
  constexpr int A_BYTES = BM * BK, S_AT = (BM + BN) * BK, STAGE = mx_stage_bytes<BM, BN>();
  constexpr int NS = ring_stages(STAGE, BM * BN);
  static_assert(NS >= 2, "the ring needs two stages");
  const int tiles_n = a.g.tiles_n;

  int tile = 0, split = 0;
  RowPiece t;
  const bool found = find_row_piece(a.offsets, a.experts, a.rows, BM, [&](int total) {
    const int tiles = (int)min((int64_t)total * tiles_n, (int64_t)(a.grid / a.splits));
    if (b >= tiles * a.splits) return -1;
    tile = xcd_remap(b, tiles * a.splits);
    split = tile / tiles;
    tile -= split * tiles;
    return tile / tiles_n;
  }, t);
  if (!found) return;
  GemmArgs p = a.g;
  if (t.e == a.experts) {   // rows of no expert: zeros (plus the residual)
    const int m0 = t.row0 + t.index * BM, m1 = min(m0 + BM, a.rows);
    const int n0 = (tile % tiles_n) * BNC, n1 = min(n0 + BNC, p.N);
    constexpr int V = 16 / ElemTraits<IoT>::bytes, W = BNC / V;
    for (int i = threadIdx.x; i < BM * W; i += 64 * WAVES) {
      const int m = m0 + i / W, n = n0 + i % W * V;
      if (m >= m1 || n >= n1) continue;
      const u32x4 zero = {0u, 0u, 0u, 0u};
      if (p.flags & 1) {
        *reinterpret_cast<u32x4*>(elem_ptr<IoT>(p.aux, m, p.ld_aux, n)) = zero;
        if (GATED) *reinterpret_cast<u32x4*>(elem_ptr<IoT>(p.aux, m, p.ld_aux, p.half + n)) = zero;
      }
      *reinterpret_cast<u32x4*>(elem_ptr<IoT>(p.C0, m, p.ldc0, n)) =
          p.res ? *reinterpret_cast<const u32x4*>(elem_ptr<IoT>(p.res, m, p.ld_res, n)) : zero;
    }
    return;
  }
  int tm, tn;
  grouped_tile(tile - t.first * tiles_n, (t.rows + BM - 1) / BM, tiles_n, p.group_m, tm, tn);
  const int64_t row0 = t.row0 + tm * BM;
  const int rows = min(t.rows - tm * BM, BM), n0 = tn * BNC;
  p.M = rows;
  p.C0 = shift<IoT>(p.C0, row0 * p.ldc0);
  p.aux = shift<IoT>(p.aux, row0 * p.ld_aux);
  p.res = shift<IoT>(p.res, row0 * p.ld_res);
  p.bias0 = shift<IoT>(p.bias0, t.e * a.bias_stride);
  p.bias1 = shift<IoT>(p.bias1, t.e * a.bias_stride);
  if (EPI == EPI_PARTIAL) p.partial += ((int64_t)split * a.rows + row0) * p.N;
  const int kbeg = split * p.k_per_split, kend = min(p.K, kbeg + p.k_per_split), nk = (kend - kbeg + BK - 1) / BK;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / 2, wn = wave % 2;

  // ---- codes: rows past the matrix are given an existing row (their products are never stored)
  using DA = KTileDma<e4m3, BM, WAVES>;   // a byte is its element
  using DB = KTileDma<e4m3, BN, WAVES>;
  DA ka;
  DB kb;
  constexpr int b_half = BN / 2;
  auto locA = [&](int r) { return make_int2(0, min(r, rows - 1)); };
  auto locB = [&](int r) {
    if constexpr (GATED) {
      return r < b_half ? make_int2(0, min(n0 + r, p.N - 1) - n0) : make_int2(1, min(n0 + r - b_half, p.N - 1) - (n0 - b_half));
    } else {
      const int n = min(n0 + r, p.N - 1);
      return make_int2(p.B1 != nullptr && n >= p.b_split ? 1 : 0, n - n0);
    }
  };
  const char* a0 = static_cast<const char*>(p.A) + row0 * p.lda;
  ka.init(lane, kbeg, a0, a0, p.lda, BM, rows == BM);
  const char* w0 = static_cast<const char*>(p.B0) + t.e * a.w_stride;
  const char* w1 = p.B1 != nullptr ? static_cast<const char*>(p.B1) + t.e * a.w_stride : nullptr;
  const char* b0 = w0 + (int64_t)n0 * p.ldb;
  const bool inner = n0 + BNC <= p.N;
  auto before = [&](int64_t rel) { return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(w1) + rel * p.ldb); };
  if constexpr (GATED) kb.init(lane, kbeg, b0, before(n0 - b_half), p.ldb, b_half, inner);
  else if (w1 != nullptr) kb.init(lane, kbeg, b0, before(n0 - p.b_split), p.ldb, p.b_split - n0, inner);
  else kb.init(lane, kbeg, b0, b0, p.ldb, BN, inner);

  // ---- scales: 16 bytes (two rows) a lane; a pair past the padded rows takes the last one (its rows are never stored)
  constexpr int SCH = (BM + BN) / 2 / WAVES;   // lanes of a wave
  const char* sc;
  int64_t sc_plane;
  {
    const int q = 2 * (wave * SCH + lane);   // the first of the two tile rows: A's, then B's
    const char* base;
    int64_t row;
    if (q < BM) {
      base = a.sa;
      row = row0 + q;
      sc_plane = a.sa_plane;
    } else {
      const int r = q - BM;
      sc_plane = a.sb_plane;
      const bool second = GATED ? r >= b_half : p.B1 != nullptr && n0 + r >= p.b_split;
      base = (second ? a.sb1 : a.sb0) + t.e * a.ws_stride;
      row = GATED ? n0 + (r >= b_half ? r - b_half : r) : second ? n0 + r - p.b_split : n0 + r;
    }
    const int64_t last = sc_plane / 8 - 2;
    sc = base + (row < last ? row : last) * 8 + (int64_t)(kbeg / BK) * sc_plane;
  }
  constexpr int N_DMA = DA::kInst + DB::kInst + 1;
  static_assert((NS - 1) * N_DMA < 64, "vmcnt range");
  const int planes = (p.K + BK - 1) / BK - kbeg / BK;
  auto issue_scales = [&](int kt, char* stage) {
    if (SCH == 64 || lane < SCH) dma16(sc + (int64_t)min(kt, planes - 1) * sc_plane, stage + S_AT + wave * SCH * 16);
  };
  // DMA d of K-step kt into ring stage st; steps past the end load zeros, and scales that are not used. fast: the step
  // is wholly in range and no row of the tile is clamped. (Without a branch: products sink below one.)
  auto issue_one = [&](int kt, int st, int d, auto fast) {
    char* stage = smem + st * STAGE;
    if (d < DA::kInst) {
      if constexpr (decltype(fast)::value) ka.issue_fast_i(stage, wave, d, kt * BK);
      else ka.issue_i(stage, wave, lane, d, kt * BK, kend - kbeg, locA);
    } else if (d < DA::kInst + DB::kInst) {
      if constexpr (decltype(fast)::value) kb.issue_fast_i(stage + A_BYTES, wave, d - DA::kInst, kt * BK);
      else kb.issue_i(stage + A_BYTES, wave, lane, d - DA::kInst, kt * BK, kend - kbeg, locB);
    } else {
      issue_scales(kt, stage);
    }
  };
  auto issue = [&](int kt, int st) {
    char* stage = smem + st * STAGE;
    ka.issue(stage, wave, lane, kt * BK, kend - kbeg, locA);
    kb.issue(stage + A_BYTES, wave, lane, kt * BK, kend - kbeg, locB);
    issue_scales(kt, stage);
  };

  const int frow = lane & 31, fhalf = lane >> 5;
  int a_base[MI], b_base[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) a_base[i] = wm * WM + i * 32;
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    if constexpr (GATED) {
      constexpr int NH = NI / 2;
      b_base[j] = j < NH ? wn * (WN / 2) + j * 32 : BN / 2 + wn * (WN / 2) + (j - NH) * 32;
    } else {
      b_base[j] = wn * WN + j * 32;
    }
  }
  u32x4 fa[2][MI], fb[2][NI];
  uint32_t sa[MI], sb[NI], na[MI], nb[NI];
  auto read_frags = [&](int st, int s, int slot) {
    const char* stage = smem + st * STAGE;
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[slot][i] = DA::read_block(stage, a_base[i], frow, 4 * fhalf + s);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[slot][j] = DB::read_block(stage + A_BYTES, b_base[j], frow, 4 * fhalf + s);
  };
  auto read_scales = [&](int st) {   // of the lane's row: the half's four bytes
    const char* stage = smem + st * STAGE + S_AT;
#pragma unroll
    for (int i = 0; i < MI; ++i) na[i] = *reinterpret_cast<const uint32_t*>(stage + (a_base[i] + frow) * 8 + 4 * fhalf);
#pragma unroll
    for (int j = 0; j < NI; ++j) nb[j] = *reinterpret_cast<const uint32_t*>(stage + (BM + b_base[j] + frow) * 8 + 4 * fhalf);
  };
  auto take_scales = [&] {
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = na[i];
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = nb[j];
  };
  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  auto mma_all = [&](auto sub) {
    constexpr int S = decltype(sub)::value;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) mx_mma<S>(fb[S & 1][j], fa[S & 1][i], sb[j], sa[i], acc[i][j]);
  };
  constexpr int N_MMA = MI * NI, N_RD = MI + NI;

#pragma unroll
  for (int s = 0; s < NS; ++s) issue(s, s);
  wait_vmcnt<(NS - 1) * N_DMA>();   // step 0 landed
  wait_lgkmcnt0();
  __builtin_amdgcn_s_barrier();
  read_frags(0, 0, 0);
  read_scales(0);
  take_scales();
  wait_lgkmcnt0();
  int cur = 0;
  auto k_step = [&](int kt, auto fast) {
    const int nxt = cur + 1 == NS ? 0 : cur + 1;
    read_frags(cur, 1, 1);
    mma_all(std::integral_constant<int, 0>{});
    interleave<N_MMA, N_RD, 0>();
    read_frags(cur, 2, 0);
    mma_all(std::integral_constant<int, 1>{});
    interleave<N_MMA, N_RD, 0>();
    read_frags(cur, 3, 1);
    mma_all(std::integral_constant<int, 2>{});
    interleave<N_MMA, N_RD, 0>();
    // step kt+1 must have landed (NS-2 younger steps may be in flight); after the barrier every wave is done reading
    // this stage, which takes step kt+NS
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<(NS - 2) * N_DMA>();
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int d = 0; d < N_DMA; ++d) issue_one(kt + NS, cur, d, fast);
    read_frags(nxt, 0, 0);
    read_scales(nxt);
    mma_all(std::integral_constant<int, 3>{});
    interleave<N_MMA, 2 * N_RD, N_DMA>();
    take_scales();
    cur = nxt;
  };
  const int nk_main = ka.interior && kb.interior ? max(0, min(nk, (kend - kbeg) / BK - NS)) : 0;
  int kt = 0;
  for (; kt < nk_main; ++kt) k_step(kt, std::true_type{});
  for (; kt < nk; ++kt) k_step(kt, std::false_type{});
  // the trailing DMAs have landed and no wave reads the ring any more: its LDS becomes the epilogue's staging area
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  __builtin_amdgcn_s_barrier();
  static_assert(mx_epilogue_bytes<BM, BN>() <= NS * STAGE, "epilogue staging must fit the ring");
  mx_epilogue<EPI, IoT, BM, BN, MI, NI>(p, acc, n0, wm, wn, lane, wave, smem);
}

template <typename IoT, int BM, int BN, int EPI>
__global__ __launch_bounds__(256, 1) void mx_kernel(const Mx4Gemm a) {
  __shared__ __attribute__((aligned(1024))) char smem[mx_ring_bytes<BM, BN>()];
  mx_tile<IoT, BM, BN, EPI>(a, blockIdx.x, smem);
}

template <typename IoT, int BM, int BN, int EPI> hipError_t launch_mx(const Mx4Gemm& a, hipStream_t s) {
  hipLaunchKernelGGL((mx_kernel<IoT, BM, BN, EPI>), dim3(a.grid), dim3(256), 0, s, a);
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
