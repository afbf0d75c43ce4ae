// One product an expert in one launch (ExpertGemm): the tile body of gemm_dma.hpp with the operands moved to an expert's rows and weights. How many rows an
// expert has is known on the device only, so a launch over rows has as many workgroups as the rows
// could need at most (every expert may end in a partial tile); each workgroup counts the experts'
// tiles from the offsets (a wave scan, no memory but the offsets) and takes one or none.
#pragma once

#include "gemm_dma.hpp"
#include "launch.hpp"

namespace gmlp {

// A piece of at most `step` rows of one expert.
struct RowPiece {
  int e;        // expert; the number of experts: rows behind the last offset
  int row0;     // the expert's first row
  int rows;     // the expert's rows
  int index;    // the piece within the expert
  int first;    // pieces of the experts before
};

// Rows of expert e (e = experts: what lies behind the last offset). Offsets are held inside [0, rows],
// so whatever they contain, no row outside the operands is named.
__device__ __forceinline__ void expert_rows(const int* offsets, int experts, int rows, int e, int& row0, int& n) {
  if (offsets == nullptr) {   // one expert with every row
    row0 = e == 0 ? 0 : rows;
    n = e == 0 ? rows : 0;
    return;
  }
  const int from = offsets[min(e, experts)], to = offsets[min(e + 1, experts)];   // one trip to memory
  row0 = min(max(from, 0), rows);
  const int end = e < experts ? min(max(to, row0), rows) : rows;
  n = e <= experts ? end - row0 : 0;
}

// Inclusive sum over the lanes up to this one: inside 16 lanes by shifted DPP operands, then the last lane of
// row 0 (and 2) added to the next row, and that of row 1 to the upper half.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

// find_row_piece with C experts a lane: lane l counts experts l C .. l C + C - 1 from C + 1 offsets loaded at once.
template <int C, int LEAST, typename Want>
__device__ __forceinline__ bool find_row_piece_of(const int* offsets, int experts, int rows, int step, Want want,
                                                  RowPiece& out) {
  const int lane = threadIdx.x & 63, e0 = lane * C;
  int at[C + 1], pieces[C], sum = 0;
  if (offsets == nullptr) {   // one expert with every row
#pragma unroll
    for (int i = 0; i <= C; ++i) at[i] = e0 + i == 0 ? 0 : rows;
  } else {
#pragma unroll
    for (int i = 0; i <= C; ++i) at[i] = offsets[min(e0 + i, experts)];
    at[0] = min(max(at[0], 0), rows);
#pragma unroll
    for (int i = 1; i <= C; ++i) {   // (whatever the offsets hold: expert_rows)
      const int from = min(max(at[i], 0), rows);
      at[i] = e0 + i <= experts ? from : rows;
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int n = max(at[i + 1] - at[i], 0);
    pieces[i] = (n + step - 1) / step;
    if constexpr (LEAST > 0) pieces[i] = e0 + i < experts ? max(pieces[i], LEAST) : 0;
    if constexpr (LEAST < 0) pieces[i] = e0 + i < experts ? max(pieces[i] - 1, 0) : 0;
    if (e0 + i > experts) pieces[i] = 0;
    sum += pieces[i];
  }
  const int incl = wave_scan(sum);
  const int k = want(__builtin_amdgcn_readlane(incl, 63));
  if (k < 0) return false;
  const uint64_t hit = __ballot(incl > k);
  if (hit == 0) return false;
  const int l = __builtin_ctzll(hit);
  int first = incl - sum, e = e0, row0 = at[0], n = max(at[1] - at[0], 0);   // of the lane's expert that has piece k
#pragma unroll
  for (int i = 1; i < C; ++i) {
    if (first + pieces[i - 1] > k || e != e0 + i - 1) continue;
    first += pieces[i - 1];
    e = e0 + i;
    row0 = at[i];
    n = max(at[i + 1] - at[i], 0);
  }
  out.e = __builtin_amdgcn_readlane(e, l);
  out.row0 = __builtin_amdgcn_readlane(row0, l);
  out.rows = __builtin_amdgcn_readlane(n, l);
  out.first = __builtin_amdgcn_readlane(first, l);
  out.index = k - out.first;
  return true;
}

// Pieces of every expert (the rows behind the last offset included) are numbered in expert order.
// want(total) -> the number of the piece wanted, or -1. Called by whole waves; every wave of a
// workgroup gets the same answer, in scalar registers. LEAST: pieces an expert has at least (the rows
// behind the last offset then have none); -1: every expert's pieces but its first are numbered (its second is piece 0
// of it, and the rows behind the last offset have none). Every tile starts with it, so it is one trip to memory and
// one scan.
template <int LEAST = 0, typename Want>
__device__ __forceinline__ bool find_row_piece(const int* offsets, int experts, int rows, int step, Want want,
                                               RowPiece& out) {
  constexpr int kTail = LEAST == 0 ? 1 : 0;   // the rows behind the last offset take a place
  if (experts <= 64 - kTail) return find_row_piece_of<1, LEAST>(offsets, experts, rows, step, want, out);
  if (experts <= 256 - kTail) return find_row_piece_of<4, LEAST>(offsets, experts, rows, step, want, out);
  return find_row_piece_of<17, LEAST>(offsets, experts, rows, step, want, out);
}

template <typename T> __device__ __forceinline__ const void* shift(const void* p, int64_t elems) {
  return p ? reinterpret_cast<const char*>(p) + elems * ElemTraits<T>::bytes : nullptr;
}
template <typename T> __device__ __forceinline__ void* shift(void* p, int64_t elems) {
  return p ? reinterpret_cast<char*>(p) + elems * ElemTraits<T>::bytes : nullptr;
}

template <typename T, int BM, int BN, int WAVES>
constexpr int expert_lds_bytes() {
  constexpr int whole = dma_ring_bytes<T, BM, BN>();
  if constexpr (WAVES == 8) return whole > dma_ring_bytes<T, BM / 2, BN>() ? whole : dma_ring_bytes<T, BM / 2, BN>();
  else return whole;
}

// Tile b of a product over rows: y = x W_e^T with a linear epilogue, or dx = dz W_e. 8-wave tiles are 256
// rows, or 128 where an expert has no more left. With split_tail the tiles of a last, at most half
// filled round of the 256 CUs run as two 128-row halves each: 32768 rows of 32 uneven experts are 6.3 rounds
// of full tiles, which without the halves take the time of 7.
template <typename T, int BM, int BN, bool BK, int EPI, int WAVES>
__device__ __forceinline__ void expert_rows_tile(const ExpertGemm& a, int b, char* smem, int splits = 1, int kps = 0,
                                                 float* part = nullptr) {
  constexpr int BNC = epi_gated(EPI) ? BN / 2 : BN;   // output columns of a tile
  constexpr bool HALVES = WAVES == 8;
  constexpr int HM = BM / 2;
  const int tiles_n = a.g.tiles_n;
  int tile = 0, half = -1, split = 0;
  RowPiece t;
  // XCD-contiguous over the tiles there are, not over the launch's upper bound
  const bool found = find_row_piece(a.offsets, a.experts, a.rows, BM, [&](int total) {
    const int tiles = (int)min((int64_t)total * tiles_n, (int64_t)(a.grid / splits));
    if (EPI == EPI_STORE_PART && splits > 1) {
      if (b >= tiles * splits) return -1;
      tile = xcd_remap(b, tiles * splits);
      split = tile / tiles;
      tile -= split * tiles;
      return tile / tiles_n;
    }
    const int rem = tiles % 256, tail = HALVES && a.split_tail && rem <= 128 && tiles > 256 ? rem : 0;
    const int whole = tiles - tail;
    if (b < whole) {
      tile = xcd_remap(b, whole);
    } else {
      if (b - whole >= 2 * tail) return -1;
      const int i = xcd_remap(b - whole, 2 * tail);
      tile = whole + i / 2;
      half = i & 1;
    }
    return tile / tiles_n;
  }, t);
  if (!found) return;
  GemmArgs p = a.g;
  if (t.e == a.experts) {   // rows of no expert: zeros (plus the residual)
    if (half > 0 || splits > 1) return;   // (the first half fills the whole tile; joining sums fills them, too)
    const int m0 = t.row0 + t.index * BM, m1 = min(m0 + BM, a.rows);
    const int n0 = (tile % tiles_n) * BNC, n1 = min(n0 + BNC, p.N);
    constexpr int V = 16 / ElemTraits<T>::bytes, W = BNC / V;
    for (int i = threadIdx.x; i < BM * W; i += 64 * WAVES) {
      const int m = m0 + i / W, n = n0 + i % W * V;
      if (m >= m1 || n >= n1) continue;
      const u32x4 zero = {0u, 0u, 0u, 0u};
      if (epi_linear(EPI) && (p.flags & 1)) {
        *reinterpret_cast<u32x4*>(elem_ptr<T>(p.aux, m, p.ld_aux, n)) = zero;
        if (epi_gated(EPI)) *reinterpret_cast<u32x4*>(elem_ptr<T>(p.aux, m, p.ld_aux, p.half + n)) = zero;
      }
      *reinterpret_cast<u32x4*>(elem_ptr<T>(p.C0, m, p.ldc0, n)) =
          epi_linear(EPI) && p.res ? *reinterpret_cast<const u32x4*>(elem_ptr<T>(p.res, m, p.ld_res, n)) : zero;
    }
    return;
  }
  // this tile's rows as a product of its own
  int tm, tn;
  grouped_tile(tile - t.first * tiles_n, (t.rows + BM - 1) / BM, tiles_n, p.group_m, tm, tn);
  const int skip = tm * BM + (half > 0 ? HM : 0);
  const int rows = min(t.rows - skip, half >= 0 ? HM : BM);
  if (rows <= 0) return;   // the second half of a tile of few rows
  const int64_t row0 = t.row0 + skip;
  p.M = rows;
  p.tiles_m = 1;
  p.A = shift<T>(p.A, row0 * p.lda);
  p.C0 = shift<T>(p.C0, row0 * p.ldc0);
  p.aux = shift<T>(p.aux, row0 * p.ld_aux);
  p.res = shift<T>(p.res, row0 * p.ld_res);
  p.B0 = shift<T>(p.B0, t.e * a.w_stride);
  p.B1 = shift<T>(p.B1, t.e * a.w_stride);
  p.bias0 = shift<T>(p.bias0, t.e * a.bias_stride);
  p.bias1 = shift<T>(p.bias1, t.e * a.bias_stride);
  if (EPI == EPI_STORE_PART && splits > 1) {   // this part of K (B stacked from B0 and B1 along it)
    const int k0 = split * kps;
    p.K = min(kps, p.K - k0);
    p.k_per_split = p.K;
    p.A = shift<T>(p.A, k0);
    if (p.B1 != nullptr && k0 >= p.b_split) {
      p.B0 = shift<T>(p.B1, (k0 - p.b_split) * p.ldb);
      p.B1 = nullptr;
      p.b_split = 1 << 30;
    } else {
      p.B0 = shift<T>(p.B0, k0 * p.ldb);
      if (p.B1 != nullptr) p.b_split -= k0;
    }
    p.partial = part + ((int64_t)split * a.rows + row0) * p.N;
  }
  if constexpr (HALVES) {
    if (rows <= HM) {
      gemm_dma_tile<T, T, HM, BN, true, BK, EPI, WAVES, true, 4>(p, tn, smem);
      return;
    }
  }
  gemm_dma_tile<T, T, BM, BN, true, BK, EPI, WAVES, true>(p, tn, smem);
}

// The first slot of expert e's partial sums: pieces of the experts before it that have more than one.
__device__ __forceinline__ int expert_slots_before(const int* offsets, int experts, int rows, int piece_rows, int e) {
  const int lane = threadIdx.x & 63;
  int slots = 0;
  for (int base = 0; base < e; base += 64) {
    int r0, n;
    expert_rows(offsets, experts, rows, base + lane, r0, n);
    int v = base + lane < e && n > piece_rows ? (n + piece_rows - 1) / piece_rows : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    slots += v;
  }
  return __builtin_amdgcn_readfirstlane(slots);
}

// Zeros into share `item` of `tiles` of the weight gradient(s) of an expert without rows: in order of memory, whatever
// the tiles are (2 rows, 50 experts of 648 x 2576 gated: the launch 134 -> 107 us).
template <typename GT>
__device__ __forceinline__ void zero_share(const GemmArgs& p, int64_t elems, int item, int tiles) {
  const int64_t pieces = elems * (int64_t)sizeof(GT) / 16, all = p.C1 != nullptr ? 2 * pieces : pieces;
  const int64_t beg = all * item / tiles, end = all * (item + 1) / tiles;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int64_t i = beg + threadIdx.x; i < end; i += blockDim.x) {
    u32x4* q = reinterpret_cast<u32x4*>(i < pieces ? p.C0 : p.C1) + (i < pieces ? i : i - pieces);
    if (p.flags & kFlagLarge) __builtin_nontemporal_store(zero, q);
    else *q = zero;
  }
}

// The share of workgroup b of the weight gradients dW_e = dz^T x over expert e's rows, or over a piece of them,
// `tiles` shares a piece: the product in p and the share's number, or -1. p.K = 0: the share is one of zeros.
template <typename T, typename GT>
__device__ __forceinline__ int expert_grad_share(const ExpertBwd& all, int b, int tiles, GemmArgs& p) {
  const ExpertGemm& a = all.dw;
  p = a.g;
  int e, row0, n, item;
  if (all.piece_rows) {
    RowPiece t;
    int tile = 0;
    const bool found = find_row_piece<1>(a.offsets, a.experts, a.rows, all.piece_rows, [&](int total) {
      const int count = (int)min((int64_t)total * tiles, (int64_t)a.grid);
      if (b >= count) return -1;
      tile = xcd_remap(b, count);
      return tile / tiles;
    }, t);
    if (!found) return -1;
    e = t.e;
    row0 = t.row0 + t.index * all.piece_rows;
    n = min(t.rows - t.index * all.piece_rows, all.piece_rows);
    item = tile - (t.first + t.index) * tiles;
    if (t.rows > all.piece_rows) {
      const int slot = expert_slots_before(a.offsets, a.experts, a.rows, all.piece_rows, e) + t.index;
      if (slot >= all.max_slots) return -1;   // offsets may be anything
      p.partial = all.part_w + (int64_t)slot * p.M * p.N;
    }
  } else {
    b = xcd_remap(b, a.grid);
    e = b / tiles;
    if (e >= a.experts) return -1;
    item = b - e * tiles;
    expert_rows(a.offsets, a.experts, a.rows, e, row0, n);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    n = __builtin_amdgcn_readfirstlane(n);
  }
  if (n == 0 && p.accumulate) return -1;
  p.C0 = shift<GT>(p.C0, e * a.w_stride);
  p.C1 = shift<GT>(p.C1, e * a.w_stride);
  p.K = p.k_per_split = n;
  p.A = shift<T>(p.A, row0 * p.lda);
  p.B0 = shift<T>(p.B0, row0 * p.ldb);
  return item;
}

template <typename T, typename GT, int BM, int BN, int WAVES>
__device__ __forceinline__ void expert_grad_tile(const ExpertBwd& all, int b, char* smem) {
  GemmArgs p;
  const int tiles = all.dw.g.tiles_m * all.dw.g.tiles_n;
  const int item = expert_grad_share<T, GT>(all, b, tiles, p);
  if (item < 0) return;
  if (p.K == 0) {
    zero_share<GT>(p, all.dw.w_stride, item, tiles);
    return;
  }
  gemm_dma_tile<T, GT, BM, BN, false, false, EPI_STORE_PART, WAVES, true>(p, item, smem);
}

// Weight gradients over few rows: a tile is one or two K-steps, so as workgroups of their own tiles are mostly
// latency (finding the rows, the first loads, the last stores: 10 us for a pair of 128 x 128 tiles of 57 rows each,
// 1.7 TB/s of gradient written). Here a workgroup keeps a strip of 128 columns of x and walks the 64-column tiles
// of dz, the DMAs two steps ahead across tiles, through a ring of three stages (24 KB each; two workgroups a CU); a
// tile's stores stay in flight over the next steps.
constexpr int kStripM = kStripTileM, kStripN = kStripTileN, kStripStages = 3;
template <typename T> constexpr int strip_lds_bytes() { return kStripStages * (kStripM + kStripN) * StepGeo<T>::ROWB; }

template <typename T, typename GT>
__device__ __forceinline__ void expert_grad_strip(const ExpertBwd& all, int b, char* smem) {
  constexpr int ES = 2, WAVES = 4, WM = kStripM / 2, WN = kStripN / 2, MI = WM / 32, NI = WN / 32;
  constexpr int KC = Mma<T>::kChunks, KMMA = 16;
  using DA = MNTileDma<kStripM, WAVES, false>;
  using DB = MNTileDma<kStripN, WAVES, false>;
  constexpr int BK = DA::KROWS, NSUB = BK / KMMA, N_DMA = DA::kInst + DB::kInst;
  constexpr int A_BYTES = kStripM * StepGeo<T>::ROWB, STAGE = (kStripM + kStripN) * StepGeo<T>::ROWB;
  static_assert(DB::KROWS == BK && BK * kStripM * ES == A_BYTES, "stage geometry");
  constexpr int RR = 16;   // rows of the epilogue's staging: it has one stage
  static_assert(epilogue_lds_bytes<kStripN, WAVES, 2, RR>() <= STAGE, "epilogue staging");
  // a whole tile's stores a wave makes (16 bytes a lane), which may be in flight when the next step is waited for
  constexpr int STORES = WM * WN * (int)sizeof(GT) / 1024;

  GemmArgs p;
  const int parts = all.strip_parts;
  const int share = expert_grad_share<T, GT>(all, b, all.dw.g.tiles_n * parts, p);
  if (share < 0) return;
  if (p.K == 0) {
    zero_share<GT>(p, all.dw.w_stride, share, all.dw.g.tiles_n * parts);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / 2, wn = wave % 2;
  const int n0 = share / parts * kStripN, part = share % parts;
  const int count = (p.tiles_m - part + parts - 1) / parts;   // tiles of this workgroup
  const int nk = (p.K + BK - 1) / BK, steps = count * nk;
  const int64_t lda = (int64_t)p.lda * ES, ldb = (int64_t)p.ldb * ES;

  DA na;
  DB nb;
  nb.init(wave, lane, reinterpret_cast<const char*>(elem_ptr<T>(p.B0, 0, p.ldb, n0)), ldb, 0, p.N - n0);
  int itile = 0, ik = 0;   // the next step to load
  auto issue = [&](char* stage) {
    if (ik == 0) {
      const int m0 = (part + itile * parts) * kStripM;
      na.init(wave, lane, reinterpret_cast<const char*>(elem_ptr<T>(p.A, 0, p.lda, m0)), lda, 0, p.M - m0);
    }
    na.issue(stage, wave, lane, ik * BK, p.K, ik * BK * lda, INT_MAX, 0);
    nb.issue(stage + A_BYTES, wave, lane, ik * BK, p.K, ik * BK * ldb, INT_MAX, 0);
    if (++ik == nk) ik = 0, ++itile;
  };
  f32x16 acc[MI][NI];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  };
  auto store = [&](int t, char* stage) {
    const int m0 = (part + t * parts) * kStripM;
    epilogue_rows<EPI_STORE_PART, GT, kStripM, kStripN, MI, NI, WAVES, 2, RR>(p, acc, m0, n0, 0, wm, wn, lane, wave, stage);
  };
  clear();
  issue(smem);
  if (steps > 1) issue(smem + STAGE);
  int cur = 0, k = 0, t = 0;
  bool stored = false;   // a whole tile's plain stores were the last thing issued
  for (int s = 0; s < steps; ++s) {
    char* stage = smem + cur * STAGE;
    // this step's DMAs have landed; the next step's, and stores made after them, may be in flight
    if (s + 1 >= steps) wait_vmcnt<0>();
    else if (stored) wait_vmcnt<N_DMA + STORES>();
    else wait_vmcnt<N_DMA>();
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();   // (and every wave is done with the stage that is loaded next)
    if (s + 2 < steps) issue(smem + (cur >= 1 ? cur - 1 : cur + 2) * STAGE);
    const int sub = min(NSUB, (p.K - k * BK + KMMA - 1) / KMMA);   // rows past the last are zeros
    auto substep = [&](int q) {
      u32x4 fa[MI][KC], fb[NI][KC];
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int c = 0; c < KC; ++c) fa[i][c] = DA::read(stage, wm * WM + i * 32, q, lane);
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int c = 0; c < KC; ++c) fb[j][c] = DB::read(stage + A_BYTES, wn * WN + j * 32, q, lane);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) Mma<T>::mma(fb[j], fa[i], acc[i][j]);
    };
    if (sub == NSUB) {   // unrolled, the reads of later substeps go ahead
#pragma unroll
      for (int q = 0; q < NSUB; ++q) substep(q);
    } else {
      for (int q = 0; q < sub; ++q) substep(q);
    }
    stored = false;
    if (++k == nk) {
      k = 0;
      wait_lgkmcnt0();
      __builtin_amdgcn_s_barrier();   // the stage becomes the epilogue's staging area
      store(t, stage);
      const int m0 = (part + t * parts) * kStripM;
      stored = p.partial == nullptr && !p.accumulate && m0 + kStripM <= p.M && n0 + kStripN <= p.N;
      clear();
      ++t;
    }
    cur = cur == 2 ? 0 : cur + 1;
  }
}

// The pieces' sums of one expert joined, 256 / runs columns by `runs` runs of pieces a workgroup (of 256 threads, or
// more that do nothing), the runs added in order. red: 256 floats. Few pieces an expert take one run: these
// workgroups share the launch's LDS size, one or two a CU, so there should be few (32 experts of 2752 columns as 5504
// workgroups of 16 columns: the backward's launch 986 us, 943 with 352 of 256).
template <typename GT>
__device__ __forceinline__ void bias_grad_block(const BiasGrad& a, int block, float* red) {
  const int runs = a.runs, cols = 256 / runs;   // powers of two
  const int lane = threadIdx.x & 63, run = threadIdx.x / cols;
  const int P = a.db1 ? 2 * a.N : a.N, blocks = (P + cols - 1) / cols;
  const int e = block / blocks, n = (block % blocks) * cols + (threadIdx.x & (cols - 1));
  // the expert's first piece: the pieces of the experts before, counted 64 experts at a time
  int first = 0;
  for (int base = 0; base < e; base += 64) {
    int r0, m;
    const int i = base + lane;
    expert_rows(a.offsets, a.experts, a.rows, i, r0, m);
    int v = i < e ? (m + a.step - 1) / a.step : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    first += v;
  }
  int row0, m;
  expert_rows(a.offsets, a.experts, a.rows, e, row0, m);
  const int pieces = (m + a.step - 1) / a.step;
  const int b = (int)((int64_t)run * pieces / runs);
  const int end = min((int)((int64_t)(run + 1) * pieces / runs), a.max_pieces - first);   // offsets may be anything
  float s = 0.0f;
  if (n < P && run < runs) {
#pragma unroll 8
    for (int i = b; i < end; ++i) s += a.sums[(int64_t)(first + i) * P + n];
  }
  if (runs > 1) {
    if (run < runs) red[threadIdx.x] = s;
    __syncthreads();
  }
  if (run != 0 || n >= P) return;
  for (int w = 1; w < runs; ++w) s += red[w * cols + threadIdx.x];
  void* db = n >= a.N ? a.db1 : a.db0;
  const int64_t at = (int64_t)e * a.N + (n >= a.N ? n - a.N : n);
  if (a.accumulate) {
    if (pieces > 0) reinterpret_cast<float*>(db)[at] += s;
  } else if constexpr (sizeof(GT) == 4) {
    reinterpret_cast<float*>(db)[at] = s;
  } else {
    reinterpret_cast<uint16_t*>(db)[at] = (uint16_t)Bits16<GT>::from_f32(s);
  }
}

template <typename T, int BM, int BN, int EPI, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 1) void expert_fwd_kernel(const ExpertGemm a) {
  __shared__ __attribute__((aligned(1024))) char smem[expert_lds_bytes<T, BM, BN, WAVES>()];
  expert_rows_tile<T, BM, BN, true, EPI, WAVES>(a, blockIdx.x, smem);
}

template <typename T, typename GT, int BM, int BN, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 1) void expert_bwd_kernel(const ExpertBwd a) {
  __shared__ __attribute__((aligned(1024))) char smem[expert_lds_bytes<T, BM, BN, WAVES>()];
  int b = blockIdx.x;
  const int first = a.dw_first ? a.dw.grid : a.dx.grid;
  if (b >= a.dx.grid + a.dw.grid) {
    bias_grad_block<GT>(a.db, b - a.dx.grid - a.dw.grid, reinterpret_cast<float*>(smem));
  } else if ((b < first) == (a.dw_first != 0)) {
    expert_grad_tile<T, GT, BM, BN, WAVES>(a, a.dw_first ? b : b - first, smem);
  } else {
    expert_rows_tile<T, BM, BN, false, EPI_STORE_PART, WAVES>(a.dx, a.dw_first ? b - first : b, smem, a.dx_splits, a.dx_kps,
                                                              a.part_x);
  }
}

// The backward with few rows an expert (ExpertBwd::strip_parts).
template <typename T, typename GT>
__global__ __launch_bounds__(256, 2) void expert_bwd_few_kernel(const ExpertBwd a) {
  constexpr int lds = expert_lds_bytes<T, 64, 128, 4>() > strip_lds_bytes<T>() ? expert_lds_bytes<T, 64, 128, 4>() : strip_lds_bytes<T>();
  __shared__ __attribute__((aligned(1024))) char smem[lds];
  int b = blockIdx.x;
  const int first = a.dw_first ? a.dw.grid : a.dx.grid;
  if (b >= a.dx.grid + a.dw.grid)
    bias_grad_block<GT>(a.db, b - a.dx.grid - a.dw.grid, reinterpret_cast<float*>(smem));
  else if ((b < first) == (a.dw_first != 0))
    expert_grad_strip<T, GT>(a, a.dw_first ? b : b - first, smem);
  else
    expert_rows_tile<T, 64, 128, false, EPI_STORE_PART, 4>(a.dx, a.dw_first ? b - first : b, smem, a.dx_splits, a.dx_kps, a.part_x);
}

template <typename T> hipError_t launch_expert_bwd_few(const ExpertBwd& a, hipStream_t s) {
  const dim3 grid(a.dx.grid + a.dw.grid + a.db.grid);
  if (a.dw.g.accumulate || a.db.accumulate) hipLaunchKernelGGL((expert_bwd_few_kernel<T, float>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((expert_bwd_few_kernel<T, T>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T, int BM, int BN, int WAVES>
hipError_t launch_expert_fwd(int epi, const ExpertGemm& a, hipStream_t s) {
  if (epi == EPI_LIN_GATED)
    hipLaunchKernelGGL((expert_fwd_kernel<T, BM, BN, EPI_LIN_GATED, WAVES>), dim3(a.grid), dim3(64 * WAVES), 0, s, a);
  else
    hipLaunchKernelGGL((expert_fwd_kernel<T, BM, BN, EPI_LIN, WAVES>), dim3(a.grid), dim3(64 * WAVES), 0, s, a);
  return hipGetLastError();
}

template <typename T, int BM, int BN, int WAVES>
hipError_t launch_expert_bwd(const ExpertBwd& a, hipStream_t s) {
  const dim3 grid(a.dx.grid + a.dw.grid + a.db.grid), block(64 * WAVES);
  if (a.dw.g.accumulate || a.db.accumulate) hipLaunchKernelGGL((expert_bwd_kernel<T, float, BM, BN, WAVES>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((expert_bwd_kernel<T, T, BM, BN, WAVES>), grid, block, 0, s, a);
  return hipGetLastError();
}

// The small tiles: 64 x 64, and 64 x 128 (64 gate and 64 up rows) for a gated forward.
template <typename T> hipError_t launch_expert_fwd_small(int epi, const ExpertGemm& a, hipStream_t s) {
  if (epi == EPI_LIN_GATED)
    hipLaunchKernelGGL((expert_fwd_kernel<T, 64, 128, EPI_LIN_GATED, 4>), dim3(a.grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((expert_fwd_kernel<T, 64, 64, EPI_LIN, 4>), dim3(a.grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

// The 16-bit experts' products of one type.
template <typename T> hipError_t expert_fwd16(int epi, TileShape tile, const ExpertGemm& a, hipStream_t s) {
  if (tile == TILE_256x256_W8) return launch_expert_fwd<T, 256, 256, 8>(epi, a, s);
  if (tile == TILE_128x128) return launch_expert_fwd<T, 128, 128, 4>(epi, a, s);
  if (tile == TILE_64x64) return launch_expert_fwd_small<T>(epi, a, s);
  return hipErrorInvalidValue;
}
template <typename T> hipError_t expert_bwd16(TileShape tile, const ExpertBwd& a, hipStream_t s) {
  if (a.strip_parts) return launch_expert_bwd_few<T>(a, s);
  if (tile == TILE_256x256_W8) return launch_expert_bwd<T, 256, 256, 8>(a, s);
  if (tile == TILE_128x128) return launch_expert_bwd<T, 128, 128, 4>(a, s);
  if (tile == TILE_64x64) return launch_expert_bwd<T, 64, 64, 4>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace gmlp
