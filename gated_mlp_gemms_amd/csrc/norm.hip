// Kernels of the norm in front of a layer (norm.h): forward with the residual's sum, backward with the column sums of
// the weight's and bias' gradients. Bound by HBM: a row is read once, held in registers as it was loaded, and written once.
#include <stdint.h>

#include <type_traits>

#include "rows.hpp"

namespace gmlp {

namespace {

// A row is taken by L threads with P pieces of 16 bytes each: piece i of thread l is number l + i L, so every load of a
// wave is one run of memory. L < 256: 256 / L rows a workgroup; else a workgroup a row.
template <int L> constexpr int norm_threads() { return L < 256 ? 256 : L; }

// The sum over a row's L threads, in every one of them. Wider rows than a wave: each wave leaves its part in `slot`, the row's
// own; a caller alternates between two slots, so that one barrier a sum is enough.
template <int L> __device__ __forceinline__ float row_sum(float v, float* slot) {
  if constexpr (L <= 64) {
    return group_sum<L>(v);
  } else {
    constexpr int W = L / 64;
    v = group_sum<64>(v);
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x % L / 64] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += slot[w];
    return s;
  }
}
// Two sums at once; `slot` holds two runs.
template <int L> __device__ __forceinline__ void row_sum2(float& a, float& b, float* slot) {
  if constexpr (L <= 64) {
    a = group_sum<L>(a);
    b = group_sum<L>(b);
  } else {
    constexpr int W = L / 64;
    const int wave = threadIdx.x % L / 64;
    a = group_sum<64>(a);
    b = group_sum<64>(b);
    if ((threadIdx.x & 63) == 0) {
      slot[wave] = a;
      slot[W + wave] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += slot[w];
      b += slot[W + w];
    }
  }
}

// The weights (or biases) of row piece c: N elements of type W, which may be wider than the row's.
template <typename W, int N> __device__ __forceinline__ void load_weights(const void* p, int64_t c, float (&v)[N]) {
  const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p) + c * N * (int64_t)sizeof(W));
  constexpr int M = Piece<W>::N;
#pragma unroll
  for (int i = 0; i < N / M; ++i) {
    float f[M];
    Piece<W>::unpack(q[i], f);
#pragma unroll
    for (int r = 0; r < M; ++r) v[i * M + r] = f[r];
  }
}

struct NormFwd {
  const u32x4* x; const u32x4* res; const void* w; const void* b;
  u32x4* y; u32x4* h; float* mean; float* rstd;
  int64_t rows;
  int pieces, layer;
  float inv_d, eps;
};

// h = x + res rounded to T, as a piece.
template <typename T> __device__ __forceinline__ u32x4 sum_piece(u32x4 a, u32x4 b) {
  constexpr int N = Piece<T>::N;
  float p[N], q[N];
  Piece<T>::unpack(a, p);
  Piece<T>::unpack(b, q);
#pragma unroll
  for (int r = 0; r < N; ++r) p[r] += q[r];
  return Piece<T>::pack(p);
}

template <typename T, typename W>
__device__ __forceinline__ u32x4 norm_piece(const NormFwd& a, int c, u32x4 h, float m, float s) {
  constexpr int N = Piece<T>::N;
  float f[N], w[N], b[N];
  Piece<T>::unpack(h, f);
#pragma unroll
  for (int r = 0; r < N; ++r) f[r] = (f[r] - m) * s;
  if (a.w != nullptr) {
    load_weights<W>(a.w, c, w);
#pragma unroll
    for (int r = 0; r < N; ++r) f[r] *= w[r];
  }
  if (a.b != nullptr) {
    load_weights<W>(a.b, c, b);
#pragma unroll
    for (int r = 0; r < N; ++r) f[r] += b[r];
  }
  return Piece<T>::pack(f);
}

template <typename T, typename W, int L, int P>
__global__ __launch_bounds__(norm_threads<L>()) void norm_fwd_kernel(const NormFwd a) {
  constexpr int N = Piece<T>::N, R = norm_threads<L>() / L;
  __shared__ float slots[2][L > 64 ? norm_threads<L>() / 64 : 1];
  const int lane = threadIdx.x % L, own = L > 64 ? threadIdx.x / L * (L / 64) : 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.rows; r0 += (int64_t)gridDim.x * R) {
    const int64_t row = r0 + threadIdx.x / L;
    const bool live = row < a.rows;
    const int64_t base = row * a.pieces;
    u32x4 h[P];
    bool in[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      in[i] = live && lane + i * L < a.pieces;
      h[i] = in[i] ? a.x[base + lane + i * L] : u32x4{0u, 0u, 0u, 0u};
    }
    if (a.res != nullptr) {
      u32x4 q[P];
#pragma unroll
      for (int i = 0; i < P; ++i) q[i] = in[i] ? a.res[base + lane + i * L] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < P; ++i) h[i] = sum_piece<T>(h[i], q[i]);
      if (a.h != nullptr) {
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (in[i]) a.h[base + lane + i * L] = h[i];
      }
    }
    float m = 0.0f;
    if (a.layer) {   // (uniform)
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float f[N];
        Piece<T>::unpack(h[i], f);
#pragma unroll
        for (int r = 0; r < N; ++r) sum += f[r];
      }
      m = row_sum<L>(sum, slots[0] + own) * a.inv_d;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float f[N], part = 0.0f;
      Piece<T>::unpack(h[i], f);
#pragma unroll
      for (int r = 0; r < N; ++r) part = __builtin_fmaf(f[r] - m, f[r] - m, part);
      sq += in[i] ? part : 0.0f;   // (what is past the row is 0, not m)
    }
    if (!a.layer && L > 64) __syncthreads();   // the other sum's barrier: every wave has read the last row's slot
    const float s = 1.0f / __builtin_sqrtf(row_sum<L>(sq, slots[1] + own) * a.inv_d + a.eps);
    if (live && lane == 0) {
      if (a.mean != nullptr) a.mean[row] = m;
      if (a.rstd != nullptr) a.rstd[row] = s;
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) a.y[base + lane + i * L] = norm_piece<T, W>(a, lane + i * L, h[i], m, s);
  }
}

constexpr int kLongThreads = 1024;

// Rows that registers do not hold: three passes over the row, the later ones from the caches. At most kLongGrid workgroups, which
// then take several rows, as item_grid's do, but at a number of rows that memory holds and a test reaches (with 2^16 and 2^20 workgroups:
// 131072 x 16392 bf16 1.84 and 1.89 ms, x 65544 9.2-9.5 and 9.2-9.6; 100000 x 32776 fp32 7.1 both).
constexpr int64_t kLongGrid = 1 << 16;
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_fwd_long_kernel(const NormFwd a) {
  constexpr int N = Piece<T>::N, L = kLongThreads;
  __shared__ float slots[2][L / 64];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * a.pieces;
    // a thread writes and reads the same pieces of h throughout
    auto piece = [&](int c) {
      const u32x4 x = a.x[base + c];
      return a.res != nullptr ? sum_piece<T>(x, a.res[base + c]) : x;
    };
    const bool keep = a.res != nullptr && a.h != nullptr;
    auto again = [&](int c) { return keep ? a.h[base + c] : piece(c); };
    float m = 0.0f;
    if (a.layer || keep) {
      float sum = 0.0f;
      for (int c = threadIdx.x; c < a.pieces; c += L) {
        const u32x4 h = piece(c);
        if (keep) a.h[base + c] = h;
        float f[N];
        Piece<T>::unpack(h, f);
#pragma unroll
        for (int r = 0; r < N; ++r) sum += f[r];
      }
      m = row_sum<L>(sum, slots[0]) * a.inv_d;
      if (!a.layer) m = 0.0f;
    } else {
      __syncthreads();
    }
    float sq = 0.0f;
    for (int c = threadIdx.x; c < a.pieces; c += L) {
      float f[N];
      Piece<T>::unpack(again(c), f);
#pragma unroll
      for (int r = 0; r < N; ++r) sq = __builtin_fmaf(f[r] - m, f[r] - m, sq);
    }
    const float s = 1.0f / __builtin_sqrtf(row_sum<L>(sq, slots[1]) * a.inv_d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = m;
      if (a.rstd != nullptr) a.rstd[row] = s;
    }
    for (int c = threadIdx.x; c < a.pieces; c += L) a.y[base + c] = norm_piece<T, W>(a, c, again(c), m, s);
  }
}

// ---- backward ------------------------------------------------------------------------------------

struct NormBwd {
  const u32x4* dy; const u32x4* h; const float* mean; const float* rstd; const void* w; const u32x4* dres;
  u32x4* dx;
  float* part;   // [gridDim.x][2][d]: column sums of dy n, then of dy, over a workgroup's rows; NULL: not formed
  int64_t rows;
  int pieces;
  float inv_d;
};

// g = dy w and n = (h - m) s of one piece.
template <typename T, typename W, int N>
__device__ __forceinline__ void grad_piece(const NormBwd& a, int c, u32x4 dy, u32x4 h, float m, float s, float (&y)[N],
                                           float (&n)[N], float (&g)[N]) {
  Piece<T>::unpack(dy, y);
  Piece<T>::unpack(h, n);
#pragma unroll
  for (int r = 0; r < N; ++r) n[r] = (n[r] - m) * s;
  if (a.w != nullptr) {
    float w[N];
    load_weights<W>(a.w, c, w);
#pragma unroll
    for (int r = 0; r < N; ++r) g[r] = y[r] * w[r];
  } else {
#pragma unroll
    for (int r = 0; r < N; ++r) g[r] = y[r];
  }
}

// dx of one piece: s (g - mean(g) - n mean(g n)) + dres; c1, c2: the means.
template <typename T, int N>
__device__ __forceinline__ u32x4 dx_piece(const float (&g)[N], const float (&n)[N], float s, float c1, float c2, bool add,
                                          u32x4 dres) {
  float o[N];
#pragma unroll
  for (int r = 0; r < N; ++r) o[r] = s * (g[r] - c1 - n[r] * c2);
  if (add) {
    float q[N];
    Piece<T>::unpack(dres, q);
#pragma unroll
    for (int r = 0; r < N; ++r) o[r] += q[r];
  }
  return Piece<T>::pack(o);
}

// A workgroup takes every gridDim-th run of R rows. A thread has the same columns in every one of them, so their sums
// over the rows stay in its registers; the R threads of a column are joined through LDS at the end, in order. The next
// rows are loaded before these are worked on.
template <typename T, typename W, int L, int P>
__global__ __launch_bounds__(norm_threads<L>()) void norm_bwd_kernel(const NormBwd a) {
  constexpr int N = Piece<T>::N, TH = norm_threads<L>(), R = TH / L;
  __shared__ float slots[2][L > 64 ? 2 * TH / 64 : 1];
  __shared__ float joined[R > 1 ? 2 * L * P * N : 1];
  const int lane = threadIdx.x % L;
  float* slot0 = slots[0] + (L > 64 ? threadIdx.x / L * (2 * L / 64) : 0);
  float* slot1 = slots[1] + (L > 64 ? threadIdx.x / L * (2 * L / 64) : 0);
  float aw[P][N], ab[P][N];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int r = 0; r < N; ++r) aw[i][r] = ab[i][r] = 0.0f;
  struct Rows {
    u32x4 dy[P], h[P], q[P];
    float m, s;
  };
  auto load = [&](int64_t r0, Rows& x) {
    const int64_t row = r0 + threadIdx.x / L;
    const bool live = row < a.rows;
    const int64_t base = row * a.pieces + lane;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = live && lane + i * L < a.pieces;
      x.dy[i] = in ? a.dy[base + i * L] : zero;
      x.h[i] = in ? a.h[base + i * L] : zero;
      x.q[i] = in && a.dres != nullptr ? a.dres[base + i * L] : zero;
    }
    x.m = live && a.mean != nullptr ? a.mean[row] : 0.0f;
    x.s = live ? a.rstd[row] : 0.0f;
  };
  Rows next;
  load((int64_t)blockIdx.x * R, next);
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.rows; r0 += (int64_t)gridDim.x * R, turn ^= 1) {
    const int64_t row = r0 + threadIdx.x / L;
    const bool live = row < a.rows;
    const Rows x = next;
    if (r0 + (int64_t)gridDim.x * R < a.rows) load(r0 + (int64_t)gridDim.x * R, next);
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!live || lane + i * L >= a.pieces) continue;
      float y[N], n[N], g[N];
      grad_piece<T, W>(a, lane + i * L, x.dy[i], x.h[i], x.m, x.s, y, n, g);
#pragma unroll
      for (int r = 0; r < N; ++r) {
        c1 += g[r];
        c2 = __builtin_fmaf(g[r], n[r], c2);
        aw[i][r] = __builtin_fmaf(y[r], n[r], aw[i][r]);
        ab[i][r] += y[r];
      }
    }
    if (a.dx == nullptr) continue;   // (uniform)
    row_sum2<L>(c1, c2, turn ? slot1 : slot0);
    c1 = a.mean != nullptr ? c1 * a.inv_d : 0.0f;
    c2 *= a.inv_d;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!live || lane + i * L >= a.pieces) continue;
      float y[N], n[N], g[N];
      grad_piece<T, W>(a, lane + i * L, x.dy[i], x.h[i], x.m, x.s, y, n, g);
      a.dx[row * a.pieces + lane + i * L] = dx_piece<T>(g, n, x.s, c1, c2, a.dres != nullptr, x.q[i]);
    }
  }
  if (a.part == nullptr) return;
  if constexpr (R > 1) {
    float* jw = joined;
    float* jb = joined + L * P * N;
    for (int k = 0; k < R; ++k) {
      if ((int)threadIdx.x / L == k) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int r = 0; r < N; ++r) {
            const int at = (i * N + r) * L + lane;   // (a thread's own words, a bank apart from its neighbour's)
            if (k > 0) {
              aw[i][r] += jw[at];
              ab[i][r] += jb[at];
            }
            if (k + 1 < R) {
              jw[at] = aw[i][r];
              jb[at] = ab[i][r];
            }
          }
      }
      __syncthreads();
    }
    if ((int)threadIdx.x / L != R - 1) return;
  }
  const int64_t d = (int64_t)a.pieces * N;
  float* pw = a.part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = lane + i * L;
    if (c >= a.pieces) continue;
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      *reinterpret_cast<f32x4*>(pw + (int64_t)c * N + 4 * k) = f32x4{aw[i][4 * k], aw[i][4 * k + 1], aw[i][4 * k + 2], aw[i][4 * k + 3]};
      *reinterpret_cast<f32x4*>(pw + d + (int64_t)c * N + 4 * k) = f32x4{ab[i][4 * k], ab[i][4 * k + 1], ab[i][4 * k + 2], ab[i][4 * k + 3]};
    }
  }
}

// Rows whose column sums registers do not hold: dx a workgroup a row in two passes, and the column sums by themselves, a
// thread a piece of the width over every gridDim.y-th row: dy and h are read three times, once from the caches. 4096 x 16384 fp32,
// residual: 223 us for 1.07 GB, 104 for 0.54 and a join of 5, where 192 would carry each byte once.
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_dx_long_kernel(const NormBwd a) {
  constexpr int N = Piece<T>::N, L = kLongThreads;
  __shared__ float slots[2][2 * L / 64];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const int64_t base = row * a.pieces;
    const float m = a.mean != nullptr ? a.mean[row] : 0.0f, s = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f, y[N], n[N], g[N];
    for (int c = threadIdx.x; c < a.pieces; c += L) {
      grad_piece<T, W>(a, c, a.dy[base + c], a.h[base + c], m, s, y, n, g);
#pragma unroll
      for (int r = 0; r < N; ++r) {
        c1 += g[r];
        c2 = __builtin_fmaf(g[r], n[r], c2);
      }
    }
    row_sum2<L>(c1, c2, slots[turn]);
    c1 = a.mean != nullptr ? c1 * a.inv_d : 0.0f;
    c2 *= a.inv_d;
    for (int c = threadIdx.x; c < a.pieces; c += L) {
      grad_piece<T, W>(a, c, a.dy[base + c], a.h[base + c], m, s, y, n, g);
      const bool add = a.dres != nullptr;
      a.dx[base + c] = dx_piece<T>(g, n, s, c1, c2, add, add ? a.dres[base + c] : u32x4{0u, 0u, 0u, 0u});
    }
  }
}
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(const NormBwd a) {
  constexpr int N = Piece<T>::N;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.pieces) return;
  float aw[N] = {}, ab[N] = {};
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float y[N], n[N];
    const float m = a.mean != nullptr ? a.mean[row] : 0.0f, s = a.rstd[row];
    Piece<T>::unpack(a.dy[row * a.pieces + c], y);
    Piece<T>::unpack(a.h[row * a.pieces + c], n);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      aw[r] = __builtin_fmaf(y[r], (n[r] - m) * s, aw[r]);
      ab[r] += y[r];
    }
  }
  const int64_t d = (int64_t)a.pieces * N;
  float* pw = a.part + (int64_t)blockIdx.y * 2 * d + (int64_t)c * N;
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    *reinterpret_cast<f32x4*>(pw + 4 * k) = f32x4{aw[4 * k], aw[4 * k + 1], aw[4 * k + 2], aw[4 * k + 3]};
    *reinterpret_cast<f32x4*>(pw + d + 4 * k) = f32x4{ab[4 * k], ab[4 * k + 1], ab[4 * k + 2], ab[4 * k + 3]};
  }
}

// The workgroups' column sums added up: 16 columns (of dweight, then of dbias) a workgroup, 4 a thread, and 64 runs of the
// parts beside one another, joined in order: of a wave's 16 by lanes, then the four waves.
// 512 parts of 4096 columns: bound by a handful of trips to memory (with 8 runs 4.7 us, with 64 3; behind a backward that has just written them 6.9).
constexpr int kJoinCols = 16;
template <typename W>
__global__ __launch_bounds__(256) void norm_join_kernel(const float* __restrict__ part, int parts, int64_t d, void* dw,
                                                        void* db, int accumulate) {
  __shared__ f32x4 sums[4][4];
  const int tx = threadIdx.x & 3, run = threadIdx.x >> 2, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * kJoinCols + tx * 4;   // d is a multiple of 4: a thread's columns are of one gradient
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < 2 * d) {
#pragma unroll 8
    for (int g = run; g < parts; g += 64) s += *reinterpret_cast<const f32x4*>(part + (int64_t)g * 2 * d + c);
  }
#pragma unroll
  for (int o = 4; o < 64; o <<= 1) {
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] += __shfl_xor(s[r], o);
  }
  if ((threadIdx.x & 63) < 4) sums[wave][tx] = s;
  __syncthreads();
  if (run != 0 || c >= 2 * d) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) s += sums[w][tx];
  void* out = c < d ? dw : db;
  if (out == nullptr) return;
  const int64_t at = c < d ? c : c - d;
  if (accumulate) {
    f32x4* o = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + at);
    *o = *o + s;
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) store1<W>(out, at + r, s[r]);
  }
}

// f(type of the rows, type of the weights)
template <typename F> hipError_t norm_types(DType dt, bool wide, F f) {
  return by_type(dt, [&](auto t) {
    if (wide) return f(t, float{});
    return f(t, t);
  });
}

template <int L, int P> struct NormShape { static constexpr int lanes = L, per = P, rows = L < 256 ? 256 / L : 1; };

// The widest rows that registers hold in the backward, and in the forward with 8 pieces a thread. There bf16 rows, and fp16 rows with
// fp32 weights, would spill (190 bytes a thread): they are long rows. Forward held, and as a long row (us): fp32 4096 x 12288 85 and
// 90, 4096 x 16384 120 and 135, 2048 x 32768 120 and 159; fp16 with its own weights 4096 x 16392 85 and 72, 4096 x 20000 90 and 87,
// 1024 x 65536 61 and 85; bf16 4096 x 16392 239 and 65, 4096 x 20000 258 and 82, 1024 x 65536 119 and 85, 16 x 20000 10.4 and 5.5; fp16 with
// fp32 weights 242 and 73, 260 and 92, 120 and 85, 10.7 and 5.6.
constexpr int kNormBwdPieces = 2048, kNormPieces = 8192;
template <typename T, typename W>
constexpr int norm_held = std::is_same<T, bf16>::value || sizeof(W) != sizeof(T) ? kNormBwdPieces : kNormPieces;

// f(NormShape) for rows of `pieces` pieces: few of them a thread, so that the backward's column sums (two fp32 an element)
// leave room for several waves, and as few lanes idle as three pieces a thread allow. 8192 rows of 4096 bf16, residual, lanes x pieces
// (us): forward 64 x 8 56.8, 128 x 4 50.0, 512 x 1 48.7; backward 64 x 8 101, 128 x 4 64, 256 x 2 62, 512 x 1 58.
template <typename F> hipError_t norm_shape(int pieces, F f) {
  if (pieces <= 16) return f(NormShape<16, 1>{});
  if (pieces <= 32) return f(NormShape<32, 1>{});
  if (pieces <= 64) return f(NormShape<64, 1>{});
  if (pieces <= 128) return f(NormShape<128, 1>{});
  if (pieces <= 192) return f(NormShape<64, 3>{});
  if (pieces <= 256) return f(NormShape<256, 1>{});
  if (pieces <= 384) return f(NormShape<128, 3>{});
  if (pieces <= 512) return f(NormShape<512, 1>{});
  if (pieces <= 768) return f(NormShape<256, 3>{});
  if (pieces <= 1024) return f(NormShape<512, 2>{});
  if (pieces <= 1536) return f(NormShape<512, 3>{});
  return f(NormShape<1024, 2>{});
}

}  // namespace

// Workgroups of a backward, a multiple of the 256 CUs that falls with the width, since each writes its column sums for the join to
// read: 2^18 / pieces rounded up to it, at most 1024; 256 for 16-bit rows beyond 768 pieces, where a workgroup has 8 waves and a
// piece's sums 64 bytes. Together the sums are at most 25 MB up to there and 34 MB at 2048 pieces; of fp32 rows half. Backward and join with
// 256, 512 and 1024 (us): 8192 rows of 4096 bf16 64 + 3, 57 + 3, 61 + 11; 4096 of 8192 63 + 4, 69 + 12, 76 + 21; 5003 of 1024 fp32
// -, 20 + 3, 17 + 3. Calls with 256 and 512: 8192 of 5120 bf16 (640 pieces) 122 and 97, 5003 of 6144 (768) 83 and 70, of 6152 75 and 80;
// 7168: 512 rows 20 and 27, 2048 41 and 49, 8192 125 and 133; 8192 of 8152 132 and 140; 8192 of 3584 fp32 (896) 104 and 98.
int norm_parts(int64_t rows, int pieces, bool fp32) {
  if (pieces > kNormBwdPieces) return (int)std::min<int64_t>(rows, 64);
  int r = 1;
  (void)norm_shape(pieces, [&](auto s) {
    r = decltype(s)::rows;
    return hipSuccess;
  });
  const int64_t most = !fp32 && pieces > 768 ? 256 : std::min<int64_t>(1024, ((1 << 18) / pieces + 255) / 256 * 256);
  return (int)std::min<int64_t>((rows + r - 1) / r, most);
}

hipError_t run_norm_fwd(DType dt, bool wide, const void* x, const void* res, const void* w, const void* b, int64_t rows,
                        int pieces, int64_t d, int layer, float eps, void* y, void* h, float* mean, float* rstd,
                        hipStream_t s) {
  const NormFwd a{static_cast<const u32x4*>(x), static_cast<const u32x4*>(res), w, b, static_cast<u32x4*>(y),
                  static_cast<u32x4*>(h), mean, rstd, rows, pieces, layer, 1.0f / (float)d, eps};
  return norm_types(dt, wide, [&](auto t, auto v) {
    using T = decltype(t);
    using W = decltype(v);
    if (pieces > norm_held<T, W>) {
      hipLaunchKernelGGL((norm_fwd_long_kernel<T, W>), dim3((unsigned)std::min(rows, kLongGrid)), dim3(kLongThreads), 0, s, a);
      return hipGetLastError();
    }
    auto launch = [&](auto shape) {
      constexpr int L = decltype(shape)::lanes, P = decltype(shape)::per, TH = norm_threads<L>();
      hipLaunchKernelGGL((norm_fwd_kernel<T, W, L, P>), dim3(item_grid(rows, TH / L)), dim3(TH), 0, s, a);
      return hipGetLastError();
    };
    if constexpr (norm_held<T, W> > kNormBwdPieces) {
      if (pieces > kNormBwdPieces) return launch(NormShape<1024, 8>{});
    }
    return norm_shape(pieces, launch);
  });
}

hipError_t run_norm_bwd(DType dt, bool wide, const void* dy, const void* h, const float* mean, const float* rstd,
                        const void* w, const void* dres, int64_t rows, int pieces, int64_t d, void* dx, void* dw,
                        void* db, int accumulate, float* part, hipStream_t s) {
  const bool sums = dw != nullptr || db != nullptr;
  const NormBwd a{static_cast<const u32x4*>(dy), static_cast<const u32x4*>(h), mean, rstd, w,
                  static_cast<const u32x4*>(dres), static_cast<u32x4*>(dx), sums ? part : nullptr, rows, pieces,
                  1.0f / (float)d};
  const int parts = norm_parts(rows, pieces, dt == DT_F32);
  return norm_types(dt, wide, [&](auto t, auto v) {
    using T = decltype(t);
    using W = decltype(v);
    hipError_t e = hipSuccess;
    if (rows == 0) {   // only the sums over no rows
    } else if (pieces > kNormBwdPieces) {
      if (dx != nullptr) {
        hipLaunchKernelGGL((norm_dx_long_kernel<T, W>), dim3(item_grid(rows, 1)), dim3(kLongThreads), 0, s, a);
        e = hipGetLastError();
      }
      if (e == hipSuccess && sums) {
        hipLaunchKernelGGL((norm_columns_kernel<T>), dim3((pieces + 255) / 256, parts), dim3(256), 0, s, a);
        e = hipGetLastError();
      }
    } else {
      e = norm_shape(pieces, [&](auto shape) {
        constexpr int L = decltype(shape)::lanes, P = decltype(shape)::per;
        hipLaunchKernelGGL((norm_bwd_kernel<T, W, L, P>), dim3(parts), dim3(norm_threads<L>()), 0, s, a);
        return hipGetLastError();
      });
    }
    if (e != hipSuccess || !sums) return e;
    hipLaunchKernelGGL((norm_join_kernel<W>), dim3((unsigned)((2 * d + kJoinCols - 1) / kJoinCols)), dim3(256), 0, s, part,
                       parts, d, dw, db, accumulate);
    return hipGetLastError();
  });
}

}  // namespace gmlp
