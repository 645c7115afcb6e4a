// Dense projection with bias, activation and residual in its epilogue, and its backward: the
// shared expert or dense branch beside the routed experts.
//
//   forward    z = X W^T + b,  out = residual + act(z)         X [M, K], W [N', K], z [M, N']
//   backward   dZ = dY act'(z),  dX = dZ W,  dW = dZ^T X,  db = sum of dZ over rows
// N' = N, except SwiGLU: N' = 2 N, W = [W_gate; W_up], act(z) = silu(z_gate) z_up.
//
// All three products run on the MFMA main loop of gemm_dense.h: X and W are K-major in the forward;
// dX reads W with its rows along the reduction, dW reads both operands so.  Reductions may end
// inside a stage (any multiple of 8).  Where the output has too few tiles for 256 CUs the
// reduction is cut into slices whose fp32 partial products a second kernel adds in slice order
// before the epilogue (k_lin_finish).
//
// Large products are bound by the matrix cores at the clock that the chip's power allows.  8192 x
// 14336 x 4096 bf16, many passes on end: 700 to 730 us without an activation (1320 to 1370 TFLOP/s, of which
// the loop alone 650), 745 to 755 with GELU (15 vector operations an element), 765 to 780 with bias and
// Z kept too; a library product of that size alone 615 to 630.  Small ones are bound by launches and the
// length of one workgroup's loop.  The two products of a large backward go out apart: together their
// last rounds filled up, but 16384 x 7168 x 4096 took 1578 us against 1537, as idle CUs leave the others
// a higher clock.
//
// The epilogue works on the fp32 accumulators: a tile half is laid out in LDS and walked in
// 16-byte chunks of a row, so that residual, saved pre-activation and output are read and written in
// whole segments and rounded once.
#include "gemm_core.h"
#include "gemm_dense.h"
#include "internal.h"
#include "lin_epi.h"
#include "skinny.h"

namespace moe {

static inline int grid8(int64_t n) { return (int)((n + 7) / 8 * 8); }

// One GEMM: C[m][n] = sum_k A(m, k) B(k, n) over red values of k, B valid for the first bred of
// them (the rest are zeros).  KM: rows contiguous along k; otherwise rows indexed by k.
struct LinGemm {
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  int m, n, red, bred;
  int MT, NT, SK, klen;  // tiles, slices and values of k per slice (a multiple of 64; fp32: 32)
  int tile;              // LIN_BIG, LIN_MID or LIN_SMALL
  bool off_lines;        // rows that do not start on 128-byte lines
  double us;             // the plan's time by the model
  float* part;           // [SK][m][n] when the output goes there
};

enum { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };            // operand layouts
enum { LIN_OUT_EPI = 0, LIN_OUT_GLU = 1, LIN_OUT_PART = 2 };  // where the tile goes

// A tile half held in LDS as fp32 rows (row r in slot r / (TM / 2)), walked in 16-byte chunks: a
// thread owns 8 columns and every 32nd row.
template <class TI>
__device__ __forceinline__ char* lin_frow(char* b0, char* b1, int r) {
  return r < TI::SPLIT ? b0 + r * TI::EPITCH : b1 + (r - TI::SPLIT) * TI::EPITCH;
}
// val(i, h): the four accumulators of row block i and column block h of the half.
template <class TI, class Val>
__device__ __forceinline__ void lin_dump(char* b0, char* b1, int wm, int wn, Val val) {
#pragma unroll
  for (int i = 0; i < TI::MI; ++i) {
    char* row = lin_frow<TI>(b0, b1, (wm * TI::MI + i) * 16 + (threadIdx.x & 15));
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<f32x4*>(row + dn_col(wn, h) * 4) = val(i, h);
  }
}
// Eight values to and from 16-byte chunks (one of bf16, two of fp32).
template <typename T> __device__ __forceinline__ void lin_st8(T* p, const float* f) {
#pragma unroll
  for (int u = 0; u < 8; u += Vec<T>::N) st16_nt(p + u, pack16<T>(f + u));
}

// Walks the staged half: row(r, c, f, res) with 8 fp32 values f of tile row r, columns c .., and 8
// of the residual (zeros without one).  Rows go in batches of KB whose residual chunks are
// requested together; res_row(r) is row r's residual at the half's first column.
template <class TI, typename T, class ResRow, class Row>
__device__ __forceinline__ void lin_walk(char* b0, char* b1, int mrows, int valid, bool has_res, ResRow res_row, Row row) {
  constexpr int NV = 8 / Vec<T>::N, KB = TI::TM_ / 32 < 4 ? TI::TM_ / 32 : 4;
  const int c = (threadIdx.x % (TI::HC / 8)) * 8, r0 = threadIdx.x / (TI::HC / 8);
  if (c >= valid) return;
#pragma unroll
  for (int k0 = 0; k0 < TI::TM_ / 32; k0 += KB) {
    u32x4 rv[KB][NV];
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        rv[k][v] = has_res ? ld16_nt(res_row(min(r0 + 32 * (k0 + k), mrows - 1)) + c + v * Vec<T>::N) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int r = r0 + 32 * (k0 + k);
      const char* p = lin_frow<TI>(b0, b1, r) + c * 4;
      const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
      float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}, rr[8];
#pragma unroll
      for (int v = 0; v < NV; ++v) unpack16<T>(rv[k][v], rr + v * Vec<T>::N);
      if (r < mrows) row(r, c, f, rr);
    }
  }
}

// One product on the dense main loop (gemm_dense.h).  SwiGLU (LIN_OUT_GLU): a tile has TN / 2 output
// columns, the B tile stacks their gate rows over their up rows, so a lane holds both of a column.
template <typename T, class TI, int MODE, bool TAIL, int OUT>
__device__ __forceinline__ void lin_tile(int lin, const LinGemm& g, const LinEpi<T>& ep, char* b0, char* b1) {
  const int per = g.MT * g.NT;
  const int sl = lin / per;
  if (sl >= g.SK) return;
  int mt, nt;
  raster_tile(lin % per, g.MT, g.NT, mt, nt);
  constexpr int HC = TI::HC, TN = OUT == LIN_OUT_GLU ? HC : 2 * HC;
  const int m0 = mt * TI::TM_, n0 = nt * TN;
  const int wave = threadIdx.x >> 6;
  const int wm = wave / TI::WN_, wn = wave % TI::WN_;
  const int k0 = sl * g.klen, klen = min(g.klen, g.red - k0), blen = max(min(g.klen, g.bred - k0), 1);
  const int mrows = min(TI::TM_, g.m - m0);
  const int64_t ldab = g.lda * (int64_t)sizeof(T), ldbb = g.ldb * (int64_t)sizeof(T);
  const char* Ab = static_cast<const char*>(g.A);
  const char* Bb = static_cast<const char*>(g.B);
  DnAcc<TI::MI> acc;
  const int nkt = (int)cdiv(klen, dn_bk<T>());
  if constexpr (MODE == LIN_DW) {
    DnMN<T, TI::TM_, TI::NW, TAIL> la;
    DnMN<T, 2 * HC, TI::NW, TAIL> lb;
    la.init(Ab + k0 * ldab + (int64_t)m0 * sizeof(T), ldab, klen, mrows);
    lb.init(Bb + k0 * ldbb + (int64_t)n0 * sizeof(T), ldbb, blen, min(2 * HC, g.n - n0));
    dn_mainloop<TI>(la, lb, nkt, acc, b0, b1, wm, wn);
  } else {
    DnK<T, TI::TM_, TI::NW, TAIL> la;
    la.init(Ab + m0 * ldab + (int64_t)k0 * sizeof(T), ldab, klen, [&](int i) { return (int64_t)min(i, mrows - 1); });
    if constexpr (MODE == LIN_DX) {
      DnMN<T, 2 * HC, TI::NW, TAIL> lb;
      lb.init(Bb + k0 * ldbb + (int64_t)n0 * sizeof(T), ldbb, blen, min(2 * HC, g.n - n0));
      dn_mainloop<TI>(la, lb, nkt, acc, b0, b1, wm, wn);
    } else {
      DnK<T, 2 * HC, TI::NW, TAIL> lb;
      const int ncols = min(TN, g.n - n0);
      // SwiGLU: the tile's upper half holds the up rows, N rows behind the gate rows
      lb.init(Bb + n0 * ldbb + (int64_t)k0 * sizeof(T), ldbb, klen,
              [&](int i) { return (int64_t)min(OUT == LIN_OUT_GLU ? i % HC : i, ncols - 1); },
              OUT == LIN_OUT_GLU ? g.n * ldbb : 0);
      dn_mainloop<TI>(la, lb, nkt, acc, b0, b1, wm, wn);
    }
  }
  constexpr int MI = TI::MI;
  if constexpr (OUT == LIN_OUT_PART) {
    float* dst = g.part + (int64_t)sl * g.m * g.n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + (j >> 1) * HC + dn_col(wn, j & 1);  // n is a multiple of 4
      if (c >= g.n) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int r = (wm * MI + i) * 16 + (threadIdx.x & 15);
        if (r < mrows) *reinterpret_cast<f32x4*>(dst + (int64_t)(m0 + r) * g.n + c) = acc.c[i][j];
      }
    }
  } else if constexpr (OUT == LIN_OUT_EPI) {
    const int cw = (threadIdx.x % (HC / 8)) * 8;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int c0 = n0 + half * HC, valid = min(HC, g.n - c0);
      if (valid <= 0) break;  // (uniform)
      lin_dump<TI>(b0, b1, wm, wn, [&](int i, int h) { return acc.c[i][2 * half + h]; });
      __syncthreads();
      const T* res = ep.res ? ep.res + m0 * ep.ldr + c0 : nullptr;
      T* out = ep.out + m0 * ep.ldo + c0;
      auto res_row = [&](int r) { return res + r * ep.ldr; };
      if constexpr (MODE == LIN_FWD) {
        float b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (ep.bias && cw < valid) {
#pragma unroll
          for (int u = 0; u < 8; ++u) b[u] = ep.bias[c0 + cw + u];
        }
        T* Z = ep.Z ? ep.Z + m0 * ep.ldz + c0 : nullptr;
        lin_by_act(ep.act, [&](auto A) {
          lin_walk<TI, T>(b0, b1, mrows, valid, res != nullptr, res_row, [&](int r, int c, float (&f)[8], const float (&rr)[8]) {
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] += b[u];
            if (Z) lin_st8(Z + r * ep.ldz + c, f);
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] = lin_act1<decltype(A)::value, T>(f[u]) + rr[u];
            lin_st8(out + r * ep.ldo + c, f);
          });
        });
      } else {
        lin_walk<TI, T>(b0, b1, mrows, valid, res != nullptr, res_row, [&](int r, int c, float (&f)[8], const float (&rr)[8]) {
#pragma unroll
          for (int u = 0; u < 8; ++u) f[u] += rr[u];
          lin_st8(out + r * ep.ldo + c, f);
        });
      }
      __syncthreads();
    }
  } else {  // SwiGLU: block 0 is the gate, block 1 the up projection of the same columns
    const int valid = min(HC, g.n - n0);
    if (ep.bias) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n0 + dn_col(wn, j & 1);
        f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
        if (c < g.n) b = *reinterpret_cast<const f32x4*>(ep.bias + (int64_t)(j >> 1) * g.n + c);
#pragma unroll
        for (int i = 0; i < MI; ++i) acc.c[i][j] += b;
      }
    }
    if (ep.Z) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lin_dump<TI>(b0, b1, wm, wn, [&](int i, int h) { return acc.c[i][2 * j + h]; });
        __syncthreads();
        lin_walk<TI, T>(b0, b1, mrows, valid, false, [&](int) { return ep.res; }, [&](int r, int c, float (&f)[8], const float (&)[8]) {
          lin_st8(ep.Z + (m0 + r) * ep.ldz + (int64_t)j * g.n + n0 + c, f);
        });
        __syncthreads();
      }
    }
    lin_dump<TI>(b0, b1, wm, wn, [&](int i, int h) {
      f32x4 v = acc.c[i][h];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = v[u] * sigmoid_f32(v[u]) * acc.c[i][2 + h][u];
      return v;
    });
    __syncthreads();
    lin_walk<TI, T>(b0, b1, mrows, valid, ep.res != nullptr, [&](int r) { return ep.res + (m0 + r) * ep.ldr + n0; },
                 [&](int r, int c, float (&f)[8], const float (&rr)[8]) {
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] += rr[u];
      lin_st8(ep.out + (m0 + r) * ep.ldo + n0 + c, f);
    });
  }
}

template <typename T, class TI, int MODE, bool TAIL, int OUT>
__global__ __launch_bounds__(TI::THREADS, TI::NW == 8 ? 1 : 2) void k_lin(LinGemm g, LinEpi<T> ep) {
  __shared__ __attribute__((aligned(1024))) char b0[TI::SLOT];
  __shared__ __attribute__((aligned(1024))) char b1[TI::SLOT];
  lin_tile<T, TI, MODE, TAIL, OUT>(xcd_remap(blockIdx.x, gridDim.x), g, ep, b0, b1);
}

// The backward's two products in one launch, where neither fills the chip: workgroups below nx take
// dX's tiles, the others dW's.
template <typename T, class TI, int OUT_X, int OUT_W>
__global__ __launch_bounds__(TI::THREADS, 2) void k_lin_pair(LinGemm gx, LinEpi<T> ex, int nx, LinGemm gw, LinEpi<T> ew) {
  __shared__ __attribute__((aligned(1024))) char b0[TI::SLOT];
  __shared__ __attribute__((aligned(1024))) char b1[TI::SLOT];
  if ((int)blockIdx.x < nx) lin_tile<T, TI, LIN_DX, true, OUT_X>(xcd_remap(blockIdx.x, nx), gx, ex, b0, b1);
  else lin_tile<T, TI, LIN_DW, true, OUT_W>(xcd_remap(blockIdx.x - nx, gridDim.x - nx), gw, ew, b0, b1);
}

// Adds the SK slices in slice order and applies the epilogue; a thread takes four consecutive
// output columns and requests the slices four at a time.  n: output columns; np: columns of the
// partial products (2 n for SwiGLU).
template <typename T>
__device__ __forceinline__ void lin_finish(int64_t i, const float* __restrict__ part, int SK, int m, int n, int np,
                                           const LinEpi<T>& ep) {
  const int cpr = n / 4;
  if (i >= (int64_t)m * cpr) return;
  const int64_t r = i / cpr;
  const int c = (int)(i - r * cpr) * 4;
  const int64_t slice = (int64_t)m * np;
  const bool glu = np != n;
  const float* p = part + r * np + c;
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f}, zu = z;
  auto ld = [](const float* q) { return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(q)); };
  int s = 0;
  for (; s + 4 <= SK; s += 4, p += 4 * slice) {
    f32x4 v[4], w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = ld(p + k * slice);
      if (glu) w[k] = ld(p + k * slice + n);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      z += v[k];
      if (glu) zu += w[k];
    }
  }
  for (; s < SK; ++s, p += slice) {
    z += ld(p);
    if (glu) zu += ld(p + n);
  }
  lin_epi4(ep, r, c, n, glu, z, zu);
}
template <typename T>
__global__ __launch_bounds__(256) void k_lin_finish(const float* __restrict__ part, int SK, int m, int n, int np,
                                                    LinEpi<T> ep) {
  lin_finish<T>((int64_t)blockIdx.x * 256 + threadIdx.x, part, SK, m, n, np, ep);
}

// db = the row blocks' sums (fp64) for 8 columns: 32 runs of row blocks, then the runs in order (many
// rows and few columns leave hundreds of row blocks: 5875 x 24 takes 735, 12 us by 8 runs).
constexpr int LIN_DB_COLS = 8, LIN_DB_RUNS = 32;
__device__ __forceinline__ void lin_db(int block, const float* __restrict__ db_part, int blocks, int np,
                                       float* __restrict__ db) {
  __shared__ double red[LIN_DB_RUNS][LIN_DB_COLS + 1];
  const int cl = threadIdx.x % LIN_DB_COLS, run = threadIdx.x / LIN_DB_COLS;
  const int c = block * LIN_DB_COLS + cl;  // np is a multiple of 8
  double v = 0.0;
#pragma unroll 8
  for (int b = run; b < blocks; b += LIN_DB_RUNS) v += (double)db_part[(int64_t)b * np + c];
  red[run][cl] = v;
  __syncthreads();
  if (run == 0) {
#pragma unroll
    for (int q = 1; q < LIN_DB_RUNS; ++q) v += red[q][cl];
    db[c] = (float)v;
  }
}
__global__ __launch_bounds__(256) void k_lin_db(const float* __restrict__ db_part, int blocks, int np,
                                                float* __restrict__ db) {
  lin_db(blockIdx.x, db_part, blocks, np, db);
}

// What is left after k_lin_pair's partial products, in one launch: dX, dW and db (when given).
struct LinDb {
  const float* part;
  int blocks, np;
  float* db;
};
template <typename T>
__global__ __launch_bounds__(256) void k_lin_finish_pair(LinGemm gx, LinEpi<T> ex, int nx, LinGemm gw, LinEpi<T> ew, int nw,
                                                         LinDb d) {
  const int b = blockIdx.x;
  if (b < nx) lin_finish<T>((int64_t)b * 256 + threadIdx.x, gx.part, gx.SK, gx.m, gx.n, gx.n, ex);
  else if (b < nx + nw) lin_finish<T>((int64_t)(b - nx) * 256 + threadIdx.x, gw.part, gw.SK, gw.m, gw.n, gw.n, ew);
  else lin_db(b - nx - nw, d.part, d.blocks, d.np, d.db);
}

// A few rows (single tokens, small decode batches): one workgroup per 16 RT rows of W, its waves
// sharing the reduction; W is streamed from memory straight into the MFMA's A operand (two batches
// of loads in flight per wave) and X, which stays in the caches, into B, NG groups of 16 rows.  The
// waves' partial tiles meet in LDS, are added in wave order, and the epilogue runs in the same
// launch.  Bound by reading W once: one row, SwiGLU, 4096 x 7168 weights 10.8 us (5.4 TB/s); 13 rows,
// 7168 x 2048 weights with a residual 8.6 us, of which a launch is about 3.
// SwiGLU with RT = 1 takes 8 gate rows and the 8 matching up rows, so that a column's two halves lie
// 32 lanes apart; with RT = 2 16 gate rows and their 16 up rows, in the same lane.
template <typename T, int NG, int RT>
struct LinStream {
  static constexpr int U = NG + RT <= 3 ? 4 : 2;  // steps per batch: two batches fit the registers
  const T* w[RT];  // lane's W rows at its k offset
  const T* x[NG];
  u32x4 wv[2][U][RT], xv[2][U][NG];
  __device__ __forceinline__ void load(int buf, int st, int last) {
    constexpr int S = DecMma<T>::S;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(st + u, last) * S;
#pragma unroll
      for (int r = 0; r < RT; ++r) wv[buf][u][r] = ld16(w[r] + k);
#pragma unroll
      for (int g = 0; g < NG; ++g) xv[buf][u][g] = ld16(x[g] + k);
    }
  }
  __device__ __forceinline__ void mma(int buf, int live, f32x4 (&acc)[RT][NG]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < live) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int g = 0; g < NG; ++g) acc[r][g] = DecMma<T>::mma(wv[buf][u][r], xv[buf][u][g], acc[r][g]);
      }
  }
  // steps [a, b), a < b: batches of U with the next batch's loads issued before the current one's
  // MFMAs; steps past b repeat the last one and are not used
  __device__ __forceinline__ void run(int a, int b, f32x4 (&acc)[RT][NG]) {
    load(0, a, b - 1);
    int st = a;
    for (; st + 2 * U < b; st += 2 * U) {  // steady state: both batches whole
      load(1, st + U, b - 1);
      mma(0, U, acc);
      load(0, st + 2 * U, b - 1);
      mma(1, U, acc);
    }
    if (st + U < b) {
      load(1, st + U, b - 1);
      mma(0, U, acc);
      mma(1, b - st - U, acc);
    } else {
      mma(0, b - st, acc);
    }
  }
};

template <typename T, int NG, int RT, bool GLU>
__global__ __launch_bounds__(512) void k_lin_skinny(const T* __restrict__ X, int64_t ldx, const T* __restrict__ W,
                                                    int m, int n, int K, LinEpi<T> ep) {
  extern __shared__ f32x4 sk_part[];  // [wave][RT][NG][64]
  constexpr int S = DecMma<T>::S, V = DecMma<T>::V;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W_ = blockDim.x >> 6;
  const int r16 = lane & 15, q = lane >> 4, ko = q * V;
  constexpr int TC = GLU ? 8 * RT : 16 * RT;  // output columns per tile
  const int c0 = blockIdx.x * TC;
  LinStream<T, NG, RT> ds;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = !GLU ? min(c0 + 16 * r + r16, n - 1)
                         : (RT == 1 ? (r16 < 8 ? c0 + r16 : n + c0 + r16 - 8) : r * n + min(c0 + r16, n - 1));
    ds.w[r] = W + (int64_t)row * K + ko;
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) ds.x[g] = X + (int64_t)min(g * 16 + r16, m - 1) * ldx + ko;
  f32x4 acc[RT][NG];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int ns = K / S, a = (int)((int64_t)ns * wave / W_), b = (int)((int64_t)ns * (wave + 1) / W_);
  if (a < b) ds.run(a, b, acc);
  if (wave == W_ - 1 && K % S) {  // the last, partial step: lanes past K supply zeros on both sides
    const bool in = ns * S + ko < K;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const u32x4 xv = in ? ld16(ds.x[g] + ns * S) : zero;
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r][g] = DecMma<T>::mma(in ? ld16(ds.w[r] + ns * S) : zero, xv, acc[r][g]);
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int g = 0; g < NG; ++g) sk_part[((wave * RT + r) * NG + g) * 64 + lane] = acc[r][g];
  __syncthreads();
  auto total = [&](int r, int g) {
    f32x4 v = sk_part[(r * NG + g) * 64 + lane];
    for (int w = 1; w < W_; ++w) v += sk_part[((w * RT + r) * NG + g) * 64 + lane];
    return v;
  };
  constexpr int ITEMS = (GLU ? 1 : RT) * NG;  // 16 x 16 (SwiGLU: 8 RT x 16) output blocks
  for (int it = wave; it < ITEMS; it += W_) {
    const int g = it % NG, r = it / NG, t = g * 16 + r16;
    if constexpr (GLU) {
      f32x4 z = total(0, g), up;
      if constexpr (RT == 1) {
#pragma unroll
        for (int u = 0; u < 4; ++u) up[u] = __shfl_xor(z[u], 32, 64);
      } else {
        up = total(1, g);
      }
      const int c = c0 + 4 * q;
      if ((RT == 2 || q < 2) && t < m && c < n) lin_epi4(ep, (int64_t)t, c, n, true, z, up);
    } else {
      const int c = c0 + 16 * r + 4 * q;
      const f32x4 z = total(r, g);
      if (t < m && c < n) lin_epi4(ep, (int64_t)t, c, n, false, z, z);
    }
  }
}

// dZ = dY act'(z) (SwiGLU: [dG | dU]) and the bias gradient's partial sums: a workgroup takes 256
// columns (32 lanes of 8) and `rows` rows (8 at a time); db_part[row block][column].  dZ may be
// null (only the sums), db_part too.  Bound by memory: 16384 x 2048 SwiGLU, 336 MB, 61 us.
template <typename T>
__global__ __launch_bounds__(256) void k_lin_dz(const T* __restrict__ dY, int64_t ldy, const T* __restrict__ Z, int m,
                                                int n, int act, int rows, T* __restrict__ dZ,
                                                float* __restrict__ db_part) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ float red[8][256 + 4];
  const int glu = act == LIN_SWIGLU, np = glu ? 2 * n : n;
  const int cl = (threadIdx.x & 31) * 8, rl = threadIdx.x >> 5;
  const int cbs = (n + 255) / 256, cb = blockIdx.x % cbs, rb = blockIdx.x / cbs;
  const int c = cb * 256 + cl;
  const int r0 = rb * rows, r1 = min(m, r0 + rows);
  float s0[8], s1[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) s0[u] = s1[u] = 0.0f;
  if (c < n) {
    for (int r = r0 + rl; r < r1; r += 8) {
      float dy[8], z[8], zu[8];
#pragma unroll
      for (int u = 0; u < 8; u += VEC) {
        unpack16<T>(ld16(dY + r * ldy + c + u), dy + u);
        if (act != LIN_NONE) unpack16<T>(ld16_nt(Z + (int64_t)r * np + c + u), z + u);
        if (glu) unpack16<T>(ld16_nt(Z + (int64_t)r * np + n + c + u), zu + u);
      }
      if (glu) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float sg = sigmoid_f32(z[u]), d = dy[u];
          dy[u] = d * zu[u] * sg * (1.0f + z[u] * (1.0f - sg));
          zu[u] = d * z[u] * sg;
          s0[u] += dy[u];
          s1[u] += zu[u];
        }
      } else {
        lin_by_act(act, [&](auto A) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            dy[u] = lin_bwd1<decltype(A)::value>(dy[u], z[u]);
            s0[u] += dy[u];
          }
        });
      }
      if (dZ) {
#pragma unroll
        for (int u = 0; u < 8; u += VEC) {
          st16(dZ + (int64_t)r * np + c + u, pack16<T>(dy + u));
          if (glu) st16(dZ + (int64_t)r * np + n + c + u, pack16<T>(zu + u));
        }
      }
    }
  }
  if (!db_part) return;
  for (int h = 0; h <= glu; ++h) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 8; ++u) red[rl][cl + u] = h ? s1[u] : s0[u];
    __syncthreads();
    const int col = cb * 256 + threadIdx.x;
    if (col < n) {
      float v = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += red[q][threadIdx.x];
      db_part[(int64_t)rb * np + h * n + col] = v;
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
// The tiles: 256 x 256 on eight waves (bf16), 128 x 128 on four with two workgroups per CU, and
// 64 x 64 on two with up to five.
enum { LIN_BIG = 256, LIN_MID = 128, LIN_SMALL = 64 };
typedef DnTile<256, 256, 2, 4> LinBig;
typedef DnTile<128, 128, 2, 2> LinMid;
typedef DnTile<64, 64, 2, 1> LinSmall;

// Tile size and slices of a product's reduction: the cheapest by a model of the time in
// microseconds, fitted to measured times.  A round of 256 large tiles takes 1.4 per stage and 10
// besides.  The smaller tiles take 4 besides and per stage: 128 x 128 0.5 where every CU has one
// workgroup and 0.95 where it has two; 64 x 64 0.29, and 0.165 per workgroup of the CU beyond that;
// where an operand is read with its rows along the reduction in a launch of two products 0.8 and
// 0.45 at least.  In fp32 a stage takes 2.05 and 3.8, or 1.05, 2.0 and 0.61 per workgroup (and
// 128 x 128 tiles 5.5 besides).  Slices cost a second launch (2.5) and 1.2 per million partial
// products written and read back.  Measured (4096 x 4096 weights, bf16; 64 x 64 | 128 x 128 tiles):
// 64 rows 12.4 us with 4 slices, 22.1 with one | 13.6 with 8, 30 with one; 256 rows 20.4 with 2 |
// 19.9 with 4, 31.7 with one; 300 x 512 x 512 6.0 | 8.7; 100 x 4096 x 512 fp32 15.2 with 2 | 18.1
// with 6; 1237 x 904 x 1544 fp32 47 with 3 | 46 with 3, 104 with one.
constexpr int kLinSlices[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
static int lin_stages(const LinGemm& g, bool bf16_) { return (int)cdiv(g.red, bf16_ ? dn_bk<bf16>() : dn_bk<float>()); }
static int64_t lin_tiles(const LinGemm& g, int tile) { return cdiv(g.m, tile) * cdiv(g.n, tile); }
// wgs workgroups of `stages` stages on tiles below the largest, out partial products in all.
static double lin_time(int tile, double wgs, int64_t stages, double out, bool bf16_, bool pair, double slow) {
  const double per = wgs / 256.0;  // workgroups per CU
  double stage, most;              // per stage; workgroups that a CU holds
  const double besides = !bf16_ && tile == LIN_MID ? 5.5 : 4.0;
  if (tile == LIN_MID) {
    stage = bf16_ ? (per > 1 ? 0.95 : (pair ? 0.8 : 0.5)) : (per > 1 ? 3.8 : 2.05);
    most = 2;
  } else {
    const double share = bf16_ ? 0.165 * slow : 0.61, least = bf16_ ? (pair ? 0.45 : 0.29) : (per > 1 ? 2.0 : 1.05);
    stage = share * per > least ? share * per : least;
    most = 5;
    if (per > most) stage = share * most;
  }
  const double rounds = per <= most ? 1.0 : per / most;
  return rounds * (stages * stage + besides) + (out > 0 ? 2.5 + 1.2e-6 * out : 0.0);
}
static void lin_set(LinGemm& g, bool bf16_, int tile, int sk) {
  g.tile = tile;
  g.MT = (int)cdiv(g.m, tile);
  g.NT = (int)cdiv(g.n, tile);
  g.klen = (int)cdiv(lin_stages(g, bf16_), sk) * (bf16_ ? dn_bk<bf16>() : dn_bk<float>());
  g.SK = g.red > 0 ? (int)cdiv(g.red, g.klen) : 1;
}
// What bf16 64 x 64 tiles lose, as they load twice as much per product as 128 x 128 ones, where the
// operands leave the L2s and where rows do not start on 128-byte lines (2560 x 1024 x 7168: 78 us on
// them, 55 on 128 x 128; 3000 x 1000 x 2000: 30.6 and 23.7).
static double lin_slow(const LinGemm& g) {
  const double mb = 2e-6 * g.red * ((double)g.m + g.n);
  return (mb > 40 ? 1.6 : mb > 24 ? 1.2 : 1.0) * (g.off_lines ? 1.3 : 1.0);
}
static void lin_plan(LinGemm& g, bool bf16_, bool may_split) {
  const int stages = lin_stages(g, bf16_);
  const double slow = lin_slow(g);
  double best = bf16_ ? cdiv(lin_tiles(g, LIN_BIG), 256) * (stages * 1.4 + 10.0) : 1e30;
  int tile = LIN_BIG, sk = 1;
  for (int t : {LIN_MID, LIN_SMALL})
    for (int q : kLinSlices) {
      if (q > 1 && (!may_split || q > stages)) break;
      const double us = lin_time(t, lin_tiles(g, t) * q, cdiv(stages, q), q > 1 ? (double)q * g.m * g.n : 0.0, bf16_, false, slow);
      if (us < best) {
        best = us;
        tile = t;
        sk = q;
      }
    }
  lin_set(g, bf16_, tile, sk);
  g.us = best;
}

// Rows per workgroup of k_lin_dz: 64 where that gives four workgroups per CU, fewer (at least 8) for
// small inputs, whose time is the length of one workgroup's row loop.
static int lin_dz_rows(const LinShape& s) {
  int rows = 64;
  while (rows > 8 && cdiv(s.N, 256) * cdiv(s.M, rows) < 1024) rows /= 2;
  return rows;
}

// Whether the forward streams W through k_lin_skinny: up to 16 rows, and up to 32 while K keeps the
// repeated reads of X short (7168 x 2048 weights, 32 rows: 10.5 us against 12.3 tiled; 4096 x 4096:
// 13.6 against 12.2).
static bool lin_is_skinny(const LinShape& s) { return s.M <= 16 || (s.M <= 32 && s.K <= 2048); }

static LinGemm lin_gemm(const LinShape& s, int mode) {
  LinGemm g{};
  const int NW = (int)(s.act == LIN_SWIGLU ? 2 * s.N : s.N);
  if (mode == LIN_FWD) {
    g.m = (int)s.M;
    g.n = NW;
    g.red = (int)s.K;
  } else if (mode == LIN_DX) {
    g.m = (int)s.M;
    g.n = (int)s.K;
    g.red = NW;
  } else {
    g.m = NW;
    g.n = (int)s.K;
    g.red = (int)s.M;
  }
  g.bred = g.red;
  g.off_lines = s.K % 64 || (mode != LIN_FWD && NW % 64);
  lin_plan(g, s.bf16, true);
  return g;
}

static size_t lin_part_bytes(const LinGemm& g) { return (size_t)g.SK * g.m * g.n * sizeof(float); }

size_t linear_fwd_workspace_bytes(const LinShape& s) {
  if (lin_is_skinny(s)) return 0;
  const LinGemm g = lin_gemm(s, LIN_FWD);
  return g.SK > 1 ? lin_part_bytes(g) : 0;
}

// The backward's two products in one launch, each cut so that no workgroup has more than `most` stages
// (a batch of many rows has a short reduction for dX and a long one for dW): where the model says
// that this beats one after the other.  Replayed from a graph: 999 x 1000 x 264, ReLU with a bias, 28.5 us in
// six launches, 18.7 in three; 12062 x 296 x 424 29 us apart, 25.5 together; 2048 x 2048 x 2048 46 and 40.
// What small tiles lose (lin_slow) counts for the pair too: on 64 x 64 tiles 12062 x 296 x 424 takes 32
// together, 3000 x 2000 x 1000 65 (49 apart), 1500 x 1000 x 2000 33 (26 together on 128 x 128).  False: one
// after the other, each with a plan of its own, in gx and gw.
static bool lin_pair_plan(const LinShape& s, LinGemm& gx, LinGemm& gw) {
  // with over four rounds of tiles each product fills the chip by itself (16384 x 512 x 2048: 91 us
  // apart, 98 together)
  if (s.M == 0 || lin_tiles(gx, LIN_MID) + lin_tiles(gw, LIN_MID) > 1024) return false;
  const double apart = gx.us + gw.us, sx_slow = lin_slow(gx), sw_slow = lin_slow(gw);
  const double slow = sx_slow > sw_slow ? sx_slow : sw_slow;  // as for the products apart
  const int sx = lin_stages(gx, s.bf16), sw = lin_stages(gw, s.bf16), longest = sx > sw ? sx : sw;
  double best = 0.9 * apart;  // (its error, within which the simpler launches stay)
  int tile = 0, most = 0;
  for (int t : {LIN_MID, LIN_SMALL})
    for (int q : kLinSlices) {
      if (q > longest) break;
      const int len = (int)cdiv(longest, q), qx = (int)cdiv(sx, len), qw = (int)cdiv(sw, len);
      const double out = (qx > 1 ? (double)qx * gx.m * gx.n : 0.0) + (qw > 1 ? (double)qw * gw.m * gw.n : 0.0);
      // the shorter product's workgroups count by their share of the longest
      const double wgs = ((double)lin_tiles(gx, t) * sx + (double)lin_tiles(gw, t) * sw) / len;
      const double us = lin_time(t, wgs, len, out, s.bf16, true, slow);
      if (us < best) {
        best = us;
        tile = t;
        most = len;
      }
    }
  if (!tile) return false;
  lin_set(gx, s.bf16, tile, (int)cdiv(sx, most));
  lin_set(gw, s.bf16, tile, (int)cdiv(sw, most));
  return true;
}

struct LinBwdWs {
  LinGemm gx, gw;  // the plans
  bool pair;
  void* dZ;
  float* db_part;
  float* part;    // of a product on its own, or dX's of a pair
  float* part_w;  // dW's of a pair
};
static size_t lin_carve_bwd(const LinShape& s, void* base, LinBwdWs* w) {
  char* b = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = b ? b + off : nullptr;
    off = align_up(off + bytes, 256);
    return p;
  };
  const int64_t NW = s.act == LIN_SWIGLU ? 2 * s.N : s.N;
  LinBwdWs q;
  q.dZ = take(s.act == LIN_NONE ? 0 : (size_t)s.M * NW * (s.bf16 ? 2 : 4));
  q.db_part = reinterpret_cast<float*>(take((size_t)cdiv(s.M, lin_dz_rows(s)) * NW * 4));
  q.gx = lin_gemm(s, LIN_DX);
  q.gw = lin_gemm(s, LIN_DW);
  q.pair = lin_pair_plan(s, q.gx, q.gw);
  const size_t px = q.gx.SK > 1 ? lin_part_bytes(q.gx) : 0, pw = q.gw.SK > 1 ? lin_part_bytes(q.gw) : 0;
  q.part_w = q.pair ? reinterpret_cast<float*>(take(pw)) : nullptr;
  const size_t alone = q.pair || px > pw ? px : pw;
  q.part = reinterpret_cast<float*>(take(alone));
  if (w) *w = q;
  return off;
}

size_t linear_bwd_workspace_bytes(const LinShape& s) { return lin_carve_bwd(s, nullptr, nullptr); }

int linear_plan(const LinShape& s, int product, int* slices, bool* paired) {
  *slices = 1;
  *paired = false;
  if (product == LIN_FWD && lin_is_skinny(s)) return 0;
  LinBwdWs w;
  LinGemm g;
  if (product == LIN_FWD) {
    g = lin_gemm(s, LIN_FWD);
  } else {
    lin_carve_bwd(s, nullptr, &w);
    g = product == LIN_DX ? w.gx : w.gw;
    *paired = w.pair;
  }
  *slices = g.SK;
  return g.tile;
}

template <typename T, class TI, int MODE, int OUT>
static void lin_launch_t(const LinGemm& g, const LinEpi<T>& ep, hipStream_t st) {
  const int grid = grid8((int64_t)g.MT * g.NT * g.SK);
  if (g.red % dn_bk<T>() || g.bred != g.red) k_lin<T, TI, MODE, true, OUT><<<grid, TI::THREADS, 0, st>>>(g, ep);
  else k_lin<T, TI, MODE, false, OUT><<<grid, TI::THREADS, 0, st>>>(g, ep);
}
template <int MODE, int OUT, typename T>
static void lin_launch(const LinGemm& g, const LinEpi<T>& ep, hipStream_t st) {
  if (g.tile == LIN_SMALL) lin_launch_t<T, LinSmall, MODE, OUT>(g, ep, st);
  else if (g.tile == LIN_MID) lin_launch_t<T, LinMid, MODE, OUT>(g, ep, st);
  else if constexpr (sizeof(T) == 2 && OUT != LIN_OUT_PART) lin_launch_t<T, LinBig, MODE, OUT>(g, ep, st);  // never sliced
}

hipError_t launch_lin_finish(const float* part, int SK, int m, int n, int np, const LinEpi<bf16>& ep, hipStream_t st) {
  k_lin_finish<bf16><<<(int)cdiv((int64_t)m * (n / 4), 256), 256, 0, st>>>(part, SK, m, n, np, ep);
  return hipGetLastError();
}

// A product whose epilogue is ep: directly, or through partial products where it is sliced.
template <int MODE, typename T>
static hipError_t lin_run(LinGemm g, float* part, const LinEpi<T>& ep, hipStream_t st) {
  if (g.m == 0) return hipSuccess;
  if (g.SK == 1) {
    if constexpr (MODE == LIN_FWD) {
      if (ep.act == LIN_SWIGLU) {
        g.n /= 2;
        g.NT = (int)cdiv(g.n, g.tile / 2);
        lin_launch<MODE, LIN_OUT_GLU>(g, ep, st);
        return hipGetLastError();
      }
    }
    lin_launch<MODE, LIN_OUT_EPI>(g, ep, st);
    return hipGetLastError();
  }
  g.part = part;
  lin_launch<MODE, LIN_OUT_PART>(g, ep, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int n = ep.act == LIN_SWIGLU ? g.n / 2 : g.n;
  k_lin_finish<T><<<(int)cdiv((int64_t)g.m * (n / 4), 256), 256, 0, st>>>(part, g.SK, g.m, n, g.n, ep);
  return hipGetLastError();
}

template <typename T>
static LinEpi<T> lin_epi(const float* bias, const void* res, int64_t ldr, void* Z, int64_t ldz, void* out, int64_t ldo,
                         int act) {
  return LinEpi<T>{bias, static_cast<const T*>(res), ldr, static_cast<T*>(Z), ldz, static_cast<T*>(out), ldo, act};
}

template <typename T, int NG, int RT>
static void lin_skinny_rt(const LinShape& s, const void* X, const void* W, const LinEpi<T>& ep, hipStream_t st) {
  const bool glu = s.act == LIN_SWIGLU;
  const int tiles = (int)cdiv(s.N, (glu ? 8 : 16) * RT);
  // waves per tile: more while a wave has over 16 steps to read, or while the grid has fewer than 6
  // waves per CU and a wave at least 8 steps (16384 x 4096 weights, one row: 32.0 us with 2 waves,
  // 26.3 with 8; 7168 x 2048: 7.6 with 4, 8.1 with 8)
  const int steps = (int)(s.K / DecMma<T>::S);
  int w = 4;
  while (w < 8 && (steps / w > 16 || (tiles * w < 1536 && steps / w >= 8))) w *= 2;
  const size_t lds = (size_t)w * RT * NG * 64 * sizeof(f32x4);
  const T* x = static_cast<const T*>(X);
  const T* wt = static_cast<const T*>(W);
  if (glu) k_lin_skinny<T, NG, RT, true><<<tiles, w * 64, lds, st>>>(x, s.ldx, wt, (int)s.M, (int)s.N, (int)s.K, ep);
  else k_lin_skinny<T, NG, RT, false><<<tiles, w * 64, lds, st>>>(x, s.ldx, wt, (int)s.M, (int)s.N, (int)s.K, ep);
}
// Two row blocks per wave halve the reads of X, where that still leaves a workgroup for nearly every CU.
template <typename T, int NG>
static void lin_skinny_ng(const LinShape& s, const void* X, const void* W, const LinEpi<T>& ep, hipStream_t st) {
  if (s.M > 1 && cdiv(s.N, s.act == LIN_SWIGLU ? 16 : 32) >= 224) lin_skinny_rt<T, NG, 2>(s, X, W, ep, st);
  else lin_skinny_rt<T, NG, 1>(s, X, W, ep, st);
}
template <typename T>
static hipError_t lin_skinny(const LinShape& s, const void* X, const void* W, const LinEpi<T>& ep, hipStream_t st) {
  if (s.M <= 16) lin_skinny_ng<T, 1>(s, X, W, ep, st);
  else lin_skinny_ng<T, 2>(s, X, W, ep, st);
  return hipGetLastError();
}

template <typename T>
static hipError_t lin_forward(const LinShape& s, const void* X, const void* W, const LinEpi<T>& ep, void* ws, hipStream_t st) {
  if (lin_is_skinny(s)) return lin_skinny(s, X, W, ep, st);
  LinGemm g = lin_gemm(s, LIN_FWD);
  g.A = X;
  g.lda = s.ldx;
  g.B = W;
  g.ldb = s.K;
  return lin_run<LIN_FWD>(g, static_cast<float*>(ws), ep, st);
}

hipError_t launch_linear(const LinShape& s, const void* X, const void* W, const float* bias, const void* residual,
                         void* Z, void* out, void* ws, hipStream_t st) {
  if (s.M == 0) return hipSuccess;
  const int64_t NW = s.act == LIN_SWIGLU ? 2 * s.N : s.N;
  if (s.bf16) return lin_forward<bf16>(s, X, W, lin_epi<bf16>(bias, residual, s.ldr, Z, NW, out, s.ldy, s.act), ws, st);
  return lin_forward<float>(s, X, W, lin_epi<float>(bias, residual, s.ldr, Z, NW, out, s.ldy, s.act), ws, st);
}

template <typename T, class TI>
static void lin_pair_launch(const LinGemm& gx, const LinEpi<T>& ex, const LinGemm& gw, const LinEpi<T>& ew, hipStream_t st) {
  const int nx = grid8((int64_t)gx.MT * gx.NT * gx.SK), grid = nx + grid8((int64_t)gw.MT * gw.NT * gw.SK);
  const bool px = gx.SK > 1, pw = gw.SK > 1;
  if (px && pw) k_lin_pair<T, TI, LIN_OUT_PART, LIN_OUT_PART><<<grid, TI::THREADS, 0, st>>>(gx, ex, nx, gw, ew);
  else if (px) k_lin_pair<T, TI, LIN_OUT_PART, LIN_OUT_EPI><<<grid, TI::THREADS, 0, st>>>(gx, ex, nx, gw, ew);
  else if (pw) k_lin_pair<T, TI, LIN_OUT_EPI, LIN_OUT_PART><<<grid, TI::THREADS, 0, st>>>(gx, ex, nx, gw, ew);
  else k_lin_pair<T, TI, LIN_OUT_EPI, LIN_OUT_EPI><<<grid, TI::THREADS, 0, st>>>(gx, ex, nx, gw, ew);
}

template <typename T>
static hipError_t lin_backward(const LinShape& s, const T* dY, const T* X, const T* W, const T* Z, T* dX, T* dW,
                               float* dbias, void* ws, hipStream_t st) {
  LinBwdWs w;
  lin_carve_bwd(s, ws, &w);
  const bool none = s.act == LIN_NONE;
  const int NW = (int)(s.act == LIN_SWIGLU ? 2 * s.N : s.N);
  const int rows = lin_dz_rows(s), blocks = (int)cdiv(s.M, rows);
  if (s.M > 0 && (dbias || (!none && (dX || dW)))) {
    k_lin_dz<T><<<(int)(cdiv(s.N, 256) * blocks), 256, 0, st>>>(dY, s.ldy, Z, (int)s.M, (int)s.N, s.act, rows,
                                                               none || !(dX || dW) ? nullptr : static_cast<T*>(w.dZ),
                                                               dbias ? w.db_part : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  LinGemm gx = w.gx, gw = w.gw;
  gx.A = gw.A = none ? static_cast<const void*>(dY) : w.dZ;
  gx.lda = gw.lda = none ? s.ldy : NW;
  gx.B = W;
  gw.B = X;
  gx.ldb = s.K;
  gw.ldb = s.ldx;
  const LinEpi<T> ex = lin_epi<T>(nullptr, nullptr, 0, nullptr, 0, dX, s.ldx, LIN_NONE);
  const LinEpi<T> ew = lin_epi<T>(nullptr, nullptr, 0, nullptr, 0, dW, s.K, LIN_NONE);
  const LinDb db{w.db_part, blocks, NW, dbias};
  // (the plan goes by the shape alone: a gradient asked for on its own has the pair's bits)
  if (w.pair && dX && dW) {
    gx.part = w.part;
    gw.part = w.part_w;
    if (gx.tile == LIN_SMALL) lin_pair_launch<T, LinSmall>(gx, ex, gw, ew, st);
    else lin_pair_launch<T, LinMid>(gx, ex, gw, ew, st);
    const int fx = gx.SK > 1 ? (int)cdiv((int64_t)gx.m * (gx.n / 4), 256) : 0;
    const int fw = gw.SK > 1 ? (int)cdiv((int64_t)gw.m * (gw.n / 4), 256) : 0;
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || fx + fw + (dbias ? 1 : 0) == 0) return e;
    k_lin_finish_pair<T><<<fx + fw + (dbias ? NW / LIN_DB_COLS : 0), 256, 0, st>>>(gx, ex, fx, gw, ew, fw, db);
    return hipGetLastError();
  }
  if (dbias) k_lin_db<<<NW / LIN_DB_COLS, 256, 0, st>>>(db.part, db.blocks, db.np, db.db);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && dX) e = lin_run<LIN_DX>(gx, w.part, ex, st);
  if (e == hipSuccess && dW) e = lin_run<LIN_DW>(gw, w.pair ? w.part_w : w.part, ew, st);
  return e;
}

hipError_t launch_linear_bwd(const LinShape& s, const void* dY, const void* X, const void* W, const void* Z, void* dX,
                             void* dW, float* dbias, void* ws, hipStream_t st) {
  if (s.bf16)
    return lin_backward<bf16>(s, static_cast<const bf16*>(dY), static_cast<const bf16*>(X), static_cast<const bf16*>(W),
                              static_cast<const bf16*>(Z), static_cast<bf16*>(dX), static_cast<bf16*>(dW), dbias, ws, st);
  return lin_backward<float>(s, static_cast<const float*>(dY), static_cast<const float*>(X), static_cast<const float*>(W),
                             static_cast<const float*>(Z), static_cast<float*>(dX), static_cast<float*>(dW), dbias, ws, st);
}

// dX += dL W_r, after the gather-sum has rounded dX to the element type: the sum is rounded twice,
// which its bound counts, where keeping the first part in fp32 would cost [T, d] floats of workspace
// and traffic.
template <typename T>
static hipError_t lin_logit_dx(LinGemm g, const Shape& s, void* dX, hipStream_t st) {
  return lin_run<LIN_DX>(g, nullptr, lin_epi<T>(nullptr, dX, s.d, nullptr, 0, dX, s.d, LIN_NONE), st);
}

hipError_t launch_logit_dx(const Shape& s, const void* dL, int E_pad, const void* W_r, void* dX, hipStream_t st) {
  LinGemm g{};
  g.A = dL;
  g.lda = E_pad;
  g.B = W_r;
  g.ldb = s.d;
  g.m = (int)s.T;
  g.n = (int)s.d;
  g.red = E_pad;
  g.bred = s.E;
  lin_plan(g, s.bf16, false);
  return s.bf16 ? lin_logit_dx<bf16>(g, s, dX, st) : lin_logit_dx<float>(g, s, dX, st);
}

}  // namespace moe
