// Dense projection with bias, activation and residual in its epilogue, and its backward: the
// shared expert or dense branch beside the routed experts.
//
//   forward    z = X W^T + b,  out = residual + act(z)         X [M, K], W [N', K], z [M, N']
//   backward   dZ = dY act'(z),  dX = dZ W,  dW = dZ^T X,  db = sum of dZ over rows
// N' = N, except SwiGLU: N' = 2 N, W = [W_gate; W_up], act(z) = silu(z_gate) z_up.
//
// All three products run on the layer's MFMA engine (gemm_core.h: bf16 on eight waves, 256 x 256
// tiles, the DMA ring; fp32 on the register-staged ring): X and W are K-major in the forward;
// dX reads W with its rows along the reduction, dW reads both operands so.  Reductions
// may end inside a stage (any multiple of 8).  Where the output has too few tiles for 256 CUs the
// reduction is cut into slices whose fp32 partial products a second kernel adds in slice order
// before the epilogue (k_lin_finish).
//
// The epilogue works on the fp32 accumulators: a tile half is laid out in LDS and walked in
// 16-byte chunks of a row, so that residual, saved pre-activation and output are read and written in
// whole segments and rounded once.
#include "gemm_core.h"
#include "internal.h"

namespace moe {

static inline int grid8(int64_t n) { return (int)((n + 7) / 8 * 8); }

enum { LIN_NONE = 0, LIN_RELU = 1, LIN_GELU = 2, LIN_SILU = 3, LIN_SWIGLU = 4 };

// act(z) of N elements in place (not SwiGLU).  GELU is the exact form z Phi(z).
template <int N>
__device__ __forceinline__ void lin_act(float* z, int act) {
  if (act == LIN_RELU) {
#pragma unroll
    for (int u = 0; u < N; ++u) z[u] = z[u] < 0.0f ? 0.0f : z[u];  // a NaN stays
  } else if (act == LIN_GELU) {
#pragma unroll
    for (int u = 0; u < N; ++u) z[u] = 0.5f * z[u] * (1.0f + erff(z[u] * 0.70710678118654752f));
  } else if (act == LIN_SILU) {
#pragma unroll
    for (int u = 0; u < N; ++u) z[u] *= sigmoid_f32(z[u]);
  }
}
__device__ __forceinline__ float lin_act_grad(float z, int act) {
  switch (act) {
    case LIN_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case LIN_GELU:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * __expf(-0.5f * z * z) * 0.39894228040143268f;
    case LIN_SILU: {
      const float s = sigmoid_f32(z);
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// What the epilogue does with z [m][n]; pointers may be null, res may be out.
template <typename T>
struct LinEpi {
  const float* bias;
  const T* res;
  int64_t ldr;
  T* Z;
  int64_t ldz;
  T* out;
  int64_t ldo;
  int act;
};

// One GEMM: C[m][n] = sum_k A(m, k) B(k, n) over red values of k, B valid for the first bred of
// them (the rest are zeros).  KM: rows contiguous along k; otherwise rows indexed by k.
struct LinGemm {
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  int m, n, red, bred;
  int MT, NT, SK, klen;  // tiles, slices and values of k per slice (a multiple of 32)
  float* part;           // [SK][m][n] when the output goes there
};

enum { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };            // operand layouts
enum { LIN_OUT_EPI = 0, LIN_OUT_GLU = 1, LIN_OUT_PART = 2 };  // where the tile goes

// The tile half held in LDS as fp32 rows (frow), walked in 16-byte chunks: thread owns 8 columns
// (tid % 16) and rows tid / 16 + 32 k.
constexpr int LIN_FROW = 128 * 4 + 16;
static_assert(64 * LIN_FROW <= LDS_BUF, "fp32 staging");
__device__ __forceinline__ char* lin_frow(LdsBufs L, int r) { return epi_buf(L, r) + (r & 63) * LIN_FROW; }

template <class Val>
__device__ __forceinline__ void lin_dump(LdsBufs L, int wm, int wn, Val val) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 v4 = {val(i, 4 * q), val(i, 4 * q + 1), val(i, 4 * q + 2), val(i, 4 * q + 3)};
      *reinterpret_cast<f32x4*>(lin_frow(L, acc_m(wm, i)) + (wn * 32 + acc_n(4 * q)) * 4) = v4;
    }
}
template <class Row>
__device__ __forceinline__ void lin_walk(LdsBufs L, int mrows, int valid, Row row) {
  const int c = (threadIdx.x & 15) * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = (int)(threadIdx.x >> 4) + 32 * k;
    if (r >= mrows || c >= valid) continue;
    const char* p = lin_frow(L, r) + c * 4;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
    float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    row(k, r, c, f);
  }
}

// bf16: eight waves, 256 x 256 tiles (SwiGLU: 128 output columns, gate rows over up rows in the B
// tile, so a lane holds both of a column).  Wave column wn has column block j at j 128 + 32 wn, so
// that block j of every wave is half j of the tile.
template <int MODE, bool TAIL, int OUT>
__global__ __launch_bounds__(GEMM8_THREADS, 1) void k_lin_w8(LinGemm g, LinEpi<bf16> ep) {
  MOE_GEMM_LDS(L);
  const int lin = xcd_remap(blockIdx.x, gridDim.x);
  const int per = g.MT * g.NT;
  const int sl = lin / per;
  if (sl >= g.SK) return;
  int mt, nt;
  raster_tile(lin % per, g.MT, g.NT, mt, nt);
  constexpr int TN = OUT == LIN_OUT_GLU ? 128 : BN;
  const int m0 = mt * BM, n0 = nt * TN;
  const int wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3;
  const int k0 = sl * g.klen, klen = min(g.klen, g.red - k0), blen = max(min(g.klen, g.bred - k0), 1);
  const int mrows = min(BM, g.m - m0);
  const int64_t ldab = g.lda * (int64_t)sizeof(bf16), ldbb = g.ldb * (int64_t)sizeof(bf16);
  const char* Ab = static_cast<const char*>(g.A);
  const char* Bb = static_cast<const char*>(g.B);
  auto bsub = [&](int j) { return j * 128 + wn * 32; };
  AccW8 acc;
  const int nkt = (int)cdiv(klen, Mma<bf16>::BK);
  typedef typename std::conditional<TAIL, KDmaW8Tail, KDmaW8>::type KD;
  auto krows = [&](auto row_ptr) {
    KD l;
    if constexpr (TAIL) l.init(row_ptr, klen);
    else l.init(row_ptr);
    return l;
  };
  auto arow = [&](int i) -> const char* { return i < mrows ? Ab + (m0 + i) * ldab + (int64_t)k0 * 2 : nullptr; };
  if constexpr (MODE == LIN_FWD) {
    auto la = krows(arow);
    auto lb = krows([&](int i) -> const char* {
      int r = n0 + i;
      if (OUT == LIN_OUT_GLU) {
        if (n0 + (i & 127) >= g.n) return nullptr;
        r = n0 + (i & 127) + (i < 128 ? 0 : g.n);
      } else if (r >= g.n) {
        return nullptr;
      }
      return Bb + r * ldbb + (int64_t)k0 * 2;
    });
    gemm_mainloop_w8_rows(la, lb, nkt, acc, L, wm, bsub, mrows);
  } else if constexpr (MODE == LIN_DX) {
    auto la = krows(arow);
    const char* bk = Bb + k0 * ldbb + (int64_t)n0 * 2;
    auto lb = mn_rows_w8([=](int k) { return bk + k * ldbb; }, blen, n0, g.n);
    gemm_mainloop_w8_rows(la, lb, nkt, acc, L, wm, bsub, mrows);
  } else {
    const char* ak = Ab + k0 * ldab + (int64_t)m0 * 2;
    const char* bk = Bb + k0 * ldbb + (int64_t)n0 * 2;
    auto la = mn_rows_w8([=](int k) { return ak + k * ldab; }, klen, m0, g.m);
    auto lb = mn_rows_w8([=](int k) { return bk + k * ldbb; }, blen, n0, g.n);
    gemm_mainloop_w8_rows(la, lb, nkt, acc, L, wm, bsub, mrows);
  }
  if constexpr (OUT == LIN_OUT_PART) {
    float* dst = g.part + (int64_t)sl * g.m * g.n;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = n0 + bsub(j) + acc_n(4 * q);  // n is a multiple of 4
        if (c >= g.n) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = acc_m(wm, i);
          if (r >= mrows) continue;
          *reinterpret_cast<f32x4*>(dst + (int64_t)(m0 + r) * g.n + c) =
              f32x4{acc.c[i][j][4 * q], acc.c[i][j][4 * q + 1], acc.c[i][j][4 * q + 2], acc.c[i][j][4 * q + 3]};
        }
      }
  } else if constexpr (OUT == LIN_OUT_EPI) {
    const int cw = (threadIdx.x & 15) * 8;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int c0 = n0 + half * 128, valid = min(128, g.n - c0);
      if (valid <= 0) break;  // (uniform)
      u32x4 rv[8];
      float b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (cw < valid) {
        if (ep.bias) {
#pragma unroll
          for (int u = 0; u < 8; ++u) b[u] = ep.bias[c0 + cw + u];
        }
        if (ep.res) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = min((int)(threadIdx.x >> 4) + 32 * k, mrows - 1);
            rv[k] = ld16_nt(ep.res + (m0 + r) * ep.ldr + c0 + cw);
          }
        }
      }
      lin_dump(L, wm, wn, [&](int i, int v) { return acc.c[i][half][v]; });
      __syncthreads();
      lin_walk(L, mrows, valid, [&](int k, int r, int c, float (&f)[8]) {
#pragma unroll
        for (int u = 0; u < 8; ++u) f[u] += b[u];
        if (ep.Z) st16_nt(ep.Z + (m0 + r) * ep.ldz + c0 + c, pack16<bf16>(f));
        lin_act<8>(f, ep.act);
        if (ep.res) {
          float rr[8];
          unpack16<bf16>(rv[k], rr);
#pragma unroll
          for (int u = 0; u < 8; ++u) f[u] += rr[u];
        }
        st16_nt(ep.out + (m0 + r) * ep.ldo + c0 + c, pack16<bf16>(f));
      });
      __syncthreads();
    }
  } else {  // SwiGLU: block 0 is the gate, block 1 the up projection of the same columns
    const int valid = min(128, g.n - n0);
    if (ep.bias) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = n0 + wn * 32 + acc_n(4 * q);
          f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
          if (c < g.n) b = *reinterpret_cast<const f32x4*>(ep.bias + (int64_t)j * g.n + c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc.c[i][j][4 * q + u] += b[u];
        }
    }
    if (ep.Z) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lin_dump(L, wm, wn, [&](int i, int v) { return acc.c[i][j][v]; });
        __syncthreads();
        lin_walk(L, mrows, valid, [&](int, int r, int c, float (&f)[8]) {
          st16_nt(ep.Z + (m0 + r) * ep.ldz + (int64_t)j * g.n + n0 + c, pack16<bf16>(f));
        });
        __syncthreads();
      }
    }
    lin_dump(L, wm, wn, [&](int i, int v) {
      const float gv = acc.c[i][0][v];
      return gv * sigmoid_f32(gv) * acc.c[i][1][v];
    });
    __syncthreads();
    lin_walk(L, mrows, valid, [&](int, int r, int c, float (&f)[8]) {
      if (ep.res) {
        float rr[8];
        unpack16<bf16>(ld16_nt(ep.res + (m0 + r) * ep.ldr + n0 + c), rr);
#pragma unroll
        for (int u = 0; u < 8; ++u) f[u] += rr[u];
      }
      st16_nt(ep.out + (m0 + r) * ep.ldo + n0 + c, pack16<bf16>(f));
    });
  }
}

// fp32: four waves, 256 x 256 tiles, the register-staged ring; a lane's accumulators 4 q .. 4 q + 3
// are four consecutive columns, one 16-byte access each.
template <int MODE, int OUT>
__global__ __launch_bounds__(GEMM_THREADS, 1) void k_lin_f32(LinGemm g, LinEpi<float> ep) {
  MOE_GEMM_LDS(L);
  const int lin = xcd_remap(blockIdx.x, gridDim.x);
  const int per = g.MT * g.NT;
  const int sl = lin / per;
  if (sl >= g.SK) return;
  int mt, nt;
  raster_tile(lin % per, g.MT, g.NT, mt, nt);
  const int m0 = mt * BM, n0 = nt * BN;
  const int wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int k0 = sl * g.klen, klen = min(g.klen, g.red - k0), blen = min(g.klen, g.bred - k0);
  const int mrows = min(BM, g.m - m0);
  const int64_t ldab = g.lda * 4, ldbb = g.ldb * 4;
  const char* Ab = static_cast<const char*>(g.A);
  const char* Bb = static_cast<const char*>(g.B);
  auto bsub = [&](int j) { return bsub_plain(wn, j); };
  WaveAcc acc;
  const int nkt = (int)cdiv(klen, Mma<float>::BK);
  auto arow = [&](int i) -> const char* { return i < mrows ? Ab + (m0 + i) * ldab + (int64_t)k0 * 4 : nullptr; };
  if constexpr (MODE == LIN_FWD) {
    RowLoaderF32Tail la, lb;
    la.init(arow, klen);
    lb.init([&](int i) -> const char* { return n0 + i < g.n ? Bb + (n0 + i) * ldbb + (int64_t)k0 * 4 : nullptr; }, klen);
    gemm_mainloop_reg(la, lb, nkt, acc, L, wm, bsub);
  } else if constexpr (MODE == LIN_DX) {
    RowLoaderF32Tail la;
    la.init(arow, klen);
    const char* bk = Bb + k0 * ldbb + (int64_t)n0 * 4;
    auto lb = mn_rows<float>([=](int k) { return bk + k * ldbb; }, blen, n0, g.n);
    gemm_mainloop_reg(la, lb, nkt, acc, L, wm, bsub);
  } else {
    const char* ak = Ab + k0 * ldab + (int64_t)m0 * 4;
    const char* bk = Bb + k0 * ldbb + (int64_t)n0 * 4;
    auto la = mn_rows<float>([=](int k) { return ak + k * ldab; }, klen, m0, g.m);
    auto lb = mn_rows<float>([=](int k) { return bk + k * ldbb; }, blen, n0, g.n);
    gemm_mainloop_reg(la, lb, nkt, acc, L, wm, bsub);
  }
  float* dst = OUT == LIN_OUT_PART ? g.part + (int64_t)sl * g.m * g.n : nullptr;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = n0 + bsub(j) + acc_n(4 * q);  // n is a multiple of 4
      if (c >= g.n) continue;
      f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
      if (OUT == LIN_OUT_EPI && ep.bias) b = *reinterpret_cast<const f32x4*>(ep.bias + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = acc_m(wm, i);
        if (r >= mrows) continue;
        f32x4 v = {acc.c[i][j][4 * q], acc.c[i][j][4 * q + 1], acc.c[i][j][4 * q + 2], acc.c[i][j][4 * q + 3]};
        if (OUT == LIN_OUT_PART) {
          *reinterpret_cast<f32x4*>(dst + (int64_t)(m0 + r) * g.n + c) = v;
          continue;
        }
        v += b;
        if (ep.Z) *reinterpret_cast<f32x4*>(ep.Z + (m0 + r) * ep.ldz + c) = v;
        float f[4] = {v[0], v[1], v[2], v[3]};
        lin_act<4>(f, ep.act);
        v = f32x4{f[0], f[1], f[2], f[3]};
        if (ep.res) v += *reinterpret_cast<const f32x4*>(ep.res + (m0 + r) * ep.ldr + c);
        *reinterpret_cast<f32x4*>(ep.out + (m0 + r) * ep.ldo + c) = v;
      }
    }
}

// Adds the SK slices in slice order and applies the epilogue; a thread takes 8 consecutive output
// columns.  n: output columns; np: columns of the partial products (2 n for SwiGLU).
template <typename T>
__global__ __launch_bounds__(256) void k_lin_finish(const float* __restrict__ part, int SK, int m, int n, int np,
                                                    LinEpi<T> ep) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int cpr = n / 8;
  if (i >= (int64_t)m * cpr) return;
  const int r = (int)(i / cpr), c = (int)(i - (int64_t)r * cpr) * 8;
  auto sum8 = [&](int col, float (&f)[8]) {
    f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
    const float* p = part + (int64_t)r * np + col;
    for (int s = 0; s < SK; ++s, p += (int64_t)m * np) {
      a += __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
      b += __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[u] = a[u];
      f[4 + u] = b[u];
    }
    if (ep.bias)
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] += ep.bias[col + u];
    if (ep.Z) {
      T* z = ep.Z + r * ep.ldz + col;
#pragma unroll
      for (int u = 0; u < 8; u += 16 / (int)sizeof(T)) st16_nt(z + u, pack16<T>(f + u));
    }
  };
  float f[8];
  sum8(c, f);
  if (np != n) {
    float up[8];
    sum8(n + c, up);
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] = f[u] * sigmoid_f32(f[u]) * up[u];
  } else {
    lin_act<8>(f, ep.act);
  }
  T* o = ep.out + r * ep.ldo + c;
#pragma unroll
  for (int u = 0; u < 8; u += 16 / (int)sizeof(T)) {
    if (ep.res) {
      float rr[16 / sizeof(T)];
      unpack16<T>(ld16(ep.res + r * ep.ldr + c + u), rr);
#pragma unroll
      for (int k = 0; k < 16 / (int)sizeof(T); ++k) f[u + k] += rr[k];
    }
    st16_nt(o + u, pack16<T>(f + u));
  }
}

// dZ = dY act'(z) (SwiGLU: [dG | dU]) and the bias gradient's partial sums: a workgroup takes 256
// columns (32 lanes of 8) and LIN_DZ_ROWS rows (8 at a time); db_part[row block][column].  dZ may
// be null (only the sums), db_part too.
constexpr int LIN_DZ_ROWS = 64;
template <typename T>
__global__ __launch_bounds__(256) void k_lin_dz(const T* __restrict__ dY, int64_t ldy, const T* __restrict__ Z, int m,
                                                int n, int act, T* __restrict__ dZ, float* __restrict__ db_part) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ float red[8][256 + 4];
  const int glu = act == LIN_SWIGLU, np = glu ? 2 * n : n;
  const int cl = (threadIdx.x & 31) * 8, rl = threadIdx.x >> 5;
  const int cbs = (n + 255) / 256, cb = blockIdx.x % cbs, rb = blockIdx.x / cbs;
  const int c = cb * 256 + cl;
  const int r0 = rb * LIN_DZ_ROWS, r1 = min(m, r0 + LIN_DZ_ROWS);
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
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (act != LIN_NONE) dy[u] *= lin_act_grad(z[u], act);
          s0[u] += dy[u];
        }
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

// db = the row blocks' sums in order (fp64): 64 columns by 4 runs of row blocks per workgroup.
__global__ __launch_bounds__(256) void k_lin_db(const float* __restrict__ db_part, int blocks, int np,
                                                float* __restrict__ db) {
  __shared__ double red[4][64];
  const int cl = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + cl;
  double v = 0.0;
  if (c < np)
    for (int b = run; b < blocks; b += 4) v += (double)db_part[(int64_t)b * np + c];
  red[run][cl] = v;
  __syncthreads();
  if (run == 0 && c < np) db[c] = (float)((red[0][cl] + red[1][cl]) + (red[2][cl] + red[3][cl]));
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
// Slices of a product's reduction: one where the tiles fill half the chip, else as many as fill
// it, each of at least four stages.
static void lin_plan(LinGemm& g, int tn, bool may_split) {
  g.MT = (int)cdiv(g.m, BM);
  g.NT = (int)cdiv(g.n, tn);
  const int64_t tiles = g.m ? (int64_t)g.MT * g.NT : 1;
  const int stages = (int)cdiv(g.red, 32);
  int sk = 1;
  if (may_split && tiles < 128) {
    sk = (int)(256 / tiles);
    if (sk > stages / 4) sk = stages / 4;
    if (sk > 64) sk = 64;
    if (sk < 1) sk = 1;
  }
  g.klen = (int)cdiv(stages, sk) * 32;
  g.SK = g.red > 0 ? (int)cdiv(g.red, g.klen) : 1;
}

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
  lin_plan(g, BN, true);
  return g;
}

// Whether the forward's SwiGLU goes through partial products: where they are split anyway, and in
// fp32, whose four-wave kernel keeps gate and up in different lanes.
static bool lin_fwd_part(const LinShape& s, const LinGemm& g) { return g.SK > 1 || (s.act == LIN_SWIGLU && !s.bf16); }

static size_t lin_part_bytes(const LinGemm& g) { return (size_t)g.SK * g.m * g.n * sizeof(float); }

size_t linear_fwd_workspace_bytes(const LinShape& s) {
  if (s.M == 0) return 0;
  const LinGemm g = lin_gemm(s, LIN_FWD);
  return lin_fwd_part(s, g) ? lin_part_bytes(g) : 0;
}

struct LinBwdWs {
  void* dZ;
  float* db_part;
  float* part;
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
  q.db_part = reinterpret_cast<float*>(take((size_t)cdiv(s.M, LIN_DZ_ROWS) * NW * 4));
  const LinGemm gx = lin_gemm(s, LIN_DX), gw = lin_gemm(s, LIN_DW);
  const size_t px = gx.SK > 1 ? lin_part_bytes(gx) : 0, pw = gw.SK > 1 ? lin_part_bytes(gw) : 0;
  q.part = reinterpret_cast<float*>(take(px > pw ? px : pw));
  if (w) *w = q;
  return off;
}

size_t linear_bwd_workspace_bytes(const LinShape& s) { return lin_carve_bwd(s, nullptr, nullptr); }

template <int MODE, int OUT>
static void lin_launch(const LinShape& s, const LinGemm& g, const LinEpi<bf16>& eb, const LinEpi<float>& ef,
                       hipStream_t st) {
  const int grid = grid8((int64_t)g.MT * g.NT * g.SK);
  if (s.bf16) {
    if (MODE != LIN_DW && g.red % 32) k_lin_w8<MODE, MODE != LIN_DW, OUT><<<grid, GEMM8_THREADS, 0, st>>>(g, eb);
    else k_lin_w8<MODE, false, OUT><<<grid, GEMM8_THREADS, 0, st>>>(g, eb);
  } else {
    if constexpr (OUT != LIN_OUT_GLU) k_lin_f32<MODE, OUT><<<grid, GEMM_THREADS, 0, st>>>(g, ef);
  }
}

// A product whose epilogue is ep: directly, or through partial products.
template <int MODE>
static hipError_t lin_run(const LinShape& s, LinGemm g, float* part, const LinEpi<bf16>& eb, const LinEpi<float>& ef,
                          bool through_part, hipStream_t st) {
  if (g.m == 0) return hipSuccess;
  if (!through_part) {
    if constexpr (MODE == LIN_FWD) {
      if (eb.act == LIN_SWIGLU) {
        g.n = (int)s.N;
        g.NT = (int)cdiv(g.n, 128);
        lin_launch<MODE, LIN_OUT_GLU>(s, g, eb, ef, st);
        return hipGetLastError();
      }
    }
    lin_launch<MODE, LIN_OUT_EPI>(s, g, eb, ef, st);
    return hipGetLastError();
  }
  g.part = part;
  lin_launch<MODE, LIN_OUT_PART>(s, g, eb, ef, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int n = eb.act == LIN_SWIGLU ? g.n / 2 : g.n;
  const int grid = (int)cdiv((int64_t)g.m * (n / 8), 256);
  if (s.bf16) k_lin_finish<bf16><<<grid, 256, 0, st>>>(part, g.SK, g.m, n, g.n, eb);
  else k_lin_finish<float><<<grid, 256, 0, st>>>(part, g.SK, g.m, n, g.n, ef);
  return hipGetLastError();
}

template <typename T>
static LinEpi<T> lin_epi(const float* bias, const void* res, int64_t ldr, void* Z, int64_t ldz, void* out, int64_t ldo,
                         int act) {
  return LinEpi<T>{bias, static_cast<const T*>(res), ldr, static_cast<T*>(Z), ldz, static_cast<T*>(out), ldo, act};
}

hipError_t launch_linear(const LinShape& s, const void* X, const void* W, const float* bias, const void* residual,
                         void* Z, void* out, void* ws, hipStream_t st) {
  if (s.M == 0) return hipSuccess;
  LinGemm g = lin_gemm(s, LIN_FWD);
  g.A = X;
  g.lda = s.ldx;
  g.B = W;
  g.ldb = s.K;
  return lin_run<LIN_FWD>(s, g, static_cast<float*>(ws), lin_epi<bf16>(bias, residual, s.ldr, Z, g.n, out, s.ldy, s.act),
                          lin_epi<float>(bias, residual, s.ldr, Z, g.n, out, s.ldy, s.act), lin_fwd_part(s, g), st);
}

hipError_t launch_linear_dz(const LinShape& s, const void* dY, const void* Z, float* dbias, void* ws, hipStream_t st) {
  LinBwdWs w;
  lin_carve_bwd(s, ws, &w);
  const int NW = (int)(s.act == LIN_SWIGLU ? 2 * s.N : s.N);
  const int blocks = (int)cdiv(s.M, LIN_DZ_ROWS);
  if (s.M > 0 && (dbias || s.act != LIN_NONE)) {
    const int grid = (int)(cdiv(s.N, 256) * blocks);
    void* dZ = s.act == LIN_NONE ? nullptr : w.dZ;
    float* db = dbias ? w.db_part : nullptr;
    if (s.bf16)
      k_lin_dz<bf16><<<grid, 256, 0, st>>>((const bf16*)dY, s.ldy, (const bf16*)Z, (int)s.M, (int)s.N, s.act, (bf16*)dZ, db);
    else
      k_lin_dz<float><<<grid, 256, 0, st>>>((const float*)dY, s.ldy, (const float*)Z, (int)s.M, (int)s.N, s.act, (float*)dZ, db);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dbias) k_lin_db<<<(int)cdiv(NW, 64), 256, 0, st>>>(w.db_part, blocks, NW, dbias);
  return hipGetLastError();
}

hipError_t launch_linear_dx(const LinShape& s, const void* dY, const void* W, void* dX, void* ws, hipStream_t st) {
  LinBwdWs w;
  lin_carve_bwd(s, ws, &w);
  LinGemm g = lin_gemm(s, LIN_DX);
  g.A = s.act == LIN_NONE ? dY : w.dZ;
  g.lda = s.act == LIN_NONE ? s.ldy : g.red;
  g.B = W;
  g.ldb = s.K;
  return lin_run<LIN_DX>(s, g, w.part, lin_epi<bf16>(nullptr, nullptr, 0, nullptr, 0, dX, s.ldx, LIN_NONE),
                         lin_epi<float>(nullptr, nullptr, 0, nullptr, 0, dX, s.ldx, LIN_NONE), g.SK > 1, st);
}

hipError_t launch_linear_dw(const LinShape& s, const void* dY, const void* X, void* dW, void* ws, hipStream_t st) {
  LinBwdWs w;
  lin_carve_bwd(s, ws, &w);
  LinGemm g = lin_gemm(s, LIN_DW);
  g.A = s.act == LIN_NONE ? dY : w.dZ;
  g.lda = s.act == LIN_NONE ? s.ldy : g.m;
  g.B = X;
  g.ldb = s.ldx;
  return lin_run<LIN_DW>(s, g, w.part, lin_epi<bf16>(nullptr, nullptr, 0, nullptr, 0, dW, s.K, LIN_NONE),
                         lin_epi<float>(nullptr, nullptr, 0, nullptr, 0, dW, s.K, LIN_NONE), g.SK > 1, st);
}

hipError_t launch_logit_dx(const Shape& s, const void* dL, int E_pad, const void* W_r, void* dX, hipStream_t st) {
  LinShape ls{};
  ls.bf16 = s.bf16;
  LinGemm g{};
  g.A = dL;
  g.lda = E_pad;
  g.B = W_r;
  g.ldb = s.d;
  g.m = (int)s.T;
  g.n = (int)s.d;
  g.red = E_pad;
  g.bred = s.E;
  lin_plan(g, BN, false);
  return lin_run<LIN_DX>(ls, g, nullptr, lin_epi<bf16>(nullptr, dX, s.d, nullptr, 0, dX, s.d, LIN_NONE),
                         lin_epi<float>(nullptr, dX, s.d, nullptr, 0, dX, s.d, LIN_NONE), false, st);
}

}  // namespace moe
