// Layer norm and RMS norm of rows, with the sum of a residual stream in front, and their backward.
//
//   s = x + r (rounded to the type),  mu = mean(s) (RMS: 0),  rstd = 1 / sqrt(mean((s - mu)^2) + eps)
//   y = (s - mu) rstd w + b
// and with xh = (s - mu) rstd, g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dsum  (RMS: without mean(g)),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// A row is held whole in the registers of `tpr` threads (a power of two, 8 .. 1024), NC chunks of 8
// elements each, so it is read once; the variance is the mean of squared differences from the mean, not a
// difference of large sums.  All sums are fp32.
#include "internal.h"

namespace moe {

// Element i of a thread's chunk j lies in column norm_col(j, i): 8 neighbours per chunk where rows are
// 16-byte aligned, else neighbours in neighbouring threads, which keeps 2- and 4-byte accesses coalesced.
template <bool ALIGNED>
__device__ __forceinline__ int norm_col(int j, int i, int tpr, int t) {
  return ALIGNED ? (j * tpr + t) * 8 + i : (j * 8 + i) * tpr + t;
}

// 8 elements as they lie in memory.
template <typename T> struct Raw8 { u32x4 v[8 / Vec<T>::N]; };

template <typename T, int NC, bool ALIGNED>
__device__ __forceinline__ void norm_load(const T* p, int cols, int tpr, int t, Raw8<T> (&r)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = norm_col<ALIGNED>(j, 0, tpr, t);
    if (ALIGNED && c + 8 <= cols) {
#pragma unroll
      for (int v = 0; v < 8 / Vec<T>::N; ++v) r[j].v[v] = ld16_nt(p + c + v * Vec<T>::N);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ci = norm_col<ALIGNED>(j, i, tpr, t);
        f[i] = ci < cols ? to_f32(p[ci]) : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < 8 / Vec<T>::N; ++v) r[j].v[v] = pack16<T>(f + v * Vec<T>::N);
    }
  }
}
template <typename T>
__device__ __forceinline__ void norm_unpack(const Raw8<T>& r, float* f) {
#pragma unroll
  for (int v = 0; v < 8 / Vec<T>::N; ++v) unpack16<T>(r.v[v], f + v * Vec<T>::N);
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ void norm_store(T* p, int cols, int tpr, int t, int j, const Raw8<T>& r) {
  const int c = norm_col<ALIGNED>(j, 0, tpr, t);
  if (ALIGNED && c + 8 <= cols) {
#pragma unroll
    for (int v = 0; v < 8 / Vec<T>::N; ++v) st16_nt(p + c + v * Vec<T>::N, r.v[v]);
  } else {
    float f[8];
    norm_unpack<T>(r, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ci = norm_col<ALIGNED>(j, i, tpr, t);
      if (ci < cols) p[ci] = from_f32<T>(f[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> norm_pack(const float* f) {
  Raw8<T> r;
#pragma unroll
  for (int v = 0; v < 8 / Vec<T>::N; ++v) r.v[v] = pack16<T>(f + v * Vec<T>::N);
  return r;
}

// Weight or bias of a thread's columns (null: the value `none`).
template <int NC, bool ALIGNED>
__device__ __forceinline__ void norm_vector(const void* p, bool wbf16, float none, int cols, int tpr, int t, float (&w)[NC * 8]) {
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = norm_col<ALIGNED>(j, i, tpr, t);
      float v = none;
      if (p && c < cols) v = wbf16 ? to_f32(static_cast<const bf16*>(p)[c]) : static_cast<const float*>(p)[c];
      w[j * 8 + i] = v;
    }
}

// Sums of a row's values over its threads, in every one of them: shuffles inside a wave, then (tpr > 64:
// the row's threads are the workgroup) the waves' sums through LDS in wave order.  The two halves of `red`
// alternate, so that a reduction writes what no wave still reads: between its write and the last read of
// the same half lies the other half's barrier.
template <int N>
__device__ __forceinline__ void norm_row_sum(float (&v)[N], int tpr, float (*red)[N][16], int& half) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    if (o < tpr) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o, WAVE);
    }
  if (tpr <= WAVE) return;
  const int waves = tpr >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[half][k][threadIdx.x >> 6] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = red[half][k][0];
    for (int q = 1; q < waves; ++q) s += red[half][k][q];
    v[k] = s;
  }
  half ^= 1;
}

struct NormFwd {
  const void *x, *res, *w, *b;
  void *sum, *y;
  float *mean, *rstd;
  int64_t rows, ldx, ldr, lds, ldy;
  int cols, tpr;
  float eps;
  bool wbf16, rms;
};

template <typename T, int NC, bool ALIGNED, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm(NormFwd a) {
  __shared__ float red[2][1][16];
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1), rpb = blockDim.x / tpr, cols = a.cols;
  const float inv = 1.0f / (float)cols;
  int half = 0;
  float w[NC * 8], b[NC * 8];
  norm_vector<NC, ALIGNED>(a.w, a.wbf16, 1.0f, cols, tpr, t, w);
  norm_vector<NC, ALIGNED>(a.b, a.wbf16, 0.0f, cols, tpr, t, b);
  // (with tpr > 64 a row is the workgroup's, so the barriers inside are reached by all of it; with several
  // rows a workgroup there are none)
  for (int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr; row < a.rows; row += (int64_t)gridDim.x * rpb) {
    Raw8<T> raw[NC];
    norm_load<T, NC, ALIGNED>(static_cast<const T*>(a.x) + row * a.ldx, cols, tpr, t, raw);
    float f[NC * 8];
    if (a.res) {
      Raw8<T> rr[NC];
      norm_load<T, NC, ALIGNED>(static_cast<const T*>(a.res) + row * a.ldr, cols, tpr, t, rr);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float u[8], v[8];
        norm_unpack<T>(raw[j], u);
        norm_unpack<T>(rr[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += v[i];
        raw[j] = norm_pack<T>(u);  // what is normalised is the rounded sum, which the backward reads
        if (a.sum) norm_store<T, ALIGNED>(static_cast<T*>(a.sum) + row * a.lds, cols, tpr, t, j, raw[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) norm_unpack<T>(raw[j], f + j * 8);
    float mu = 0.0f;
    if (!a.rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) s[0] += f[i];  // (columns past the row hold zeros)
      norm_row_sum<1>(s, tpr, red, half);
      mu = s[0] * inv;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = norm_col<ALIGNED>(j, i, tpr, t) < cols ? f[j * 8 + i] - mu : 0.0f;
        f[j * 8 + i] = d;
        q[0] = fmaf(d, d, q[0]);
      }
    norm_row_sum<1>(q, tpr, red, half);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv, a.eps));
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j * 8 + i] = fmaf(f[j * 8 + i] * rstd, w[j * 8 + i], b[j * 8 + i]);
      norm_store<T, ALIGNED>(y, cols, tpr, t, j, norm_pack<T>(f + j * 8));
    }
  }
}

struct NormBwd {
  const void *dy, *s, *w, *dsum;
  const float *mean, *rstd;
  void* dx;       // may be null
  float* part;    // [workgroups][dw, db][cols], or null
  int64_t rows, ldy, lds, ldr, ldx;
  int cols, tpr;
  bool wbf16, rms;
};

// Every thread keeps its columns' parts of dw and db over the rows it takes; a workgroup adds those of
// its row groups in LDS and writes one partial row, which k_norm_wgrad adds up in a fixed order.
template <typename T, int NC, bool ALIGNED, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm_bwd(NormBwd a) {
  __shared__ float red[2][2][16];
  __shared__ float add[THREADS <= 256 ? 256 * 8 : 1];
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1), rpb = blockDim.x / tpr, cols = a.cols;
  const float inv = 1.0f / (float)cols;
  int half = 0;
  float w[NC * 8], dw[NC * 8], db[NC * 8];
  norm_vector<NC, ALIGNED>(a.w, a.wbf16, 1.0f, cols, tpr, t, w);
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr; row < a.rows; row += (int64_t)gridDim.x * rpb) {
    Raw8<T> rdy[NC], rs[NC], rd[NC];
    norm_load<T, NC, ALIGNED>(static_cast<const T*>(a.dy) + row * a.ldy, cols, tpr, t, rdy);
    norm_load<T, NC, ALIGNED>(static_cast<const T*>(a.s) + row * a.lds, cols, tpr, t, rs);
    const bool has_dsum = a.dsum && a.dx;
    if (has_dsum) norm_load<T, NC, ALIGNED>(static_cast<const T*>(a.dsum) + row * a.ldr, cols, tpr, t, rd);
    const float mu = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float g[8], x[8];
      norm_unpack<T>(rdy[j], g);
      norm_unpack<T>(rs[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = j * 8 + i;
        const float xh = norm_col<ALIGNED>(j, i, tpr, t) < cols ? (x[i] - mu) * rstd : 0.0f;
        dw[k] = fmaf(g[i], xh, dw[k]);
        db[k] += g[i];
        const float gw = g[i] * w[k];
        v[0] += gw;
        v[1] = fmaf(gw, xh, v[1]);
      }
    }
    if (!a.dx) continue;  // (uniform)
    norm_row_sum<2>(v, tpr, red, half);
    const float m1 = a.rms ? 0.0f : v[0] * inv, m2 = v[1] * inv;
    T* dx = static_cast<T*>(a.dx) + row * a.ldx;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float g[8], x[8], d[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      norm_unpack<T>(rdy[j], g);
      norm_unpack<T>(rs[j], x);
      if (has_dsum) norm_unpack<T>(rd[j], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (x[i] - mu) * rstd;
        d[i] = fmaf(rstd, fmaf(-xh, m2, fmaf(g[i], w[j * 8 + i], -m1)), d[i]);
      }
      norm_store<T, ALIGNED>(dx, cols, tpr, t, j, norm_pack<T>(d));
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k ? db[j * 8 + i] : dw[j * 8 + i];
      if (THREADS <= 256 && rpb > 1) {  // add the workgroup's row groups, in their order
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) add[i * 256 + threadIdx.x] = v[i];
        __syncthreads();
        if ((int)threadIdx.x < tpr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] = add[i * 256 + t];
            for (int q = 1; q < rpb; ++q) v[i] += add[i * 256 + q * tpr + t];
          }
        }
      }
      if ((int)threadIdx.x < tpr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = norm_col<ALIGNED>(j, i, tpr, t);
          if (c < cols) part[k * cols + c] = v[i];
        }
      }
    }
}

// dw and db: the workgroups' partial rows added in fp64, 8 runs of them per column, then the runs.
constexpr int NORM_WG_COLS = 32, NORM_WG_RUNS = 8;
__global__ __launch_bounds__(256) void k_norm_wgrad(const float* __restrict__ part, int parts, int cols, float* dw, float* db) {
  __shared__ double red[NORM_WG_RUNS][NORM_WG_COLS + 1];
  const int cl = threadIdx.x % NORM_WG_COLS, run = threadIdx.x / NORM_WG_COLS;
  const int c = blockIdx.x * NORM_WG_COLS + cl;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;  // (uniform)
  double v = 0.0;
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * cols + c;
#pragma unroll 8
    for (int q = run; q < parts; q += NORM_WG_RUNS) v += (double)p[(int64_t)q * 2 * cols];
  }
  red[run][cl] = v;
  __syncthreads();
  if (run == 0 && c < cols) {
#pragma unroll
    for (int q = 1; q < NORM_WG_RUNS; ++q) v += red[q][cl];
    out[c] = (float)v;
  }
}

// Threads per row: NC = ceil(cols / (8 tpr)) chunks each.
static int norm_tpr(int64_t cols, int64_t rows) {
  const int64_t chunks = cdiv(cols, 8);
  int tpr = 8;
  const int most = rows >= 1024 ? 4 : 1;  // few rows: as many threads as there are chunks
  while (tpr < 1024 && cdiv(chunks, tpr) > (tpr < 64 ? 1 : most)) tpr *= 2;
  return tpr;
}
static int norm_threads(int tpr) { return tpr > 256 ? tpr : tpr > 64 ? tpr : 256; }
static int norm_grid(int64_t rows, int tpr, int most) {
  const int64_t need = cdiv(rows, norm_threads(tpr) / tpr);
  return (int)(need < most ? need : most);
}
constexpr int NORM_FWD_GRID = 2048, NORM_BWD_GRID = 1024;  // workgroups

template <typename T, int NC, bool ALIGNED>
static void norm_go(const NormFwd& a, int grid, int threads, hipStream_t st) {
  if constexpr (NC <= 4)  // (more chunks only with 1024 threads a row)
    if (threads <= 256) return k_norm<T, NC, ALIGNED, 256><<<grid, threads, 0, st>>>(a);
  k_norm<T, NC, ALIGNED, 1024><<<grid, threads, 0, st>>>(a);
}
template <typename T, int NC, bool ALIGNED>
static void norm_go(const NormBwd& a, int grid, int threads, hipStream_t st) {
  if constexpr (NC <= 4)
    if (threads <= 256) return k_norm_bwd<T, NC, ALIGNED, 256><<<grid, threads, 0, st>>>(a);
  k_norm_bwd<T, NC, ALIGNED, 1024><<<grid, threads, 0, st>>>(a);
}
template <typename T, bool ALIGNED, class Args>
static void norm_chunks(const Args& a, int grid, int threads, hipStream_t st) {
  const int nc = (int)cdiv(a.cols, 8 * a.tpr);
  if (nc <= 1) norm_go<T, 1, ALIGNED>(a, grid, threads, st);
  else if (nc <= 2) norm_go<T, 2, ALIGNED>(a, grid, threads, st);
  else if (nc <= 3) norm_go<T, 3, ALIGNED>(a, grid, threads, st);
  else if (nc <= 4) norm_go<T, 4, ALIGNED>(a, grid, threads, st);
  else norm_go<T, 8, ALIGNED>(a, grid, threads, st);
}
template <class Args>
static hipError_t norm_launch(const Args& a, bool is_bf16, bool aligned, int grid, hipStream_t st) {
  const int threads = norm_threads(a.tpr);
  if (is_bf16) {
    if (aligned) norm_chunks<bf16, true>(a, grid, threads, st);
    else norm_chunks<bf16, false>(a, grid, threads, st);
  } else {
    if (aligned) norm_chunks<float, true>(a, grid, threads, st);
    else norm_chunks<float, false>(a, grid, threads, st);
  }
  return hipGetLastError();
}

hipError_t launch_norm(const NormShape& s, const void* x, const void* residual, const void* weight, const void* bias,
                       void* sum, void* y, float* mean, float* rstd, hipStream_t st) {
  if (s.rows == 0) return hipSuccess;
  NormFwd a;
  a.x = x; a.res = residual; a.w = weight; a.b = bias;
  a.sum = sum; a.y = y; a.mean = s.rms ? nullptr : mean; a.rstd = rstd;
  a.rows = s.rows; a.ldx = s.ldx; a.ldr = s.ldr; a.lds = s.lds; a.ldy = s.ldy;
  a.cols = (int)s.cols;
  a.tpr = norm_tpr(s.cols, s.rows);
  a.eps = s.eps; a.wbf16 = s.wbf16; a.rms = s.rms;
  const int64_t vec = s.bf16 ? 8 : 4;
  const bool aligned = s.ldx % vec == 0 && s.ldy % vec == 0 && (!residual || s.ldr % vec == 0) && (!sum || s.lds % vec == 0);
  return norm_launch(a, s.bf16, aligned, norm_grid(s.rows, a.tpr, NORM_FWD_GRID), st);
}

size_t norm_bwd_workspace_bytes(const NormShape& s) {
  const int tpr = norm_tpr(s.cols, s.rows);
  return (size_t)norm_grid(s.rows, tpr, NORM_BWD_GRID) * 2 * s.cols * sizeof(float);
}

hipError_t launch_norm_bwd(const NormShape& s, const void* dy, const void* sum, const void* weight, const float* mean,
                           const float* rstd, const void* dsum, void* dx, float* dweight, float* dbias, void* ws,
                           hipStream_t st) {
  const int tpr = norm_tpr(s.cols, s.rows), grid = norm_grid(s.rows, tpr, NORM_BWD_GRID);
  const bool vectors = dweight || dbias;
  float* part = static_cast<float*>(ws);
  if (s.rows > 0) {
    NormBwd a;
    a.dy = dy; a.s = sum; a.w = weight; a.dsum = dsum; a.mean = mean; a.rstd = rstd;
    a.dx = dx; a.part = vectors ? part : nullptr;
    a.rows = s.rows; a.ldy = s.ldy; a.lds = s.lds; a.ldr = s.ldr; a.ldx = s.ldx;
    a.cols = (int)s.cols; a.tpr = tpr; a.wbf16 = s.wbf16; a.rms = s.rms;
    const int64_t vec = s.bf16 ? 8 : 4;
    const bool aligned = s.ldy % vec == 0 && s.lds % vec == 0 && (!dx || s.ldx % vec == 0) && (!dsum || s.ldr % vec == 0);
    const hipError_t e = norm_launch(a, s.bf16, aligned, grid, st);
    if (e != hipSuccess) return e;
  }
  if (!vectors) return hipSuccess;
  k_norm_wgrad<<<dim3((unsigned)cdiv(s.cols, NORM_WG_COLS), 2), 256, 0, st>>>(part, s.rows > 0 ? grid : 0, (int)s.cols, dweight, dbias);
  return hipGetLastError();
}

}  // namespace moe
