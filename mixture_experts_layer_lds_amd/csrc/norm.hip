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
//
// Bound by memory: the forward reads x and r and writes s and y once, the backward reads dy, s and dsum and
// writes dx.  32768 x 7168 bf16: forward 1.88 GB in 327 us (5.7 TB/s), backward 1.88 GB in 319 us (5.9 TB/s); 32768 x
// 1536 backward 78 us (5.1 TB/s: the partial rows and the second launch are 5 us of it).  What brought them there: the
// next row requested while one is reduced, a grid that just fills the chip (norm_grid), lane sums by DPP.  One row of
// 7168 is a launch: 3.3 us on the GPU.  A backward of some hundred rows is bound by its chain of launch, row, sums and
// second launch: 999 x 1003 fp32 12.8 us, 3 at the rate of a copy.
#include "internal.h"

namespace moe {

// Rows are accessed in 16 bytes whatever their alignment (their strides may be any; 30000 x 1600 bf16 of stride
// 1603 by elements took 704 us, so 89, dense ones 70): with a part of a chunk at the row's end, or in whole chunks throughout.
enum { NORM_PART = 0, NORM_WHOLE = 1 };
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
__device__ __forceinline__ u32x4 norm_ld16(const void* p) {
  return __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ void norm_st16(void* p, u32x4 v) { __builtin_nontemporal_store(v, static_cast<u32x4_any*>(p)); }

// The first column of a thread's chunk j, 8 neighbours.
__device__ __forceinline__ int norm_col(int j, int tpr, int t) { return (j * tpr + t) * 8; }

// 8 elements as they lie in memory.
template <typename T> struct Raw8 { u32x4 v[8 / Vec<T>::N]; };

// Columns behind the row hold zeros.
template <typename T, int MODE>
__device__ __forceinline__ Raw8<T> norm_load1(const T* p, int cols, int tpr, int t, int j) {
  constexpr int NV = 8 / Vec<T>::N;
  const int c = norm_col(j, tpr, t);
  Raw8<T> r;
  if constexpr (MODE == NORM_WHOLE) {
#pragma unroll
    for (int v = 0; v < NV; ++v) r.v[v] = u32x4{0u, 0u, 0u, 0u};
    if (c < cols) {
#pragma unroll
      for (int v = 0; v < NV; ++v) r.v[v] = norm_ld16(p + c + v * Vec<T>::N);
    }
    return r;
  }
  if (c + 8 <= cols) {
#pragma unroll
    for (int v = 0; v < NV; ++v) r.v[v] = norm_ld16(p + c + v * Vec<T>::N);
    return r;
  }
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ci = norm_col(j, tpr, t) + i;
      if (ci < cols) f[i] = to_f32(p[ci]);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) r.v[v] = pack16<T>(f + v * Vec<T>::N);
  return r;
}
template <typename T, int NC, int MODE>
__device__ __forceinline__ void norm_load(const T* p, int cols, int tpr, int t, Raw8<T> (&r)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) r[j] = norm_load1<T, MODE>(p, cols, tpr, t, j);
}
template <typename T>
__device__ __forceinline__ void norm_unpack(const Raw8<T>& r, float* f) {
#pragma unroll
  for (int v = 0; v < 8 / Vec<T>::N; ++v) unpack16<T>(r.v[v], f + v * Vec<T>::N);
}
template <typename T, int MODE>
__device__ __forceinline__ void norm_store(T* p, int cols, int tpr, int t, int j, const Raw8<T>& r) {
  const int c = norm_col(j, tpr, t);
  if (c >= cols) return;
  if (MODE == NORM_WHOLE || (MODE == NORM_PART && c + 8 <= cols)) {
#pragma unroll
    for (int v = 0; v < 8 / Vec<T>::N; ++v) norm_st16(p + c + v * Vec<T>::N, r.v[v]);
  } else {
    float f[8];
    norm_unpack<T>(r, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ci = norm_col(j, tpr, t) + i;
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

// Weight or bias of a thread's chunk j (null: the value `none`).
template <int MODE>
__device__ __forceinline__ void norm_vector(const void* p, bool wbf16, float none, int cols, int tpr, int t, int j, float* w) {
  const int c0 = norm_col(j, tpr, t);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = none;
  if (!p || c0 >= cols) return;
  if (MODE == NORM_WHOLE || c0 + 8 <= cols) {
    if (wbf16) {
      unpack16<bf16>(ld16(static_cast<const bf16*>(p) + c0), w);
    } else {
      unpack16<float>(ld16(static_cast<const float*>(p) + c0), w);
      unpack16<float>(ld16(static_cast<const float*>(p) + c0 + 4), w + 4);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = norm_col(j, tpr, t) + i;
    if (c < cols) w[i] = wbf16 ? to_f32(static_cast<const bf16*>(p)[c]) : static_cast<const float*>(p)[c];
  }
}

// Sum of v over groups of `tpr` neighbouring lanes (a power of two, 8 .. 64), in every lane: mirrored and
// swapped lanes, no trip through LDS.
template <int CTRL> __device__ __forceinline__ float norm_dpp(float v) {
  return v + __uint_as_float(dpp_src<CTRL, 0xf, 0xf>(__float_as_uint(v)));
}
__device__ __forceinline__ float norm_lane_sum(float v, int tpr) {
  v = norm_dpp<0xb1>(v);   // quad_perm 1 0 3 2
  v = norm_dpp<0x4e>(v);   // quad_perm 2 3 0 1
  v = norm_dpp<0x141>(v);  // row_half_mirror
  if (tpr >= 16) v = norm_dpp<0x140>(v);  // row_mirror
  if (tpr >= 32) {
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if (tpr >= 64) {
    auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// Sums of a row's values over its threads, in every one of them: inside a wave, then (tpr > 64:
// the row's threads are the workgroup) the waves' sums through LDS in wave order.  The two halves of `red`
// alternate, so that a reduction writes what no wave still reads: between its write and the last read of
// the same half lies the other half's barrier.
template <int N>
__device__ __forceinline__ void norm_row_sum(float (&v)[N], int tpr, float (*red)[N][16], int& half) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = norm_lane_sum(v[k], tpr);
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

// 1 / sqrt(q / n + eps) for a row's sum of squares q, inv = 1 / n.  Squares that leave fp32's range (elements over
// 2^64, or of 2^-50 and less with an eps that does not hide them) are summed once more, as squares(s) of elements times
// a power of two s: any finite row has its deviation.  v is the same in all threads of a row.
template <class Squares>
__device__ __forceinline__ float norm_rstd(float q, float inv, float eps, Squares squares) {
  const float v = fmaf(q, inv, eps);
  if (v >= 0x1p-100f && v <= 3.4028235e38f) return 1.0f / sqrtf(v);
  const float s = v < 1.0f ? 0x1p100f : 0x1p-76f;
  return s / sqrtf(fmaf(squares(s), inv, eps * s * s));
}
// A row's mean from its sum s; where that left fp32's range, from sum(2^-20), the sum of elements times 2^-20.
template <class Sum>
__device__ __forceinline__ float norm_mean(float s, float inv, Sum sum) {
  if (fabsf(s) <= 3.4028235e38f) return s * inv;
  return sum(0x1p-20f) * inv * 0x1p20f;
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

template <typename T, int NC, int MODE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm(NormFwd a) {
  __shared__ float red[2][1][16];
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1), rpb = blockDim.x / tpr, cols = a.cols;
  const float inv = 1.0f / (float)cols;
  const bool res = a.res != nullptr;
  int half = 0;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  constexpr bool AHEAD = THREADS < 1024;  // (128 registers do not hold the next row too)
  Raw8<T> raw[NC], rr[NC];
  auto load = [&](int64_t r) {
    if (r >= a.rows) return;
    norm_load<T, NC, MODE>(static_cast<const T*>(a.x) + r * a.ldx, cols, tpr, t, raw);
    if (res) norm_load<T, NC, MODE>(static_cast<const T*>(a.res) + r * a.ldr, cols, tpr, t, rr);
  };
  if constexpr (AHEAD) load(row);
  float w[NC * 8], b[NC * 8];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    norm_vector<MODE>(a.w, a.wbf16, 1.0f, cols, tpr, t, j, w + j * 8);
    norm_vector<MODE>(a.b, a.wbf16, 0.0f, cols, tpr, t, j, b + j * 8);
  }
  // (with tpr > 64 a row is the workgroup's, so the barriers inside are reached by all of it; with several
  // rows a workgroup there are none)
  for (; row < a.rows; row += step) {
    if constexpr (!AHEAD) load(row);
    float f[NC * 8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      norm_unpack<T>(raw[j], f + j * 8);
      if (res) {
        float v[8];
        norm_unpack<T>(rr[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j * 8 + i] += v[i];
        const Raw8<T> sum = norm_pack<T>(f + j * 8);  // what is normalised is the rounded sum, which the backward reads
        if (a.sum) norm_store<T, MODE>(static_cast<T*>(a.sum) + row * a.lds, cols, tpr, t, j, sum);
        norm_unpack<T>(sum, f + j * 8);
      }
    }
    if constexpr (AHEAD) load(row + step);  // the next row arrives while this one is reduced
    float mu = 0.0f;
    if (!a.rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) s[0] += f[i];  // (columns past the row hold zeros)
      norm_row_sum<1>(s, tpr, red, half);
      mu = norm_mean(s[0], inv, [&](float scale) {
        float z[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NC * 8; ++i) z[0] = fmaf(f[i], scale, z[0]);
        norm_row_sum<1>(z, tpr, red, half);
        return z[0];
      });
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = norm_col(j, tpr, t) + i < cols ? f[j * 8 + i] - mu : 0.0f;
        f[j * 8 + i] = d;
        q[0] = fmaf(d, d, q[0]);
      }
    norm_row_sum<1>(q, tpr, red, half);
    const float rstd = norm_rstd(q[0], inv, a.eps, [&](float scale) {
      float z[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC * 8; ++i) z[0] = fmaf(f[i] * scale, f[i] * scale, z[0]);
      norm_row_sum<1>(z, tpr, red, half);
      return z[0];
    });
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j * 8 + i] = fmaf(f[j * 8 + i] * rstd, w[j * 8 + i], b[j * 8 + i]);
      norm_store<T, MODE>(y, cols, tpr, t, j, norm_pack<T>(f + j * 8));
    }
  }
}

// Rows that the registers do not hold: 1024 threads a row, which is read three times (for the mean, the squares
// and the result; after the first from the caches, mostly), as the vectors are for each row.
template <typename T, int MODE>
__global__ __launch_bounds__(1024) void k_norm_long(NormFwd a) {
  __shared__ float red[2][1][16];
  const int tpr = 1024, t = threadIdx.x, cols = a.cols, nc = (cols + 8191) / 8192;
  const float inv = 1.0f / (float)cols;
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.lds : nullptr;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    // chunk j of x + r, rounded
    auto added = [&](int j, float (&f)[8]) {
      norm_unpack<T>(norm_load1<T, MODE>(x, cols, tpr, t, j), f);
      if (!r) return;
      float v[8];
      norm_unpack<T>(norm_load1<T, MODE>(r, cols, tpr, t, j), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += v[i];
      const Raw8<T> s = norm_pack<T>(f);
      norm_unpack<T>(s, f);
    };
    // the same once more: from sum where it is kept, as sum may lie where x or r was
    auto again = [&](int j, float (&f)[8]) {
      if (sum) norm_unpack<T>(norm_load1<T, MODE>(sum, cols, tpr, t, j), f);
      else added(j, f);
    };
    float s[1] = {0.0f};
    for (int j = 0; j < nc; ++j) {
      float f[8];
      added(j, f);
      if (sum) norm_store<T, MODE>(sum, cols, tpr, t, j, norm_pack<T>(f));
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += f[i];
    }
    norm_row_sum<1>(s, tpr, red, half);
    const float mu = a.rms ? 0.0f : norm_mean(s[0], inv, [&](float scale) {
      float z[1] = {0.0f};
      for (int j = 0; j < nc; ++j) {
        float f[8];
        again(j, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[0] = fmaf(f[i], scale, z[0]);
      }
      norm_row_sum<1>(z, tpr, red, half);
      return z[0];
    });
    auto squares = [&](float scale) {
      float z[1] = {0.0f};
      for (int j = 0; j < nc; ++j) {
        float f[8];
        again(j, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = norm_col(j, tpr, t) + i < cols ? (f[i] - mu) * scale : 0.0f;
          z[0] = fmaf(d, d, z[0]);
        }
      }
      norm_row_sum<1>(z, tpr, red, half);
      return z[0];
    };
    const float rstd = norm_rstd(squares(1.0f), inv, a.eps, squares);
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int j = 0; j < nc; ++j) {
      float f[8], w[8], b[8];
      again(j, f);
      norm_vector<MODE>(a.w, a.wbf16, 1.0f, cols, tpr, t, j, w);
      norm_vector<MODE>(a.b, a.wbf16, 0.0f, cols, tpr, t, j, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fmaf((f[i] - mu) * rstd, w[i], b[i]);
      norm_store<T, MODE>(y, cols, tpr, t, j, norm_pack<T>(f));
    }
  }
}

struct NormBwd {
  const void *dy, *s, *w, *dsum;
  const float *mean, *rstd;
  void* dx;       // may be null
  float* part;    // [workgroups][dw, db][pitch], or null
  int64_t rows, ldy, lds, ldr, ldx;
  int cols, tpr, pitch;
  bool wbf16, rms;
};

// Every thread keeps its columns' parts of dw and db over the rows it takes; a workgroup adds those of
// its row groups in LDS and writes one partial row, which k_norm_wgrad adds up in a fixed order.
template <typename T, int NC, int MODE, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm_bwd(NormBwd a) {
  __shared__ float red[2][2][16];
  __shared__ float add[THREADS <= 256 ? 256 * 8 : 1];
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1), rpb = blockDim.x / tpr, cols = a.cols;
  const float inv = 1.0f / (float)cols;
  const bool has_dsum = a.dsum && a.dx;
  int half = 0;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  Raw8<T> ndy[NC], ns[NC], nd[NC];
  float nmu = 0.0f, nrstd = 0.0f;
  auto load = [&](int64_t r) {
    if (r >= a.rows) return;
    norm_load<T, NC, MODE>(static_cast<const T*>(a.dy) + r * a.ldy, cols, tpr, t, ndy);
    norm_load<T, NC, MODE>(static_cast<const T*>(a.s) + r * a.lds, cols, tpr, t, ns);
    if (has_dsum) norm_load<T, NC, MODE>(static_cast<const T*>(a.dsum) + r * a.ldr, cols, tpr, t, nd);
    nmu = a.rms ? 0.0f : a.mean[r];
    nrstd = a.rstd[r];
  };
  load(row);
  float w[NC * 8], dw[NC * 8], db[NC * 8];
#pragma unroll
  for (int j = 0; j < NC; ++j) norm_vector<MODE>(a.w, a.wbf16, 1.0f, cols, tpr, t, j, w + j * 8);
#pragma unroll
  for (int i = 0; i < NC * 8; ++i) dw[i] = db[i] = 0.0f;
  for (; row < a.rows; row += step) {
    Raw8<T> rdy[NC], rs[NC], rd[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      rdy[j] = ndy[j];
      rs[j] = ns[j];
      if (has_dsum) rd[j] = nd[j];
    }
    const float mu = nmu, rstd = nrstd;
    load(row + step);  // the next row arrives while this one is reduced
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float g[8], x[8];
      norm_unpack<T>(rdy[j], g);
      norm_unpack<T>(rs[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = j * 8 + i;
        const float xh = norm_col(j, tpr, t) + i < cols ? (x[i] - mu) * rstd : 0.0f;
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
      norm_store<T, MODE>(dx, cols, tpr, t, j, norm_pack<T>(d));
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.pitch;
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
      if ((int)threadIdx.x >= tpr) continue;
      const int c = norm_col(j, tpr, t);
      if (c < cols) {  // (a partial row is whole chunks)
        st16(part + k * a.pitch + c, pack16<float>(v));
        st16(part + k * a.pitch + c + 4, pack16<float>(v + 4));
      }
    }
}

// dx of rows that the registers do not hold: 1024 threads a row, which is read twice (the second time from the
// caches, mostly), as the weights are.
template <typename T, int MODE>
__global__ __launch_bounds__(1024) void k_norm_bwd_long(NormBwd a) {
  __shared__ float red[2][2][16];
  const int tpr = 1024, t = threadIdx.x, cols = a.cols, nc = (cols + 8191) / 8192;
  const float inv = 1.0f / (float)cols;
  int half = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.ldy;
    const T* s = static_cast<const T*>(a.s) + row * a.lds;
    const T* ds = a.dsum ? static_cast<const T*>(a.dsum) + row * a.ldr : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.ldx;
    const float mu = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
    float v[2] = {0.0f, 0.0f};
    auto chunk = [&](int j, float (&gw)[8], float (&xh)[8]) {
      norm_unpack<T>(norm_load1<T, MODE>(dy, cols, tpr, t, j), gw);
      norm_unpack<T>(norm_load1<T, MODE>(s, cols, tpr, t, j), xh);
      float w[8];
      norm_vector<MODE>(a.w, a.wbf16, 1.0f, cols, tpr, t, j, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gw[i] *= w[i];
        xh[i] = norm_col(j, tpr, t) + i < cols ? (xh[i] - mu) * rstd : 0.0f;
      }
    };
    for (int j = 0; j < nc; ++j) {
      float gw[8], xh[8];
      chunk(j, gw, xh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[0] += gw[i];
        v[1] = fmaf(gw[i], xh[i], v[1]);
      }
    }
    norm_row_sum<2>(v, tpr, red, half);
    const float m1 = a.rms ? 0.0f : v[0] * inv, m2 = v[1] * inv;
    for (int j = 0; j < nc; ++j) {
      float gw[8], xh[8], d[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      chunk(j, gw, xh);
      if (ds) norm_unpack<T>(norm_load1<T, MODE>(ds, cols, tpr, t, j), d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-xh[i], m2, gw[i] - m1), d[i]);
      norm_store<T, MODE>(dx, cols, tpr, t, j, norm_pack<T>(d));
    }
  }
}

// dw and db of rows too long for k_norm_bwd's registers: one column a thread, a run of rows a workgroup.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_cols(NormBwd a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  const int64_t r0 = a.rows * blockIdx.y / gridDim.y, r1 = a.rows * (blockIdx.y + 1) / gridDim.y;
  const T* dy = static_cast<const T*>(a.dy) + c;
  const T* s = static_cast<const T*>(a.s) + c;
  float dw = 0.0f, db = 0.0f;
#pragma unroll 8
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_f32(dy[r * a.ldy]), x = to_f32(s[r * a.lds]);
    dw = fmaf(g, (x - (a.rms ? 0.0f : a.mean[r])) * a.rstd[r], dw);
    db += g;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.pitch;
  part[c] = dw;
  part[a.pitch + c] = db;
}

// dw and db: the workgroups' partial rows added in fp64, 32 runs of them per column, then the runs (512 rows of 1003:
// 2 us less than 8 runs, whose trips to memory follow one another).
constexpr int NORM_WG_COLS = 32, NORM_WG_RUNS = 32;
__global__ __launch_bounds__(NORM_WG_COLS * NORM_WG_RUNS) void k_norm_wgrad(const float* __restrict__ part, int parts, int cols,
                                                                           int pitch, float* dw, float* db) {
  __shared__ double red[NORM_WG_RUNS][NORM_WG_COLS + 1];
  const int cl = threadIdx.x % NORM_WG_COLS, run = threadIdx.x / NORM_WG_COLS;
  const int c = blockIdx.x * NORM_WG_COLS + cl;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;  // (uniform)
  double v = 0.0;
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * pitch + c;
#pragma unroll 8
    for (int q = run; q < parts; q += NORM_WG_RUNS) v += (double)p[(int64_t)q * 2 * pitch];
  }
  red[run][cl] = v;
  __syncthreads();
  if (run == 0 && c < cols) {
#pragma unroll
    for (int q = 1; q < NORM_WG_RUNS; ++q) v += red[q][cl];
    out[c] = (float)v;
  }
}

// Threads per row and with them the chunks of 8 columns per thread: a few rows take as many threads as there
// are chunks (two a thread with 512 threads: one row of 7168 3.8 us, 4.1 with 1024); many rows up to three chunks
// a thread (two with 512 threads), so that the lanes are busy, a row's sums cross few waves and the registers still
// hold the next row.  So 256 threads go with 1 to 3 chunks, 512 with 1 or 2, 1024 (rows over 8192, forward) with 2.
// `many`: in the forward 256 rows (999 x 1536 bf16 4.6 us, one chunk a thread 5.3), in the backward 1024 (999 x
// 1003 fp32 14.9 us, with three chunks 17.4: fewer threads hold the sums of the vectors' gradients).
constexpr int NORM_FWD_MANY = 256, NORM_BWD_MANY = 1024;
static int norm_tpr(int64_t cols, int64_t rows, int many) {
  const int64_t chunks = cdiv(cols, 8);
  int tpr = 8;
  while (tpr < 1024 && cdiv(chunks, tpr) > (tpr == 512 ? 2 : rows < many || tpr < 64 ? 1 : 3)) tpr *= 2;
  return tpr;
}
static int norm_threads(int tpr) { return tpr > 64 ? tpr : 256; }
// Workgroups, which walk the rows: eight waves a CU, or sixteen where a row takes 1024 threads; more of them only spread the
// accesses over more of memory's pages (32768 x 7168 forward 327 us with 256 of 512 threads, 345 with 512; 16384 x 4096
// 89 us with 512 of 256 threads, 93 with 1024).  128 threads (many rows of over 1536 columns) are two waves: bf16 rows take 1024
// workgroups (32768 x 2048 88 us, backward 98; with 512 109 and 118), fp32 rows, twice the bytes, 512 (16384 x 2048 104 us,
// backward 104; with 1024 112 and 113), and so does a backward with less than four rows for each of 1024, since each
// leaves a partial row of the vectors' gradients (2048 x 2048 bf16 17.7 us; with 1024 21.8).
static int norm_grid(int64_t rows, int tpr, bool is_bf16, bool backward) {
  const int threads = norm_threads(tpr);
  int64_t most = threads >= 512 ? 256 : 512;
  if (threads == 128 && is_bf16 && (!backward || rows >= 4 * 1024)) most = 1024;
  const int64_t need = cdiv(rows, threads / tpr);
  return (int)(need < most ? need : most);
}
// Rows that the registers of 1024 threads do not hold: of the forward, and of the backward, where the vectors'
// gradients are held too.
static bool norm_fwd_long(int64_t cols) { return cols > 16 * 1024; }
static bool norm_bwd_long(int64_t cols) { return cols > 8 * 1024; }

template <typename T, int NC, int MODE>
static void norm_go(const NormFwd& a, int grid, int threads, hipStream_t st) {
  if (threads <= 256) k_norm<T, NC, MODE, 256><<<grid, threads, 0, st>>>(a);
  else if constexpr (NC <= 2) {
    if (threads <= 512) k_norm<T, NC, MODE, 512><<<grid, threads, 0, st>>>(a);
    else if constexpr (NC == 2) k_norm<T, NC, MODE, 1024><<<grid, threads, 0, st>>>(a);
  }
}
template <typename T, int NC, int MODE>
static void norm_go(const NormBwd& a, int grid, int threads, hipStream_t st) {
  if (threads <= 256) k_norm_bwd<T, NC, MODE, 256><<<grid, threads, 0, st>>>(a);
  else if constexpr (NC <= 2) k_norm_bwd<T, NC, MODE, 512><<<grid, threads, 0, st>>>(a);
}
template <typename T, int MODE>
static bool norm_go_long(const NormFwd& a, int grid, hipStream_t st) {
  if (!norm_fwd_long(a.cols)) return false;
  k_norm_long<T, MODE><<<grid, 1024, 0, st>>>(a);
  return true;
}
template <typename T, int MODE>
static bool norm_go_long(const NormBwd& a, int grid, hipStream_t st) {
  if (!norm_bwd_long(a.cols)) return false;
  k_norm_bwd_long<T, MODE><<<grid, 1024, 0, st>>>(a);
  return true;
}
template <typename T, int MODE, class Args>
static void norm_chunks(const Args& a, int grid, int threads, hipStream_t st) {
  if (norm_go_long<T, MODE>(a, grid, st)) return;
  const int nc = (int)cdiv(a.cols, 8 * a.tpr);
  if (nc <= 1) norm_go<T, 1, MODE>(a, grid, threads, st);
  else if (nc <= 2) norm_go<T, 2, MODE>(a, grid, threads, st);
  else norm_go<T, 3, MODE>(a, grid, threads, st);
}
template <class Args>
static hipError_t norm_launch(const Args& a, bool is_bf16, int grid, hipStream_t st) {
  const int threads = norm_threads(a.tpr), mode = a.cols % 8 ? NORM_PART : NORM_WHOLE;
  if (is_bf16) {
    if (mode == NORM_WHOLE) norm_chunks<bf16, NORM_WHOLE>(a, grid, threads, st);
    else norm_chunks<bf16, NORM_PART>(a, grid, threads, st);
  } else {
    if (mode == NORM_WHOLE) norm_chunks<float, NORM_WHOLE>(a, grid, threads, st);
    else norm_chunks<float, NORM_PART>(a, grid, threads, st);
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
  a.tpr = norm_tpr(s.cols, s.rows, NORM_FWD_MANY);
  a.eps = s.eps; a.wbf16 = s.wbf16; a.rms = s.rms;
  return norm_launch(a, s.bf16, norm_grid(s.rows, a.tpr, s.bf16, false), st);
}

static int norm_pitch(int64_t cols) { return (int)align_up((size_t)cols, 8); }
size_t norm_bwd_workspace_bytes(const NormShape& s) {
  const int tpr = norm_tpr(s.cols, s.rows, NORM_BWD_MANY);
  return (size_t)norm_grid(s.rows, tpr, s.bf16, true) * 2 * norm_pitch(s.cols) * sizeof(float);
}

hipError_t launch_norm_bwd(const NormShape& s, const void* dy, const void* sum, const void* weight, const float* mean,
                           const float* rstd, const void* dsum, void* dx, float* dweight, float* dbias, void* ws,
                           hipStream_t st) {
  const int tpr = norm_tpr(s.cols, s.rows, NORM_BWD_MANY), grid = norm_grid(s.rows, tpr, s.bf16, true);
  const bool vectors = dweight || dbias;
  float* part = static_cast<float*>(ws);
  if (s.rows > 0) {
    NormBwd a;
    a.dy = dy; a.s = sum; a.w = weight; a.dsum = dsum; a.mean = mean; a.rstd = rstd;
    a.dx = dx; a.part = vectors ? part : nullptr;
    a.rows = s.rows; a.ldy = s.ldy; a.lds = s.lds; a.ldr = s.ldr; a.ldx = s.ldx;
    a.cols = (int)s.cols; a.tpr = tpr; a.pitch = norm_pitch(s.cols); a.wbf16 = s.wbf16; a.rms = s.rms;
    const bool long_rows = norm_bwd_long(s.cols);
    hipError_t e = hipSuccess;
    if (vectors && long_rows) {  // (first: dx may take the place of dy or s)
      const dim3 cols((unsigned)cdiv(s.cols, 256), (unsigned)grid);
      if (s.bf16) k_norm_cols<bf16><<<cols, 256, 0, st>>>(a);
      else k_norm_cols<float><<<cols, 256, 0, st>>>(a);
      e = hipGetLastError();
    }
    if (e == hipSuccess && (dx || !long_rows)) e = norm_launch(a, s.bf16, grid, st);
    if (e != hipSuccess) return e;
  }
  if (!vectors) return hipSuccess;
  k_norm_wgrad<<<dim3((unsigned)cdiv(s.cols, NORM_WG_COLS), 2), NORM_WG_COLS * NORM_WG_RUNS, 0, st>>>(
      part, s.rows > 0 ? grid : 0, (int)s.cols, norm_pitch(s.cols), dweight, dbias);
  return hipGetLastError();
}

}  // namespace moe
