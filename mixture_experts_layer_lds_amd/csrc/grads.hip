// The global norm of many gradient tensors, and their scaling down to a largest norm.
//
//   N = sqrt(sum over tensors and elements of g^2),  c = max_norm / N where N > max_norm, else 1,  out = c g
//
// The tensors are described by a table that the host makes once (GradEntry per tensor, then the tensor of each
// chunk of GRAD_CHUNK elements), so that a pass over any number of them is one launch.  A fixed grid of workgroups
// walks the chunks, each thread adding its squares in fp64 (which neither overflow nor vanish for any fp32
// value), and leaves one partial sum per workgroup.  The scaling kernel's workgroups each add the partial sums,
// all in the same order, so no launch stands between the two passes.
//
// Bound by memory: 151M bf16 gradients take 141 us for two reads and one write (906 MB, 6.4 TB/s, the second read
// mostly from the cache: 51 us for the squares, 91 for the scaling), a few MB the two launches (9 us).
#include <algorithm>
#include <memory>
#include <new>

#include "internal.h"

namespace moe {

constexpr int GRAD_GRID = 1024;     // workgroups

enum { GRAD_BF16 = 1 };

// 16 bytes of any tensor: they need no more than an element's alignment.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
__device__ __forceinline__ u32x4 grad_ld16(const void* p) { return *static_cast<const u32x4_any*>(p); }
__device__ __forceinline__ u32x4 grad_ld16_nt(const void* p) {
  return __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ void grad_st16_nt(void* p, u32x4 v) { __builtin_nontemporal_store(v, static_cast<u32x4_any*>(p)); }

__device__ __forceinline__ double grad_block_sum(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, WAVE);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int q = 1; q < (int)blockDim.x >> 6; ++q) v += red[q];
  return v;
}

template <typename T>
__device__ __forceinline__ double grad_square(const T* p, int n) {
  constexpr int VEC = Vec<T>::N, U = 4;
  double v = 0.0;
  const int step = 256 * VEC;
  int k = threadIdx.x * VEC;
  for (; k + (U - 1) * step + VEC <= n; k += U * step) {
    u32x4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = grad_ld16(p + k + u * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[VEC];
      unpack16<T>(r[u], f);
#pragma unroll
      for (int q = 0; q < VEC; ++q) v = fma((double)f[q], (double)f[q], v);
    }
  }
  for (; k + VEC <= n; k += step) {
    float f[VEC];
    unpack16<T>(grad_ld16(p + k), f);
#pragma unroll
    for (int q = 0; q < VEC; ++q) v = fma((double)f[q], (double)f[q], v);
  }
  for (int i = n / VEC * VEC + threadIdx.x; i < n; i += 256) {
    const double x = (double)to_f32(p[i]);
    v = fma(x, x, v);
  }
  return v;
}

// o = p c[0] c[1]
template <typename T>
__device__ __forceinline__ void grad_scale(const T* p, T* o, int n, const float (&c)[2]) {
  constexpr int VEC = Vec<T>::N, U = 4;
  const int step = 256 * VEC;
  int k = threadIdx.x * VEC;
  for (; k + (U - 1) * step + VEC <= n; k += U * step) {
    u32x4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = grad_ld16_nt(p + k + u * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[VEC];
      unpack16<T>(r[u], f);
#pragma unroll
      for (int q = 0; q < VEC; ++q) f[q] = f[q] * c[0] * c[1];
      grad_st16_nt(o + k + u * step, pack16<T>(f));
    }
  }
  for (; k + VEC <= n; k += step) {
    float f[VEC];
    unpack16<T>(grad_ld16_nt(p + k), f);
#pragma unroll
    for (int q = 0; q < VEC; ++q) f[q] = f[q] * c[0] * c[1];
    grad_st16_nt(o + k, pack16<T>(f));
  }
  for (int i = n / VEC * VEC + threadIdx.x; i < n; i += 256) o[i] = from_f32<T>(to_f32(p[i]) * c[0] * c[1]);
}

// f(entry, first element of the chunk, elements in it)
template <class F>
__device__ __forceinline__ void grad_chunks(const GradEntry* __restrict__ table, const int32_t* __restrict__ tensor, int chunks, F f) {
  int next = (int)blockIdx.x < chunks ? tensor[blockIdx.x] : 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const GradEntry g = table[__builtin_amdgcn_readfirstlane(next)];
    if (c + (int)gridDim.x < chunks) next = tensor[c + gridDim.x];
    const int64_t at = (int64_t)(c - g.first) * GRAD_CHUNK, left = g.n - at;
    f(g, at, (int)(left < GRAD_CHUNK ? left : GRAD_CHUNK));
  }
}

__global__ __launch_bounds__(256) void k_grad_square(const GradEntry* table, const int32_t* tensor, int chunks, double* part) {
  __shared__ double red[4];
  double v = 0.0;
  grad_chunks(table, tensor, chunks, [&](const GradEntry& g, int64_t at, int n) {
    if (g.kind & GRAD_BF16) v += grad_square<bf16>(static_cast<const bf16*>(g.src) + at, n);
    else v += grad_square<float>(static_cast<const float*>(g.src) + at, n);
  });
  v = grad_block_sum(v, red);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// The sum of the partial sums, in one order in every workgroup.
__device__ __forceinline__ double grad_total(const double* part, int parts, double* red) {
  double v = 0.0;
#pragma unroll
  for (int i = 0; i < GRAD_GRID / 256; ++i) {
    const int k = threadIdx.x + 256 * i;
    v += k < parts ? part[k] : 0.0;
  }
  return grad_block_sum(v, red);
}

__global__ __launch_bounds__(256) void k_grad_norm(const double* part, int parts, float* norm) {
  __shared__ double red[4];
  const double v = grad_total(part, parts, red);
  if (threadIdx.x == 0) *norm = (float)sqrt(v);
}

__global__ __launch_bounds__(256) void k_grad_scale(const GradEntry* table, const int32_t* tensor, int chunks, const double* part,
                                                    int parts, const float* norm_in, float* norm, double max_norm) {
  __shared__ double red[4];
  const double n = part ? sqrt(grad_total(part, parts, red)) : (double)*norm_in;
  if (part && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // a norm that is not a finite fp32 number (as the caller sees it) leaves the values as they are
  const bool cut = n > max_norm && (float)n < __builtin_inff();
  // a factor below fp32's normal range (a norm of 1e36 cut to 1e-6) would lose its digits: then it goes in two, the first a
  // power of two
  const double f = cut ? max_norm / n : 1.0;
  const bool two = f < 0x1p-126;
  const float c[2] = {two ? 0x1p-126f : 1.0f, (float)(two ? f * 0x1p126 : f)};
  grad_chunks(table, tensor, chunks, [&](const GradEntry& g, int64_t at, int m) {
    if (!cut && g.src == g.dst) return;
    if (g.kind & GRAD_BF16) grad_scale<bf16>(static_cast<const bf16*>(g.src) + at, static_cast<bf16*>(g.dst) + at, m, c);
    else grad_scale<float>(static_cast<const float*>(g.src) + at, static_cast<float*>(g.dst) + at, m, c);
  });
}

static int grad_grid(int chunks) { return chunks < GRAD_GRID ? chunks : GRAD_GRID; }

size_t grad_workspace_bytes() { return GRAD_GRID * sizeof(double); }

int grad_table(const GradTensor* list, int count, void* host) {
  GradEntry* e = static_cast<GradEntry*>(host);
  int32_t* tensor = reinterpret_cast<int32_t*>(e + count);
  int chunks = 0;
  for (int i = 0; i < count; ++i) {
    e[i] = GradEntry{list[i].src, list[i].dst, list[i].n, chunks, list[i].bf16 ? GRAD_BF16 : 0};
    for (int64_t c = cdiv(list[i].n, GRAD_CHUNK); c > 0; --c) tensor[chunks++] = i;
  }
  return chunks;
}

// Two tensors (sources or destinations, but for one's own two in the same place) that share bytes.
bool grad_overlap(const GradTensor* list, int count, int* first, int* second) {
  struct Span {
    uintptr_t a, b;
    int i;
  };
  const std::unique_ptr<Span[]> s(new (std::nothrow) Span[2 * (size_t)count + 1]);
  if (!s) return false;
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    const uintptr_t bytes = (uintptr_t)list[i].n * (list[i].bf16 ? 2 : 4);
    if (bytes == 0) continue;
    const uintptr_t src = reinterpret_cast<uintptr_t>(list[i].src), dst = reinterpret_cast<uintptr_t>(list[i].dst);
    s[n++] = Span{src, src + bytes, i};
    if (dst != src) s[n++] = Span{dst, dst + bytes, i};
  }
  std::sort(s.get(), s.get() + n, [](const Span& x, const Span& y) { return x.a < y.a; });
  for (size_t k = 1; k < n; ++k)
    if (s[k].a < s[k - 1].b) {
      *first = s[k - 1].i;
      *second = s[k].i;
      return true;
    }
  return false;
}

static const int32_t* grad_tensors(const void* table, int count) {
  return reinterpret_cast<const int32_t*>(static_cast<const GradEntry*>(table) + count);
}

static hipError_t grad_squares(const void* table, int count, int chunks, double* part, hipStream_t st) {
  if (chunks == 0) return hipSuccess;
  k_grad_square<<<grad_grid(chunks), 256, 0, st>>>(static_cast<const GradEntry*>(table), grad_tensors(table, count), chunks, part);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const void* table, int count, int chunks, float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  const hipError_t e = grad_squares(table, count, chunks, part, st);
  if (e != hipSuccess) return e;
  k_grad_norm<<<1, 256, 0, st>>>(part, grad_grid(chunks), norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const void* table, int count, int chunks, double max_norm, const float* norm_in, float* norm, void* ws,
                            hipStream_t st) {
  if (chunks == 0) return norm_in ? hipSuccess : launch_grad_norm(table, count, 0, norm, ws, st);
  double* part = norm_in ? nullptr : static_cast<double*>(ws);
  if (!norm_in) {
    const hipError_t e = grad_squares(table, count, chunks, part, st);
    if (e != hipSuccess) return e;
  }
  const int grid = grad_grid(chunks);
  k_grad_scale<<<grid, 256, 0, st>>>(static_cast<const GradEntry*>(table), grad_tensors(table, count), chunks, part, grid, norm_in, norm, max_norm);
  return hipGetLastError();
}

}  // namespace moe
