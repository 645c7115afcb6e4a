// The global norm of many gradient tensors, and their scaling down to a largest norm.
//
//   N = sqrt(sum over tensors and elements of g^2),  c = max_norm / N where N > max_norm, else 1,  out = c g
//
// The tensors' addresses and lengths travel in the kernels' arguments, GRAD_TENSORS of them a launch, so a
// call needs no table in device memory and a captured graph holds its own.  Tensors are cut into chunks of
// GRAD_CHUNK elements; a fixed grid of workgroups walks them, each thread adding its squares in fp64
// (whose squares neither overflow nor vanish for any fp32 value), and leaves one partial sum per workgroup.
// The scaling kernel's workgroups each add the partial sums, all in the same order, so no launch stands
// between the two passes.
#include "internal.h"

namespace moe {

constexpr int GRAD_TENSORS = 112;   // per launch: 3.4 KB of kernel arguments
constexpr int GRAD_CHUNK = 8192;    // elements
constexpr int GRAD_GRID = 2048;     // workgroups over all launches of a pass (more where launches are many)

struct GradTable {
  const void* src[GRAD_TENSORS];
  void* dst[GRAD_TENSORS];
  int64_t n[GRAD_TENSORS];
  int32_t first[GRAD_TENSORS + 1];  // first chunk of each tensor, and the number of chunks
  uint8_t kind[GRAD_TENSORS];       // GRAD_BF16 | GRAD_ALIGNED
  int32_t count;
};
enum { GRAD_BF16 = 1, GRAD_ALIGNED = 2 };

// The tensor that chunk c belongs to: the last one whose first chunk is not behind it.
__device__ __forceinline__ int grad_find(const GradTable& g, int c) {
  int lo = 0, hi = g.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

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
__device__ __forceinline__ double grad_square(const T* p, int n, bool aligned) {
  constexpr int VEC = Vec<T>::N, U = 4;
  double v = 0.0;
  int i = 0;
  if (aligned) {
    const int step = 256 * VEC;
    int k = threadIdx.x * VEC;
    for (; k + (U - 1) * step + VEC <= n; k += U * step) {
      u32x4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ld16(p + k + u * step);
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
      unpack16<T>(ld16(p + k), f);
#pragma unroll
      for (int q = 0; q < VEC; ++q) v = fma((double)f[q], (double)f[q], v);
    }
    i = n / VEC * VEC;
  }
  for (int k = i + threadIdx.x; k < n; k += 256) {
    const double x = (double)to_f32(p[k]);
    v = fma(x, x, v);
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void grad_scale(const T* p, T* o, int n, bool aligned, float c) {
  constexpr int VEC = Vec<T>::N, U = 4;
  int i = 0;
  if (aligned) {
    const int step = 256 * VEC;
    int k = threadIdx.x * VEC;
    for (; k + (U - 1) * step + VEC <= n; k += U * step) {
      u32x4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ld16_nt(p + k + u * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[VEC];
        unpack16<T>(r[u], f);
#pragma unroll
        for (int q = 0; q < VEC; ++q) f[q] *= c;
        st16_nt(o + k + u * step, pack16<T>(f));
      }
    }
    for (; k + VEC <= n; k += step) {
      float f[VEC];
      unpack16<T>(ld16_nt(p + k), f);
#pragma unroll
      for (int q = 0; q < VEC; ++q) f[q] *= c;
      st16_nt(o + k, pack16<T>(f));
    }
    i = n / VEC * VEC;
  }
  for (int k = i + threadIdx.x; k < n; k += 256) o[k] = from_f32<T>(to_f32(p[k]) * c);
}

// f(tensor, first element of the chunk, elements in it)
template <class F>
__device__ __forceinline__ void grad_chunks(const GradTable& g, F f) {
  const int chunks = g.first[g.count];
  int t = -1;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    if (t < 0 || c >= g.first[t + 1]) t = grad_find(g, c);
    const int64_t at = (int64_t)(c - g.first[t]) * GRAD_CHUNK;
    const int64_t left = g.n[t] - at;
    f(t, at, (int)(left < GRAD_CHUNK ? left : GRAD_CHUNK));
  }
}

__global__ __launch_bounds__(256) void k_grad_square(GradTable g, double* part) {
  __shared__ double red[4];
  double v = 0.0;
  grad_chunks(g, [&](int t, int64_t at, int n) {
    const bool al = g.kind[t] & GRAD_ALIGNED;
    if (g.kind[t] & GRAD_BF16) v += grad_square<bf16>(static_cast<const bf16*>(g.src[t]) + at, n, al);
    else v += grad_square<float>(static_cast<const float*>(g.src[t]) + at, n, al);
  });
  v = grad_block_sum(v, red);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// The sum of the partial sums, in one order in every workgroup.
__device__ __forceinline__ double grad_total(const double* part, int parts, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) v += part[i];
  return grad_block_sum(v, red);
}

__global__ __launch_bounds__(256) void k_grad_norm(const double* part, int parts, float* norm) {
  __shared__ double red[4];
  const double v = grad_total(part, parts, red);
  if (threadIdx.x == 0) *norm = (float)sqrt(v);
}

__global__ __launch_bounds__(256) void k_grad_scale(GradTable g, const double* part, int parts, const float* norm_in, float* norm,
                                                    double max_norm) {
  __shared__ double red[4];
  const double n = part ? sqrt(grad_total(part, parts, red)) : (double)*norm_in;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // a norm that is not a finite fp32 number (as the caller sees it) leaves the values as they are
  const bool cut = n > max_norm && (float)n < __builtin_inff();
  const float c = cut ? (float)(max_norm / n) : 1.0f;
  grad_chunks(g, [&](int t, int64_t at, int m) {
    if (!cut && g.src[t] == g.dst[t]) return;
    const bool al = g.kind[t] & GRAD_ALIGNED;
    if (g.kind[t] & GRAD_BF16)
      grad_scale<bf16>(static_cast<const bf16*>(g.src[t]) + at, static_cast<bf16*>(g.dst[t]) + at, m, al, c);
    else
      grad_scale<float>(static_cast<const float*>(g.src[t]) + at, static_cast<float*>(g.dst[t]) + at, m, al, c);
  });
}

// Launches of a pass over the list: f(table, grid) for every GRAD_TENSORS tensors that have elements.
static int grad_launches(int count) { return (int)cdiv(count, GRAD_TENSORS); }
static int grad_grid(int chunks, int count) {
  const int share = (int)cdiv(GRAD_GRID, grad_launches(count));
  const int most = share < 256 ? 256 : share;
  return chunks < most ? chunks : most;
}
template <class F>
static hipError_t grad_pass(const GradTensor* list, int count, F f) {
  for (int i = 0; i < count; i += GRAD_TENSORS) {
    GradTable g;
    g.count = 0;
    int chunks = 0;
    for (int k = i; k < count && k < i + GRAD_TENSORS; ++k) {
      if (list[k].n == 0) continue;
      const int q = g.count++;
      const uintptr_t both = reinterpret_cast<uintptr_t>(list[k].src) | reinterpret_cast<uintptr_t>(list[k].dst);
      g.src[q] = list[k].src;
      g.dst[q] = list[k].dst;
      g.n[q] = list[k].n;
      g.first[q] = chunks;
      g.kind[q] = (uint8_t)((list[k].bf16 ? GRAD_BF16 : 0) | (both % 16 == 0 ? GRAD_ALIGNED : 0));
      chunks += (int)cdiv(list[k].n, GRAD_CHUNK);
    }
    if (g.count == 0) continue;
    g.first[g.count] = chunks;
    f(g, grad_grid(chunks, count));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t grad_workspace_bytes(int count) {
  const int per = grad_grid(0x7fffffff, count < 1 ? 1 : count);
  return (size_t)per * (count < 1 ? 1 : grad_launches(count)) * sizeof(double);
}

static hipError_t grad_squares(const GradTensor* list, int count, double* part, int* parts, hipStream_t st) {
  *parts = 0;
  return grad_pass(list, count, [&](const GradTable& g, int grid) {
    k_grad_square<<<grid, 256, 0, st>>>(g, part + *parts);
    *parts += grid;
  });
}

hipError_t launch_grad_norm(const GradTensor* list, int count, float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  int parts = 0;
  const hipError_t e = grad_squares(list, count, part, &parts, st);
  if (e != hipSuccess) return e;
  k_grad_norm<<<1, 256, 0, st>>>(part, parts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTensor* list, int count, double max_norm, const float* norm_in, float* norm, void* ws,
                            hipStream_t st) {
  double* part = norm_in ? nullptr : static_cast<double*>(ws);
  int parts = 0;
  if (!norm_in) {
    const hipError_t e = grad_squares(list, count, part, &parts, st);
    if (e != hipSuccess) return e;
  }
  bool first = true;
  const hipError_t e = grad_pass(list, count, [&](const GradTable& g, int grid) {
    k_grad_scale<<<grid, 256, 0, st>>>(g, part, parts, norm_in, first && !norm_in ? norm : nullptr, max_norm);
    first = false;
  });
  if (e != hipSuccess || !first || norm_in) return e;
  k_grad_norm<<<1, 256, 0, st>>>(part, 0, norm);  // no elements at all
  return hipGetLastError();
}

}  // namespace moe
