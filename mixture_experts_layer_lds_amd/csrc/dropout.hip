// Dropout with an optional residual sum: out = residual + keep(x) * scale, the mask recomputed
// from the counter (philox.h) and never stored.  The same kernel without a residual is its
// gradient: d x = keep(d out) * scale.
//
// One thread takes one group of eight columns of a row (one generator call): 16 bytes of bf16 or
// two 16-byte chunks of fp32 where rows are 16-byte aligned; a row's last group may be partial and
// goes element by element, as do all groups of rows that are not aligned.  A dropped element is
// selected away, not multiplied by zero, so it adds nothing even where x is infinite or NaN.
// Bound by memory (x and residual read once, out written once): 32768 x 7168 bf16, 940 MB, 150 us
// (6.3 TB/s; a library copy of 2 GiB reaches 4.9); 257 x 1003 fp32 rows with a residual 3.7 us, a launch's
// length.  16 random bits an element keep the generator at 20 products of 32 x 32 -> 64 bits per group of
// eight, 2.5 an element, below what memory takes.
#include "internal.h"
#include "philox.h"

namespace moe {

template <typename T, bool RES, bool ALIGNED>
__global__ __launch_bounds__(256) void k_dropout(const T* x, int64_t ldx, const T* res, int64_t ldr, T* out,
                                                 int64_t ldo, uint32_t groups, uint32_t per_row, int cols,
                                                 DropArgs a) {
  const PhiloxKey key = philox_key(a.rng);
  constexpr int VEC = 16 / sizeof(T);
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < groups; i += gridDim.x * 256u) {
    const uint32_t row = i / per_row, g = i - row * per_row;
    const int c0 = (int)g * 8, n = min(8, cols - c0);
    const T* xp = x + (int64_t)row * ldx + c0;
    const T* rp = RES ? res + (int64_t)row * ldr + c0 : nullptr;
    T* op = out + (int64_t)row * ldo + c0;
    if (ALIGNED && n == 8) {
      u32x4 xv[8 / VEC], rv[8 / VEC];
#pragma unroll
      for (int j = 0; j < 8 / VEC; ++j) {
        xv[j] = ld16_nt(xp + j * VEC);
        if (RES) rv[j] = ld16_nt(rp + j * VEC);
      }
      const u32x4 w = philox10(key, g, row);
#pragma unroll
      for (int j = 0; j < 8 / VEC; ++j) {
        float f[VEC], r[VEC];
        unpack16<T>(xv[j], f);
        if (RES) unpack16<T>(rv[j], r);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float y = drop_keep(w, j * VEC + k, a.threshold) ? f[k] * a.scale : 0.0f;
          f[k] = RES ? y + r[k] : y;
        }
        st16_nt(op + j * VEC, pack16<T>(f));
      }
    } else {
      const u32x4 w = philox10(key, g, row);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= n) break;
        const float y = drop_keep(w, k, a.threshold) ? to_f32(xp[k]) * a.scale : 0.0f;
        op[k] = from_f32<T>(RES ? y + to_f32(rp[k]) : y);
      }
    }
  }
}

template <typename T, bool RES>
static void dropout_for(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* res, int64_t ldr, void* out,
                        int64_t ldo, const DropArgs& a, hipStream_t st) {
  const uint32_t per_row = (uint32_t)cdiv(cols, 8), groups = (uint32_t)rows * per_row;
  const int grid = (int)cdiv((int64_t)groups, 256);
  constexpr int64_t VEC = 16 / sizeof(T);
  const bool aligned = ldx % VEC == 0 && ldo % VEC == 0 && (!RES || ldr % VEC == 0);
  const T* xt = static_cast<const T*>(x);
  const T* rt = static_cast<const T*>(res);
  T* ot = static_cast<T*>(out);
  if (aligned) k_dropout<T, RES, true><<<grid, 256, 0, st>>>(xt, ldx, rt, ldr, ot, ldo, groups, per_row, (int)cols, a);
  else k_dropout<T, RES, false><<<grid, 256, 0, st>>>(xt, ldx, rt, ldr, ot, ldo, groups, per_row, (int)cols, a);
}

hipError_t launch_dropout(bool is_bf16, int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual,
                          int64_t ldr, void* out, int64_t ldo, const DropArgs& a, hipStream_t st) {
  if (is_bf16) {
    if (residual) dropout_for<bf16, true>(rows, cols, x, ldx, residual, ldr, out, ldo, a, st);
    else dropout_for<bf16, false>(rows, cols, x, ldx, residual, ldr, out, ldo, a, st);
  } else {
    if (residual) dropout_for<float, true>(rows, cols, x, ldx, residual, ldr, out, ldo, a, st);
    else dropout_for<float, false>(rows, cols, x, ldx, residual, ldr, out, ldo, a, st);
  }
  return hipGetLastError();
}

}  // namespace moe
