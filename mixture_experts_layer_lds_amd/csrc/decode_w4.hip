// The MoE layer for a few tokens with 4-bit expert weights (w4.h): router logits, top-K with softmax, the
// chosen experts' SwiGLU FFNs, the weighted combine.
//
// A few short launches on the caller's stream, not one with grid-wide barriers: a launch that waits for
// the one before costs about 2 us, a barrier of the whole chip and the phases' uneven ends cost more.
//
// By pairs (few tokens for the experts, so that hardly two choose the same one): three launches.
//   1. router logits, the reduction cut into slices whose sums the next launch adds;
//   2. gate/up: a workgroup takes 16 columns of one (token, choice) pair.  Its first wave finds the pair's
//      expert from the token's logits while the others copy the token to LDS, so that top-K needs no launch;
//      one workgroup of a token writes its logits, choices and weights;
//   3. down: a workgroup takes 16 output columns of a token, its waves the token's experts; their results are
//      added in ascending expert order with their weights, in LDS.
// DeepSeek-V3-shaped layer, T = 1, fp4: 4.8 + 32 + 18 us for 191 MB (up at 3.9 TB/s, down at 3.7: each launch has
// some 3 us of choosing, first loads and sums in which no codes arrive); fine-grained layer, T = 8, int4/64: 3.7 + 12 + 7.
// By experts (more tokens): five launches.  1. router logits, which also clear the experts' counters; 2. top-K,
// each pair appended to its expert's list (the order inside a list reaches no value); 3. gate/up and
// 4. down on groups of 16 of an expert's tokens; 5. combine in ascending expert order.
// d = 7168, n = 2048, E = 64, T = 16, fp4: 312 us for 1.33 GB, 4.3 TB/s.
#include <cmath>

#include "internal.h"
#include "skinny.h"
#include "topk_wave.h"
#include "w4.h"

namespace moe {

struct DecW4 {
  const bf16 *X, *W_r;
  const float* bias;
  const uint8_t *gate, *up, *down;
  const uint8_t *s_gate, *s_up, *s_down;
  float* logits;
  int32_t* topk_idx;
  float* topk_w;
  bf16* out;
  int32_t* cnt;   // [E]
  int32_t* list;  // [E][T] pair ids t * K + k
  bf16* act;      // [T * K][n], the activation rounded as in the layer's other forms: the MFMAs of down take bf16
  float* y;       // [T * K][d]
  float* part;    // [slices][T][E] sums of slices of the router logits (one slice: they are the logits)
  int T, d, n, E, K, slices;
};

// ---- 1. router logits: a workgroup takes 16 experts, up to 48 tokens and a slice of d, its waves share it ----
constexpr int DW_LOGIT_WAVES = 4, DW_NG = 3, DW_SLICES = 8;

template <int NG>
__device__ __forceinline__ void dw_logit_rows(const bf16* wrow, const bf16* const* xrow, int a, int b, f32x4* acc) {
  const int ko = ((threadIdx.x & 63) >> 4) * DecMma<bf16>::V;
  DecStream<bf16, NG> ds;
  ds.w = wrow + ko;
#pragma unroll
  for (int g = 0; g < NG; ++g) ds.x[g] = xrow[g] + ko;
  dec_stream<bf16, NG>(ds, a, b, acc);
}

__global__ __launch_bounds__(DW_LOGIT_WAVES * 64) void k_dw4_logits(DecW4 a, bool lists) {
  __shared__ f32x4 red[DW_LOGIT_WAVES][DW_NG][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  if (lists && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int i = threadIdx.x; i < a.E; i += DW_LOGIT_WAVES * 64) a.cnt[i] = 0;
  const int e0 = blockIdx.x * 16, g0 = blockIdx.y * DW_NG;
  const int ng = min(DW_NG, (a.T + 15) / 16 - g0);
  const bf16* wrow = a.W_r + (int64_t)min(e0 + r16, a.E - 1) * a.d;
  const bf16* xrow[DW_NG];
#pragma unroll
  for (int g = 0; g < DW_NG; ++g) xrow[g] = a.X + (int64_t)min((g0 + g) * 16 + r16, a.T - 1) * a.d;
  f32x4 acc[DW_NG];
#pragma unroll
  for (int g = 0; g < DW_NG; ++g) acc[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int ns = a.d / DecMma<bf16>::S, parts = gridDim.z * DW_LOGIT_WAVES, p = blockIdx.z * DW_LOGIT_WAVES + wave;
  const int s0 = ns * p / parts, s1 = ns * (p + 1) / parts;
  if (ng == 3) dw_logit_rows<3>(wrow, xrow, s0, s1, acc);
  else if (ng == 2) dw_logit_rows<2>(wrow, xrow, s0, s1, acc);
  else dw_logit_rows<1>(wrow, xrow, s0, s1, acc);
#pragma unroll
  for (int g = 0; g < DW_NG; ++g) red[wave][g][lane] = acc[g];
  __syncthreads();
  if (wave < ng) {
    f32x4 v = red[0][wave][lane];
    for (int w = 1; w < DW_LOGIT_WAVES; ++w) v += red[w][wave][lane];
    const int t = (g0 + wave) * 16 + r16;
    const bool whole = gridDim.z == 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + 4 * q + i;
      if (t >= a.T || e >= a.E) continue;
      if (whole) a.logits[(int64_t)t * a.E + e] = v[i] + (a.bias ? a.bias[e] : 0.0f);
      else a.part[((int64_t)blockIdx.z * a.T + t) * a.E + e] = v[i];
    }
  }
}

// The first K choices of token t by one wave; lane k returns the k-th expert.  WRITE (then K is the layer's):
// also writes the logits where they lie in slices, the choices and the weights.
template <int EJ, bool WRITE>
__device__ __forceinline__ int dw_choose_ej(const DecW4& a, int t, int K) {
  const int lane = threadIdx.x & 63;
  int e;
  float v;
  wave_select<EJ>([&](int i) {
    const int64_t at = (int64_t)t * a.E + i;
    if (a.slices == 1) return a.logits[at];
    float p[DW_SLICES];
#pragma unroll
    for (int s = 0; s < DW_SLICES; ++s) p[s] = s < a.slices ? a.part[(int64_t)s * a.T * a.E + at] : 0.0f;
    float l = p[0];
#pragma unroll
    for (int s = 1; s < DW_SLICES; ++s) l += p[s];
    if (a.bias) l += a.bias[i];
    if (WRITE) a.logits[at] = l;
    return l;
  }, a.E, K, e, v);
  if (WRITE) {
    const float ex = lane < K ? __expf(v - __shfl(v, 0, WAVE)) : 0.0f;
    const float sum = wave_sum(ex);
    if (lane < K) {
      a.topk_idx[(int64_t)t * K + lane] = e;
      a.topk_w[(int64_t)t * K + lane] = ex / sum;
    }
  }
  return e;
}
template <bool WRITE>
__device__ __forceinline__ int dw_choose(const DecW4& a, int t, int K) {
  if (a.E <= 128) return dw_choose_ej<2, WRITE>(a, t, K);
  if (a.E <= 256) return dw_choose_ej<4, WRITE>(a, t, K);
  return dw_choose_ej<16, WRITE>(a, t, K);
}

// A token's choices by expert id: order[r] is the choice of the r-th smallest expert.  mine: lane k holds the k-th
// choice; no two are the same.
__device__ __forceinline__ void dw_order(int mine, int K, int (&order)[16]) {
  const int lane = threadIdx.x & 63;
  int rank = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < K) rank += __builtin_amdgcn_readlane(mine, k) < mine ? 1 : 0;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    order[r] = r < K ? (int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < K && rank == r) | (1ull << 63)) : 0;
}

// ---- by pairs ----
// gate/up of a pair: 16 gate rows and their up rows
template <int FMT, int G, bool XLDS>
__global__ __launch_bounds__(256) void k_dw4_up_pair(DecW4 a) {
  extern __shared__ __attribute__((aligned(16))) char dw_lds[];
  __shared__ int chosen;
  typedef W4Stream<FMT, G, 1, 2, 1, XLDS ? W4_XLDS : W4_XMEM, 1> Stream;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W_ = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int pair = blockIdx.y, t = pair / a.K, k = pair - t * a.K, j0 = blockIdx.x * 16;
  const bf16* x = a.X + (int64_t)t * a.d;
  bf16* xl = reinterpret_cast<bf16*>(dw_lds);
  const int nb = w4_blocks(a.d), b0 = nb * wave / W_, b1 = nb * (wave + 1) / W_;
  W4Stage<1> stage;
  if constexpr (XLDS) stage.request(x, xl, b0 * W4_BLOCK, min(b1 * W4_BLOCK, a.d));
  if (wave == 0) {
    const int e = blockIdx.x == 0 && k == 0 ? dw_choose<true>(a, t, a.K) : dw_choose<false>(a, t, k + 1);
    if (lane == k) chosen = e;
  }
  if constexpr (XLDS) stage.write();
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(chosen);
  const int64_t row = (int64_t)e * a.n + j0 + r16;
  Stream ws;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    ws.w[r] = (r == 0 ? a.gate : a.up) + row * (a.d / 2) + 16 * q;
    ws.s[r] = (r == 0 ? a.s_gate : a.s_up) + (FMT == W4_INT ? row * 2 : row * 4 + q);
  }
  ws.plane = (int64_t)a.E * a.n * (FMT == W4_INT ? 2 : 4);
  ws.x[0] = (XLDS ? xl : x) + Stream::XQ * q;
  ws.K = a.d;
  f32x4 acc[2][1] = {{{0.0f, 0.0f, 0.0f, 0.0f}}, {{0.0f, 0.0f, 0.0f, 0.0f}}};
  if (b0 < b1) ws.run(b0, b1, acc);
  __syncthreads();
  float* res = reinterpret_cast<float*>(dw_lds);  // [wave][gate, up][16]
  if (q < 2) res[(wave * 2 + q) * 16 + r16] = q == 0 ? acc[0][0][0] : acc[1][0][0];
  __syncthreads();
  if (threadIdx.x < 16) {
    float g = 0.0f, u = 0.0f;
    for (int w = 0; w < W_; ++w) {
      g += res[w * 32 + threadIdx.x];
      u += res[w * 32 + 16 + threadIdx.x];
    }
    a.act[(int64_t)pair * a.n + j0 + threadIdx.x] = from_f32<bf16>(g * sigmoid_f32(g) * u);
  }
}

// down and combine of a token: 16 output columns, `splits` waves per choice
template <int FMT, int G, bool XLDS>
__global__ __launch_bounds__(1024) void k_dw4_down_pair(DecW4 a, int splits) {
  extern __shared__ __attribute__((aligned(16))) char dw_lds[];
  typedef W4Stream<FMT, G, 1, 1, 1, XLDS ? W4_XLDS : W4_XMEM, 1> Stream;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int t = blockIdx.y, c0 = blockIdx.x * 16, k = wave / splits, part = wave - k * splits;
  const int64_t choice = (int64_t)t * a.K + min(lane, a.K - 1);
  const int ids = a.topk_idx[choice];
  const float weights = a.topk_w[choice];
  const bf16* x = a.act + ((int64_t)t * a.K + k) * a.n;
  bf16* xl = reinterpret_cast<bf16*>(dw_lds) + (int64_t)k * a.n;
  const int nb = w4_blocks(a.n), b0 = nb * part / splits, b1 = nb * (part + 1) / splits;
  W4Stage<4> stage;
  if constexpr (XLDS) stage.request(x, xl, b0 * W4_BLOCK, min(b1 * W4_BLOCK, a.n));
  const int64_t row = (int64_t)__builtin_amdgcn_readlane(ids, k) * a.d + c0 + r16;
  Stream ws;
  ws.w[0] = a.down + row * (a.n / 2) + 16 * q;
  ws.s[0] = a.s_down + (FMT == W4_INT ? row * 2 : row * 4 + q);
  ws.plane = (int64_t)a.E * a.d * (FMT == W4_INT ? 2 : 4);
  ws.x[0] = (XLDS ? xl : x) + Stream::XQ * q;
  ws.K = a.n;
  f32x4 acc[1][1] = {{{0.0f, 0.0f, 0.0f, 0.0f}}};
  if (b0 < b1)
    ws.run(b0, b1, acc, [&] {
      if constexpr (XLDS) stage.write();
    });
  __syncthreads();
  float* res = reinterpret_cast<float*>(dw_lds);  // [wave][16]
  if (q == 0) res[wave * 16 + r16] = acc[0][0][0];
  __syncthreads();
  if (wave == 0) {
    int order[16];
    dw_order(ids, a.K, order);
    float o = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (r < a.K) {
        float y = 0.0f;
        for (int s = 0; s < splits; ++s) y += res[(order[r] * splits + s) * 16 + r16];
        o = fmaf(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weights), order[r])), y, o);
      }
    if (lane < 16) a.out[(int64_t)t * a.d + c0 + lane] = from_f32<bf16>(o);
  }
}

// ---- by experts ----
__global__ __launch_bounds__(256) void k_dw4_topk(DecW4 a) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= a.T) return;
  const int e = dw_choose<true>(a, t, a.K);
  if (lane < a.K) a.list[(int64_t)e * a.T + atomicAdd(&a.cnt[e], 1)] = t * a.K + lane;  // (a token picks an expert at most once)
}

// A tile of an expert against groups of 16 of its tokens, the waves sharing the reduction.  UP: 8 RT gate rows
// and their up rows -> act; else 16 RT rows of W_down -> y.
constexpr int DW_RT = 4, DW_EXPERT_WAVES = 4;
template <int FMT, int G, bool UP>
__global__ __launch_bounds__(512) void k_dw4_expert(DecW4 a) {
  extern __shared__ __attribute__((aligned(16))) char dw_lds[];
  constexpr int RT = DW_RT, H = RT / 2, TILE = 256;
  typedef W4Stream<FMT, G, 1, RT, 4, W4_XLINE, 1> Stream;
  static_assert(RT * TILE * 4 == W4_XSLOT, "a wave's tokens and results take the same place");
  const int e = blockIdx.y, c = __builtin_amdgcn_readfirstlane(a.cnt[e]);
  if (c == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W_ = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int rows = UP ? a.n : a.d, K = UP ? a.d : a.n;  // of an expert; multiples of 64, as the tiles' columns divide
  const int c0 = blockIdx.x * (UP ? 16 * H : 16 * RT);
  const int32_t* lst = a.list + (int64_t)e * a.T;
  Stream ws;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t row = (int64_t)e * rows + c0 + 16 * (UP ? r % H : r) + r16;
    const uint8_t* w = UP ? (r < H ? a.gate : a.up) : a.down;
    const uint8_t* s = UP ? (r < H ? a.s_gate : a.s_up) : a.s_down;
    ws.w[r] = w + row * (K / 2) + 16 * q;
    ws.s[r] = s + (FMT == W4_INT ? row * 2 : row * 4 + q);
  }
  ws.plane = (int64_t)a.E * rows * (FMT == W4_INT ? 2 : 4);
  ws.K = K;
  const int nb = w4_blocks(K), b0 = nb * wave / W_, b1 = nb * (wave + 1) / W_;
  ws.xb = reinterpret_cast<const char*>(UP ? a.X : a.act);
  ws.xs = dw_lds + wave * W4_XSLOT;
  float* res = reinterpret_cast<float*>(dw_lds);  // [wave][RT][token][16]
  for (int g0 = 0; g0 < c; g0 += 16) {
    if (g0 > 0) __syncthreads();  // (the last group's results, where the waves put their tokens, have been read)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = lst[min(g0 + 4 * i + q, c - 1)];
      ws.xo[0][i] = (uint32_t)(UP ? pair / a.K : pair) * (uint32_t)(K * 2) + 16 * r16;  // (below 2^31: T <= 1024, K <= 16)
    }
    f32x4 acc[RT][1];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (b0 < b1) ws.run(b0, b1, acc);
    w4_lds_order();
#pragma unroll
    for (int r = 0; r < RT; ++r) w4_put<4>(res + (wave * RT + r) * TILE, acc[r][0]);
    __syncthreads();
    auto total = [&](int r, int at) {
      const float* p = res + r * TILE + at;
      f32x4 v = *reinterpret_cast<const f32x4*>(p);
      for (int w = 1; w < W_; ++w) v += *reinterpret_cast<const f32x4*>(p + w * RT * TILE);
      return v;
    };
    constexpr int QUADS = UP ? 4 * H : 4 * RT;  // of a token's columns
    for (int it = threadIdx.x; it < 16 * QUADS; it += blockDim.x) {
      const int quad = it % QUADS, tok = it / QUADS, col = c0 + 4 * quad, r = quad >> 2, at = tok * 16 + 4 * (quad & 3);
      if (g0 + tok >= c) continue;
      const int64_t to = lst[g0 + tok];
      if constexpr (UP) {
        const f32x4 g = total(r, at), u = total(r + H, at);
        f32x4 h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = g[i] * sigmoid_f32(g[i]) * u[i];
        dec_store4<bf16>(a.act + to * a.n + col, h);
      } else {
        *reinterpret_cast<f32x4*>(a.y + to * a.d + col) = total(r, at);
      }
    }
  }
}

__global__ __launch_bounds__(256) void k_dw4_combine(DecW4 a) {
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
  int order[16];
  dw_order(a.topk_idx[(int64_t)t * a.K + min((int)threadIdx.x & 63, a.K - 1)], a.K, order);
  if (c >= a.d) return;
  f32x4 yv[16];
  float wv[16];
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (r < a.K) {
      const int64_t p = (int64_t)t * a.K + order[r];
      wv[r] = a.topk_w[p];
      yv[r] = *reinterpret_cast<const f32x4*>(a.y + p * a.d + c);
    }
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (r < a.K) s += wv[r] * yv[r];
  dec_store4<bf16>(a.out + (int64_t)t * a.d + c, s);
}

constexpr int64_t DW_LDS = 65536;

// Whether the call goes by pairs: that saves two launches, and reads an expert again for every further pair
// that chose it (from the caches, mostly).  Where half as many pairs as experts at most are routed pairs are never
// slower (d = 7168, n = 2048, E = 64, T = 4: 154 and 161 us), beyond that the expected repeated bytes decide: d =
// 1536, n = 256, E = 128, K = 8 int4 takes 32 and 41 us at T = 16 (28 MB), 42 and 45 at 24 (54 MB), 50 and 46 at 32
// (86 MB); d = 7168, n = 2048, E = 64 289 and 259 at T = 8 (514 MB).
static bool dw4_pairs(const Shape& s) {
  const double P = (double)s.T * s.K, E = s.E;
  if (P > 1024) return false;
  const double again = P - E * (1.0 - pow(1.0 - 1.0 / E, P));
  return s.T == 1 || 2 * P <= E || again * 1.5 * (double)s.n * (double)s.d <= 64e6;
}

template <int FMT, int G>
static hipError_t dw4_run(const DecW4& a, bool pairs, hipStream_t st) {
  const dim3 lg((unsigned)cdiv(a.E, 16), (unsigned)cdiv(a.T, 16 * DW_NG), (unsigned)a.slices);
  k_dw4_logits<<<lg, DW_LOGIT_WAVES * 64, 0, st>>>(a, !pairs);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pairs) {
    const int nb = w4_blocks(a.d);
    int waves = 4;
    while (waves > 1 && nb / waves < 3) waves /= 2;
    const dim3 ug((unsigned)(a.n / 16), (unsigned)(a.T * a.K));
    const int64_t xl = (int64_t)a.d * 2;
    if (xl <= DW_LDS) k_dw4_up_pair<FMT, G, true><<<ug, waves * 64, xl < 1024 ? 1024 : xl, st>>>(a);
    else k_dw4_up_pair<FMT, G, false><<<ug, waves * 64, 1024, st>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    // waves per choice: up to 8 waves in all, so that the chip holds three workgroups a CU
    const int nd = w4_blocks(a.n);
    int splits = 1;
    while (a.K * splits * 2 <= 8 && nd / (splits * 2) >= 4) splits *= 2;
    const dim3 dg((unsigned)(a.d / 16), (unsigned)a.T);
    const int64_t al = (int64_t)a.K * a.n * 2;
    if (al <= DW_LDS) k_dw4_down_pair<FMT, G, true><<<dg, a.K * splits * 64, al < 1024 ? 1024 : al, st>>>(a, splits);
    else k_dw4_down_pair<FMT, G, false><<<dg, a.K * splits * 64, 1024, st>>>(a, splits);
    return hipGetLastError();
  }
  k_dw4_topk<<<(unsigned)cdiv(a.T, 4), 256, 0, st>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  auto waves_of = [](int K) {
    int w = DW_EXPERT_WAVES;
    while (w > 1 && w4_blocks(K) / w < 2) w /= 2;
    return w;
  };
  const int wu = waves_of(a.d), wd = waves_of(a.n), lds = DW_RT * 1024;  // per wave
  k_dw4_expert<FMT, G, true><<<dim3((unsigned)(a.n / (8 * DW_RT)), (unsigned)a.E), wu * 64, wu * lds, st>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_dw4_expert<FMT, G, false><<<dim3((unsigned)(a.d / (16 * DW_RT)), (unsigned)a.E), wd * 64, wd * lds, st>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_dw4_combine<<<dim3((unsigned)cdiv(a.d, 1024), (unsigned)a.T), 256, 0, st>>>(a);
  return hipGetLastError();
}

static size_t dw_align(size_t b) { return (b + 255) / 256 * 256; }
hipError_t launch_decode_w4(const Shape& s, const void* X, const void* W_r, const float* bias, const W4View& W_gate,
                            const W4View& W_up, const W4View& W_down, float* logits, int32_t* topk_idx, float* topk_w, void* out,
                            void* ws, hipStream_t st) {
  DecW4 a;
  a.X = static_cast<const bf16*>(X);
  a.W_r = static_cast<const bf16*>(W_r);
  a.bias = bias;
  a.gate = W_gate.codes;
  a.up = W_up.codes;
  a.down = W_down.codes;
  a.s_gate = static_cast<const uint8_t*>(W_gate.scales);
  a.s_up = static_cast<const uint8_t*>(W_up.scales);
  a.s_down = static_cast<const uint8_t*>(W_down.scales);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.out = static_cast<bf16*>(out);
  a.T = (int)s.T; a.d = (int)s.d; a.n = (int)s.n; a.E = s.E; a.K = s.K;
  char* w = static_cast<char*>(ws);  // (moe_decode's workspace holds more)
  a.cnt = reinterpret_cast<int32_t*>(w);
  w += dw_align((size_t)s.E * 4);
  a.act = reinterpret_cast<bf16*>(w);
  w += dw_align((size_t)s.T * s.K * s.n * 2);
  a.list = reinterpret_cast<int32_t*>(w);
  w += dw_align((size_t)s.E * s.T * 4);
  a.y = reinterpret_cast<float*>(w);
  // slices of the logits lie where y will be written, by pairs over the unused lists too; each has at least 8
  // steps of the reduction
  const bool pairs = dw4_pairs(s);
  a.part = pairs ? reinterpret_cast<float*>(a.list) : a.y;
  const int64_t room = (int64_t)s.K * s.d + (pairs ? s.E : 0);  // floats per token
  a.slices = 1;
  while (a.slices < DW_SLICES && s.d / 32 / (a.slices * 2) >= 8 && (int64_t)s.E * a.slices * 2 <= room) a.slices *= 2;
  if (W_gate.format == W4_FP) return dw4_run<W4_FP, 32>(a, pairs, st);
  if (W_gate.group == 32) return dw4_run<W4_INT, 32>(a, pairs, st);
  if (W_gate.group == 64) return dw4_run<W4_INT, 64>(a, pairs, st);
  return dw4_run<W4_INT, 128>(a, pairs, st);
}

}  // namespace moe
