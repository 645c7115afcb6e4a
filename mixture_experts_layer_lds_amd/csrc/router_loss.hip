// Router losses: the balance loss with its per-expert counts, the z-loss, and their gradient with
// respect to the logits.
//
// With p_t = softmax(logits_t) over all experts, l_t = log sum exp(logits_t), c_se the picks of
// expert e among sequence s's top-K choices, T_s its counting tokens, P_se = sum_t p_te over
// them and N = sum_s T_s:
//   balance = sum_s (T_s / N) E sum_e (c_se / (K T_s)) (P_se / T_s),   z = (1 / N) sum_t l_t^2
//   d balance / d logits_te = E / (K T_s N) p_te (c_se - sum_j c_sj p_tj),  d z = 2 l_t p_te / N
// A sequence is a run of tokens seq_off[s] .. seq_off[s+1] - 1; a token counts if it lies in one
// and its mask byte is not zero.
//
// Forward: one workgroup per chunk of 64 tokens reads the logits once (the only large operand).
// Where a chunk holds several sequences it is cut into pieces, and the piece of chunk c and
// sequence s leaves its partial sums in slot c + s: along the tokens either c or s grows from one
// piece to the next, so slots never collide, and the number of pieces needs no host knowledge.  A
// second launch adds the slots of a sequence in chunk order (in 64 bits), and its last workgroup
// forms the two losses.  No floating-point atomics: the order of every sum is fixed.
//
// A token is taken by G lanes, each holding up to 4 NV of its logits (four consecutive ones per
// 16-byte load where E is a multiple of 4), so that a wave reads whole rows whatever E is; the
// row's maximum and sum are exchanged within the G lanes.  Probabilities, sums and statistics are
// fp32; the sums over chunks are fp64.
#include "internal.h"

namespace moe {

constexpr int RL_CHUNK = 64;     // tokens per workgroup
constexpr int RL_THREADS = 256;
constexpr int RL_WAVES = RL_THREADS / 64;
constexpr int RL_JOIN_COLS = 32;      // columns per workgroup of the joining launch
constexpr int RL_JOIN_THREADS = 1024;

struct RlossWs {
  unsigned* ticket;  // workgroups of the joining launch that have finished
  float* prob;       // [slots][E]
  int32_t* cnt;      // [slots][E]
  int32_t* tok;      // [slots]
  float* z;          // [slots]
  double* bal;       // [n_seq][column blocks]
  double* zs;        // [n_seq]
};

static int64_t rl_chunks(int64_t T) { return cdiv(T, RL_CHUNK); }
static int rl_colblocks(int E) { return (E + RL_JOIN_COLS - 1) / RL_JOIN_COLS; }

static size_t rl_carve(void* base, int64_t T, int E, int n_seq, RlossWs* w) {
  char* b = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = b ? b + off : nullptr;
    off = align_up(off + bytes, 256);
    return p;
  };
  const size_t slots = (size_t)(rl_chunks(T) + n_seq);
  RlossWs q;
  q.ticket = reinterpret_cast<unsigned*>(take(sizeof(unsigned)));
  q.prob = reinterpret_cast<float*>(take(slots * E * 4));
  q.cnt = reinterpret_cast<int32_t*>(take(slots * E * 4));
  q.tok = reinterpret_cast<int32_t*>(take(slots * 4));
  q.z = reinterpret_cast<float*>(take(slots * 4));
  q.bal = reinterpret_cast<double*>(take((size_t)n_seq * rl_colblocks(E) * 8));
  q.zs = reinterpret_cast<double*>(take((size_t)n_seq * 8));
  if (w) *w = q;
  return off;
}

size_t router_loss_workspace_bytes(int64_t T, int E, int n_seq) { return rl_carve(nullptr, T, E, n_seq, nullptr); }

// Sequence s's bounds, kept within [0, T] so that a bad table reads nothing out of bounds.
__device__ __forceinline__ int rl_off(const int32_t* seq_off, int s, int T) {
  return seq_off ? min(max(seq_off[s], 0), T) : (s ? T : 0);
}

// The piece of the chunk [.., end) that starts at token t: its sequence (-1: outside all of them)
// and its end.
__device__ __forceinline__ int rl_piece(const int32_t* seq_off, int n_seq, int T, int t, int end, int& stop) {
  int lo = 0, hi = n_seq;  // the first s with seq_off[s + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (rl_off(seq_off, mid + 1, T) > t) hi = mid;
    else lo = mid + 1;
  }
  if (lo >= n_seq) {
    stop = end;
    return -1;
  }
  const int b = rl_off(seq_off, lo, T);
  if (t < b) {
    stop = min(end, b);
    return -1;
  }
  stop = min(end, max(rl_off(seq_off, lo + 1, T), t + 1));
  return lo;
}

__device__ __forceinline__ float rl_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896f); }

// A lane's share of a row of E logits: element i of 4 NV sits in column col(i).
template <int G, int NV, bool V4>
struct RlRow {
  static constexpr int N = 4 * NV;
  __device__ static int col(int li, int i) { return V4 ? (li + G * (i >> 2)) * 4 + (i & 3) : li + G * i; }
  __device__ static void load(const float* row, int li, int E, float (&x)[N]) {
    if constexpr (V4) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (li + G * j) * 4;
        const f32x4 v = c < E ? *reinterpret_cast<const f32x4*>(row + c)
                              : f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < 4; ++u) x[4 * j + u] = v[u];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = li + G * i < E ? row[li + G * i] : -INFINITY;
    }
  }
  __device__ static void store(float* row, int li, int E, const float (&x)[N]) {
    if constexpr (V4) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (li + G * j) * 4;
        if (c < E) __builtin_nontemporal_store(f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]}, reinterpret_cast<f32x4*>(row + c));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (li + G * i < E) row[li + G * i] = x[i];
    }
  }
};
template <int G>
__device__ __forceinline__ float rl_group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int G>
__device__ __forceinline__ float rl_group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

template <int G, int NV, bool V4>
__global__ __launch_bounds__(RL_THREADS) void k_rloss_part(const float* __restrict__ logits,
                                                           const int32_t* __restrict__ topk_idx, int T, int E, int K,
                                                           int n_seq, const int32_t* __restrict__ seq_off,
                                                           const uint8_t* __restrict__ mask, float* __restrict__ lse,
                                                           RlossWs w) {
  using Row = RlRow<G, NV, V4>;
  constexpr int N = Row::N, TPW = 64 / G;
  extern __shared__ float rl_lds[];  // [waves][E] probability sums, [E] counts
  int* hist = reinterpret_cast<int*>(rl_lds + RL_WAVES * E);
  __shared__ float sz[RL_WAVES];
  __shared__ int sn[RL_WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane % G, grp = lane / G;
  const int t_begin = blockIdx.x * RL_CHUNK, t_end = min(T, t_begin + RL_CHUNK);
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0u;
  for (int a = t_begin, b; a < t_end; a = b) {
    const int s = rl_piece(seq_off, n_seq, T, a, t_end, b);
    for (int e = threadIdx.x; e < E; e += RL_THREADS) hist[e] = 0;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    int n = 0;
    for (int t = a + wave * TPW + grp; t < b; t += RL_WAVES * TPW) {  // uniform within a group of G lanes
      float x[N];
      Row::load(logits + (int64_t)t * E, li, E, x);
      float m = x[0];
#pragma unroll
      for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
      m = rl_group_max<G>(m);
      // a row of -infinity only (every expert masked) has no probabilities: its sum is zero, its
      // log-sum-exp -infinity, and it adds to neither loss; a NaN or +infinity makes the row NaN
      m = m == -INFINITY ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = rl_exp(x[i] - m);
        sum += x[i];
      }
      sum = rl_group_sum<G>(sum);
      const float l = m + __logf(sum);
      if (li == 0) lse[t] = l;
      if (s >= 0 && (!mask || mask[t])) {
        ++n;
        if (sum != 0.0f) {
          const float inv = 1.0f / sum;
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] += x[i] * inv;
          z += l * l;
        }
      }
    }
    if (s < 0) continue;  // (uniform) tokens outside every sequence only get their log-sum-exp
    __syncthreads();      // the histogram is clear
    for (int i = threadIdx.x; i < (b - a) * K; i += RL_THREADS) {
      const int t = a + i / K;
      const int e = topk_idx[(int64_t)a * K + i];
      if ((uint32_t)e < (uint32_t)E && (!mask || mask[t])) atomicAdd(&hist[e], 1);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int o = G; o < 64; o <<= 1) acc[i] += __shfl_xor(acc[i], o, 64);
      if (grp == 0 && Row::col(li, i) < E) rl_lds[wave * E + Row::col(li, i)] = acc[i];
    }
    // every lane of a group holds its tokens' count and z: take one lane per group
    z = wave_sum(li == 0 ? z : 0.0f);
    n = wave_sum_i(li == 0 ? n : 0);
    if (lane == 0) {
      sz[wave] = z;
      sn[wave] = n;
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += RL_THREADS) {
      w.prob[slot * E + e] = (rl_lds[e] + rl_lds[E + e]) + (rl_lds[2 * E + e] + rl_lds[3 * E + e]);
      w.cnt[slot * E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      w.z[slot] = (sz[0] + sz[1]) + (sz[2] + sz[3]);
      w.tok[slot] = sn[0] + sn[1] + sn[2] + sn[3];
    }
    __syncthreads();  // the LDS is free for the next piece
  }
}

// Adds a sequence's slots in chunk order: 32 columns by 32 runs of chunks per workgroup, then the
// runs in order.  The last workgroup to finish forms the losses.
__global__ __launch_bounds__(RL_JOIN_THREADS) void k_rloss_join(int T, int E, int K, int n_seq,
                                                                const int32_t* __restrict__ seq_off, RlossWs w,
                                                                int32_t* __restrict__ seq_tokens,
                                                                int32_t* __restrict__ seq_counts,
                                                                float* __restrict__ prob_sum, float* __restrict__ loss) {
  constexpr int RUNS = RL_JOIN_THREADS / RL_JOIN_COLS;
  __shared__ double sp[RUNS][RL_JOIN_COLS + 1];
  __shared__ int sc[RUNS][RL_JOIN_COLS + 1];
  __shared__ double rz[16], rb[16];
  __shared__ long long rn[16];
  __shared__ int last;
  const int cbs = (E + RL_JOIN_COLS - 1) / RL_JOIN_COLS;
  const int s = blockIdx.x / cbs, cb = blockIdx.x % cbs;
  const int lo = rl_off(seq_off, s, T), hi = rl_off(seq_off, s + 1, T);
  const int c0 = lo / RL_CHUNK, c1 = hi > lo ? (hi - 1) / RL_CHUNK + 1 : c0;  // chunks c0 .. c1 - 1
  const int ci = threadIdx.x % RL_JOIN_COLS, run = threadIdx.x / RL_JOIN_COLS;
  const int e = cb * RL_JOIN_COLS + ci;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double p = 0.0;
  int cnt = 0;
  if (e < E)
    for (int c = c0 + run; c < c1; c += RUNS) {
      const int64_t i = (int64_t)(c + s) * E + e;
      p += (double)w.prob[i];
      cnt += w.cnt[i];
    }
  sp[run][ci] = p;
  sc[run][ci] = cnt;
  if (cb == 0) {  // the sequence's tokens and z sum
    double z = 0.0;
    long long n = 0;
    for (int c = c0 + (int)threadIdx.x; c < c1; c += RL_JOIN_THREADS) {
      z += (double)w.z[c + s];
      n += w.tok[c + s];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      z += __shfl_xor(z, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if (lane == 0) {
      rz[wave] = z;
      rn[wave] = n;
    }
  }
  __syncthreads();
  if (threadIdx.x < RL_JOIN_COLS) {
    double ps = 0.0;
    int cs = 0;
    for (int r = 0; r < RUNS; ++r) {
      ps += sp[r][ci];
      cs += sc[r][ci];
    }
    if (e < E) {
      prob_sum[(int64_t)s * E + e] = (float)ps;
      seq_counts[(int64_t)s * E + e] = cs;
    }
    double bsum = e < E ? ps * (double)cs : 0.0;
#pragma unroll
    for (int o = RL_JOIN_COLS / 2; o > 0; o >>= 1) bsum += __shfl_xor(bsum, o, 64);
    if (threadIdx.x == 0) w.bal[(int64_t)s * cbs + cb] = bsum;
  }
  if (cb == 0 && threadIdx.x == 0) {
    double z = 0.0;
    long long n = 0;
    for (int q = 0; q < 16; ++q) {
      z += rz[q];
      n += rn[q];
    }
    w.zs[s] = z;
    seq_tokens[s] = (int)n;
  }
  // the last workgroup sums over the sequences
  __syncthreads();
  if (threadIdx.x == 0) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    const unsigned v = __hip_atomic_fetch_add(w.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = v == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  double bsum = 0.0, zsum = 0.0;
  long long n = 0;
  for (int q = threadIdx.x; q < n_seq; q += RL_JOIN_THREADS) {
    double bq = 0.0;
    for (int k = 0; k < cbs; ++k) bq += w.bal[(int64_t)q * cbs + k];
    const int tq = seq_tokens[q];
    if (tq > 0) bsum += bq / (double)tq;
    zsum += w.zs[q];
    n += tq;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    bsum += __shfl_xor(bsum, o, 64);
    zsum += __shfl_xor(zsum, o, 64);
    n += __shfl_xor(n, o, 64);
  }
  if (lane == 0) {
    rb[wave] = bsum;
    rz[wave] = zsum;
    rn[wave] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bsum = zsum = 0.0;
    n = 0;
    for (int q = 0; q < 16; ++q) {
      bsum += rb[q];
      zsum += rz[q];
      n += rn[q];
    }
    loss[0] = n ? (float)(bsum * (double)E / ((double)K * (double)n)) : 0.0f;
    loss[1] = n ? (float)(zsum / (double)n) : 0.0f;
  }
}

// dLogits, piece by piece as the forward.  The counts enter less their mean K T_s / E: the
// probabilities of a row sum to one, so the mean drops out of the difference, and without it the
// difference of two nearly equal numbers would lose the leading bits.
template <int G, int NV, bool V4>
__global__ __launch_bounds__(RL_THREADS) void k_rloss_bwd(const float* __restrict__ dloss,
                                                          const float* __restrict__ logits, int T, int E, int K,
                                                          int n_seq, const int32_t* __restrict__ seq_off,
                                                          const uint8_t* __restrict__ mask,
                                                          const int32_t* __restrict__ seq_tokens,
                                                          const int32_t* __restrict__ seq_counts,
                                                          const float* __restrict__ lse, float* __restrict__ dLogits) {
  using Row = RlRow<G, NV, V4>;
  constexpr int N = Row::N, TPW = 64 / G;
  __shared__ long long rn[RL_WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane % G, grp = lane / G;
  const int t_begin = blockIdx.x * RL_CHUNK, t_end = min(T, t_begin + RL_CHUNK);
  long long n = 0;
  for (int q = threadIdx.x; q < n_seq; q += RL_THREADS) n += seq_tokens[q];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  if (lane == 0) rn[wave] = n;
  __syncthreads();
  n = rn[0] + rn[1] + rn[2] + rn[3];
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = dloss[0] * inv_n * (float)E / (float)K, gz = dloss[1] * 2.0f * inv_n;
  for (int a = t_begin, b; a < t_end; a = b) {
    const int s = rl_piece(seq_off, n_seq, T, a, t_end, b);
    float ex[N];
    float coef = 0.0f;
    if (s >= 0) {
      const int ts = seq_tokens[s];
      coef = ts > 0 ? gb / (float)ts : 0.0f;
      const float mean = (float)((double)K * (double)ts / (double)E);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = Row::col(li, i);
        ex[i] = c < E ? (float)seq_counts[(int64_t)s * E + c] - mean : 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) ex[i] = 0.0f;
    }
    for (int t = a + wave * TPW + grp; t < b; t += RL_WAVES * TPW) {
      const float l = lse[t];
      float x[N];
      if (s >= 0 && (!mask || mask[t]) && l != -INFINITY) {
        Row::load(logits + (int64_t)t * E, li, E, x);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i] = rl_exp(x[i] - l);
          dot += x[i] * ex[i];
        }
        dot = rl_group_sum<G>(dot);
        const float zt = gz * l;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= coef * (ex[i] - dot) + zt;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.0f;
      }
      Row::store(dLogits + (int64_t)t * E, li, E, x);
    }
  }
}

// Lanes per token and 4-logit chunks per lane for E: one chunk where that leaves few idle lanes,
// else up to four.  V4 needs 16-byte aligned rows.
template <class F>
static void rl_dispatch(int E, F f) {
#define RL_CASE(GG, NN) (E % 4 == 0 ? f.template operator()<GG, NN, true>() : f.template operator()<GG, NN, false>())
  const int q = (E + 3) / 4;  // chunks per row
  if (q <= 2) RL_CASE(2, 1);
  else if (q <= 4) RL_CASE(4, 1);
  else if (q <= 8) RL_CASE(8, 1);
  else if (q <= 16) RL_CASE(16, 1);
  else if (q <= 32) RL_CASE(16, 2);
  else if (q <= 48) RL_CASE(16, 3);
  else if (q <= 64) RL_CASE(32, 2);
  else if (q <= 96) RL_CASE(32, 3);
  else if (q <= 128) RL_CASE(64, 2);
  else RL_CASE(64, 4);
#undef RL_CASE
}

namespace {
struct RlossFwd {
  const float* logits;
  const int32_t* topk_idx;
  int T, E, K, n_seq;
  const int32_t* seq_off;
  const uint8_t* mask;
  float* lse;
  RlossWs w;
  hipStream_t st;
  template <int G, int NV, bool V4>
  void operator()() const {
    k_rloss_part<G, NV, V4><<<(int)rl_chunks(T), RL_THREADS, (size_t)(RL_WAVES + 1) * E * 4, st>>>(
        logits, topk_idx, T, E, K, n_seq, seq_off, mask, lse, w);
  }
};
struct RlossBwd {
  const float *dloss, *logits;
  int T, E, K, n_seq;
  const int32_t* seq_off;
  const uint8_t* mask;
  const int32_t *seq_tokens, *seq_counts;
  const float* lse;
  float* dLogits;
  hipStream_t st;
  template <int G, int NV, bool V4>
  void operator()() const {
    k_rloss_bwd<G, NV, V4><<<(int)rl_chunks(T), RL_THREADS, 0, st>>>(dloss, logits, T, E, K, n_seq, seq_off, mask,
                                                                      seq_tokens, seq_counts, lse, dLogits);
  }
};
}  // namespace

hipError_t launch_router_loss(const float* logits, const int32_t* topk_idx, int64_t T, int E, int K, int n_seq,
                              const int32_t* seq_off, const uint8_t* mask, int32_t* seq_tokens, int32_t* seq_counts,
                              float* prob_sum, float* lse, float* loss, void* ws, hipStream_t st) {
  RlossWs w;
  rl_carve(ws, T, E, n_seq, &w);
  rl_dispatch(E, RlossFwd{logits, topk_idx, (int)T, E, K, n_seq, seq_off, mask, lse, w, st});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_rloss_join<<<n_seq * rl_colblocks(E), RL_JOIN_THREADS, 0, st>>>((int)T, E, K, n_seq, seq_off, w, seq_tokens,
                                                                    seq_counts, prob_sum, loss);
  return hipGetLastError();
}

hipError_t launch_router_loss_bwd(const float* dloss, const float* logits, int64_t T, int E, int K, int n_seq,
                                  const int32_t* seq_off, const uint8_t* mask, const int32_t* seq_tokens,
                                  const int32_t* seq_counts, const float* lse, float* dLogits, hipStream_t st) {
  rl_dispatch(E, RlossBwd{dloss, logits, (int)T, E, K, n_seq, seq_off, mask, seq_tokens, seq_counts, lse, dLogits, st});
  return hipGetLastError();
}

}  // namespace moe
