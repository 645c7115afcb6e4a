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
// Forward: one workgroup per chunk of tokens (32 or 64, more where rows are short) reads the logits
// once (the only large operand); it requests the whole chunk, its choices and the sequence
// table together before it uses any, since at these sizes the length of the chain of dependent
// loads, not their bytes, sets the time.
// Where a chunk holds several sequences it is cut into pieces, and the piece of chunk c and
// sequence s leaves its partial sums in slot c + s: along the tokens either c or s grows from one
// piece to the next, so slots never collide, and the number of pieces needs no host knowledge.  A
// second launch adds the slots of a sequence in chunk order (in 64 bits), and its last workgroup
// forms the two losses.  Where one chunk holds the whole batch, its workgroup writes the results
// itself and there is no second launch.  No floating-point atomics: the order of every sum is fixed.
// Measured: 16384 x 256 in 7 sequences 16.2 us (9.8 and 6.0 for the two launches; the 17.4 MB would
// take 3.5), 256 x 8 in one launch 5.2; backward 32768 x 384, 101 MB, 19.3 us (5.2 TB/s).
//
// A token is taken by G lanes, each holding up to 4 NV of its logits (four consecutive ones per
// 16-byte load where E is a multiple of 4), so that a wave reads whole rows whatever E is; the
// row's maximum and sum are exchanged within the G lanes.  Probabilities, sums and statistics are
// fp32; the sums over chunks are fp64.
#include "internal.h"

namespace moe {

constexpr int RL_BWD_CHUNK = 64;  // tokens per workgroup of the backward, less where T gives under two per CU
constexpr int RL_JOIN_THREADS = 512;  // (1024 threads in both launches: 16384 x 256 16.7 us, 15.9 so)
constexpr int RL_MAX_WAVES = 16;
constexpr int RL_JOIN_COLS = 32;      // columns per workgroup of the joining launch
constexpr int RL_JOIN_SEQS = 1 << 16; // sequences per grid row of it (a grid's x extent stays below 2^32 threads)
constexpr int RL_BWD_THREADS = 256;
// A chunk of more than RL_FEW pieces leaves those of up to RL_SHORT rounds of a wave's tokens to single
// waves: a piece that the whole workgroup takes costs two to three barriers and as many LDS round
// trips whatever its length (35 tokens of 379 logits in 46 sequences: 84 us so, 21 by waves; 64 x 128 in
// 64: 130 against 17).
constexpr int RL_FEW = 3;
constexpr int RL_SHORT = 8;

struct RlossWs {
  unsigned* ticket;  // workgroups of the joining launch that have finished
  float* prob;       // [slots][E]
  int32_t* cnt;      // [slots][E]
  int32_t* tok;      // [slots]
  float* z;          // [slots]
  double* bal;       // [n_seq][column blocks]
  double* zs;        // [n_seq]
};

// Lanes per token (G) and 4-logit chunks per lane (NV) for E: the fewest idle lanes, at most 16
// logits a lane.
struct RlLayout {
  int G, NV;
};
static RlLayout rl_layout(int E) {
  const int q = (E + 3) / 4;  // chunks per row
  if (q <= 2) return {2, 1};
  if (q <= 4) return {4, 1};
  if (q <= 8) return {8, 1};
  if (q <= 16) return {16, 1};
  if (q <= 32) return {16, 2};
  if (q <= 48) return {16, 3};
  if (q <= 64) return {32, 2};
  if (q <= 96) return {32, 3};
  if (q <= 128) return {64, 2};
  return {64, 4};
}
// The forward's workgroup: 16 waves where it holds the whole batch (one per short sequence), else 8.
// It takes its chunk in steps of a token per lane group; where rows are long and the longer chunks
// still give every CU one, twice as many (fewer sums to join: 32768 x 384 22.7 us against 26.4, but
// 4096 x 256 in 64 sequences 23.6 against 19.6).
__host__ __device__ constexpr int rl_waves(bool one) { return one ? 16 : 8; }
__host__ __device__ constexpr int rl_steps(int G, bool longer) { return G > 16 ? (longer ? G / 8 : G / 16) : 1; }
__host__ __device__ constexpr int rl_chunk(int G, bool one, bool longer) { return rl_waves(one) * (64 / G) * rl_steps(G, longer); }
struct RlGrid {
  bool one, longer;
  int chunk;
};
static RlGrid rl_grid(int64_t T, int E) {
  const int G = rl_layout(E).G;
  if (T <= rl_chunk(G, true, false)) return {true, false, rl_chunk(G, true, false)};
  const bool longer = G > 16 && cdiv(T, rl_chunk(G, false, true)) >= 256;
  return {false, longer, rl_chunk(G, false, longer)};
}
static int64_t rl_chunks(int64_t T, int E) { return cdiv(T, rl_grid(T, E).chunk); }
static int rl_colblocks(int E) { return (E + RL_JOIN_COLS - 1) / RL_JOIN_COLS; }

static size_t rl_carve(void* base, int64_t T, int E, int n_seq, RlossWs* w) {
  char* b = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = b ? b + off : nullptr;
    off = align_up(off + bytes, 256);
    return p;
  };
  const size_t slots = (size_t)(rl_chunks(T, E) + n_seq);
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

// The first sequence from lo on that ends after token t (n_seq: none).  off(s) gives the table's
// entries.
template <class Off>
__device__ __forceinline__ int rl_find(Off off, int n_seq, int t, int lo) {
  int hi = n_seq;
  if (lo < hi && off(lo + 1) > t) return lo;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off(mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
// The piece of a chunk that starts at token t: its sequence (-1: outside all of them) and its end,
// at most `end`.  lo: a sequence that does not lie behind t; left at the one found.
template <class Off>
__device__ __forceinline__ int rl_piece(Off off, int n_seq, int t, int end, int& stop, int& lo) {
  lo = rl_find(off, n_seq, t, lo);
  if (lo >= n_seq) {
    stop = end;
    return -1;
  }
  const int b = off(lo);
  if (t < b) {
    stop = min(end, b);
    return -1;
  }
  stop = min(end, max(off(lo + 1), t + 1));
  return lo;
}

// The next piece of more than `least` tokens from token a on, among the sequences s0 .. s1 of a
// chunk: a wave looks at 64 sequences at once.  Its sequence (-1: none), a and b.
template <class Off>
__device__ __forceinline__ int rl_long_piece(Off off, int s0, int s1, int begin, int end, int least, int& a, int& b) {
  for (int base = s0; base <= s1; base += 64) {
    const int s = base + (int)(threadIdx.x & 63), c = min(s, s1);
    const int lo = max(off(c), begin), hi = min(off(c + 1), end);
    const uint64_t hit = __builtin_amdgcn_ballot_w64(s <= s1 && lo >= a && hi - lo > least);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      a = __shfl(lo, l, 64);
      b = __shfl(hi, l, 64);
      return base + l;
    }
  }
  return -1;
}

// The sequence table in LDS where it fits, else read in place.
constexpr int RL_TABLE = 1024;
struct RlTable {
  int off[RL_TABLE + 1];
};
__device__ __forceinline__ void rl_table_load(RlTable& L, const int32_t* seq_off, int n_seq, int T) {
  if (n_seq <= RL_TABLE)
    for (int i = threadIdx.x; i <= n_seq; i += blockDim.x) L.off[i] = rl_off(seq_off, i, T);
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
// Exchange within aligned groups of 2, 4, 8 and 16 lanes by DPP (quad permutations, then mirrors of
// half rows and rows, whose lanes already agree), between 16-lane rows by shuffles: an add with a
// DPP operand costs a few cycles, a shuffle an LDS round trip, and these chains are what a token's
// softmax waits for.
template <int CTRL>
__device__ __forceinline__ float rl_dpp(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xf, 0xf, true));
}
template <int G, class Op>
__device__ __forceinline__ float rl_group(float v, Op op) {
  if (G >= 2) v = op(v, rl_dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  if (G >= 4) v = op(v, rl_dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  if (G >= 8) v = op(v, rl_dpp<0x141>(v));   // row_half_mirror
  if (G >= 16) v = op(v, rl_dpp<0x140>(v));  // row_mirror
  if (G >= 32) v = op(v, __shfl_xor(v, 16, 64));
  if (G >= 64) v = op(v, __shfl_xor(v, 32, 64));
  return v;
}
template <int G>
__device__ __forceinline__ float rl_group_sum(float v) {
  return rl_group<G>(v, [](float a, float b) { return a + b; });
}
template <int G>
__device__ __forceinline__ float rl_group_max(float v) {
  return rl_group<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// The softmax of a token's row in place; returns the log-sum-exp, and in l2 its square.  A row of
// -infinity only (every expert masked) has no probabilities: its sum is zero, its log-sum-exp
// -infinity, and it adds to neither loss; a NaN or +infinity makes the row NaN.
template <int G, int N>
__device__ __forceinline__ float rl_softmax(float (&x)[N], float& l2) {
  float m = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) m = fmaxf(m, x[k]);
  m = rl_group_max<G>(m);
  m = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[k] = rl_exp(x[k] - m);
    sum += x[k];
  }
  sum = rl_group_sum<G>(sum);
  const float l = m + __logf(sum);
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  l2 = sum != 0.0f ? l * l : 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] *= inv;
  return l;
}

// What a wave's lanes have put into LDS is there for its other lanes.
__device__ __forceinline__ void rl_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  __builtin_amdgcn_wave_barrier();
}

// What one workgroup of the joining launch leaves for the last: stored and loaded past the caches of
// the XCDs (agent scope), so that no cache has to be written back or invalidated as a whole.
template <typename V>
__device__ __forceinline__ void rl_put(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V rl_get(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Where the sums end up.
struct RlossOut {
  int32_t* seq_tokens;
  int32_t* seq_counts;
  float* prob_sum;
  float* loss;
};

constexpr int RL_RUNS = RL_JOIN_THREADS / RL_JOIN_COLS;
struct RlJoinLds {
  double p[RL_JOIN_THREADS / 64][RL_JOIN_COLS];
  int c[RL_JOIN_THREADS / 64][RL_JOIN_COLS];
  double z[RL_MAX_WAVES], b[RL_MAX_WAVES];
  long long n[RL_MAX_WAVES];
  int last;
};

__device__ __forceinline__ void rl_write_loss(const RlossOut& o, int E, int K, double bal, double z, long long n) {
  o.loss[0] = n ? (float)(bal * (double)E / ((double)K * (double)n)) : 0.0f;
  o.loss[1] = n ? (float)(z / (double)n) : 0.0f;
}

// Adds sequence s's slots for columns block cb in a fixed order: 32 columns by 16 runs of chunks, then
// the runs by waves (two each).  Also the sequence's tokens and z sum when cb is 0.
__device__ __forceinline__ void rl_join(RlJoinLds& L, int s, int cb, int chunk, int T, int E,
                                        const int32_t* __restrict__ seq_off, const RlossWs& w, const RlossOut& o) {
  const int cbs = (E + RL_JOIN_COLS - 1) / RL_JOIN_COLS;
  const int lo = rl_off(seq_off, s, T), hi = rl_off(seq_off, s + 1, T);
  const int c0 = lo / chunk, c1 = hi > lo ? (hi - 1) / chunk + 1 : c0;  // chunks c0 .. c1 - 1
  const int ci = threadIdx.x % RL_JOIN_COLS, run = threadIdx.x / RL_JOIN_COLS;
  const int e = cb * RL_JOIN_COLS + ci;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double p = 0.0;
  int cnt = 0;
  if (e < E) {
#pragma unroll 4
    for (int c = c0 + run; c < c1; c += RL_RUNS) {
      const int64_t i = (int64_t)(c + s) * E + e;
      p += (double)w.prob[i];
      cnt += w.cnt[i];
    }
  }
  p += __shfl_xor(p, 32, 64);
  cnt += __shfl_xor(cnt, 32, 64);
  if (lane < 32) {
    L.p[wave][ci] = p;
    L.c[wave][ci] = cnt;
  }
  if (cb == 0) {
    double z = 0.0;
    long long n = 0;
    for (int c = c0 + (int)threadIdx.x; c < c1; c += RL_JOIN_THREADS) {
      z += (double)w.z[c + s];
      n += w.tok[c + s];
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) {
      z += __shfl_xor(z, k, 64);
      n += __shfl_xor(n, k, 64);
    }
    if (lane == 0) {
      L.z[wave] = z;
      L.n[wave] = n;
    }
  }
  __syncthreads();
  if (threadIdx.x < RL_JOIN_COLS) {
    double ps = 0.0;
    int cs = 0;
#pragma unroll
    for (int r = 0; r < RL_JOIN_THREADS / 64; ++r) {
      ps += L.p[r][ci];
      cs += L.c[r][ci];
    }
    if (e < E) {
      o.prob_sum[(int64_t)s * E + e] = (float)ps;
      o.seq_counts[(int64_t)s * E + e] = cs;
    }
    double bsum = e < E ? ps * (double)cs : 0.0;
#pragma unroll
    for (int k = RL_JOIN_COLS / 2; k > 0; k >>= 1) bsum += __shfl_xor(bsum, k, 64);
    if (threadIdx.x == 0) rl_put(&w.bal[(int64_t)s * cbs + cb], bsum);
  }
  if (cb == 0 && threadIdx.x == 64) {
    double z = 0.0;
    long long n = 0;
    for (int q = 0; q < RL_JOIN_THREADS / 64; ++q) {
      z += L.z[q];
      n += L.n[q];
    }
    rl_put(&w.zs[s], z);
    rl_put(&o.seq_tokens[s], (int32_t)n);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0);  // this wave's stores have arrived
  __syncthreads();
}

// The two losses from the sequences' sums (one workgroup), cbs of them per sequence in w.bal.
__device__ __forceinline__ void rl_losses(RlJoinLds& L, int E, int K, int n_seq, int cbs, const RlossWs& w, const RlossOut& o) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double bsum = 0.0, zsum = 0.0;
  long long n = 0;
  for (int q = threadIdx.x; q < n_seq; q += blockDim.x) {
    const int tq = rl_get(&o.seq_tokens[q]);
    double bq = 0.0;
    for (int k = 0; k < cbs; ++k) bq += rl_get(&w.bal[(int64_t)q * cbs + k]);
    const double zq = rl_get(&w.zs[q]);
    if (tq > 0) {  // (a sequence without tokens may have left no sums)
      bsum += bq / (double)tq;
      zsum += zq;
      n += tq;
    }
  }
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) {
    bsum += __shfl_xor(bsum, k, 64);
    zsum += __shfl_xor(zsum, k, 64);
    n += __shfl_xor(n, k, 64);
  }
  if (lane == 0) {
    L.b[wave] = bsum;
    L.z[wave] = zsum;
    L.n[wave] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bsum = zsum = 0.0;
    n = 0;
    for (int q = 0; q < (int)blockDim.x / 64; ++q) {
      bsum += L.b[q];
      zsum += L.z[q];
      n += L.n[q];
    }
    rl_write_loss(o, E, K, bsum, zsum, n);
  }
}

template <int G, int NV, bool V4, bool ONE, bool LONGER>
__global__ __launch_bounds__(rl_waves(ONE) * 64) void k_rloss_part(const float* __restrict__ logits,
                                                           const int32_t* __restrict__ topk_idx, int T, int E, int K,
                                                           int n_seq, const int32_t* __restrict__ seq_off,
                                                           const uint8_t* __restrict__ mask, float* __restrict__ lse,
                                                           RlossWs w, RlossOut o) {
  using Row = RlRow<G, NV, V4>;
  constexpr int N = Row::N, TPW = 64 / G, WAVES = rl_waves(ONE), THREADS = 64 * WAVES;
  constexpr int STEPS = rl_steps(G, LONGER), CHUNK = rl_chunk(G, ONE, LONGER);
  extern __shared__ float rl_lds[];  // [waves][E] probability sums, [E] counts
  int* hist = reinterpret_cast<int*>(rl_lds + WAVES * E);
  __shared__ float sz[WAVES];
  __shared__ int sn[WAVES];
  __shared__ double sb[WAVES];
  __shared__ RlTable tab;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane % G, grp = lane / G;
  const int t_begin = blockIdx.x * CHUNK, t_end = min(T, t_begin + CHUNK);
  // everything the chunk needs is requested here
  float x[STEPS][N];
  bool live[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int t = min(t_begin + (i * WAVES + wave) * TPW + grp, T - 1);
    Row::load(logits + (int64_t)t * E, li, E, x[i]);
    live[i] = !mask || mask[t];
  }
  const int picks = (t_end - t_begin) * K;  // the chunk's choices, one per thread and round
  const int first = (int)threadIdx.x < picks ? topk_idx[(int64_t)t_begin * K + threadIdx.x] : -1;
  const int first_t = t_begin + (int)threadIdx.x / K;
  const bool first_live = !mask || ((int)threadIdx.x < picks && mask[first_t]);
  rl_table_load(tab, seq_off, n_seq, T);
  if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0u;
  for (int e = threadIdx.x; e < E; e += THREADS) hist[e] = 0;
  if constexpr (ONE) {  // sequences without tokens have no piece
    for (int i = threadIdx.x; i < n_seq * E; i += THREADS) {
      const int s = i / E;
      if (rl_off(seq_off, s + 1, T) <= rl_off(seq_off, s, T)) {
        o.prob_sum[i] = 0.0f;
        o.seq_counts[i] = 0;
        if (i == s * E) o.seq_tokens[s] = 0;
      }
    }
  }
  // softmax of every token of the chunk
  float l2[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const float l = rl_softmax<G>(x[i], l2[i]);
    const int t = t_begin + (i * WAVES + wave) * TPW + grp;
    if (li == 0 && t < t_end) lse[t] = l;
  }
  __syncthreads();
  auto off = [&](int s) { return n_seq <= RL_TABLE ? tab.off[s] : rl_off(seq_off, s, T); };
  double bsum = 0.0, zsum = 0.0;  // ONE: thread 0's sums over the sequences
  long long nsum = 0;
  // a chunk of many pieces: the workgroup takes the longer ones, its waves one short one each
  const int s0 = __builtin_amdgcn_readfirstlane(rl_find(off, n_seq, t_begin, 0));
  const bool many = n_seq - s0 > RL_FEW && off(s0 + RL_FEW) < t_end;
  const int s1 = many ? __builtin_amdgcn_readfirstlane(min(rl_find(off, n_seq, t_end - 1, s0), n_seq - 1)) : s0;
  int at = s0;
  for (int a = t_begin, b; a < t_end; a = b) {
    int s;
    if (many) {
      s = rl_long_piece(off, s0, s1, t_begin, t_end, RL_SHORT * TPW, a, b);
      if (s < 0) break;
    } else {
      s = rl_piece(off, n_seq, a, t_end, b, at);
      if (s < 0) continue;  // (uniform) tokens outside every sequence only get their log-sum-exp
    }
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.0f;
    float z = 0.0f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int t = t_begin + (i * WAVES + wave) * TPW + grp;
      if (t >= a && t < b && live[i]) {
        ++n;
        z += l2[i];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += x[i][k];
      }
    }
    if ((int)threadIdx.x < picks && first_t >= a && first_t < b && (uint32_t)first < (uint32_t)E && first_live)
      atomicAdd(&hist[first], 1);
    for (int i = threadIdx.x + THREADS; i < picks; i += THREADS) {
      const int t = t_begin + i / K, e = topk_idx[(int64_t)t_begin * K + i];
      if (t >= a && t < b && (uint32_t)e < (uint32_t)E && (!mask || mask[t])) atomicAdd(&hist[e], 1);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
      for (int h = G; h < 64; h <<= 1) acc[k] += __shfl_xor(acc[k], h, 64);
      if (grp == 0 && Row::col(li, k) < E) rl_lds[wave * E + Row::col(li, k)] = acc[k];
    }
    // every lane of a group holds its tokens' count and z: take one lane per group
    z = rl_group_sum<64>(li == 0 ? z : 0.0f);
    n = (int)rl_group_sum<64>(li == 0 ? (float)n : 0.0f);
    if (lane == 0) {
      sz[wave] = z;
      sn[wave] = n;
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    double bal = 0.0;
    for (int e = threadIdx.x; e < E; e += THREADS) {
      float v = 0.0f;
#pragma unroll
      for (int q = 0; q < WAVES; ++q) v += rl_lds[q * E + e];
      const int c = hist[e];
      hist[e] = 0;
      if constexpr (ONE) {
        o.prob_sum[(int64_t)s * E + e] = v;
        o.seq_counts[(int64_t)s * E + e] = c;
        bal += (double)v * (double)c;
      } else {
        w.prob[slot * E + e] = v;
        w.cnt[slot * E + e] = c;
      }
    }
    if constexpr (ONE) {
#pragma unroll
      for (int h = 32; h > 0; h >>= 1) bal += __shfl_xor(bal, h, 64);
      if (lane == 0) sb[wave] = bal;
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      float zs = 0.0f;
      int ns = 0;
#pragma unroll
      for (int q = 0; q < WAVES; ++q) {
        zs += sz[q];
        ns += sn[q];
      }
      if constexpr (ONE) {
        double bs = 0.0;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) bs += sb[q];
        if (many) {
          rl_put(&w.bal[s], bs);
          rl_put(&w.zs[s], (double)zs);
          rl_put(&o.seq_tokens[s], (int32_t)ns);
        } else {
          o.seq_tokens[s] = ns;
          if (ns > 0) bsum += bs / (double)ns;
          zsum += (double)zs;
          nsum += ns;
        }
      } else {
        w.z[slot] = zs;
        w.tok[slot] = ns;
      }
    }
    __syncthreads();  // the LDS is free for the next piece
  }
  if (many) {
    int* cnt = reinterpret_cast<int*>(rl_lds) + wave * E;  // the wave's own counts
    for (int s = s0 + wave; s <= s1; s += WAVES) {
      const int a = __builtin_amdgcn_readfirstlane(max(off(s), t_begin)), b = __builtin_amdgcn_readfirstlane(min(off(s + 1), t_end));
      if (b <= a || b - a > RL_SHORT * TPW) continue;
      rl_wave_sync();  // (the last piece's counts have been read)
      for (int e = lane; e < E; e += 64) cnt[e] = 0;
      rl_wave_sync();
      const int32_t* pick = topk_idx + (int64_t)a * K;
      for (int i = lane; i < (b - a) * K; i += 64) {
        const int e = pick[i];
        if ((uint32_t)e < (uint32_t)E && (!mask || mask[a + i / K])) atomicAdd(&cnt[e], 1);
      }
      float acc[N];
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = 0.0f;
      float z = 0.0f, n = 0.0f;
      for (int t0 = a; t0 < b; t0 += TPW) {
        const int t = min(t0 + grp, b - 1);
        float y[N], q;
        Row::load(logits + (int64_t)t * E, li, E, y);
        rl_softmax<G>(y, q);
        if (t0 + grp < b && (!mask || mask[t])) {
          n += 1.0f;
          z += q;
#pragma unroll
          for (int k = 0; k < N; ++k) acc[k] += y[k];
        }
      }
      rl_wave_sync();  // the counts are whole
      const int64_t slot = ONE ? (int64_t)s : (int64_t)blockIdx.x + s;
      float* prob = (ONE ? o.prob_sum : w.prob) + slot * E;
      int32_t* out_cnt = (ONE ? o.seq_counts : w.cnt) + slot * E;
      double bal = 0.0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int h = G; h < 64; h <<= 1) acc[k] += __shfl_xor(acc[k], h, 64);
        const int e = Row::col(li, k);
        if (grp == 0 && e < E) {
          const int c = cnt[e];
          prob[e] = acc[k];
          out_cnt[e] = c;
          if (ONE) bal += (double)acc[k] * (double)c;
        }
      }
      z = rl_group_sum<64>(li == 0 ? z : 0.0f);
      n = rl_group_sum<64>(li == 0 ? n : 0.0f);
      if constexpr (ONE) {
#pragma unroll
        for (int h = 32; h > 0; h >>= 1) bal += __shfl_xor(bal, h, 64);
      }
      if (lane == 0) {
        if constexpr (ONE) {
          rl_put(&w.bal[s], bal);
          rl_put(&w.zs[s], (double)z);
          rl_put(&o.seq_tokens[s], (int32_t)n);
        } else {
          w.z[slot] = z;
          w.tok[slot] = (int)n;
        }
      }
    }
    if constexpr (ONE) {
      __shared__ RlJoinLds L;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
      __builtin_amdgcn_s_waitcnt(0);  // this wave's sums have arrived
      __syncthreads();
      rl_losses(L, E, K, n_seq, 1, w, o);
    }
  } else if (ONE && threadIdx.x == 0) {
    rl_write_loss(o, E, K, bsum, zsum, nsum);
  }
}

// The joining launch, one workgroup per sequence and block of 32 columns; the last one to finish
// forms the losses.
__global__ __launch_bounds__(RL_JOIN_THREADS) void k_rloss_join(int T, int E, int K, int n_seq, int chunk,
                                                           const int32_t* __restrict__ seq_off, RlossWs w, RlossOut o) {
  __shared__ RlJoinLds L;
  const int cbs = (E + RL_JOIN_COLS - 1) / RL_JOIN_COLS;
  const int s = blockIdx.y * RL_JOIN_SEQS + blockIdx.x / cbs;
  if (s >= n_seq) return;
  rl_join(L, s, blockIdx.x % cbs, chunk, T, E, seq_off, w, o);
  if (threadIdx.x == 0) {
    const unsigned v = __hip_atomic_fetch_add(w.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    L.last = v == (unsigned)(n_seq * cbs) - 1;
  }
  __syncthreads();
  if (!L.last) return;
  rl_losses(L, E, K, n_seq, cbs, w, o);
}

// dLogits.  A group of lanes keeps its sequence's counts as long as its tokens stay in it.  The
// counts enter less their mean K T_s / E: the probabilities of a row sum to one, so the mean drops
// out of the difference, and without it the difference of two nearly equal numbers would lose the
// leading bits.
template <int G, int NV, bool V4>
__global__ __launch_bounds__(RL_BWD_THREADS) void k_rloss_bwd(const float* __restrict__ dloss,
                                                          const float* __restrict__ logits, int T, int E, int K,
                                                          int n_seq, const int32_t* __restrict__ seq_off,
                                                          const uint8_t* __restrict__ mask,
                                                          const int32_t* __restrict__ seq_tokens,
                                                          const int32_t* __restrict__ seq_counts,
                                                          const float* __restrict__ lse, float* __restrict__ dLogits,
                                                          int chunk) {
  using Row = RlRow<G, NV, V4>;
  constexpr int N = Row::N, TPW = 64 / G, WAVES = RL_BWD_THREADS / 64;
  __shared__ long long rn[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane % G, grp = lane / G;
  const int t_begin = blockIdx.x * chunk, t_end = min(T, t_begin + chunk);
  __shared__ RlTable tab;
  rl_table_load(tab, seq_off, n_seq, T);
  auto off = [&](int s) { return n_seq <= RL_TABLE ? tab.off[s] : rl_off(seq_off, s, T); };
  long long n = 0;
  for (int q = threadIdx.x; q < n_seq; q += RL_BWD_THREADS) n += seq_tokens[q];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  if (lane == 0) rn[wave] = n;
  __syncthreads();
  n = rn[0] + rn[1] + rn[2] + rn[3];
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = dloss[0] * inv_n * (float)E / (float)K, gz = dloss[1] * 2.0f * inv_n;
  int s = -1, stop = t_begin, at = 0;  // the sequence of this lane group's tokens before `stop`
  float ex[N], coef = 0.0f;
  for (int t = t_begin + wave * TPW + grp; t < t_end; t += WAVES * TPW) {
    float x[N];
    Row::load(logits + (int64_t)t * E, li, E, x);
    const float l = lse[t];
    const bool live = !mask || mask[t];
    if (t >= stop) {
      s = rl_piece(off, n_seq, t, T, stop, at);
      if (s >= 0) {
        const int ts = seq_tokens[s];
        coef = ts > 0 ? gb / (float)ts : 0.0f;
        const float mean = (float)((double)K * (double)ts / (double)E);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = Row::col(li, i);
          ex[i] = c < E ? (float)seq_counts[(int64_t)s * E + c] - mean : 0.0f;
        }
      }
    }
    if (s >= 0 && live && l != -INFINITY) {
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

// Calls f<G, NV, V4> for E's layout; V4 needs 16-byte aligned rows.
template <class F>
static void rl_dispatch(int E, F f) {
  const RlLayout l = rl_layout(E);
#define RL_CASE(GG, NN) \
  if (l.G == GG && l.NV == NN) return E % 4 == 0 ? f.template operator()<GG, NN, true>() : f.template operator()<GG, NN, false>()
  RL_CASE(2, 1);
  RL_CASE(4, 1);
  RL_CASE(8, 1);
  RL_CASE(16, 1);
  RL_CASE(16, 2);
  RL_CASE(16, 3);
  RL_CASE(32, 2);
  RL_CASE(32, 3);
  RL_CASE(64, 2);
  RL_CASE(64, 4);
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
  RlossOut o;
  hipStream_t st;
  template <int G, int NV, bool V4>
  void operator()() const {
    const RlGrid g = rl_grid(T, E);
    const int grid = (int)cdiv(T, g.chunk), threads = 64 * rl_waves(g.one);
    const size_t lds = (size_t)(rl_waves(g.one) + 1) * E * 4;
    auto go = [&](auto kernel) {
      kernel<<<grid, threads, lds, st>>>(logits, topk_idx, T, E, K, n_seq, seq_off, mask, lse, w, o);
    };
    if (g.one) return go(k_rloss_part<G, NV, V4, true, false>);
    if constexpr (G > 16)
      if (g.longer) return go(k_rloss_part<G, NV, V4, false, true>);
    go(k_rloss_part<G, NV, V4, false, false>);
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
    constexpr int LEAST = RL_BWD_THREADS / G;  // one token per lane group
    int chunk = RL_BWD_CHUNK > LEAST ? RL_BWD_CHUNK : LEAST;
    while (chunk > LEAST && cdiv(T, chunk) < 512) chunk /= 2;
    k_rloss_bwd<G, NV, V4><<<(int)cdiv(T, chunk), RL_BWD_THREADS, 0, st>>>(dloss, logits, T, E, K, n_seq, seq_off, mask,
                                                                      seq_tokens, seq_counts, lse, dLogits, chunk);
  }
};
}  // namespace

hipError_t launch_router_loss(const float* logits, const int32_t* topk_idx, int64_t T, int E, int K, int n_seq,
                              const int32_t* seq_off, const uint8_t* mask, int32_t* seq_tokens, int32_t* seq_counts,
                              float* prob_sum, float* lse, float* loss, void* ws, hipStream_t st) {
  RlossWs w;
  rl_carve(ws, T, E, n_seq, &w);
  const RlossOut o{seq_tokens, seq_counts, prob_sum, loss};
  rl_dispatch(E, RlossFwd{logits, topk_idx, (int)T, E, K, n_seq, seq_off, mask, lse, w, o, st});
  const hipError_t e = hipGetLastError();
  const RlGrid g = rl_grid(T, E);
  if (e != hipSuccess || g.one) return e;
  const dim3 join((unsigned)((n_seq < RL_JOIN_SEQS ? n_seq : RL_JOIN_SEQS) * rl_colblocks(E)), (unsigned)cdiv(n_seq, RL_JOIN_SEQS));
  k_rloss_join<<<join, RL_JOIN_THREADS, 0, st>>>((int)T, E, K, n_seq, g.chunk, seq_off, w, o);
  return hipGetLastError();
}

hipError_t launch_router_loss_bwd(const float* dloss, const float* logits, int64_t T, int E, int K, int n_seq,
                                  const int32_t* seq_off, const uint8_t* mask, const int32_t* seq_tokens,
                                  const int32_t* seq_counts, const float* lse, float* dLogits, hipStream_t st) {
  rl_dispatch(E, RlossBwd{dloss, logits, (int)T, E, K, n_seq, seq_off, mask, seq_tokens, seq_counts, lse, dLogits, st});
  return hipGetLastError();
}

}  // namespace moe
