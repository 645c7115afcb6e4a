// MFMA main loop for the dense projection (bf16): C[m][n] = sum_k A(m, k) B(k, n) on TM x TN tiles, each
// wave 32 MI x 64 of it, K in stages of 64.
//
// Against the grouped engine's ring of four 32-k stages (gemm_core.h), a stage here is 64 k deep:
// a K-major operand row then contributes whole 128-byte lines (half lines are what limits the
// loads there).  Two stages fill the LDS, so the loop frees a stage early instead of holding it: a
// wave has read all four k-steps' fragments into registers by the stage's middle, a barrier makes
// the slot free, and the stage two ahead is loaded into it beside the remaining MFMAs.  A second
// barrier publishes the next stage before the last k-step, whose MFMAs cover the first fragment
// reads of that stage.
//
//   K-major operand (rows contiguous along k): [rows][128 B]; 16-byte chunk c of row r sits at slot
//     c ^ ((r >> 1) & 7): the 16 rows read together cover all 64 banks.
//   MN-major operand (rows indexed by k): [64 k][2 COLS B]; chunk c of k-row k sits at slot
//     c ^ (4 (k & 3)) and fragments are read with the transposing ds_read_b64_tr_b16, as in the
//     grouped engine.
// Rows and columns past the matrix repeat a valid one: their products land in results that are
// never stored.  k past the reduction's end (only with TAIL, in the last stage) comes from a zero
// page on both sides.
//
// Accumulators are those of the grouped engine: the MFMA computes the transposed block, so
// register v of block (i, j) holds row 32 i + lane % 32 of the wave and column bsub(j) + acc_n(v),
// column block j of wave column wn at j TN / 2 + 32 wn: half j of the tile holds every wave's
// block j.
#pragma once

#include "gemm_core.h"

namespace moe {

constexpr int DN_BK = 64;

// Lane address in the last, partial stage: the zero page where the lane's k is past the end.
__device__ __forceinline__ const char* dn_pick(const char* p, uint64_t mask) {
  const uint64_t live = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)mask) |
                        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(mask >> 32)) << 32;
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t zero = reinterpret_cast<uint64_t>(g_zero_page) + (threadIdx.x & 63) * 16;
  uint32_t sl = (uint32_t)a, sh = (uint32_t)(a >> 32);
  asm("v_cndmask_b32_e64 %0, %1, %0, %2" : "+v"(sl) : "v"((uint32_t)zero), "s"(live));
  asm("v_cndmask_b32_e64 %0, %1, %0, %2" : "+v"(sh) : "v"((uint32_t)(zero >> 32)), "s"(live));
  return reinterpret_cast<const char*>(((uint64_t)sh << 32) | sl);
}

// K-major operand of ROWS rows, loaded by NW waves: wave w instruction q fills rows 8 (q NW + w) ..
// + 7 (lane l: row l / 8, slot l % 8).  base: the tile's first row at the first k; row(i): the
// source row of tile row i relative to base (at most 255); the upper half of the tile's rows lies
// `up` bytes further (whole instructions each).
template <int ROWS, int NW, bool TAIL>
struct DnK {
  static constexpr int NQ = ROWS / 8 / NW;
  const char* base;
  int64_t up;
  uint32_t off[NQ];
  int last;       // TAIL: the last stage
  uint64_t live;  // TAIL: lanes whose chunk lies inside the row there
  template <class Row>
  __device__ void init(const char* b, int64_t ldb, int klen, Row row, int64_t upper = 0) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int chunk = (lane & 7) ^ ((w * 4 + (lane >> 4)) & 7);  // (row >> 1) & 7: NW is a multiple of 2
    base = b;
    up = upper;
#pragma unroll
    for (int q = 0; q < NQ; ++q) off[q] = (uint32_t)(row((q * NW + w) * 8 + (lane >> 3)) * ldb) + chunk * 16;
    if (TAIL) {
      last = (klen + DN_BK - 1) / DN_BK - 1;
      live = __builtin_amdgcn_ballot_w64(last * DN_BK + chunk * 8 < klen);
    }
  }
  __device__ void issue(int s, int q, char* dst) const {
    const int w = threadIdx.x >> 6;
    const int su = __builtin_amdgcn_readfirstlane(s);
    const char* p = base + (int64_t)su * 128 + (q >= NQ / 2 ? up : 0) + off[q];
    if (TAIL) p = dn_pick(p, su == last ? live : ~0ull);
    dma16(p, dst + (q * NW + w) * 1024);
  }
  // A lane's fragment of row block b (32 rows) and k-step ks lies at (base ^ 32 ks) + 4096 b.
  __device__ static uint32_t lane_base(int row0) {
    const int lane = threadIdx.x & 63, r = lane & 31;
    return (row0 + r) * 128 + (((lane >> 5) ^ ((r >> 1) & 7)) * 16);
  }
  template <int STEP>  // STEP: rows between blocks
  __device__ static bf16x8 frag(const char* t, uint32_t base, int b, int ks) {
    return *reinterpret_cast<const bf16x8*>(t + (base ^ (ks * 32)) + b * STEP * 128);
  }
};

// MN-major operand of COLS columns: an instruction fills 512 / COLS k-rows.  base: element (first
// column, first k); cols: how many columns are valid (a multiple of 8).
template <int COLS, int NW, bool TAIL>
struct DnMN {
  static constexpr int PITCH = COLS * 2, RPI = 1024 / PITCH, NQ = DN_BK / RPI / NW, LPR = 64 / RPI;
  const char* base;
  int64_t ld;
  uint32_t off;
  int kl, klen;  // lane's k-row in instruction 0
  __device__ void init(const char* b, int64_t ldb, int klen_, int cols) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    kl = w * RPI + lane / LPR;
    const int chunk = (lane % LPR) ^ (4 * (kl & 3));
    base = b;
    ld = ldb;
    off = (uint32_t)(kl * ldb) + min(chunk * 16, cols * 2 - 16);
    klen = klen_;
  }
  __device__ void issue(int s, int q, char* dst) const {
    const int w = threadIdx.x >> 6;
    const int k0 = __builtin_amdgcn_readfirstlane(s) * DN_BK + q * NW * RPI;
    const char* p = base + (int64_t)k0 * ld + off;
    if (TAIL) p = dn_pick(p, __builtin_amdgcn_ballot_w64(k0 + kl < klen));
    dma16(p, dst + (q * NW + w) * 1024);
  }
  // A lane's fragment of column block b and k-step ks: two reads at ((base ^ 2 STEP b) + 32 PITCH
  // ks / 2) and four k-rows on, for blocks STEP = 32 columns apart; farther ones (a multiple of
  // 128) add.
  __device__ static uint32_t lane_base(int mn0) {
    const int lane = threadIdx.x & 63;
    const int g = lane >> 4, i = lane & 15;
    const int k = (g >> 1) * 8 + (i >> 2);
    const int mn = mn0 + (g & 1) * 16 + 4 * (i & 3);
    return k * PITCH + ((mn >> 3) ^ (4 * (k & 3))) * 16 + (mn & 7) * 2;
  }
  template <int STEP>
  __device__ static bf16x8 frag(const char* t, uint32_t base, int b, int ks) {
    const char* p = t + (STEP % 128 == 0 ? base + b * STEP * 2 : base ^ (b * STEP * 2)) + ks * 16 * PITCH;
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p);
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * PITCH));
    const v4i16 both[2] = {lo, hi};
    bf16x8 r;
    __builtin_memcpy(&r, both, 16);
    return r;
  }
};

template <int MI>
struct DnAcc {
  f32x16 c[MI][2];
};
template <int MI>
struct DnFrag {
  bf16x8 a[MI], b[2];
};

// TM x TN tiles; WM x WN waves of 32 MI rows x 64 columns (two blocks of 32, see above).
template <int TM, int TN, int WM, int WN>
struct DnTile {
  static constexpr int TM_ = TM, WN_ = WN, SPLIT = TM / 2;
  static constexpr int NW = WM * WN, THREADS = 64 * NW, MI = TM / WM / 32;
  static constexpr int A_BYTES = TM * 128, STAGE = (TM + TN) * 128;
  static constexpr int HC = TN / 2;          // columns per tile half
  static constexpr int EPITCH = HC * 4 + 16; // fp32 staging row of a tile half
  static constexpr int SLOT = STAGE > TM / 2 * EPITCH ? STAGE : TM / 2 * EPITCH;
  static_assert(HC == WN * 32, "two column blocks per wave");
};

// A wave's LDS bases of its A and B fragments in a slot.
struct DnLds {
  uint32_t a, b;
};
template <class TI, class AL, class BL>
__device__ __forceinline__ void dn_frags(const char* slot, int ks, const DnLds& d, DnFrag<TI::MI>& F) {
#pragma unroll
  for (int j = 0; j < 2; ++j) F.b[j] = BL::template frag<TI::HC>(slot + TI::A_BYTES, d.b, j, ks);
#pragma unroll
  for (int i = 0; i < TI::MI; ++i) F.a[i] = AL::template frag<32>(slot, d.a, i, ks);
}
template <int FROM, int TO, int MI>
__device__ __forceinline__ void dn_mma(const DnFrag<MI>& F, DnAcc<MI>& acc) {
#pragma unroll
  for (int p = FROM; p < TO; ++p)
    acc.c[p >> 1][p & 1] = Mma<bf16>::mma(F.b[p & 1], F.a[p >> 1], acc.c[p >> 1][p & 1]);
}

// One k-step's MFMA blocks FROM .. NB - 1 with DMA instructions N0 .. N1 - 1 spread between them.
template <int FROM, int N0, int N1, int MI, class Issue>
__device__ __forceinline__ void dn_mma_issue(const DnFrag<MI>& F, DnAcc<MI>& acc, Issue issue) {
  constexpr int NB = 2 * MI;
#pragma unroll
  for (int p = FROM; p < NB; ++p) {
#pragma unroll
    for (int n = N0; n < N1; ++n)
      if (FROM + (n - N0) * (NB - FROM) / (N1 - N0) == p) {
        issue(n);
        __builtin_amdgcn_sched_barrier(0);
      }
    acc.c[p >> 1][p & 1] = Mma<bf16>::mma(F.b[p & 1], F.a[p >> 1], acc.c[p >> 1][p & 1]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One stage.  F0 holds its k-step 0 (read beside the previous stage's last MFMAs).  Half of stage
// s + 2 goes out beside k-step 2, the other half beside k-step 3.
template <class TI, class AL, class BL>
__device__ __forceinline__ void dn_step(const AL& la, const BL& lb, int s, int nkt, char* cur, const char* next,
                                        DnLds& d, DnFrag<TI::MI>& F0, DnAcc<TI::MI>& acc) {
  constexpr int MI = TI::MI, NB = 2 * MI;  // blocks per k-step
  constexpr int NI = AL::NQ + BL::NQ;      // DMA instructions per wave and stage
  DnFrag<MI> F1, F2, F3;
  auto issue = [&](int n) {
    const int r = min(s + 2, nkt - 1);  // past the end the last stage again: the waits count on it
    if (n < AL::NQ) la.issue(r, n, cur);
    else lb.issue(r, n - AL::NQ, cur + TI::A_BYTES);
  };
  // the bases are opaque here, so that the fragments' addresses are formed at their reads instead
  // of being kept in registers across the loop
  asm volatile("" : "+v"(d.a), "+v"(d.b));
  dn_mma<0, 1>(F0, acc);
  __builtin_amdgcn_sched_barrier(0);
  dn_frags<TI, AL, BL>(cur, 1, d, F1);
  dn_frags<TI, AL, BL>(cur, 2, d, F2);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<1, NB>(F0, acc);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<0, 1>(F1, acc);
  __builtin_amdgcn_sched_barrier(0);
  dn_frags<TI, AL, BL>(cur, 3, d, F3);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<1, NB>(F1, acc);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read the whole stage
  ring_barrier();                      // so has every wave: its slot is free
  __builtin_amdgcn_sched_barrier(0);
  dn_mma_issue<0, 0, NI / 2>(F2, acc, issue);
  wait_vmcnt<NI / 2>();  // stage s + 1 has landed: only half of stage s + 2 was issued after it
  ring_barrier();
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<0, 1>(F3, acc);
  __builtin_amdgcn_sched_barrier(0);
  dn_frags<TI, AL, BL>(next, 0, d, F0);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma_issue<1, NI / 2, NI>(F3, acc, issue);
}

// The main loop over nkt stages, accumulating from zero; ends with the LDS free.
template <class TI, class AL, class BL>
__device__ __forceinline__ void dn_mainloop(const AL& la, const BL& lb, int nkt, DnAcc<TI::MI>& acc, char* b0, char* b1,
                                            int wm, int wn) {
#pragma unroll
  for (int i = 0; i < TI::MI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc.c[i][j][v] = 0.0f;
  if (nkt <= 0) return;
  const int r1 = min(1, nkt - 1);
#pragma unroll
  for (int q = 0; q < AL::NQ; ++q) la.issue(0, q, b0);
#pragma unroll
  for (int q = 0; q < BL::NQ; ++q) lb.issue(0, q, b0 + TI::A_BYTES);
#pragma unroll
  for (int q = 0; q < AL::NQ; ++q) la.issue(r1, q, b1);
#pragma unroll
  for (int q = 0; q < BL::NQ; ++q) lb.issue(r1, q, b1 + TI::A_BYTES);
  wait_vmcnt<AL::NQ + BL::NQ>();
  ring_barrier();
  DnFrag<TI::MI> F0;
  DnLds d{AL::lane_base(wm * TI::MI * 32), BL::lane_base(wn * 32)};
  dn_frags<TI, AL, BL>(b0, 0, d, F0);
  int s = 0;
  for (; s + 2 <= nkt; s += 2) {
    dn_step<TI>(la, lb, s, nkt, b0, b1, d, F0, acc);
    dn_step<TI>(la, lb, s + 1, nkt, b1, b0, d, F0, acc);
  }
  if (s < nkt) dn_step<TI>(la, lb, s, nkt, b0, b1, d, F0, acc);
  __syncthreads();  // drains the trailing loads; the LDS is free for the epilogue
}

}  // namespace moe
