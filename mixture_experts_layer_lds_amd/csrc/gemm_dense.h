// MFMA main loop for the dense projection: C[m][n] = sum_k A(m, k) B(k, n) on TM x TN tiles, each wave
// 16 MI x 64 of it, K in stages of 128 bytes per row (64 bf16 or 32 fp32 values).
//
// Against the grouped engine's ring of four 32-k stages (gemm_core.h), a bf16 stage here is 64 k deep:
// a K-major operand row then contributes whole 128-byte lines (half lines are what limits the
// loads there).  Two stages fill the LDS, so the loop frees a stage early instead of holding it: a
// wave reads all of a stage's fragments within its first quarter, a barrier makes the slot
// free, and the stage two ahead is loaded into it beside the next half's MFMAs.  A second barrier
// publishes the next stage inside the last quarter, whose other MFMAs cover that stage's first
// fragment reads.  The MFMA is 16x16x32, which moves half the accumulator registers per product
// of 32x32x16: the chip's power sets the clock here, so what the loop moves costs as much as what
// it waits for.  Measured on an 8192 x 14336 x 4096 product, loop alone: 1328 TFLOP/s with
// 32x32x16 (2580 cycles per stage of 2048 MFMA cycles at 1.69 GHz), 1460 with 16x16x32 (2684 at
// 1.92 GHz), 1480 with the slot freed after the first quarter instead of the half (2522); 1725
// when a timing-only copy leaves the refills out.
//
//   K-major operand (rows contiguous along k): [rows][128 B]; 16-byte chunk c of row r sits at slot
//     c ^ ((r >> 1) & 7): the 16 rows read together cover all 64 banks.
//   MN-major operand (rows indexed by k): [64 or 32 k][COLS values]; chunk c of k-row k sits at slot
//     c ^ swz(k).  bf16 fragments are read with the transposing ds_read_b64_tr_b16 (see the grouped
//     engine): 32 lanes read two chunks each of k-rows 0 .. 3 and 8 .. 11, and the swizzle gives
//     those eight rows distinct banks.  fp32 fragments are four 4-byte reads, 16 columns of the
//     k-rows i, i + 4, i + 8 and i + 12 each, the four rows in distinct banks.
// fp32 runs through the same stages and fragments (16 bytes of a row are four k of an fp32 operand,
// eight of a bf16 one): one 16x16x32 bf16 MFMA becomes four 16x16x4 fp32 ones, element i of every
// lane's chunk in the i-th, which pairs the same k on both sides.
// Rows and columns past the matrix repeat a valid one: their products land in results that are
// never stored.  k past the reduction's end (only with TAIL, in the last stage) comes from a zero
// page on both sides.
#pragma once

#include "gemm_core.h"

namespace moe {

template <typename T> __host__ __device__ constexpr int dn_bk() { return 128 / (int)sizeof(T); }

template <typename T> struct DnMma;
template <> struct DnMma<bf16> {
  typedef bf16x8 frag;
  __device__ static f32x4 mma(frag a, frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  // swizzle of k-row k of an MN-major operand of PITCH bytes per k-row (128: two rows to 256 bytes)
  template <int PITCH>
  __device__ static int swz(int k) {
    return PITCH == 128 ? (2 * ((k >> 1) & 1)) ^ (4 * ((k >> 3) & 1)) : (4 * (k & 3)) ^ (2 * ((k >> 3) & 1));
  }
};
template <> struct DnMma<float> {
  typedef f32x4 frag;
  __device__ static f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
  template <int PITCH>
  __device__ static int swz(int k) { return 4 * ((k >> 2) & 3); }
};

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

// The wave's number and a uniform address as scalars: a DMA's LDS address and its global base then
// take no vector register (kept in them, they made the dW loop spill).
__device__ __forceinline__ int dn_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
__device__ __forceinline__ const char* dn_uniform(const char* p) {
  uint64_t a = reinterpret_cast<uint64_t>(p);
  asm("" : "+s"(a));
  return reinterpret_cast<const char*>(a);
}

// K-major operand of ROWS rows, loaded by NW waves: wave w instruction q fills rows 8 (q NW + w) ..
// + 7 (lane l: row l / 8, slot l % 8).  base: the tile's first row at the first k; row(i): the
// source row of tile row i relative to base (at most 255); the upper half of the tile's rows lies
// `up` bytes further (whole instructions each).
template <typename T, int ROWS, int NW, bool TAIL>
struct DnK {
  typedef typename DnMma<T>::frag Frag;
  static constexpr bool PARTIAL = TAIL;
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
      last = (klen + dn_bk<T>() - 1) / dn_bk<T>() - 1;
      live = __builtin_amdgcn_ballot_w64(last * dn_bk<T>() + chunk * (16 / (int)sizeof(T)) < klen);
    }
  }
  template <bool END>
  __device__ void issue(int s, int q, char* dst) const {
    const int w = dn_wave();
    const int su = __builtin_amdgcn_readfirstlane(s);
    const char* p = dn_uniform(base + (int64_t)su * 128 + (q >= NQ / 2 ? up : 0)) + off[q];
    if (TAIL && END) p = dn_pick(p, su == last ? live : ~0ull);
    dma16(p, dst + (q * NW + w) * 1024);
  }
  // A lane's fragment (16 rows x 64 bytes) of the rows `at` further and k-step ks lies at
  // (base ^ 64 ks) + 128 at.
  __device__ static uint32_t lane_base(int row0) {
    const int lane = threadIdx.x & 63, r = lane & 15;
    return (row0 + r) * 128 + (((lane >> 4) ^ ((r >> 1) & 7)) * 16);
  }
  __device__ static Frag frag(const char* t, uint32_t base, int at, int ks) {
    return *reinterpret_cast<const Frag*>(t + (base ^ (ks * 64)) + at * 128);
  }
};

// MN-major operand of COLS columns: an instruction fills RPI k-rows.  base: element (first column,
// first k); cols: how many columns are valid (a multiple of 8).
template <typename T, int COLS, int NW, bool TAIL>
struct DnMN {
  typedef typename DnMma<T>::frag Frag;
  static constexpr bool PARTIAL = TAIL;
  static constexpr int SZ = (int)sizeof(T), PITCH = COLS * SZ, RPI = 1024 / PITCH, LPR = 64 / RPI;
  static constexpr int NQ = dn_bk<T>() / RPI / NW;
  const char* base;
  int64_t ld;
  uint32_t off[2];  // of even and odd instructions (8 or 16 k-rows apart: at most two swizzles)
  int kl, klen;     // lane's k-row in instruction 0
  __device__ void init(const char* b, int64_t ldb, int klen_, int cols) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    kl = w * RPI + lane / LPR;
    base = b;
    ld = ldb;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int chunk = (lane % LPR) ^ DnMma<T>::template swz<PITCH>(kl + q * NW * RPI);
      off[q] = (uint32_t)(kl * ldb) + min(chunk * 16, cols * SZ - 16);
    }
    klen = klen_;
  }
  template <bool END>
  __device__ void issue(int s, int q, char* dst) const {
    const int w = dn_wave();
    const int k0 = __builtin_amdgcn_readfirstlane(s) * dn_bk<T>() + q * NW * RPI;
    const char* p = dn_uniform(base + (int64_t)k0 * ld) + off[q & 1];
    if (TAIL && END) p = dn_pick(p, __builtin_amdgcn_ballot_w64(k0 + kl < klen));
    dma16(p, dst + (q * NW + w) * 1024);
  }
  // A lane's fragment (16 columns x 64 bytes of k) of the columns `at` further (a multiple of 16 that
  // shares no bit with the base's column before the swizzle) and k-step ks, at base ^ (SZ at).
  __device__ static uint32_t lane_base(int mn0) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    if constexpr (SZ == 2) {
      const int k = g * 8 + (i >> 2), mn = mn0 + 4 * (i & 3);
      return k * PITCH + ((mn >> 3) ^ DnMma<T>::template swz<PITCH>(k)) * 16 + (mn & 7) * 2;
    } else {
      const int k = g * 4, mn = mn0 + i;
      return k * PITCH + ((mn >> 2) ^ DnMma<T>::template swz<PITCH>(k)) * 16 + (mn & 3) * 4;
    }
  }
  __device__ static Frag frag(const char* t, uint32_t base, int at, int ks) {
    const char* p = t + (base ^ (at * SZ)) + ks * (dn_bk<T>() / 2) * PITCH;
    if constexpr (SZ == 2) {
      const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p);
      const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * PITCH));
      const v4i16 both[2] = {lo, hi};
      Frag r;
      __builtin_memcpy(&r, both, 16);
      return r;
    } else {
      Frag r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const float*>(p + i * PITCH);
      return r;
    }
  }
};

// Accumulators of a wave: MI x 4 blocks of 16 x 16.  The MFMA computes the transposed block, so
// register v of block (i, 2 j + h) holds row 16 i + lane % 16 of the wave and column
// dn_col(j, h, v) of the tile.
template <int MI>
struct DnAcc {
  f32x4 c[MI][4];
};

// TM x TN tiles; WM x WN waves of 16 MI rows x 64 columns: 32 columns in each tile half.
template <int TM, int TN, int WM, int WN>
struct DnTile {
  static constexpr int TM_ = TM, WN_ = WN, SPLIT = TM / 2;
  static constexpr int NW = WM * WN, THREADS = 64 * NW, MI = TM / WM / 16, MH = MI / 2;
  static constexpr int A_BYTES = TM * 128, STAGE = (TM + TN) * 128;
  static constexpr int HC = TN / 2;          // columns per tile half
  static constexpr int EPITCH = HC * 4 + 16; // fp32 staging row of a tile half
  static constexpr int SLOT = STAGE > TM / 2 * EPITCH ? STAGE : TM / 2 * EPITCH;
  static_assert(HC == WN * 32, "two 16-column blocks of each half per wave");
};
// Column within its tile half of a lane's four accumulators of block 2 j + h.
__device__ __forceinline__ int dn_col(int wn, int h) { return wn * 32 + h * 16 + ((threadIdx.x & 63) >> 4) * 4; }

// A wave's LDS bases of its A and B fragments in a slot.
struct DnLds {
  uint32_t a, b;
};
// Fragments of one k-step: B whole, A in two halves of MH row blocks.
template <class TI, class Frag> struct DnFragA { Frag f[TI::MH]; };
template <class Frag> struct DnFragB { Frag f[4]; };
template <class TI, class AL>
__device__ __forceinline__ void dn_read_a(const char* slot, int ks, int half, const DnLds& d, DnFragA<TI, typename AL::Frag>& F) {
#pragma unroll
  for (int i = 0; i < TI::MH; ++i) F.f[i] = AL::frag(slot, d.a, (half * TI::MH + i) * 16, ks);
}
template <class TI, class BL>
__device__ __forceinline__ void dn_read_b(const char* slot, int ks, const DnLds& d, DnFragB<typename BL::Frag>& F) {
#pragma unroll
  for (int j = 0; j < 4; ++j) F.f[j] = BL::frag(slot + TI::A_BYTES, d.b, (j >> 1) * TI::HC + (j & 1) * 16, ks);
}

// The 4 MH MFMA blocks of one half k-step, FROM .. TO - 1 of them, with DMA instructions N0 ..
// N1 - 1 spread between them.
template <class TI, int HALF, int FROM, int TO, int N0 = 0, int N1 = 0, class Frag, class Issue>
__device__ __forceinline__ void dn_mma(const DnFragA<TI, Frag>& A, const DnFragB<Frag>& B, DnAcc<TI::MI>& acc, Issue issue) {
  typedef DnMma<typename std::conditional<std::is_same<Frag, bf16x8>::value, bf16, float>::type> M;
#pragma unroll
  for (int p = FROM; p < TO; ++p) {
#pragma unroll
    for (int n = N0; n < N1; ++n)
      if (FROM + (n - N0) * (TO - FROM) / (N1 > N0 ? N1 - N0 : 1) == p) {
        __builtin_amdgcn_sched_barrier(0);
        issue(n);
        __builtin_amdgcn_sched_barrier(0);
      }
    f32x4& c = acc.c[HALF * TI::MH + (p >> 2)][p & 3];
    c = M::mma(B.f[p & 3], A.f[p >> 2], c);
  }
}

// One stage: two k-steps, each in two halves (the upper and the lower half of the wave's
// rows), four quarters of 4 MH MFMAs.  B0 and A0 hold the first quarter's fragments (read beside
// the previous stage's last MFMAs); the others are read between the first quarter's MFMAs, and
// stage s + 2 goes out beside the second and third quarter.  END: that stage may be the last one.
template <class TI, bool END, class AL, class BL>
__device__ __forceinline__ void dn_step(const AL& la, const BL& lb, int s, int nkt, char* cur, const char* next,
                                        DnLds& d, DnFragA<TI, typename AL::Frag>& A0, DnFragB<typename AL::Frag>& B0,
                                        DnAcc<TI::MI>& acc) {
  constexpr int NM = 4 * TI::MH;
  constexpr int NI = AL::NQ + BL::NQ;  // DMA instructions per wave and stage
  const int r = END ? min(s + 2, nkt - 1) : s + 2;  // past the end the last stage again: the waits count on it
  auto issue = [&](int n) {
    if (n < AL::NQ) la.template issue<END>(r, n, cur);
    else lb.template issue<END>(r, n - AL::NQ, cur + TI::A_BYTES);
  };
  // the bases are opaque here, so that the fragments' addresses are formed at their reads instead
  // of being kept in registers across the loop
  asm volatile("" : "+v"(d.a), "+v"(d.b));
  DnFragA<TI, typename AL::Frag> A1, A2, A3;
  DnFragB<typename AL::Frag> B1;
  dn_mma<TI, 0, 0, 1>(A0, B0, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  dn_read_a<TI, AL>(cur, 0, 1, d, A1);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 0, 1, NM / 4>(A0, B0, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" : "+v"(d.a), "+v"(d.b));
  dn_read_b<TI, BL>(cur, 1, d, B1);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 0, NM / 4, 7 * NM / 16>(A0, B0, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  dn_read_a<TI, AL>(cur, 1, 0, d, A2);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 0, 7 * NM / 16, 10 * NM / 16>(A0, B0, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" : "+v"(d.a));
  dn_read_a<TI, AL>(cur, 1, 1, d, A3);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 0, 10 * NM / 16, NM>(A0, B0, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read the whole stage
  ring_barrier();                      // so has every wave: its slot is free
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 1, 0, NM, 0, NI / 2>(A1, B0, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 0, 0, NM, NI / 2, NI>(A2, B1, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 1, 0, NM / 4>(A3, B1, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<NI>();
  ring_barrier();
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 1, NM / 4, NM / 4 + 1>(A3, B1, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
  dn_read_b<TI, BL>(next, 0, d, B0);
  dn_read_a<TI, AL>(next, 0, 0, d, A0);
  __builtin_amdgcn_sched_barrier(0);
  dn_mma<TI, 1, NM / 4 + 1, NM>(A3, B1, acc, issue);
  __builtin_amdgcn_sched_barrier(0);
}

// The main loop over nkt stages, accumulating from zero; ends with the LDS free.
template <class TI, class AL, class BL>
__device__ __forceinline__ void dn_mainloop(const AL& la, const BL& lb, int nkt, DnAcc<TI::MI>& acc, char* b0, char* b1,
                                            int wm, int wn) {
#pragma unroll
  for (int i = 0; i < TI::MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc.c[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (nkt <= 0) return;
  const int r1 = min(1, nkt - 1);
#pragma unroll
  for (int q = 0; q < AL::NQ; ++q) la.template issue<true>(0, q, b0);
#pragma unroll
  for (int q = 0; q < BL::NQ; ++q) lb.template issue<true>(0, q, b0 + TI::A_BYTES);
#pragma unroll
  for (int q = 0; q < AL::NQ; ++q) la.template issue<true>(r1, q, b1);
#pragma unroll
  for (int q = 0; q < BL::NQ; ++q) lb.template issue<true>(r1, q, b1 + TI::A_BYTES);
  wait_vmcnt<AL::NQ + BL::NQ>();
  ring_barrier();
  DnFragA<TI, typename AL::Frag> A0;
  DnFragB<typename AL::Frag> B0;
  DnLds d{AL::lane_base(wm * TI::MI * 16), BL::lane_base(wn * 32)};
  dn_read_b<TI, BL>(b0, 0, d, B0);
  dn_read_a<TI, AL>(b0, 0, 0, d, A0);
  int s = 0;
  // the steps that load no last stage, apart where that takes the selection of addresses off them
  // (8190 x 4000 x 4096 backward 540 -> 445 us)
  if constexpr (AL::PARTIAL)
    for (; s + 4 < nkt; s += 2) {
      dn_step<TI, false>(la, lb, s, nkt, b0, b1, d, A0, B0, acc);
      dn_step<TI, false>(la, lb, s + 1, nkt, b1, b0, d, A0, B0, acc);
    }
  for (; s + 2 <= nkt; s += 2) {
    dn_step<TI, true>(la, lb, s, nkt, b0, b1, d, A0, B0, acc);
    dn_step<TI, true>(la, lb, s + 1, nkt, b1, b0, d, A0, B0, acc);
  }
  if (s < nkt) dn_step<TI, true>(la, lb, s, nkt, b0, b1, d, A0, B0, acc);
  __syncthreads();  // drains the trailing loads; the LDS is free for the epilogue
}

}  // namespace moe
