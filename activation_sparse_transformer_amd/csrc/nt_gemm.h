// Products C = A B^T on MFMA (32x32x16).  An operand is held in
// one of three forms:
//  - kBf16:    one bfloat16 part, as bfloat16 tensors are;
//  - kHalves:  two half-precision parts hi + lo of a float32 value times a power of
//              two that brings the matrix (or row) below 2^15.  Both round to 11 bits,
//              so |lo| <= 2^-11 |v| and hi + lo is within 2^-23 of v (2^-24 in the
//              mean), or within 2^-25 (2^-39 of the largest) where lo is subnormal;
//              MFMA keeps subnormal inputs.  Of the four products lo lo, 2^-24 of the
//              whole in the mean and at most 2^-22, is left out: three products, where
//              three bfloat16 parts would take six for the same 24 bits and MFMA's own
//              float32 form sixteen times one.  MFMA cuts a sum's last bits at every
//              step, so the two small products go over the whole of K first and the
//              large one last: no more cuts at the sum's full size than a product of
//              one part has.
//  - kHalf:    the hi part alone, within 2^-11 of v.
//  - kRaw:     float32 as it lies, for few rows, where a pass over the other operand
//              to split it would cost as much as the product: fragments are split into
//              three bfloat16 parts (8 + 8 + 8 bits, of any exponent) as they leave
//              LDS (B's, which all waves share, once a stage by the workgroup), six
//              products, the five small ones in accumulators of their own.
// A product's form is that of both operands, or one of a mixed pair: kMixed, A in kHalf
// and B in kHalves, and kBf16Two, A in kBf16 and B as two bfloat16 parts.
//
// Operands are [parts][rows][ld], K along a row (rows past the end read the last row
// and feed outputs that no epilogue stores), or turned, [parts][depth][ld] with K along
// the column (rows, a multiple of 8, are then columns of that).  K past `depth`, a
// multiple of 8 where it runs along rows, reads zeros.  A kRaw operand is addressed in
// 16-bit units: ld and a straight operand's depth count two per float.
#pragma once

#include <algorithm>

#include "common.h"

namespace twell {
namespace nt {

constexpr int kStep = 64;  // K elements of one LDS stage

enum Form { kBf16, kHalf, kHalves, kMixed, kBf16Two, kRaw };
constexpr int parts_of(Form f) { return f == kHalves ? 2 : 1; }
constexpr bool two_parts_of_b(Form f) { return f == kMixed || f == kBf16Two; }
constexpr int products_of(Form f) { return f == kHalves ? 3 : two_parts_of_b(f) ? 2 : 1; }
constexpr bool is_bf16(Form f) { return f == kBf16 || f == kBf16Two; }

struct Operand {
  const uint16_t* p;
  int64_t part;  // elements between parts
  int64_t ld;    // elements between rows (turned: between steps of K)
  int rows;
  int depth;     // K
};

__device__ const uint4 kZeros = {0, 0, 0, 0};  // what K past an operand's depth reads

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) int i32x4_t;

// Rows of 64 elements in LDS, the 16-byte chunk kc of row r at position kc ^
// swizzle(r): the 32 rows x 2 chunks of a fragment read fall on distinct banks.
__device__ __forceinline__ int swizzle(int r) { return (r ^ (r >> 3)) & 7; }
__device__ __forceinline__ int tile_offset(int r, int kc) {
  return r * kStep + ((kc ^ swizzle(r)) << 3);
}

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct Config {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int STAGES = STAGES_;
  static constexpr int NW = WAVES_M * WAVES_N, NT = NW * kWave;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;  // a wave's tile
  static constexpr int FM = WTM / 32, FN = WTN / 32;            // its 32x32 blocks
  static constexpr int A_ISSUE = BM / (8 * NW), B_ISSUE = BN / (8 * NW);  // copies a stage
  static constexpr int STAGE = (BM + BN) * kStep;  // elements
  static_assert(A_ISSUE * 8 * NW == BM && B_ISSUE * 8 * NW == BN, "whole 1 KB copies per wave");
  static_assert(FM * 32 == WTM && FN * 32 == WTN, "32x32 blocks");
};

// Copies of one operand to a stage: instruction i of a wave fills 1 KB; lane l fetches
// the chunk that belongs at LDS position l.  SIZE: the block's rows.
template <int SIZE, int NW, bool TURNED>
struct Copies;

template <int SIZE, int NW>
struct Copies<SIZE, NW, false> {  // 8 rows of 64 elements each
  static constexpr int ISSUE = SIZE / (8 * NW);
  const uint16_t* src[ISSUE];
  int left;  // of K
  static __device__ __forceinline__ int chunk(int i) {
    const int r = (threadIdx.x / kWave + NW * i) * 8 + lane_id() / 8;
    return ((lane_id() & 7) ^ swizzle(r)) * 8;
  }
  __device__ __forceinline__ Copies(const Operand& o, int r0, int k0) : left(o.depth - k0) {
#pragma unroll
    for (int i = 0; i < ISSUE; ++i) {
      const int r = (threadIdx.x / kWave + NW * i) * 8 + lane_id() / 8;
      src[i] = o.p + static_cast<int64_t>(min(r0 + r, o.rows - 1)) * o.ld + k0 + chunk(i);
    }
  }
  __device__ __forceinline__ void issue(int k, int64_t part, uint16_t* tile) const {
    const int wave = threadIdx.x / kWave;
    if (k + kStep <= left) {
#pragma unroll
      for (int i = 0; i < ISSUE; ++i)
        __builtin_amdgcn_global_load_lds(src[i] + part + k, tile + (wave + NW * i) * 512, 16, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < ISSUE; ++i)
        __builtin_amdgcn_global_load_lds(
            k + chunk(i) < left ? src[i] + part + k : reinterpret_cast<const uint16_t*>(&kZeros),
            tile + (wave + NW * i) * 512, 16, 0, 0);
    }
  }
};

// A turned operand's stage: 64 lines (k) of SIZE elements, the 32-byte chunk c of line k
// at position c ^ turned_swizzle(k): the 4 lines x 64 bytes that 32 lanes of a transpose
// read take fall on distinct ones of the 64 banks.
__device__ __forceinline__ int turned_swizzle(int k) { return (k & 3) << 1 | (k >> 3 & 1); }
template <int SIZE>
__device__ __forceinline__ int turned_offset(int k, int r) {
  return k * SIZE + ((((r >> 4) ^ turned_swizzle(k)) & (SIZE / 16 - 1)) << 4) + (r & 15);
}

template <int SIZE, int NW>
struct Copies<SIZE, NW, true> {  // 512 / SIZE lines each
  static constexpr int ISSUE = SIZE / (8 * NW);
  const uint16_t* src[ISSUE];
  int line[ISSUE];
  int64_t ld;
  int left;  // of K
  __device__ __forceinline__ Copies(const Operand& o, int r0, int k0)
      : ld(o.ld), left(o.depth - k0) {
    const int lane = lane_id(), wave = threadIdx.x / kWave;
#pragma unroll
    for (int i = 0; i < ISSUE; ++i) {
      line[i] = (wave + NW * i) * (512 / SIZE) + lane * 8 / SIZE;
      const int at = lane * 8 % SIZE;
      const int r = (((at >> 4) ^ turned_swizzle(line[i])) & (SIZE / 16 - 1)) * 16 + (at & 15);
      src[i] = o.p + static_cast<int64_t>(k0) * ld + min(r0 + r, o.rows - 8);
    }
  }
  __device__ __forceinline__ void issue(int k, int64_t part, uint16_t* tile) const {
    const int wave = threadIdx.x / kWave;
    const uint16_t* const zeros = reinterpret_cast<const uint16_t*>(&kZeros);
    const bool whole = k + kStep <= left;
#pragma unroll
    for (int i = 0; i < ISSUE; ++i) {
      const uint16_t* const p = src[i] + part + (line[i] + k) * ld;
      __builtin_amdgcn_global_load_lds(whole || line[i] + k < left ? p : zeros,
                                       tile + (wave + NW * i) * 512, 16, 0, 0);
    }
  }
};

// Floats, a stage of 32 lines of SIZE as they lie: a lane's reads of a column are spread
// over the banks by the lanes' columns.  k counts floats.
template <int SIZE, int NW>
struct RawTurnedCopies {
  static constexpr int ISSUE = SIZE / (8 * NW);
  const uint16_t* src[ISSUE];
  int64_t ld;
  int left;
  static __device__ __forceinline__ int line(int i) {
    return (threadIdx.x / kWave + NW * i) * (256 / SIZE) + lane_id() * 4 / SIZE;
  }
  __device__ __forceinline__ RawTurnedCopies(const Operand& o, int r0, int k0)
      : ld(o.ld), left(o.depth - k0) {
#pragma unroll
    for (int i = 0; i < ISSUE; ++i)
      src[i] = o.p + (k0 + line(i)) * ld + 2 * min(r0 + lane_id() * 4 % SIZE, o.rows - 4);
  }
  __device__ __forceinline__ void issue(int k, uint16_t* tile) const {
    const int wave = threadIdx.x / kWave;
#pragma unroll
    for (int i = 0; i < ISSUE; ++i) {
      const uint16_t* p = src[i] + k * ld;
      if (line(i) + k >= left) p = reinterpret_cast<const uint16_t*>(&kZeros);
      __builtin_amdgcn_global_load_lds(p, tile + (wave + NW * i) * 512, 16, 0, 0);
    }
  }
};

typedef __attribute__((address_space(3))) uint16_t lds_u16;
__device__ __forceinline__ uint32_t lds_address(const uint16_t* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u16*)p));
}

// LDS byte offsets, within a stage, of a lane's fragments of the block of 32 rows from r0.
// K along rows: of 16-wide K step ks, a 16-byte read.  Turned: of step 0; lanes 16 h + L
// of a half hold rows 16 h + L, a transpose read of 16 lanes takes lines k .. k + 3 of 16
// rows, lane L pointing at line k + L / 4, row 4 (L % 4), and a fragment is two of them,
// 4 lines apart.  Steps are 16 lines apart: 4 and 16 lines on, the swizzle is the same.
__device__ __forceinline__ uint32_t straight_at(int r0, int ks) {
  return 2u * tile_offset(r0 + (lane_id() & 31), ks * 2 + (lane_id() >> 5));
}
template <int SIZE>
__device__ __forceinline__ uint32_t turned_at(int r0) {
  const int l = lane_id(), L = l & 15;
  return 2u * turned_offset<SIZE>((l >> 5) * 8 + L / 4, r0 + ((l >> 4) & 1) * 16 + 4 * (L & 3));
}

typedef __attribute__((ext_vector_type(2))) int i32x2_t;
__device__ __forceinline__ i32x4_t joined(i32x2_t a, i32x2_t b) {
  return i32x4_t{a[0], a[1], b[0], b[1]};
}

// The fragments of all K steps of a turned stage, of one block of rows.  The transpose
// reads are asm, as the compiler puts a wait for every copy in flight before its own.
template <int SIZE>
__device__ __forceinline__ void read_turned(uint32_t at, i32x4_t (&f)[4]) {
  i32x2_t v[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%9\n\t"
      "ds_read_b64_tr_b16 %2, %8 offset:%10\n\t"
      "ds_read_b64_tr_b16 %3, %8 offset:%11\n\t"
      "ds_read_b64_tr_b16 %4, %8 offset:%12\n\t"
      "ds_read_b64_tr_b16 %5, %8 offset:%13\n\t"
      "ds_read_b64_tr_b16 %6, %8 offset:%14\n\t"
      "ds_read_b64_tr_b16 %7, %8 offset:%15\n\t"
      "s_waitcnt lgkmcnt(0)\n\t"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]),
        "=&v"(v[7])
      : "v"(at), "n"(8 * SIZE), "n"(32 * SIZE), "n"(40 * SIZE), "n"(64 * SIZE), "n"(72 * SIZE),
        "n"(96 * SIZE), "n"(104 * SIZE)
      : "memory");
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) f[ks] = joined(v[2 * ks], v[2 * ks + 1]);
}

// The fragments of all K steps of a stage at `tile`, of BLOCKS blocks of rows from r0.
template <int SIZE, int BLOCKS, bool TURNED>
__device__ __forceinline__ void read_stage(const uint16_t* tile, int r0,
                                           i32x4_t (&f)[BLOCKS][4]) {
#pragma unroll
  for (int i = 0; i < BLOCKS; ++i) {
    if constexpr (TURNED) {
      read_turned<SIZE>(lds_address(tile) + turned_at<SIZE>(r0 + 32 * i), f[i]);
    } else {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        f[i][ks] = *reinterpret_cast<const i32x4_t*>(reinterpret_cast<const char*>(tile) +
                                                     straight_at(r0 + 32 * i, ks));
    }
  }
}

// The steps of a contraction: a product of parts after another, each over the whole
// of K, in the order lo hi (kHalves), hi lo, hi hi.
template <Form F>
struct Walk {
  int64_t part_a, part_b;
  int end;  // of K
  int k = 0, left = products_of(F) - 1;
  __device__ __forceinline__ void next() {
    k += kStep;
    if (products_of(F) > 1 && k == end) {
      k = 0;
      --left;
    }
  }
  __device__ __forceinline__ int64_t a() const { return F == kHalves && left == 2 ? part_a : 0; }
  __device__ __forceinline__ int64_t b() const {
    return products_of(F) > 1 && left == 1 ? part_b : 0;
  }
};

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
template <Form F>
__device__ __forceinline__ f32x16_t mfma(i32x4_t a, i32x4_t b, f32x16_t c) {
  if constexpr (is_bf16(F))
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// All but the last N copies of every wave landed, and every wave is done with its
// LDS reads so far.
template <int N>
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// acc = A[m0 .., k0 .. k0 + 64 ksteps) B[n0 .., the same]^T.  `lds`: STAGES stages.
// Copies run STAGES - 1 stages ahead of the products.
template <class CF, Form F, bool TA, bool TB>
__device__ __forceinline__ void mainloop(const Operand& A, int m0, const Operand& B, int n0, int k0,
                                         int ksteps, uint16_t* lds,
                                         f32x16_t (&acc)[CF::FM][CF::FN]) {
#pragma unroll
  for (int i = 0; i < CF::FM; ++i)
#pragma unroll
    for (int j = 0; j < CF::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const Copies<CF::BM, CF::NW, TA> a_copies(A, m0, k0);
  const Copies<CF::BN, CF::NW, TB> b_copies(B, n0, k0);
  const int wave = threadIdx.x / kWave;
  const int ra = wave / CF::WAVES_N * CF::WTM, rb = wave % CF::WAVES_N * CF::WTN;
  constexpr int AHEAD = CF::STAGES - 1, COPIES = CF::A_ISSUE + CF::B_ISSUE;
  const int steps = ksteps * products_of(F);
  Walk<F> walk{A.part, B.part, ksteps * kStep};
  int fill = 0;  // the stage that the next copies go to
  auto copy = [&]() {
    uint16_t* stage = lds + fill * CF::STAGE;
    a_copies.issue(walk.k, walk.a(), stage);
    b_copies.issue(walk.k, walk.b(), stage + CF::BM * kStep);
    walk.next();
    fill = fill + 1 == CF::STAGES ? 0 : fill + 1;
  };
  for (int s = 0; s < AHEAD && s < steps; ++s) copy();
  int cur = 0;
  for (int s = 0; s < steps; ++s) {
    // stages s + 1 .. s + AHEAD - 1 may be in flight; near the end there are fewer
    if (s + AHEAD <= steps) meet<(AHEAD - 1) * COPIES>();
    else meet<0>();
    if (s + AHEAD < steps) copy();
    const uint16_t* sA = lds + cur * CF::STAGE;
    const uint16_t* sB = sA + CF::BM * kStep;
    i32x4_t a[CF::FM][4], b[CF::FN][4];
    read_stage<CF::BM, CF::FM, TA>(sA, ra, a);
    read_stage<CF::BN, CF::FN, TB>(sB, rb, b);
#pragma unroll
    for (int ks = 0; ks < kStep / 16; ++ks)
#pragma unroll
      for (int i = 0; i < CF::FM; ++i)
#pragma unroll
        for (int j = 0; j < CF::FN; ++j) acc[i][j] = mfma<F>(a[i][ks], b[j][ks], acc[i][j]);
    cur = cur + 1 == CF::STAGES ? 0 : cur + 1;
  }
  __syncthreads();  // the stages are free for the epilogue
}

// ---- The same for waves of 64 rows and 128 or 64 columns (2 x 4 or 2 x 2 blocks),
// software-pipelined.  Each 16-wide K step is one asm block: the MFMAs of the fragments in
// hand with the LDS reads of the next step's fragments between them, and a wait for those
// reads at its end (no read is in flight when the block ends).  The MFMAs of a stage's last
// step run behind the next stage's barrier, beside the reads of its first step.  Same
// products in the same order as mainloop.
template <int FN>
struct Fragments {
  i32x4_t a[2], b[FN];
};
template <int FN>
struct Addresses {  // LDS addresses of the next fragments (turned: of K step 0)
  uint32_t a[2], b[FN];
};

// The reads of fragment `f` (a0, a1, b0 .. b3) at address p##f
#define NT_READ(f) "ds_read_b128 %[n" #f "], %[p" #f "]\n\t"
#define NT_READ_TURNED(f, lo, hi)                                     \
  "ds_read_b64_tr_b16 %[n" #f "], %[p" #f "] offset:%[" #lo "]\n\t"  \
  "ds_read_b64_tr_b16 %[h" #f "], %[p" #f "] offset:%[" #hi "]\n\t"
#define NT_READ_TA(f) NT_READ_TURNED(f, lo_a, hi_a)
#define NT_READ_TB(f) NT_READ_TURNED(f, lo_b, hi_b)
// Operand lists, with 2 and with 4 blocks of columns
#define NT_ACC2                                                                               \
  [c00] "+v"(c[0][0]), [c01] "+v"(c[0][1]), [c10] "+v"(c[1][0]), [c11] "+v"(c[1][1])
#define NT_ACC4                                                                               \
  NT_ACC2, [c02] "+v"(c[0][2]), [c03] "+v"(c[0][3]), [c12] "+v"(c[1][2]), [c13] "+v"(c[1][3])
#define NT_OUT_A [na0] "=&v"(nxt.a[0]), [na1] "=&v"(nxt.a[1])
#define NT_OUT_B2 [nb0] "=&v"(nxt.b[0]), [nb1] "=&v"(nxt.b[1])
#define NT_OUT_B4 NT_OUT_B2, [nb2] "=&v"(nxt.b[2]), [nb3] "=&v"(nxt.b[3])
#define NT_OUT_TA [na0] "=&v"(la[0]), [ha0] "=&v"(ha[0]), [na1] "=&v"(la[1]), [ha1] "=&v"(ha[1])
#define NT_OUT_TB2 [nb0] "=&v"(lb[0]), [hb0] "=&v"(hb[0]), [nb1] "=&v"(lb[1]), [hb1] "=&v"(hb[1])
#define NT_OUT_TB4                                                                            \
  NT_OUT_TB2, [nb2] "=&v"(lb[2]), [hb2] "=&v"(hb[2]), [nb3] "=&v"(lb[3]), [hb3] "=&v"(hb[3])
#define NT_CUR2 [a0] "v"(cur.a[0]), [a1] "v"(cur.a[1]), [b0] "v"(cur.b[0]), [b1] "v"(cur.b[1])
#define NT_CUR4 NT_CUR2, [b2] "v"(cur.b[2]), [b3] "v"(cur.b[3])
#define NT_AT2                                                                                \
  [pa0] "v"(at.a[0]), [pa1] "v"(at.a[1]), [pb0] "v"(at.b[0]), [pb1] "v"(at.b[1]),             \
      [lo_a] "n"(32 * KS * CF::BM), [hi_a] "n"(32 * KS * CF::BM + 8 * CF::BM),                \
      [lo_b] "n"(32 * KS * CF::BN), [hi_b] "n"(32 * KS * CF::BN + 8 * CF::BN)
#define NT_AT4 NT_AT2, [pb2] "v"(at.b[2]), [pb3] "v"(at.b[3])
#define NT_STEP2(MFMA, RA, RB, OUT_A, OUT_B)                                                  \
  asm volatile(RA(a0) MFMA " %[c00], %[a0], %[b0], %[c00]\n\t" RA(a1) MFMA                    \
               " %[c01], %[a0], %[b1], %[c01]\n\t" RB(b0) MFMA                                \
               " %[c10], %[a1], %[b0], %[c10]\n\t" RB(b1) MFMA                                \
               " %[c11], %[a1], %[b1], %[c11]\n\ts_waitcnt lgkmcnt(0)\n\t"                    \
               : NT_ACC2, OUT_A, OUT_B##2                                                     \
               : NT_CUR2, NT_AT2                                                              \
               : "memory")
#define NT_STEP4(MFMA, RA, RB, OUT_A, OUT_B)                                                  \
  asm volatile(RA(a0) MFMA " %[c00], %[a0], %[b0], %[c00]\n\t" RA(a1) MFMA                    \
               " %[c01], %[a0], %[b1], %[c01]\n\t" RB(b0) MFMA                                \
               " %[c02], %[a0], %[b2], %[c02]\n\t" RB(b1) MFMA                                \
               " %[c03], %[a0], %[b3], %[c03]\n\t" RB(b2) MFMA                                \
               " %[c10], %[a1], %[b0], %[c10]\n\t" RB(b3) MFMA                                \
               " %[c11], %[a1], %[b1], %[c11]\n\t" MFMA " %[c12], %[a1], %[b2], %[c12]\n\t"   \
               MFMA " %[c13], %[a1], %[b3], %[c13]\n\ts_waitcnt lgkmcnt(0)\n\t"               \
               : NT_ACC4, OUT_A, OUT_B##4                                                     \
               : NT_CUR4, NT_AT4                                                              \
               : "memory")
#define NT_LOAD2(RA, RB, OUT_A, OUT_B)                                                        \
  asm volatile(RA(a0) RA(a1) RB(b0) RB(b1) "s_waitcnt lgkmcnt(0)\n\t"                         \
               : OUT_A, OUT_B##2                                                              \
               : NT_AT2                                                                       \
               : "memory")
#define NT_LOAD4(RA, RB, OUT_A, OUT_B)                                                        \
  asm volatile(RA(a0) RA(a1) RB(b0) RB(b1) RB(b2) RB(b3) "s_waitcnt lgkmcnt(0)\n\t"           \
               : OUT_A, OUT_B##4                                                              \
               : NT_AT4                                                                       \
               : "memory")
#define NT_FORMS(DO, ...)                                                                     \
  if constexpr (TA && TB) DO(__VA_ARGS__ NT_READ_TA, NT_READ_TB, NT_OUT_TA, NT_OUT_TB);       \
  else if constexpr (TA) DO(__VA_ARGS__ NT_READ_TA, NT_READ, NT_OUT_TA, NT_OUT_B);            \
  else DO(__VA_ARGS__ NT_READ, NT_READ, NT_OUT_A, NT_OUT_B)
#define NT_BF16 "v_mfma_f32_32x32x16_bf16"
#define NT_F16 "v_mfma_f32_32x32x16_f16"

// The MFMAs of cur beside the reads of nxt, K step KS of its stage.  First: the reads alone.
template <class CF, Form F, bool TA, bool TB, int KS, bool FIRST = false>
__device__ __forceinline__ void pipe_step(f32x16_t (&c)[2][CF::FN], const Fragments<CF::FN>& cur,
                                          Fragments<CF::FN>& nxt, const Addresses<CF::FN>& at) {
  static_assert(TA || !TB, "no product turns its columns alone");
  i32x2_t la[2], ha[2], lb[CF::FN], hb[CF::FN];
  if constexpr (CF::FN == 4) {
    if constexpr (FIRST) { NT_FORMS(NT_LOAD4); }
    else if constexpr (is_bf16(F)) { NT_FORMS(NT_STEP4, NT_BF16,); }
    else { NT_FORMS(NT_STEP4, NT_F16,); }
  } else {
    if constexpr (FIRST) { NT_FORMS(NT_LOAD2); }
    else if constexpr (is_bf16(F)) { NT_FORMS(NT_STEP2, NT_BF16,); }
    else { NT_FORMS(NT_STEP2, NT_F16,); }
  }
  if constexpr (TA) {
#pragma unroll
    for (int i = 0; i < 2; ++i) nxt.a[i] = joined(la[i], ha[i]);
  }
  if constexpr (TB) {
#pragma unroll
    for (int j = 0; j < CF::FN; ++j) nxt.b[j] = joined(lb[j], hb[j]);
  }
}
#undef NT_READ
#undef NT_READ_TURNED
#undef NT_READ_TA
#undef NT_READ_TB
#undef NT_ACC2
#undef NT_ACC4
#undef NT_OUT_A
#undef NT_OUT_B2
#undef NT_OUT_B4
#undef NT_OUT_TA
#undef NT_OUT_TB2
#undef NT_OUT_TB4
#undef NT_CUR2
#undef NT_CUR4
#undef NT_AT2
#undef NT_AT4
#undef NT_STEP2
#undef NT_STEP4
#undef NT_LOAD2
#undef NT_LOAD4
#undef NT_FORMS
#undef NT_BF16
#undef NT_F16

// VALU writes of the accumulators before MFMAs in asm, and MFMA results before VALU
// reads: the accumulators are operands, so neither moves across the wait.
template <int FN>
__device__ __forceinline__ void settle(f32x16_t (&c)[2][FN]) {
#pragma unroll
  for (int j = 0; j < FN; j += 2)
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15"
                 : "+v"(c[0][j]), "+v"(c[0][j + 1]), "+v"(c[1][j]), "+v"(c[1][j + 1]));
}

template <class CF, Form F, bool TA, bool TB>
__device__ __forceinline__ void mainloop_pipe(const Operand& A, int m0, const Operand& B, int n0,
                                              int k0, int ksteps, uint16_t* lds,
                                              f32x16_t (&acc)[2][CF::FN]) {
  static_assert(CF::FM == 2 && (CF::FN == 4 || CF::FN == 2) && CF::STAGES == 2, "a wave's blocks");
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < CF::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int steps = ksteps * products_of(F);
  if (steps == 0) return;
  settle(acc);
  const Copies<CF::BM, CF::NW, TA> a_copies(A, m0, k0);
  const Copies<CF::BN, CF::NW, TB> b_copies(B, n0, k0);
  const int wave = threadIdx.x / kWave;
  const int ra = wave / CF::WAVES_N * CF::WTM, rb = wave % CF::WAVES_N * CF::WTN;
  const uint32_t base_a = lds_address(lds), base_b = base_a + 2 * CF::BM * kStep;
  Addresses<CF::FN> first[4];  // in stage 0, of each K step (turned: the same)
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      first[ks].a[i] =
          base_a + (TA ? turned_at<CF::BM>(ra + 32 * i) : straight_at(ra + 32 * i, ks));
#pragma unroll
    for (int j = 0; j < CF::FN; ++j)
      first[ks].b[j] =
          base_b + (TB ? turned_at<CF::BN>(rb + 32 * j) : straight_at(rb + 32 * j, ks));
  }
  Walk<F> walk{A.part, B.part, ksteps * kStep};
  auto copy = [&](int stage) {
    uint16_t* to = lds + stage * CF::STAGE;
    a_copies.issue(walk.k, walk.a(), to);
    b_copies.issue(walk.k, walk.b(), to + CF::BM * kStep);
    walk.next();
  };
  Fragments<CF::FN> f0, f1;
  copy(0);
  meet<0>();
  if (steps > 1) copy(1);
  pipe_step<CF, F, TA, TB, 0, true>(acc, f1, f0, first[0]);
  pipe_step<CF, F, TA, TB, 1>(acc, f0, f1, first[1]);
  pipe_step<CF, F, TA, TB, 2>(acc, f1, f0, first[2]);
  pipe_step<CF, F, TA, TB, 3>(acc, f0, f1, first[3]);
  for (int s = 1; s < steps; ++s) {  // f1: the fragments of the last K step of stage s - 1
    meet<0>();
    if (s + 1 < steps) copy((s + 1) & 1);
    const uint32_t shift = static_cast<uint32_t>(s & 1) * (CF::STAGE * 2);
    Addresses<CF::FN> at[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
      for (int i = 0; i < 2; ++i) at[ks].a[i] = first[ks].a[i] + shift;
#pragma unroll
      for (int j = 0; j < CF::FN; ++j) at[ks].b[j] = first[ks].b[j] + shift;
    }
    pipe_step<CF, F, TA, TB, 0>(acc, f1, f0, at[0]);
    pipe_step<CF, F, TA, TB, 1>(acc, f0, f1, at[1]);
    pipe_step<CF, F, TA, TB, 2>(acc, f1, f0, at[2]);
    pipe_step<CF, F, TA, TB, 3>(acc, f0, f1, at[3]);
  }
  settle(acc);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < CF::FN; ++j) acc[i][j] = mfma<F>(f1.a[i], f1.b[j], acc[i][j]);
  __syncthreads();  // the stages are free for the epilogue
}

// Three bfloat16 parts of 8 floats.  The first ends at the largest bfloat16, as a larger
// float32 would round to an infinity there.
__device__ __forceinline__ void split3(const float (&v)[8], i32x4_t (&part)[3]) {
  typedef __attribute__((ext_vector_type(2))) float f32x2_t;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a = v[2 * k], b = v[2 * k + 1];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      constexpr float kMost = 0x1.fep127f;
      const f32x2_t in = p > 0 ? f32x2_t{a, b}
                               : f32x2_t{__builtin_amdgcn_fmed3f(a, -kMost, kMost),
                                         __builtin_amdgcn_fmed3f(b, -kMost, kMost)};
      const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(in, bf16x2_t));
      part[p][k] = static_cast<int>(w);
      a -= __uint_as_float(w << 16);
      b -= __uint_as_float(w & 0xffff0000u);
    }
  }
}

// 8 floats from 8 c on of K of a raw stage: of row r of a straight one, column r of a
// turned one.
__device__ __forceinline__ void read_straight8(const uint16_t* tile, int r, int c,
                                               float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // not as a float4: the compiler then waits for every copy in flight first
    const i32x4_t q = *reinterpret_cast<const i32x4_t*>(tile + tile_offset(r, c * 2 + h));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * h + k] = __int_as_float(q[k]);
  }
}
template <int SIZE>
__device__ __forceinline__ void read_turned8(const uint16_t* tile, int r, int c, float (&v)[8]) {
  const float* p = reinterpret_cast<const float*>(tile) + c * 8 * SIZE + r;
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = p[k * SIZE];
}

template <int SIZE, int NW, bool TURNED>
struct RawCopies : Copies<SIZE, NW, false> {
  using Copies<SIZE, NW, false>::Copies;
  __device__ __forceinline__ void issue(int step, uint16_t* tile) const {
    Copies<SIZE, NW, false>::issue(step * kStep, 0, tile);
  }
};
template <int SIZE, int NW>
struct RawCopies<SIZE, NW, true> : RawTurnedCopies<SIZE, NW> {
  // k0 in 16-bit units, as the straight operand's
  __device__ __forceinline__ RawCopies(const Operand& o, int r0, int k0)
      : RawTurnedCopies<SIZE, NW>(o, r0, k0 / 2) {}
  __device__ __forceinline__ void issue(int step, uint16_t* tile) const {
    RawTurnedCopies<SIZE, NW>::issue(step * (kStep / 2), tile);
  }
};

// Elements that kRaw's B parts take in LDS behind the stages: [3][BN][32], the 16-byte
// chunk c of a row at position c ^ row / 4.
template <class CF, Form F>
constexpr int extra_lds() {
  return F == kRaw ? 3 * CF::BN * 32 : 0;
}
__device__ __forceinline__ int raw_part_offset(int row, int c) {
  return row * 32 + ((c ^ ((row >> 2) & 3)) << 3);
}

// mainloop for kRaw: stages of 32 floats of K.
template <class CF, bool TA>
__device__ __forceinline__ void mainloop_raw(const Operand& A, int m0, const Operand& B, int n0,
                                             int k0, int ksteps, uint16_t* lds,
                                             f32x16_t (&acc)[CF::FM][CF::FN]) {
  f32x16_t small[CF::FM][CF::FN];
#pragma unroll
  for (int i = 0; i < CF::FM; ++i)
#pragma unroll
    for (int j = 0; j < CF::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = small[i][j][r] = 0.f;
  static_assert(CF::NT == 256 && CF::BN * 4 <= CF::NT, "8 floats of B a thread");
  const RawCopies<CF::BM, CF::NW, TA> a_copies(A, m0, k0);
  const RawCopies<CF::BN, CF::NW, false> b_copies(B, n0, k0);
  uint16_t* const parts = lds + CF::STAGES * CF::STAGE;
  const int wave = threadIdx.x / kWave, lane = lane_id() & 31, half = lane_id() >> 5;
  const int ra = wave / CF::WAVES_N * CF::WTM + lane, rb = wave % CF::WAVES_N * CF::WTN + lane;
  constexpr int AHEAD = CF::STAGES - 1, COPIES = CF::A_ISSUE + CF::B_ISSUE;
  int fill = 0, ahead = 0;
  auto copy = [&]() {
    uint16_t* stage = lds + fill * CF::STAGE;
    a_copies.issue(ahead, stage);
    b_copies.issue(ahead, stage + CF::BM * kStep);
    ++ahead;
    fill = fill + 1 == CF::STAGES ? 0 : fill + 1;
  };
  for (int s = 0; s < AHEAD && s < ksteps; ++s) copy();
  int cur = 0;
  for (int s = 0; s < ksteps; ++s) {
    if (s + AHEAD <= ksteps) meet<(AHEAD - 1) * COPIES>();
    else meet<0>();
    if (s + AHEAD < ksteps) copy();
    const uint16_t* sA = lds + cur * CF::STAGE;
    const uint16_t* sB = sA + CF::BM * kStep;
    if (static_cast<int>(threadIdx.x) < CF::BN * 4) {
      const int row = threadIdx.x / 4, c = threadIdx.x % 4;
      float v[8];
      read_straight8(sB, row, c, v);
      i32x4_t part[3];
      split3(v, part);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<i32x4_t*>(parts + p * CF::BN * 32 + raw_part_offset(row, c)) = part[p];
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      i32x4_t a[CF::FM][3], b[CF::FN][3];
#pragma unroll
      for (int i = 0; i < CF::FM; ++i) {
        float v[8];
        if constexpr (TA) read_turned8<CF::BM>(sA, ra + 32 * i, ks * 2 + half, v);
        else read_straight8(sA, ra + 32 * i, ks * 2 + half, v);
        split3(v, a[i]);
      }
#pragma unroll
      for (int j = 0; j < CF::FN; ++j)
#pragma unroll
        for (int p = 0; p < 3; ++p)
          b[j][p] = *reinterpret_cast<const i32x4_t*>(
              parts + p * CF::BN * 32 + raw_part_offset(rb + 32 * j, ks * 2 + half));
#pragma unroll
      for (int i = 0; i < CF::FM; ++i)
#pragma unroll
        for (int j = 0; j < CF::FN; ++j) {
          small[i][j] = mfma<kBf16>(a[i][0], b[j][2], small[i][j]);
          small[i][j] = mfma<kBf16>(a[i][2], b[j][0], small[i][j]);
          small[i][j] = mfma<kBf16>(a[i][1], b[j][1], small[i][j]);
          small[i][j] = mfma<kBf16>(a[i][0], b[j][1], small[i][j]);
          small[i][j] = mfma<kBf16>(a[i][1], b[j][0], small[i][j]);
          acc[i][j] = mfma<kBf16>(a[i][0], b[j][0], acc[i][j]);
        }
    }
    cur = cur + 1 == CF::STAGES ? 0 : cur + 1;
  }
#pragma unroll
  for (int i = 0; i < CF::FM; ++i)
#pragma unroll
    for (int j = 0; j < CF::FN; ++j) acc[i][j] += small[i][j];
  __syncthreads();  // the stages are free for the epilogue
}

template <class CF, Form F, bool TA = false, bool TB = false>
__device__ __forceinline__ void multiply(const Operand& A, int m0, const Operand& B, int n0, int k0,
                                         int ksteps, uint16_t* lds,
                                         f32x16_t (&acc)[CF::FM][CF::FN]) {
  if constexpr (F == kRaw)
    mainloop_raw<CF, TA>(A, m0, B, n0, k0, ksteps, lds, acc);
  else if constexpr (CF::FM == 2)
    mainloop_pipe<CF, F, TA, TB>(A, m0, B, n0, k0, ksteps, lds, acc);
  else
    mainloop<CF, F, TA, TB>(A, m0, B, n0, k0, ksteps, lds, acc);
}

// Element (i, r) of a lane's accumulators is row block_row<CF>() + row_of(i, r),
// element j column block_col<CF>() + 32 j of the block.
template <class CF>
__device__ __forceinline__ int block_row() {
  return threadIdx.x / kWave / CF::WAVES_N * CF::WTM + 4 * (lane_id() >> 5);
}
__device__ __forceinline__ constexpr int row_of(int i, int r) {
  return i * 32 + (r >> 2) * 8 + (r & 3);
}
template <class CF>
__device__ __forceinline__ int block_col() {
  return threadIdx.x / kWave % CF::WAVES_N * CF::WTN + (lane_id() & 31);
}

// Workgroups are dealt round-robin to the 8 XCDs: workgroup b of `total` takes place
// run_of(b, total), so that each XCD gets a contiguous run of places.
__device__ __forceinline__ int run_of(int b, int total) {
  const int each = total / 8, more = total % 8, x = b % 8;
  return x * each + min(x, more) + b / 8;
}

// Tile t of m_blocks x n_blocks, in groups of 4 row blocks, so that tiles running
// together share operands in an XCD's L2.
__device__ __forceinline__ void tile_of(int t, int m_blocks, int n_blocks, int& mb, int& nb) {
  const int per_group = 4 * n_blocks;
  const int g = t / per_group, in = t - g * per_group;
  const int rows = min(4, m_blocks - g * 4);
  mb = g * 4 + in % rows;
  nb = in / rows;
}

// Tile t of those with mb <= nb, column by column.
__device__ __forceinline__ void triangle_of(int t, int& mb, int& nb) {
  nb = static_cast<int>((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
  while (nb * (nb + 1) / 2 > t) --nb;
  while ((nb + 1) * (nb + 2) / 2 <= t) ++nb;
  mb = t - nb * (nb + 1) / 2;
}

// The parts of v (scaled already), the larger first.
template <Form F>
__device__ __forceinline__ void split(float v, uint16_t (&part)[parts_of(F)]) {
  if constexpr (F == kBf16) {
    part[0] = ElemTraits<uint16_t>::from_f32(v);
  } else {
    const _Float16 hi = static_cast<_Float16>(v);
    part[0] = __builtin_bit_cast(uint16_t, hi);
    if constexpr (F == kHalves) {
      // an infinity or NaN is hi's alone
      const bool finite = (part[0] & 0x7c00u) != 0x7c00u;
      part[1] = __builtin_bit_cast(
          uint16_t, static_cast<_Float16>(finite ? v - static_cast<float>(hi) : 0.f));
    }
  }
}

// The exponent e by which a matrix or row of largest magnitude m is scaled: 2^14 <= m
// 2^e < 2^15 (at most 126, so that 2^e and 2^-e are normal numbers; m = 0 and non-finite
// m: 0).
__device__ __forceinline__ int exponent_for(float m) {
  const int b = static_cast<int>(__float_as_uint(m) >> 23) & 0xff;
  return b == 0xff || m == 0.f ? 0 : min(14 + 127 - max(b, 1), 126);
}
__device__ __forceinline__ float power_of_two(int e) { return ldexpf(1.f, e); }

// Stores of 8 consecutive values of a line: value (col, row ..) of slice `slice` of a
// product's K.
struct SumStore {  // float sums of every slice, added to what is there where `add`
  float* out;      // [slices][cols][pitch]
  int pitch, cols;
  bool add;
  __device__ __forceinline__ void operator()(int slice, int col, int row, float (&v)[8]) const {
    float* to = out + (static_cast<int64_t>(slice) * cols + col) * pitch + row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4* at = reinterpret_cast<float4*>(to) + h;
      float4 q = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      if (add) {
        const float4 old = *at;
        q = make_float4(q.x + old.x, q.y + old.y, q.z + old.z, q.w + old.w);
      }
      *at = q;
    }
  }
};
template <typename E>
struct ElementStore {  // one slice, times 2^(exponent - exponent_for(*amax)) where amax is given
  E* out;              // [cols][pitch]
  int pitch;
  const float* amax;
  int exponent;
  __device__ __forceinline__ void operator()(int, int col, int row, float (&v)[8]) const {
    E* to = out + static_cast<int64_t>(col) * pitch + row;
    if (amax != nullptr) {
      const float f = power_of_two(exponent - exponent_for(*amax));
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= f;
    }
    if constexpr (sizeof(E) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = ElemTraits<uint16_t>::from_f32(v[2 * k]) |
               static_cast<uint32_t>(ElemTraits<uint16_t>::from_f32(v[2 * k + 1])) << 16;
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
};

// C[col][row] = A[row] . B[col], rows < `pitch` (a multiple of 8, not under A.rows; what
// lies past A.rows is undefined), col < cols, over one slice of K per blockIdx.y, handed to
// `store`.  n_blocks == 0: C is symmetric, and only the tiles of m_blocks x m_blocks with
// rows up to the columns' are formed.
template <class CF, Form F, bool TA, bool TB, class Store>
__global__ __launch_bounds__(CF::NT) void product_kernel(Operand A, Operand B, int ksteps,
                                                         int m_blocks, int n_blocks, int cols,
                                                         int pitch, Store store) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[CF::STAGES * CF::STAGE + extra_lds<CF, F>()];
  int mb, nb;
  const int slices = gridDim.y, tiles = gridDim.x;
  // an XCD's run lies in one slice, or a few: its share of K stays in its L2
  const int place = run_of(blockIdx.y * tiles + blockIdx.x, slices * tiles);
  const int slice = place / tiles, t = place - slice * tiles;
  if (n_blocks == 0) triangle_of(t, mb, nb);
  else tile_of(t, m_blocks, n_blocks, mb, nb);
  const int s0 = static_cast<int>(static_cast<int64_t>(slice) * ksteps / slices);
  const int s1 = static_cast<int>(static_cast<int64_t>(slice + 1) * ksteps / slices);
  f32x16_t acc[CF::FM][CF::FN];
  multiply<CF, F, TA, TB>(A, mb * CF::BM, B, nb * CF::BN, s0 * kStep, s1 - s0, lds, acc);
  // 32 columns of every wave at a time through LDS, so that lines are stored whole: the
  // 16-byte chunk c of column col at position c ^ col, in two buffers taken in turn
  constexpr int CHUNKS = CF::BM / 4, COLS = CF::WAVES_N * 32;
  static_assert((CF::FN > 1 ? 2 : 1) * COLS * CF::BM * 2 <= CF::STAGES * CF::STAGE, "buffers fit");
  const int wave_cols = threadIdx.x / kWave % CF::WAVES_N * 32 + (lane_id() & 31);
#pragma unroll
  for (int j = 0; j < CF::FN; ++j) {
    float* buffer = reinterpret_cast<float*>(lds) + (j & 1) * COLS * CF::BM;
#pragma unroll
    for (int i = 0; i < CF::FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = (block_row<CF>() + row_of(i, 4 * q)) / 4;
        const f32x16_t& v = acc[i][j];
        *reinterpret_cast<float4*>(buffer + wave_cols * CF::BM +
                                   ((c ^ wave_cols) & (CHUNKS - 1)) * 4) =
            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    __syncthreads();
    for (int e = threadIdx.x; e < COLS * CHUNKS / 2; e += CF::NT) {
      const int at = e / (CHUNKS / 2), c = e % (CHUNKS / 2) * 2;
      const int col = nb * CF::BN + at / 32 * CF::WTN + j * 32 + at % 32;
      const int row = mb * CF::BM + c * 4;
      if (col >= cols || row >= pitch) continue;
      const float* from = buffer + at * CF::BM;
      const float4 p = *reinterpret_cast<const float4*>(from + ((c ^ at) & (CHUNKS - 1)) * 4);
      const float4 q = *reinterpret_cast<const float4*>(from + (((c + 1) ^ at) & (CHUNKS - 1)) * 4);
      float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
      store(slice, col, row, v);
    }
  }
}

// ---------------------------------------------------------------- host side
typedef Config<256, 256, 4, 2, 2> Big;
typedef Config<128, 128, 2, 2, 2> Mid;
typedef Config<128, 32, 4, 1, 4> Bare;  // at most 32 columns
// kRaw: two workgroups (with 64 columns) or three a CU, which is worth more than a
// third stage (9005 x 2376 by 39: 31 us, 42 with one workgroup of three stages)
typedef Config<128, 64, 4, 1, 2> RawFew;
typedef Config<128, 32, 4, 1, 2> RawBare;
constexpr int kFewColumns = 64;

inline int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }
inline int64_t blocks(int64_t n, int b) { return (n + b - 1) / b; }

enum Tile { kBare, kFew, kMid, kBig };
template <class Call>
hipError_t with_raw_tile(Tile t, const Call& f) {
  return t == kBare ? f(RawBare()) : f(RawFew());
}
template <class Call>
hipError_t with_wide_tile(Tile t, const Call& f) {
  return t == kMid ? f(Mid()) : f(Big());
}
inline int tile_rows(Tile t) { return t == kBig ? 256 : 128; }
inline int tile_cols(Tile t) { return t == kBig ? 256 : t == kMid ? 128 : t == kFew ? 64 : 32; }

// How a product of `rows` x `cols` over `steps` stages is cut: its tile, and slices of K.
struct Cut {
  Tile tile;
  int slices;
  double us;  // what it should take (wide_cut)
};
// At most kFewColumns columns: the narrowest tile, and slices until four workgroups a CU
// are there (two run at a time), of at least 4 stages.
inline Cut few_cut(int64_t rows, int64_t cols, int64_t steps, int64_t most_slices) {
  const Tile t = cols <= 32 ? kBare : kFew;
  const int64_t most = std::clamp<int64_t>(steps / 4, 1, most_slices);
  return {t, static_cast<int>(std::clamp<int64_t>(1024 / blocks(rows, tile_rows(t)), 1, most)), 0};
}
// Else the cheaper of 256 x 256 tiles (one workgroup a CU, 2.1 us a stage, 6 us to fill and
// to store) and 128 x 128 ones (one a CU 0.78 us a stage, two 1.25, 4 us), with as many
// slices as pay for writing and adding up their float32 sums (5 TB/s); `whole`: one slice
// writes none.
inline Cut wide_cut(int64_t rows, int64_t cols, int64_t steps, int most_slices, bool triangle,
                    bool whole) {
  Cut best{kMid, 1, 1e300};
  for (const Tile t : {kBig, kMid}) {
    const int64_t mb = blocks(rows, tile_rows(t)), nb = blocks(cols, tile_cols(t));
    const int64_t tiles = triangle ? mb * (mb + 1) / 2 : mb * nb;
    for (int s = 1; s <= most_slices && s <= std::max<int64_t>(steps / 4, 1); ++s) {
      const double each = static_cast<double>(blocks(steps, s));
      const int64_t groups = tiles * s;
      double us;
      if (t == kBig) us = blocks(groups, 256) * (each * 2.1 + 6);
      else if (groups <= 256) us = each * 0.78 + 4;
      else us = blocks(groups, 512) * (each * 1.25 + 4);
      if (s > 1 || !whole) us += static_cast<double>(s) * tiles * tile_rows(t) * tile_cols(t) * 8 / 5e6;
      if (us < best.us) best = {t, s, us};
      if (groups > 1024) break;
    }
  }
  return best;
}

struct Carve {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = reinterpret_cast<T*>(base + used);
    used += (count * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

}  // namespace nt
}  // namespace twell
