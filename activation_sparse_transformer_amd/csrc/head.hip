// The output head's log probabilities without its logits, and their gradient.
//
// z[v][n] = scale * w[v] . x[n] is formed a tile at a time on MFMA, with the
// vocabulary along the tile's rows: a lane then holds one token's column, and the
// running maximum m and sum of exp(z - m) of a tile cost no lane exchange but the
// one between the wave's halves.  The forward pass keeps {m, s} per tile and token
// and joins them:  lse = m + log s,  logp = z_target - lse.
//
// The gradient takes the vocabulary in pieces, so that what it keeps of the logits
// stays a part of them.  Per piece, with p = exp(z - m) / s and g = scale * dlogp:
//   dl[n][v] = g[n] (1[v = target] - p)     from z formed again
//   dx += dl w,   dw = dl^T x
// With bfloat16 x and w, dl is held in bfloat16: its rounding, at most 2^-8 of each element,
// is of the size of dx's and dw's own (4096 x 2048 x 32768: 0.0022 from float64 with random
// dlogp, the results' rounding alone 0.0017; two parts would double the products of dx and dw).
// With few rows, where it costs next to nothing, it is two parts (few_rows).  With float32 ones every operand is two half-precision parts
// (nt_gemm.h), w scaled by its largest element, x by each row's; dl / g lies in [-1, 1]
// and is scaled by 2^15, with g taken into dx at the end and into the x of dw: a dl / g is
// within 2^-40, so that a token of p < 2^-18 has fewer than 22 bits of its row of dw, and one
// of p < 2^-41 in every row none.  With few
// rows, where reading w is what the call costs, float32 operands and dl stay float32, and
// z is formed with K cut in slices where the vocabulary alone gives too few workgroups to
// keep the memory busy, so it goes through the workspace (n_rows of a piece of it).
// Both products read w, x and dl as they lie, turning fragments with LDS transpose
// reads where K runs along a column.
#include <algorithm>
#include <cfloat>
#include <numeric>
#include <type_traits>

#include "nt_gemm.h"
#include "train_kernels.h"

namespace twell {
namespace {

using namespace nt;

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ int64_t target_of(const void* targets, int index_bytes, int64_t n) {
  return index_bytes == 8 ? static_cast<const int64_t*>(targets)[n]
                          : static_cast<const int32_t*>(targets)[n];
}

// v of the lane with the other half's rows of the same column
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

constexpr int kDlExponent = 15;  // of dl / g in halves

__device__ __forceinline__ bool has_target(const void* targets, int index_bytes, int vocab,
                                           int64_t n) {
  const int64_t t = target_of(targets, index_bytes, n);
  return t >= 0 && t < vocab;
}

// ---------------------------------------------------------------- operand parts
// 8 scaled values from column c of a row of parts; `part`: elements between parts.
template <Form F>
__device__ __forceinline__ void put_run(uint16_t* row, int64_t part, int c, const float (&v)[8]) {
  constexpr int P = parts_of(F);
  uint32_t w[P][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t lo[P], hi[P];
    nt::split<F>(v[2 * k], lo);
    nt::split<F>(v[2 * k + 1], hi);
#pragma unroll
    for (int p = 0; p < P; ++p) w[p][k] = lo[p] | static_cast<uint32_t>(hi[p]) << 16;
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
    *reinterpret_cast<uint4*>(row + p * part + c) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

template <typename E>
__device__ __forceinline__ void load_run(const E* p, float (&v)[8]) {
  if constexpr (sizeof(E) == 2) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// The largest finite magnitude of v and m
__device__ __forceinline__ float max_finite(float m, float v) {
  v = fabsf(v);
  return v < INFINITY ? fmaxf(m, v) : m;
}
__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
  for (int h = 32; h > 0; h /= 2) m = fmaxf(m, __shfl_xor(m, h));
  return m;
}

__global__ void head_clear_kernel(float* amax) { amax[threadIdx.x] = 0.f; }

// *amax = max(*amax, the largest finite magnitude of src): an order-free atomic on the
// bits of non-negative floats.  4 runs a lane at a time; at most kAmaxGroups workgroups, as
// their atomics are on one address.
constexpr int kAmaxRuns = 4 * 256, kAmaxGroups = 1024;
__global__ __launch_bounds__(256) void head_amax_kernel(const float* __restrict__ src,
                                                        int64_t runs, float* amax) {
  __shared__ float lds[4];
  float m = 0.f;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAmaxRuns + threadIdx.x; i < runs;
       i += static_cast<int64_t>(gridDim.x) * kAmaxRuns) {
    float v[4][8] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * 256 < runs) load_run(src + (i + u * 256) * 8, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max_finite(m, v[u][k]);
  }
  m = wave_max(m);
  if (lane_id() == 0) lds[threadIdx.x / kWave] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    m = fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
    // most workgroups find a larger one there already
    if (m > __hip_atomic_load(amax, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
      atomicMax(reinterpret_cast<int*>(amax), __float_as_int(m));
  }
}

// Bound by memory, with the head_amax pass before: 49999 x 1000 45 us for the largest element
// (4.5 TB/s) and 72 for the parts (5.5 TB/s), of 2170 that the gradient takes.
// Halves [2][rows][ld] of a piece of w, src [rows][d], scaled by *amax; columns past d
// are zeros.
__global__ __launch_bounds__(256) void head_w_kernel(const float* __restrict__ src, int64_t rows,
                                                     int d, int ld, const float* amax,
                                                     uint16_t* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = i / (ld / 8);
  const int c = static_cast<int>(i % (ld / 8)) * 8;
  if (row >= rows) return;
  float v[8] = {};
  if (c < d) load_run(src + row * d + c, v);
  const float f = power_of_two(exponent_for(*amax));
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= f;
  put_run<kHalves>(out + row * ld, rows * ld, c, v);
}

// Halves [2][rows][ld] of x, a wave a row, scaled by the row's largest element; in
// factor[row], positive and finite, what makes z of its products with w's halves: scale and
// both powers of two undone.  Where that would be under 2^-126 the row's scale is held back
// (its parts then carry less of z, 2^-133 at most each product); past float32 it ends at the
// largest one, so that 0 stays 0.  For the gradient (dlogp not null) also amax[1] = the
// largest of |scale dlogp x| over rows with a target.  amax[0]: w's.
__global__ __launch_bounds__(256) void head_x_kernel(HeadArgs a, int ld,
                                                     const float* __restrict__ dlogp,
                                                     float* __restrict__ factor, float* amax,
                                                     uint16_t* __restrict__ out) {
  __shared__ float largest[4];
  const int wave = threadIdx.x / kWave;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (lane_id() == 0) largest[wave] = 0.f;
  if (row < a.n_rows) {
    const float* src = static_cast<const float*>(a.x) + row * a.d;
    float m = 0.f;
    for (int c = lane_id() * 8; c < a.d; c += kWave * 8) {
      float v[8];
      load_run(src + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max_finite(m, v[k]);
    }
    m = wave_max(m);
    const int ew = exponent_for(amax[0]);
    const int e = min(exponent_for(m), 126 + ilogbf(a.scale) - ew);
    const float f = power_of_two(e);
    if (lane_id() == 0) {
      factor[row] = static_cast<float>(
          fmin(ldexp(static_cast<double>(a.scale), -(e + ew)), static_cast<double>(FLT_MAX)));
      if (dlogp != nullptr && has_target(a.targets, a.index_bytes, a.vocab, row))
        largest[wave] = max_finite(0.f, dlogp[row] * a.scale * m);
    }
    for (int c = lane_id() * 8; c < ld; c += kWave * 8) {
      float v[8] = {};
      if (c < a.d) load_run(src + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= f;
      put_run<kHalves>(out + row * ld, a.n_rows * ld, c, v);
    }
  }
  if (dlogp == nullptr) return;
  __syncthreads();  // one atomic for the four rows: they are on one address
  if (threadIdx.x == 0)
    atomicMax(reinterpret_cast<int*>(amax + 1),
              __float_as_int(fmaxf(fmaxf(largest[0], largest[1]), fmaxf(largest[2], largest[3]))));
}

// dw's x, [parts][n_rows][d], a wave a row: rows without a target are zeros (whatever x
// holds there meets gradients of zero, and a NaN must not spread).  Halves: scale * dlogp
// * x, scaled by *amax; else x as it is.
template <Form F>
__global__ __launch_bounds__(256) void head_gx_kernel(HeadArgs a, const float* __restrict__ dlogp,
                                                      const float* amax,
                                                      uint16_t* __restrict__ out) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  if (row >= a.n_rows) return;
  const bool live = has_target(a.targets, a.index_bytes, a.vocab, row);
  typedef std::conditional_t<F == kBf16, uint16_t, float> E;
  const E* src = static_cast<const E*>(a.x) + row * a.d;
  float f = 1.f, g = 1.f;
  if constexpr (F == kHalves) {
    f = power_of_two(exponent_for(*amax));
    if (live) g = dlogp[row] * a.scale;
  }
  for (int c = lane_id() * 8; c < a.d; c += kWave * 8) {
    float v[8] = {};
    if (live) load_run(src + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * g * f;
    put_run<F>(out + row * a.d, a.n_rows * a.d, c, v);
  }
}

// z of a sum, rounded before anything is taken from it: a multiply-add with -m would leave
// m's own rounding, |z| 2^-25, in the exponent, and make e^(z - m) infinite for z past 2^32.
__device__ __forceinline__ float z_of(float sum, float f) {
#pragma clang fp contract(off)
  return sum * f;
}
// exp(z - m) of a z formed again: at most 1, also where it was summed in another order than
// the forward pass's.  A row with a NaN is NaN by its sum.
__device__ __forceinline__ float exp_again(float z, float m) {
  return __builtin_amdgcn_exp2f(fminf(z - m, 0.f) * kLog2e);
}

// What a column of accumulators is multiplied by to be z: positive, so that the -infinity of
// a row past the vocabulary's end stays one.
template <Form F, class Args>
__device__ __forceinline__ float z_factor(const Args& a, int64_t n) {
  if constexpr (F == kHalves) return n < a.x.rows ? a.factor[n] : 1.f;
  return a.scale;
}

// ---------------------------------------------------------------- forward
// Many rows: bound by MFMA and the clocks under it.  4096 x 2048 x 32768 bf16 takes 475 us in
// all, 1.16 PFLOP/s (a plain library product of 8192^3 reaches 1.17); the statistics are a
// subtraction, a multiply, an exp2 and an add per z, behind the products.
struct StatsArgs {
  Operand w, x;      // w: a piece of the vocabulary, from column v0
  int v0, vocab;     // whole vocabulary
  int ksteps;
  float scale;
  const float* factor;  // halves: per row of x
  const void* targets;
  int index_bytes;
  float2* parts;     // [tiles][n], this piece's first tile onwards
  float* target_z;   // [n], z of the target, written by the tile that holds it
};

template <class CF, Form F>
__global__ __launch_bounds__(CF::NT) void head_stats_kernel(StatsArgs a, int m_blocks,
                                                            int n_blocks) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[CF::STAGES * CF::STAGE];
  int mb, nb;
  nt::tile_of(nt::run_of(blockIdx.x, gridDim.x), m_blocks, n_blocks, mb, nb);
  f32x16_t acc[CF::FM][CF::FN];
  nt::multiply<CF, F>(a.w, mb * CF::BM, a.x, nb * CF::BN, 0, a.ksteps, lds, acc);
  const int row0 = mb * CF::BM + nt::block_row<CF>();
  const int half = lane_id() >> 5;
  const int wave_row = row0 - 4 * half;  // the wave's first row
  const bool full = (mb + 1) * CF::BM <= a.w.rows;
  float2* joint = reinterpret_cast<float2*>(lds);  // [WAVES_M][BN]
  const int wm = threadIdx.x / kWave / CF::WAVES_N;
#pragma unroll
  for (int j = 0; j < CF::FN; ++j) {
    const int col = nt::block_col<CF>() + 32 * j;
    const int n = nb * CF::BN + col;
    const float f = z_factor<F>(a, n);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < CF::FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (!full && row0 + nt::row_of(i, r) >= a.w.rows) acc[i][j][r] = -INFINITY;
        m = fmaxf(m, acc[i][j][r]);
      }
    m = fmaxf(m, other_half(m));
    // z - max z from the sums' difference: 0 at the largest, never above
    const float base = m == -INFINITY ? 0.f : m, f2 = fminf(f * kLog2e, FLT_MAX);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CF::FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) s += __builtin_amdgcn_exp2f((acc[i][j][r] - base) * f2);
    s += other_half(s);
    m = z_of(m, f);
    if (half == 0) joint[wm * CF::BN + col] = make_float2(m, s);
    // the target's z, where this wave's rows hold it
    int64_t t = -1;
    if (n < a.x.rows) {
      t = target_of(a.targets, a.index_bytes, n);
      t = t >= 0 && t < a.vocab ? t - a.v0 - wave_row : -1;
    }
    const bool mine = t >= 0 && t < CF::WTM && wave_row + t < a.w.rows &&
                      ((static_cast<int>(t) >> 2) & 1) == half;
    if (wave_ballot(mine) != 0) {
      const int rel = static_cast<int>(t) - 4 * half;
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < CF::FM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (rel == nt::row_of(i, r)) z = acc[i][j][r];
      if (mine) a.target_z[n] = z_of(z, f);
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < CF::BN; col += CF::NT) {
    const int n = nb * CF::BN + col;
    if (n >= a.x.rows) continue;
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < CF::WAVES_M; ++w) m = fmaxf(m, joint[w * CF::BN + col].x);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < CF::WAVES_M; ++w) {
      const float2 p = joint[w * CF::BN + col];
      s += p.y * __builtin_amdgcn_exp2f((p.x - base) * kLog2e);
    }
    a.parts[static_cast<int64_t>(mb) * a.x.rows + n] = make_float2(m, s);
  }
}

// {m, s} of two disjoint sets of columns, as one.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float base = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * __builtin_amdgcn_exp2f((a.x - base) * kLog2e) +
                            b.y * __builtin_amdgcn_exp2f((b.x - base) * kLog2e));
}

struct RowResults {
  const void* targets;
  int index_bytes, vocab;
  float *logp, *lse;
  float2* stats;
};
__device__ __forceinline__ void finish_row(const RowResults& o, int64_t n, float2 p,
                                           const float* target_z) {
  const float base = p.x == -INFINITY ? 0.f : p.x;
  const float log_s = logf(p.y);  // -inf for a row with nothing left
  o.stats[n] = p;
  o.lse[n] = base + log_s;
  float lp = 0.f;
  // a row with nothing left: z - lse would be -inf + inf
  if (has_target(o.targets, o.index_bytes, o.vocab, n))
    lp = p.x == -INFINITY && p.y == 0.f ? -INFINITY : *target_z - base - log_s;
  o.logp[n] = lp;
}

// Joins the tiles' {m, s} of 16 tokens a workgroup, in 16 streams of tiles: 6 us of 475 at
// 4096 tokens and 128 tiles.
__global__ __launch_bounds__(256) void head_join_kernel(const float2* __restrict__ parts,
                                                        int tiles, int64_t n_rows,
                                                        const float* __restrict__ target_z,
                                                        RowResults o) {
  __shared__ float2 joint[16][16];
  const int col = threadIdx.x % 16, stream = threadIdx.x / 16;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + col;
  float2 p = make_float2(-INFINITY, 0.f);
  if (n < n_rows)
    for (int t = stream; t < tiles; t += 16) p = join(p, parts[t * n_rows + n]);
  joint[stream][col] = p;
  __syncthreads();
  if (stream != 0 || n >= n_rows) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) p = join(p, joint[w][col]);
  finish_row(o, n, p, target_z + n);
}

// ---------------------------------------------------------------- few rows
// At most 64 (few_rows): reading w bounds them.  16 x 4096 x 131072 bf16 194 us, of which the
// product 183 (5.9 TB/s; a plain read reaches 6.9), the statistics of z from the workspace 6
// and joining 5.  64 x 128 x 1000 float32 gradient: 31 us, five launches of which none fills
// the card.
// z of 4 columns from v: the slices' sums in their order, times scale.
struct FewZ {
  const float* sums;  // [slices][n_rows][pitch]
  int slices, pitch;
  int rows, v0;       // of the vocabulary
  float scale;
};
__device__ __forceinline__ float4 few_z(const FewZ& z, int64_t n_rows, int64_t n, int v) {
  float4 t = make_float4(0, 0, 0, 0);
#pragma unroll 8
  for (int s = 0; s < z.slices; ++s) {
    const float4 q = *reinterpret_cast<const float4*>(z.sums + (s * n_rows + n) * z.pitch + v);
    t = make_float4(t.x + q.x, t.y + q.y, t.z + q.z, t.w + q.w);
  }
  return make_float4(z_of(t.x, z.scale), z_of(t.y, z.scale), z_of(t.z, z.scale),
                     z_of(t.w, z.scale));
}

// {m, s} of kFewChunk columns of a row a workgroup: to parts, or, where one holds the whole
// vocabulary, the row's results.
constexpr int kFewChunk = 4096;
__global__ __launch_bounds__(256) void head_few_stats_kernel(FewZ z, int64_t n_rows,
                                                             float2* __restrict__ parts,
                                                             float* __restrict__ target_z,
                                                             RowResults o) {
  __shared__ float2 joint[4];
  const int64_t n = blockIdx.y;
  const int64_t t = target_of(o.targets, o.index_bytes, n) - z.v0;
  float v[kFewChunk / 1024][4];
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < kFewChunk / 1024; ++u) {
    const int c = blockIdx.x * kFewChunk + (u * 256 + threadIdx.x) * 4;
    const bool some = c < z.rows;
    const float4 q = some ? few_z(z, n_rows, n, c) : make_float4(0, 0, 0, 0);
    v[u][0] = q.x, v[u][1] = q.y, v[u][2] = q.z, v[u][3] = q.w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c + k >= z.rows) v[u][k] = -INFINITY;
      else if (c + k == t) target_z[n] = v[u][k];
      m = fmaxf(m, v[u][k]);
    }
  }
  const float base = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < kFewChunk / 1024; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k) s += __builtin_amdgcn_exp2f((v[u][k] - base) * kLog2e);
  float2 p = make_float2(m, s);
#pragma unroll
  for (int h = 1; h < kWave; h *= 2)
    p = join(p, make_float2(__shfl_xor(p.x, h), __shfl_xor(p.y, h)));
  if (lane_id() == 0) joint[threadIdx.x / kWave] = p;
  __threadfence_block();
  __syncthreads();
  if (threadIdx.x != 0) return;
  p = join(join(joint[0], joint[1]), join(joint[2], joint[3]));
  if (parts != nullptr) parts[blockIdx.x * n_rows + n] = p;
  else finish_row(o, n, p, target_z + n);
}

// ---------------------------------------------------------------- gradient
// Part p of two values, packed.
template <Form F>
__device__ __forceinline__ uint32_t pack_part(float a, float b, int p) {
  if constexpr (F == kBf16) {
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
  } else {
    _Float16 x = static_cast<_Float16>(a), y = static_cast<_Float16>(b);
    if (p == 1) {  // what the first part leaves; |a| is at most 2^15, or NaN
      x = static_cast<_Float16>(a == a ? a - static_cast<float>(x) : 0.f);
      y = static_cast<_Float16>(b == b ? b - static_cast<float>(y) : 0.f);
    }
    return __builtin_bit_cast(uint16_t, x) |
           static_cast<uint32_t>(__builtin_bit_cast(uint16_t, y)) << 16;
  }
}

// Many rows: z formed again and dl in its place: 4096 x 2048 x 16384 bf16 285 us, 0.96
// PFLOP/s (the statistics pass 250): the epilogue's exponentials, and dl's 134 MB through LDS.
// In halves the epilogue of 256 x 256 tiles spills 22 registers (92 bytes a lane).
struct DlArgs {
  Operand w, x;
  int v0, vocab;
  int ksteps;
  float scale;
  const float* factor;  // halves: per row of x
  const void* targets;
  int index_bytes;
  const float2* stats;
  const float* dlogp;
  uint16_t* dl;  // [parts][n][ldv]
  int ldv;
};

template <class CF, Form F>
__global__ __launch_bounds__(CF::NT) void head_dl_kernel(DlArgs a, int m_blocks, int n_blocks) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[CF::STAGES * CF::STAGE];
  int mb, nb;
  nt::tile_of(nt::run_of(blockIdx.x, gridDim.x), m_blocks, n_blocks, mb, nb);
  f32x16_t acc[CF::FM][CF::FN];
  nt::multiply<CF, F>(a.w, mb * CF::BM, a.x, nb * CF::BN, 0, a.ksteps, lds, acc);
  const int row0 = mb * CF::BM + nt::block_row<CF>();
  const int half = lane_id() >> 5;
  const int wave_row = row0 - 4 * half;  // the wave's first row
  const bool full = (mb + 1) * CF::BM <= a.w.rows;
  const int64_t n_rows = a.x.rows;
#pragma unroll
  for (int j = 0; j < CF::FN; ++j) {
    const int n = nb * CF::BN + nt::block_col<CF>() + 32 * j;
    const float f = z_factor<F>(a, n);
    float g = 0.f, m = 0.f, share = 0.f;  // share = -g / sum
    int t = -1;  // the target, of the wave's rows
    bool given = false;
    if (n < n_rows) {
      const int64_t target = target_of(a.targets, a.index_bytes, n);
      const float2 st = a.stats[n];
      given = target >= 0 && target < a.vocab && !(st.x == -INFINITY && st.y == 0.f);
      if (given) {
        t = static_cast<int>(target) - a.v0 - wave_row;
        g = F == kHalves ? power_of_two(kDlExponent) : a.dlogp[n] * a.scale;
        m = st.x;
        share = -g / st.y;
      }
    }
#pragma unroll
    for (int i = 0; i < CF::FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float e = exp_again(z_of(acc[i][j][r], f), m);
        acc[i][j][r] = given && (full || row0 + nt::row_of(i, r) < a.w.rows) ? share * e : 0.f;
      }
    const bool mine = t >= 0 && t < CF::WTM && wave_row + t < a.w.rows && ((t >> 2) & 1) == half;
    if (wave_ballot(mine) != 0) {
      const int rel = mine ? t - 4 * half : -1;
#pragma unroll
      for (int i = 0; i < CF::FM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (rel == nt::row_of(i, r)) acc[i][j][r] += g;
    }
  }
  // a part at a time through LDS, so that its rows are stored whole: the 16-byte chunk c
  // of row n at position c ^ n, which spreads the 32 rows of a write over the banks
  constexpr int CHUNKS = CF::BM / 8;
  static_assert(CF::BM * CF::BN <= CF::STAGES * CF::STAGE, "the tile fits the stages");
#pragma unroll
  for (int p = 0; p < parts_of(F); ++p) {
    if (p > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < CF::FN; ++j) {
      const int col = nt::block_col<CF>() + 32 * j;
#pragma unroll
      for (int i = 0; i < CF::FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = nt::block_row<CF>() + nt::row_of(i, 4 * q);
          uint32_t w[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            w[k] = pack_part<F>(acc[i][j][4 * q + 2 * k], acc[i][j][4 * q + 2 * k + 1], p);
          *reinterpret_cast<uint2*>(lds + col * CF::BM + (((row >> 3) ^ col) & (CHUNKS - 1)) * 8 +
                                    (row & 7)) = make_uint2(w[0], w[1]);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < CF::BN * CHUNKS; e += CF::NT) {
      const int col = e / CHUNKS, c = e % CHUNKS;
      const int64_t n = nb * CF::BN + col;
      const int v = mb * CF::BM + c * 8;
      if (n < n_rows && v < a.ldv)
        *reinterpret_cast<uint4*>(a.dl + (p * n_rows + n) * a.ldv + v) =
            *reinterpret_cast<const uint4*>(lds + col * CF::BM + ((c ^ col) & (CHUNKS - 1)) * 8);
    }
  }
}

// dx = the sum of the slices, rounded: 4 elements a lane, the slices in 4 streams; rows
// without a target zero, also where an infinity of w met their dl.  Halves: times scale *
// dlogp of the row and the powers of two undone.  The grid is two-dimensional: a launch
// holds fewer than 2^32 lanes along one.
template <typename E, Form F>
__global__ __launch_bounds__(256) void head_dx_kernel(HeadArgs a, const float* __restrict__ sums,
                                                      int slices, const float* __restrict__ dlogp,
                                                      const float* amax, E* __restrict__ dx) {
  __shared__ float4 joint[3][64];
  const int64_t elems = a.n_rows * a.d;
  const int at = threadIdx.x % 64, stream = threadIdx.x / 64;
  const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t i = (block * 64 + at) * 4;
  float4 v = make_float4(0, 0, 0, 0);
  if (i < elems)
#pragma unroll 8
    for (int s = stream; s < slices; s += 4) {
      const float4 q = *reinterpret_cast<const float4*>(sums + s * elems + i);
      v = make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w);
    }
  if (slices > 1) {
    if (stream > 0) joint[stream - 1][at] = v;
    __syncthreads();
    if (stream == 0)
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const float4 q = joint[w][at];
        v = make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w);
      }
  }
  if (stream != 0 || i >= elems) return;
  const int64_t n = i / a.d;
  const bool given = has_target(a.targets, a.index_bytes, a.vocab, n);
  if (!given) v = make_float4(0, 0, 0, 0);
  if constexpr (F == kHalves) {
    // in double: neither factor alone need leave v in float32's range
    const double f = given ? ldexp(static_cast<double>(dlogp[n]) * a.scale,
                                   -kDlExponent - exponent_for(*amax)) : 0.0;
    v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
  if constexpr (sizeof(E) == 2)
    *reinterpret_cast<uint2*>(dx + i) = make_uint2(pack_part<kBf16>(v.x, v.y, 0),
                                                   pack_part<kBf16>(v.z, v.w, 0));
  else
    *reinterpret_cast<float4*>(dx + i) = v;
}

// Few rows: bfloat16 parts of dl that the products take, and of the x of dw.
template <Form F>
constexpr int kFewDlParts = F == kRaw ? 3 : 2;
template <Form F>
constexpr int kFewXParts = F == kRaw ? 3 : 1;

// Few rows: dl of 64 columns of the vocabulary a workgroup, for dx (raw: float [n_rows]
// [ldv]; bfloat16: two parts of that) and for dw (parts [rows][kn], kn the rows rounded up
// to 16).
template <Form F>
__global__ __launch_bounds__(256) void head_few_dl_kernel(HeadArgs a, FewZ z,
                                                          const float2* __restrict__ stats,
                                                          const float* __restrict__ dlogp,
                                                          uint16_t* __restrict__ dl, int ldv,
                                                          uint16_t* __restrict__ dlt, int kn) {
  constexpr int PARTS = kFewDlParts<F>;
  __shared__ float tile[kFewColumns][65];
  const int n_rows = static_cast<int>(a.n_rows);
  const int c = threadIdx.x % 16 * 4, v = blockIdx.x * 64 + c;
#pragma unroll
  for (int u = 0; u < kFewColumns / 16; ++u) {
    const int n = u * 16 + threadIdx.x / 16;
    float d[4] = {};
    if (n < n_rows) {
      const int64_t t = target_of(a.targets, a.index_bytes, n);
      const float2 st = stats[n];
      const bool given = t >= 0 && t < a.vocab && !(st.x == -INFINITY && st.y == 0.f);
      if (given && v < z.rows) {
        const float g = dlogp[n] * a.scale, share = -g / st.y;
        const float4 q = few_z(z, n_rows, n, v);
        const float zs[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[k] = share * exp_again(zs[k], st.x);
          if (v + k == t - z.v0) d[k] += g;
          if (v + k >= z.rows) d[k] = 0.f;
        }
      }
      if constexpr (F == kRaw) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(dl) + static_cast<int64_t>(n) * ldv +
                                   v) = make_float4(d[0], d[1], d[2], d[3]);
      } else {
        float e[4] = {d[0], d[1], d[2], d[3]};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint2 w = make_uint2(pack_part<kBf16>(e[0], e[1], 0),
                                     pack_part<kBf16>(e[2], e[3], 0));
          *reinterpret_cast<uint2*>(dl + (static_cast<int64_t>(p) * n_rows + n) * ldv + v) = w;
          e[0] -= __uint_as_float(w.x << 16), e[1] -= __uint_as_float(w.x & 0xffff0000u);
          e[2] -= __uint_as_float(w.y << 16), e[3] -= __uint_as_float(w.y & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) tile[n][c + k] = d[k];
  }
  __syncthreads();
  const int col = threadIdx.x / 4, n0 = threadIdx.x % 4 * 16;
  const int64_t row = blockIdx.x * 64 + col;
  if (row >= z.rows || n0 >= kn) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = tile[n0 + h * 8 + k][col];
    i32x4_t part[3];
    split3(e, part);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
      *reinterpret_cast<i32x4_t*>(dlt + (static_cast<int64_t>(p) * z.rows + row) * kn + n0 +
                                  h * 8) = part[p];
  }
}

// Few rows: dw[v][c] = sum over n of dl[n][v] x[n][c] over the rows n with a target, 128
// columns c a workgroup.  x's parts stay in LDS; a wave takes 32 v at a time, with 4 c to a
// lane (columns 4 l + j of block j), so that a lane stores 4 adjacent ones: what bounds it
// is writing dw.
template <Form F>
__global__ __launch_bounds__(256) void head_few_dw_kernel(HeadArgs a, const uint16_t* __restrict__ dlt,
                                                          int rows, int kn, void* __restrict__ out) {
  constexpr int PA = kFewDlParts<F>, PB = kFewXParts<F>;
  constexpr int PITCH = kFewColumns + 8;
  __shared__ __attribute__((aligned(16))) uint16_t lds[PB][128][PITCH];
  typedef std::conditional_t<F == kBf16, uint16_t, float> E;
  const int c0 = blockIdx.x * 128;
  const uint64_t given =
      wave_ballot(lane_id() < a.n_rows && has_target(a.targets, a.index_bytes, a.vocab, lane_id()));
  // x[8 rows from n0][column], transposed
  for (int e = threadIdx.x; e < 128 * (kn / 8); e += 256) {
    const int col = e % 128, n0 = e / 128 * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int n = n0 + k;
      const bool live = (given >> n & 1) != 0 && c0 + col < a.d;
      v[k] = live ? ElemTraits<E>::to_f32(static_cast<const E*>(a.x)[static_cast<int64_t>(n) * a.d +
                                                                    c0 + col])
                  : 0.f;
    }
    i32x4_t part[3];
    split3(v, part);
    const int place = col % 4 * 32 + col / 4;  // column 4 l + j in row 32 j + l
#pragma unroll
    for (int p = 0; p < PB; ++p) *reinterpret_cast<i32x4_t*>(&lds[p][place][n0]) = part[p];
  }
  __syncthreads();
  const int l = lane_id() & 31, half = lane_id() >> 5;
  const int waves = gridDim.y * 4;
  i32x4_t f[kFewColumns / 16][PA];
  const auto load = [&](int v0) {
    const int v = min(v0 + l, rows - 1);
#pragma unroll
    for (int ks = 0; ks < kFewColumns / 16; ++ks)
      if (ks * 16 < kn)
#pragma unroll
        for (int p = 0; p < PA; ++p)
          f[ks][p] = *reinterpret_cast<const i32x4_t*>(
              dlt + (static_cast<int64_t>(p) * rows + v) * kn + ks * 16 + half * 8);
  };
  const int first = (blockIdx.y * 4 + threadIdx.x / kWave) * 32;
  if (first < rows) load(first);
  for (int v0 = first; v0 < rows; v0 += waves * 32) {
    f32x16_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
#pragma unroll
    for (int ks = 0; ks < kFewColumns / 16; ++ks)
      if (ks * 16 < kn)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          i32x4_t b[PB];
#pragma unroll
          for (int p = 0; p < PB; ++p)
            b[p] = *reinterpret_cast<const i32x4_t*>(&lds[p][32 * j + l][ks * 16 + half * 8]);
          // the small products first; those under 2^-24 are left out
#pragma unroll
          for (int sum = 2; sum >= 0; --sum)
#pragma unroll
            for (int p = 0; p < PA; ++p)
              if (sum - p >= 0 && sum - p < PB) acc[j] = mfma<kBf16>(f[ks][p], b[sum - p], acc[j]);
        }
    if (v0 + waves * 32 < rows) load(v0 + waves * 32);
    if (c0 + 4 * l >= a.d) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = v0 + 4 * half + row_of(0, r);
      if (row >= rows) continue;
      const int64_t at = static_cast<int64_t>(row) * a.d + c0 + 4 * l;
      if constexpr (F == kBf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
            make_uint2(pack_part<kBf16>(acc[0][r], acc[1][r], 0),
                       pack_part<kBf16>(acc[2][r], acc[3][r], 0));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) =
            make_float4(acc[0][r], acc[1][r], acc[2][r], acc[3][r]);
    }
  }
}

__global__ __launch_bounds__(256) void head_zero_kernel(uint4* p, int64_t count) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- sizes
// Columns of the vocabulary taken at a time: all where the forward pass reads w in place,
// else as many as keep what is made per column within `budget`, in equal pieces.
int64_t most_of(size_t per_column, size_t budget) {
  return std::max<int64_t>(budget / per_column / 256 * 256, 1024);
}
int equal_pieces(int vocab, int64_t most) {
  const int64_t pieces = blocks(vocab, static_cast<int>(std::min<int64_t>(most, vocab)));
  return static_cast<int>(std::min<int64_t>(blocks(blocks(vocab, static_cast<int>(pieces)), 256) * 256, vocab));
}
int piece_of(int vocab, size_t per_column, size_t budget) {
  return equal_pieces(vocab, most_of(per_column, budget));
}
// The same, or, if us(columns) promises less for it, the most columns of which 256 x 256
// tiles of n rows fill the CUs without a rest, and a smaller last piece (2001 x 1000 x 49999
// float32: 734 us forward with pieces of 32768, 793 with two of 25088; gradient 2145 with
// pieces of 16384, 2216 with four of 12544).
template <class Us>
int piece_of(int vocab, size_t per_column, size_t budget, int64_t n, const Us& us) {
  const int64_t most = most_of(per_column, budget);
  const int equal = equal_pieces(vocab, most);
  const int64_t unit = 65536 / std::gcd(blocks(n, 256), int64_t{256});
  if (equal >= vocab || most < unit) return equal;
  const int filled = static_cast<int>(most / unit * unit);
  const auto all = [&](int piece) {
    const int rest = vocab % piece;
    return vocab / piece * us(piece) + (rest > 0 ? us(rest) : 0.0);
  };
  return all(filled) < all(equal) ? filled : equal;
}

constexpr int kAmax = 2;  // largest magnitudes: of w, of scale * dlogp * x

// Whether the kernels of few rows take a call.  float32: where w's parts cost more than the
// products (64 x 1024 x 32768: 53 us forward and 178 for the gradient, 135 and 252 with the
// kernels of many rows).  bfloat16, whose operands lie ready: forward 16 x 4096 x 131072 195 us
// and 202, 33 x 1024 x 32768 28 and 27, 64 31 and 28; gradient 16 x 512 x 8000 25 and 31, 16 x
// 1024 x 32768 57 and 65, 16 x 2048 x 50001 195 and 170, 32 x 1024 x 32768 71 and 68.
bool few_rows(const HeadArgs& a, int elem_bytes, bool backward) {
  if (elem_bytes == 4) return a.n_rows <= kFewColumns;
  if (!backward) return a.n_rows <= 32;
  return a.n_rows <= 16 && static_cast<int64_t>(a.vocab) * a.d <= 1 << 25;
}

// The form of the operands; and the stages of a product over k.
Form form_of(int elem_bytes, int64_t n) {
  return elem_bytes == 2 ? kBf16 : n <= kFewColumns ? kRaw : kHalves;
}
int stages(Form f, int64_t k) { return static_cast<int>(blocks(k, f == kRaw ? 32 : 64)); }

// Few rows, forward and backward: z of a piece of the vocabulary through the workspace.
struct FewPlan {
  int piece, kn;
  Cut z_cut, dx_cut;
  float *z, *target_z, *sums;
  float2* parts;
  uint16_t *dl, *dlt;
  size_t bytes;
};
constexpr size_t kFewPiece = size_t{96} << 20;  // bytes of w that the Infinity Cache still
                                                // holds when dx reads them
FewPlan few_plan(const HeadArgs& a, int elem_bytes, bool backward, void* ws) {
  FewPlan p{};
  const Form f = form_of(elem_bytes, a.n_rows);
  const size_t n = a.n_rows;
  p.piece = backward ? piece_of(a.vocab, static_cast<size_t>(a.d) * elem_bytes, kFewPiece)
                     : piece_of(a.vocab, 4 * n, size_t{64} << 20);
  p.kn = static_cast<int>(blocks(n, 16) * 16);
  p.z_cut = few_cut(p.piece, n, stages(f, a.d), 32);
  const size_t ldv = up64(p.piece);
  Carve c{static_cast<char*>(ws)};
  p.z = c.take<float>(p.z_cut.slices * n * ldv);
  if (backward) {
    // the slices' sums, written and read, stay under a quarter of w
    p.dx_cut = few_cut(a.d, n, stages(f, ldv) * (f == kBf16 ? 2 : 1),
                       std::clamp<int64_t>(ldv * elem_bytes / (32 * n), 8, 128));
    p.dl = c.take<uint16_t>(2 * n * ldv);  // floats, or two parts
    p.dlt = c.take<uint16_t>((f == kRaw ? 3 : 2) * ldv * p.kn);
    p.sums = c.take<float>(p.dx_cut.slices * n * a.d);
  } else {
    // pieces but the last are whole chunks
    p.parts = c.take<float2>(blocks(a.vocab, kFewChunk) * n + blocks(a.vocab, p.piece) * n);
    p.target_z = c.take<float>(n);
  }
  p.bytes = c.used;
  return p;
}

struct ForwardPlan {
  int piece, tiles;
  Tile tile;
  uint16_t *xp, *wp;
  float *amax, *factor;
  float2* parts;
  float* target_z;
  size_t bytes;
};
ForwardPlan forward_plan(const HeadArgs& a, int elem_bytes, void* ws) {
  ForwardPlan p{};
  const Form f = form_of(elem_bytes, a.n_rows);
  const size_t ld = up64(a.d), part_bytes = 2 * parts_of(f) * ld;
  // pieces but the last are whole tiles
  const int steps = stages(f, a.d) * products_of(f);
  const auto cut = [&](int columns) { return wide_cut(columns, a.n_rows, steps, 1, false, true); };
  p.piece = f == kHalves ? piece_of(a.vocab, part_bytes, size_t{128} << 20, a.n_rows,
                                    [&](int columns) { return cut(columns).us; })
                         : a.vocab;
  p.tile = cut(p.piece).tile;
  p.tiles = static_cast<int>(blocks(a.vocab, tile_rows(p.tile)));
  Carve c{static_cast<char*>(ws)};
  p.parts = c.take<float2>(static_cast<size_t>(p.tiles) * a.n_rows);
  p.target_z = c.take<float>(a.n_rows);
  if (f == kHalves) {
    p.amax = c.take<float>(kAmax);
    p.factor = c.take<float>(a.n_rows);
    p.xp = c.take<uint16_t>(part_bytes / 2 * a.n_rows);
    p.wp = c.take<uint16_t>(part_bytes / 2 * p.piece);
  }
  p.bytes = c.used;
  return p;
}

// The cuts of the gradient's products over a piece of the vocabulary.
Cut dl_cut(const HeadArgs& a, Form f, int columns) {
  return wide_cut(columns, a.n_rows, stages(f, a.d) * products_of(f), 1, false, true);
}
Cut dw_cut(const HeadArgs& a, Form f, int columns) {
  return wide_cut(a.d, columns, stages(f, a.n_rows) * products_of(f), 1, false, true);
}
Cut dx_cut(const HeadArgs& a, Form f, int columns) {  // K is the piece: in slices
  return wide_cut(a.d, a.n_rows, stages(f, up64(columns)) * products_of(f), 32, false, false);
}

struct BackwardPlan {
  int piece;
  Cut dx_cut;
  uint16_t *xp, *wp, *gx, *dl;
  float *amax, *factor, *sums;
  size_t bytes;
};
BackwardPlan backward_plan(const HeadArgs& a, int elem_bytes, void* ws) {
  BackwardPlan p{};
  const Form f = form_of(elem_bytes, a.n_rows);
  const size_t P = parts_of(f), ld = up64(a.d), n = a.n_rows;
  p.piece = piece_of(a.vocab, 2 * P * n + (f == kHalves ? 2 * P * ld : 0), size_t{192} << 20, n,
                     [&](int columns) {
                       return dl_cut(a, f, columns).us + dw_cut(a, f, columns).us +
                              dx_cut(a, f, columns).us;
                     });
  const size_t ldv = up64(p.piece);
  p.dx_cut = dx_cut(a, f, p.piece);
  Carve c{static_cast<char*>(ws)};
  p.gx = c.take<uint16_t>(P * n * a.d);
  p.dl = c.take<uint16_t>(P * n * ldv);
  p.sums = c.take<float>(p.dx_cut.slices * n * a.d);
  if (f == kHalves) {
    p.amax = c.take<float>(kAmax);
    p.factor = c.take<float>(n);
    p.xp = c.take<uint16_t>(P * ld * n);
    p.wp = c.take<uint16_t>(P * ld * p.piece);
  }
  p.bytes = c.used;
  return p;
}

// ---------------------------------------------------------------- launches
// The operand x, in place or as parts in xp; halves: amax of w (and of the gradient's x)
// on the way.
template <Form F>
Operand x_operand(const HeadArgs& a, const float* dlogp, float* amax, float* factor, uint16_t* xp,
                  hipStream_t s) {
  const int n = static_cast<int>(a.n_rows), units = F == kRaw ? 2 * a.d : a.d;
  if (F != kHalves) return Operand{static_cast<const uint16_t*>(a.x), 0, units, n, units};
  const int ld = static_cast<int>(up64(a.d));
  head_clear_kernel<<<1, kAmax, 0, s>>>(amax);
  const int64_t runs = static_cast<int64_t>(a.vocab) * a.d / 8;
  head_amax_kernel<<<static_cast<uint32_t>(std::min<int64_t>(blocks(runs, kAmaxRuns), kAmaxGroups)),
                     256, 0, s>>>(
      static_cast<const float*>(a.w), runs, amax);
  head_x_kernel<<<static_cast<uint32_t>(blocks(n, 4)), 256, 0, s>>>(a, ld, dlogp, factor, amax,
                                                                   xp);
  return Operand{xp, a.n_rows * ld, ld, n, ld};
}

// The operand of columns [v0, v0 + rows) of the vocabulary.
template <Form F>
Operand w_operand(const HeadArgs& a, int64_t v0, int rows, const float* amax, uint16_t* wp,
                  hipStream_t s) {
  const int units = F == kRaw ? 2 * a.d : a.d;
  if (F != kHalves)
    return Operand{static_cast<const uint16_t*>(a.w) + v0 * units, 0, units, rows, units};
  const int ld = static_cast<int>(up64(a.d));
  head_w_kernel<<<static_cast<uint32_t>(blocks(static_cast<int64_t>(rows) * (ld / 8), 256)), 256, 0,
                  s>>>(static_cast<const float*>(a.w) + v0 * a.d, rows, a.d, ld, amax, wp);
  return Operand{wp, static_cast<int64_t>(rows) * ld, ld, rows, ld};
}

RowResults row_results(const HeadArgs& a, float* logp, float* lse, float* stats) {
  return RowResults{a.targets, a.index_bytes, a.vocab, logp, lse, reinterpret_cast<float2*>(stats)};
}

dim3 dx_grid(const HeadArgs& a) {
  const int64_t all = blocks(a.n_rows * a.d, 256), across = std::min<int64_t>(all, 1 << 20);
  return dim3(static_cast<uint32_t>(across),
              static_cast<uint32_t>(blocks(all, static_cast<int>(across))));
}

template <Form F>
hipError_t forward(const HeadArgs& a, void* ws, float* logp, float* lse, float* stats,
                   hipStream_t s) {
  const ForwardPlan p = forward_plan(a, F == kBf16 ? 2 : 4, ws);
  const int n = static_cast<int>(a.n_rows);
  const Operand x = x_operand<F>(a, nullptr, p.amax, p.factor, p.xp, s);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const Operand w = w_operand<F>(a, v0, rows, p.amax, p.wp, s);
    const StatsArgs k{w, x, static_cast<int>(v0), a.vocab, stages(F, a.d), a.scale,
                      p.factor, a.targets, a.index_bytes,
                      p.parts + v0 / tile_rows(p.tile) * a.n_rows, p.target_z};
    const hipError_t e = with_wide_tile(p.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(rows, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      head_stats_kernel<CF, F><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(k, mb, nb);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  head_join_kernel<<<static_cast<uint32_t>(blocks(n, 16)), 256, 0, s>>>(
      p.parts, p.tiles, a.n_rows, p.target_z, row_results(a, logp, lse, stats));
  return hipGetLastError();
}

template <Form F>
hipError_t backward(const HeadArgs& a, const float* stats, const float* dlogp, void* ws, void* dx,
                    void* dw, hipStream_t s) {
  typedef std::conditional_t<F == kBf16, uint16_t, float> E;
  const BackwardPlan p = backward_plan(a, sizeof(E), ws);
  const int n = static_cast<int>(a.n_rows);
  const float* const amax_w = F == kHalves ? p.amax : nullptr;
  const float* const amax_x = F == kHalves ? p.amax + 1 : nullptr;
  const Operand x = x_operand<F>(a, dlogp, p.amax, p.factor, p.xp, s);
  head_gx_kernel<F><<<static_cast<uint32_t>(blocks(n, 4)), 256, 0, s>>>(a, dlogp, amax_x, p.gx);
  const Operand gx{p.gx, a.n_rows * a.d, a.d, a.d, n};
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const int ldv = static_cast<int>(up64(rows));
    const Operand w = w_operand<F>(a, v0, rows, amax_w, p.wp, s);
    const DlArgs k{w, x, static_cast<int>(v0), a.vocab, stages(F, a.d), a.scale, p.factor,
                   a.targets, a.index_bytes, reinterpret_cast<const float2*>(stats), dlogp, p.dl,
                   ldv};
    hipError_t e = with_wide_tile(dl_cut(a, F, rows).tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(rows, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      head_dl_kernel<CF, F><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(k, mb, nb);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    // dx: K is the vocabulary, along w's columns; dw: K is the rows, along dl's and gx's
    const int64_t dl_part = a.n_rows * ldv;
    const Operand wt{w.p, w.part, w.ld, a.d, rows};
    const Operand dl{p.dl, dl_part, ldv, n, ldv};
    const Operand dlt{p.dl, dl_part, ldv, ldv, n};
    e = with_wide_tile(p.dx_cut.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      product_kernel<CF, F, true, false>
          <<<dim3(static_cast<uint32_t>(mb) * nb, p.dx_cut.slices), CF::NT, 0, s>>>(
              wt, dl, stages(F, ldv), mb, nb, n, a.d, SumStore{p.sums, a.d, n, v0 > 0});
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    e = with_wide_tile(dw_cut(a, F, rows).tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM));
      const int nb = static_cast<int>(blocks(rows, CF::BN));
      product_kernel<CF, F, true, true><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(
          gx, dlt, stages(F, n), mb, nb, rows, a.d,
          ElementStore<E>{static_cast<E*>(dw) + v0 * a.d, a.d, amax_x, -kDlExponent});
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  head_dx_kernel<E, F><<<dx_grid(a), 256, 0, s>>>(
      a, p.sums, p.dx_cut.slices, dlogp, amax_w, static_cast<E*>(dx));
  return hipGetLastError();
}

template <Form F, class Call>
hipError_t with_form_tile(Tile t, const Call& f) {
  if constexpr (F == kRaw) return with_raw_tile(t, f);
  else return f(Bare());  // at most 32 rows
}

// Few rows: z = x w^T of a piece, in slices of K.
template <Form F>
hipError_t few_z_product(const HeadArgs& a, const FewPlan& p, int64_t v0, int rows,
                         hipStream_t s) {
  const Operand x = x_operand<F>(a, nullptr, nullptr, nullptr, nullptr, s);
  const Operand w = w_operand<F>(a, v0, rows, nullptr, nullptr, s);
  return with_form_tile<F>(p.z_cut.tile, [&](auto cf) {
    typedef decltype(cf) CF;
    const int mb = static_cast<int>(blocks(rows, CF::BM));
    const int pitch = static_cast<int>(up64(rows));
    product_kernel<CF, F, false, false><<<dim3(mb, p.z_cut.slices), CF::NT, 0, s>>>(
        w, x, stages(F, a.d), mb, 1, x.rows, pitch, SumStore{p.z, pitch, x.rows, false});
    return hipGetLastError();
  });
}

FewZ few_z_of(const HeadArgs& a, const FewPlan& p, int64_t v0, int rows) {
  return FewZ{p.z, p.z_cut.slices, static_cast<int>(up64(rows)), rows, static_cast<int>(v0),
              a.scale};
}

template <Form F>
hipError_t few_forward(const HeadArgs& a, void* ws, float* logp, float* lse, float* stats,
                       hipStream_t s) {
  const FewPlan p = few_plan(a, F == kBf16 ? 2 : 4, false, ws);
  const RowResults o = row_results(a, logp, lse, stats);
  const bool whole = a.vocab <= kFewChunk;
  int chunks = 0;
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const hipError_t e = few_z_product<F>(a, p, v0, rows, s);
    if (e != hipSuccess) return e;
    const int more = static_cast<int>(blocks(rows, kFewChunk));
    head_few_stats_kernel<<<dim3(more, static_cast<uint32_t>(a.n_rows)), 256, 0, s>>>(
        few_z_of(a, p, v0, rows), a.n_rows, whole ? nullptr : p.parts + chunks * a.n_rows,
        p.target_z, o);
    chunks += more;
  }
  if (!whole)
    head_join_kernel<<<static_cast<uint32_t>(blocks(a.n_rows, 16)), 256, 0, s>>>(
        p.parts, chunks, a.n_rows, p.target_z, o);
  return hipGetLastError();
}

template <Form F>
hipError_t few_backward(const HeadArgs& a, const float* stats, const float* dlogp, void* ws,
                        void* dx, void* dw, hipStream_t s) {
  typedef std::conditional_t<F == kBf16, uint16_t, float> E;
  const FewPlan p = few_plan(a, sizeof(E), true, ws);
  const int n = static_cast<int>(a.n_rows), per = F == kRaw ? 2 : 1;  // 16-bit units a place
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const int ldv = static_cast<int>(up64(rows));
    hipError_t e = few_z_product<F>(a, p, v0, rows, s);
    if (e != hipSuccess) return e;
    head_few_dl_kernel<F><<<ldv / 64, 256, 0, s>>>(a, few_z_of(a, p, v0, rows),
                                                   reinterpret_cast<const float2*>(stats), dlogp,
                                                   p.dl, ldv, p.dlt, p.kn);
    // dx: K is the vocabulary, along w's columns
    const Operand wt{w_operand<F>(a, v0, rows, nullptr, nullptr, s).p, 0,
                     static_cast<int64_t>(per) * a.d, a.d, rows};
    const Operand dl{p.dl, a.n_rows * ldv, static_cast<int64_t>(per) * ldv, n, per * ldv};
    e = with_form_tile<F>(p.dx_cut.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM));
      product_kernel<CF, F == kBf16 ? kBf16Two : F, true, false>
          <<<dim3(mb, p.dx_cut.slices), CF::NT, 0, s>>>(wt, dl, stages(F, ldv), mb, 1, n, a.d,
                                                        SumStore{p.sums, a.d, n, v0 > 0});
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    // a wave takes 32 of the vocabulary at a time: two workgroups a CU, which load x once
    const int64_t across = blocks(a.d, 128), down = blocks(rows, 128);
    const uint32_t groups = static_cast<uint32_t>(
        std::clamp<int64_t>(blocks(512, static_cast<int>(across)), 1, std::min<int64_t>(down, 32768)));
    head_few_dw_kernel<F><<<dim3(static_cast<uint32_t>(across), groups), 256, 0, s>>>(
        a, p.dlt, rows, p.kn, static_cast<E*>(dw) + v0 * a.d);
  }
  head_dx_kernel<E, F><<<dx_grid(a), 256, 0, s>>>(
      a, p.sums, p.dx_cut.slices, dlogp, nullptr, static_cast<E*>(dx));
  return hipGetLastError();
}

}  // namespace

size_t head_forward_bytes(const HeadArgs& a, int elem_bytes) {
  if (a.n_rows == 0) return 0;
  return few_rows(a, elem_bytes, false) ? few_plan(a, elem_bytes, false, nullptr).bytes
                                        : forward_plan(a, elem_bytes, nullptr).bytes;
}
size_t head_backward_bytes(const HeadArgs& a, int elem_bytes) {
  if (a.n_rows == 0) return 0;
  return few_rows(a, elem_bytes, true) ? few_plan(a, elem_bytes, true, nullptr).bytes
                                       : backward_plan(a, elem_bytes, nullptr).bytes;
}

hipError_t launch_head_forward(const HeadArgs& a, int elem_bytes, void* ws, float* logp,
                               float* lse, float* stats, hipStream_t s) {
  if (a.n_rows == 0) return hipSuccess;
  const bool few = few_rows(a, elem_bytes, false);
  switch (form_of(elem_bytes, a.n_rows)) {
    case kRaw: return few_forward<kRaw>(a, ws, logp, lse, stats, s);
    case kHalves: return forward<kHalves>(a, ws, logp, lse, stats, s);
    default:
      return few ? few_forward<kBf16>(a, ws, logp, lse, stats, s)
                 : forward<kBf16>(a, ws, logp, lse, stats, s);
  }
}

hipError_t launch_head_backward(const HeadArgs& a, int elem_bytes, const float* stats,
                                const float* dlogp, void* ws, void* dx, void* dw, hipStream_t s) {
  if (a.n_rows == 0) {
    const int64_t count = static_cast<int64_t>(a.vocab) * a.d * elem_bytes / 16;
    head_zero_kernel<<<static_cast<uint32_t>(std::min<int64_t>(blocks(count, 256), 1 << 20)), 256,
                       0, s>>>(static_cast<uint4*>(dw), count);
    return hipGetLastError();
  }
  const bool few = few_rows(a, elem_bytes, true);
  switch (form_of(elem_bytes, a.n_rows)) {
    case kRaw: return few_backward<kRaw>(a, stats, dlogp, ws, dx, dw, s);
    case kHalves: return backward<kHalves>(a, stats, dlogp, ws, dx, dw, s);
    default:
      return few ? few_backward<kBf16>(a, stats, dlogp, ws, dx, dw, s)
                 : backward<kBf16>(a, stats, dlogp, ws, dx, dw, s);
  }
}

}  // namespace twell
