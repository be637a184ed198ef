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
// With bfloat16 x and w, dl is held in bfloat16: its rounding, 2^-9 of each element,
// is of the size of dx's and dw's own (with few rows, where it costs next to nothing,
// as two parts).  With float32 ones every operand is two half-precision parts
// (nt_gemm.h), w scaled by its largest element, x by each row's; dl / g lies in [-1, 1]
// and is scaled by 2^14, with g taken into dx at the end and into the x of dw.  With few
// rows, where reading w is what the call costs, float32 operands and dl stay float32.
// Both products read w, x and dl as they lie, turning fragments with LDS transpose
// reads where K runs along a column.
#include <algorithm>
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

constexpr int kDlExponent = 14;  // of dl / g in halves

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
// bits of non-negative floats.  4 runs a lane, one workgroup after another.
constexpr int kAmaxRuns = 4 * 256;
__global__ __launch_bounds__(256) void head_amax_kernel(const float* __restrict__ src,
                                                        int64_t runs, float* amax) {
  __shared__ float lds[4];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kAmaxRuns + threadIdx.x;
  float v[4][8] = {};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (i0 + u * 256 < runs) load_run(src + (i0 + u * 256) * 8, v[u]);
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max_finite(m, v[u][k]);
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

// Halves [2][rows][ld] of x, a wave a row, scaled by the row's largest element, what undoes
// it in undo[row]; and, for the gradient (dlogp not null), *amax = the largest of
// |scale dlogp x| over rows with a target.
__global__ __launch_bounds__(256) void head_x_kernel(HeadArgs a, int ld,
                                                     const float* __restrict__ dlogp,
                                                     float* __restrict__ undo, float* amax,
                                                     uint16_t* __restrict__ out) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  if (row >= a.n_rows) return;
  const float* src = static_cast<const float*>(a.x) + row * a.d;
  float m = 0.f;
  for (int c = lane_id() * 8; c < a.d; c += kWave * 8) {
    float v[8];
    load_run(src + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max_finite(m, v[k]);
  }
  m = wave_max(m);
  const int e = exponent_for(m);
  const float f = power_of_two(e);
  if (lane_id() == 0) {
    undo[row] = power_of_two(-e);
    if (dlogp != nullptr && has_target(a.targets, a.index_bytes, a.vocab, row))
      atomicMax(reinterpret_cast<int*>(amax),
                __float_as_int(max_finite(0.f, dlogp[row] * a.scale * m)));
  }
  for (int c = lane_id() * 8; c < ld; c += kWave * 8) {
    float v[8] = {};
    if (c < a.d) load_run(src + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
    put_run<kHalves>(out + row * ld, a.n_rows * ld, c, v);
  }
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
    if constexpr (F == kRaw) {
      float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + row * a.d + c);
      to[0] = make_float4(v[0], v[1], v[2], v[3]);
      to[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * g * f;
      put_run<F>(out + row * a.d, a.n_rows * a.d, c, v);
    }
  }
}

// What a column of accumulators is multiplied by to be z: scale, and the powers of two
// of both operands undone.
template <Form F, class Args>
__device__ __forceinline__ float z_factor(const Args& a, int64_t n) {
  if constexpr (F == kHalves)
    return a.scale * (n < a.x.rows ? a.undo[n] : 0.f) * power_of_two(-exponent_for(*a.amax));
  return a.scale;
}

// ---------------------------------------------------------------- forward
struct StatsArgs {
  Operand w, x;      // w: a piece of the vocabulary, from column v0
  int v0, vocab;     // whole vocabulary
  int ksteps;
  float scale;
  const float *amax, *undo;  // halves: of w, and per row of x
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
    m = fmaxf(m, other_half(m)) * f;
    const float base = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CF::FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], f, -base) * kLog2e);
    s += other_half(s);
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
      if (mine) a.target_z[n] = z * f;
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

// Joins the tiles' {m, s} of 16 tokens a workgroup, in 16 streams of tiles.
__global__ __launch_bounds__(256) void head_join_kernel(const float2* __restrict__ parts,
                                                        int tiles, int64_t n_rows,
                                                        const void* __restrict__ targets,
                                                        int index_bytes, int vocab,
                                                        const float* __restrict__ target_z,
                                                        float* __restrict__ logp,
                                                        float* __restrict__ lse,
                                                        float2* __restrict__ stats) {
  __shared__ float2 joint[16][16];
  const int col = threadIdx.x % 16, stream = threadIdx.x / 16;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + col;
  float m = -INFINITY, s = 0.f;
  if (n < n_rows)
    for (int t = stream; t < tiles; t += 16) {
      const float2 p = parts[t * n_rows + n];
      const float top = fmaxf(m, p.x);
      const float base = top == -INFINITY ? 0.f : top;
      s = s * __builtin_amdgcn_exp2f((m - base) * kLog2e) +
          p.y * __builtin_amdgcn_exp2f((p.x - base) * kLog2e);
      m = top;
    }
  joint[stream][col] = make_float2(m, s);
  __syncthreads();
  if (stream != 0 || n >= n_rows) return;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < 16; ++w) m = fmaxf(m, joint[w][col].x);
  const float base = m == -INFINITY ? 0.f : m;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w)
    s += joint[w][col].y * __builtin_amdgcn_exp2f((joint[w][col].x - base) * kLog2e);
  const float log_s = logf(s);  // -inf for a row with nothing left
  const int64_t t = target_of(targets, index_bytes, n);
  stats[n] = make_float2(m, s);
  lse[n] = base + log_s;
  float lp = 0.f;
  // a row with nothing left: z - lse would be -inf + inf
  if (t >= 0 && t < vocab) lp = m == -INFINITY && s == 0.f ? -INFINITY : target_z[n] - base - log_s;
  logp[n] = lp;
}

// ---------------------------------------------------------------- gradient
// Part p of two values, packed.
template <Form F>
__device__ __forceinline__ uint32_t pack_part(float a, float b, int p) {
  if constexpr (F == kBf16) {
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
    if (p == 1)  // what the first part leaves
      w = __builtin_bit_cast(
          uint32_t, __builtin_convertvector(f32x2_t{a - __uint_as_float(w << 16),
                                                    b - __uint_as_float(w & 0xffff0000u)},
                                            bf16x2_t));
    return w;
  } else {
    _Float16 x = static_cast<_Float16>(a), y = static_cast<_Float16>(b);
    if (p == 1) {  // what the first part leaves; |a| is at most 2^14, or NaN
      x = static_cast<_Float16>(a == a ? a - static_cast<float>(x) : 0.f);
      y = static_cast<_Float16>(b == b ? b - static_cast<float>(y) : 0.f);
    }
    return __builtin_bit_cast(uint16_t, x) |
           static_cast<uint32_t>(__builtin_bit_cast(uint16_t, y)) << 16;
  }
}

struct DlArgs {
  Operand w, x;
  int v0, vocab;
  int ksteps;
  float scale;
  const float *amax, *undo;  // halves: of w, and per row of x
  const void* targets;
  int index_bytes;
  const float2* stats;
  const float* dlogp;
  uint16_t* dl;  // [parts][n][ldv]; raw: float [n][ldv]
  int ldv;
};

template <class CF, Form F, int PARTS>
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
        const float e = __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], f, -m) * kLog2e);
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
  if constexpr (F == kRaw) {
#pragma unroll
    for (int j = 0; j < CF::FN; ++j) {
      const int n = nb * CF::BN + nt::block_col<CF>() + 32 * j;
#pragma unroll
      for (int i = 0; i < CF::FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int v = row0 + nt::row_of(i, 4 * q);
          if (n < n_rows && v < a.ldv)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.dl) + n * int64_t{a.ldv} + v) =
                make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]);
        }
    }
    return;
  }
  // a part at a time through LDS, so that its rows are stored whole: the 16-byte chunk c
  // of row n at position c ^ n, which spreads the 32 rows of a write over the banks
  constexpr int CHUNKS = CF::BM / 8;
  static_assert(CF::BM * CF::BN <= CF::STAGES * CF::STAGE, "the tile fits the stages");
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
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

// dx = the sum of the slices, rounded; 8 elements a lane.  Halves: times scale * dlogp
// of the row and the powers of two undone.
template <typename E, Form F>
__global__ __launch_bounds__(256) void head_dx_kernel(HeadArgs a, const float* __restrict__ sums,
                                                      int slices, const float* __restrict__ dlogp,
                                                      const float* amax, E* __restrict__ dx) {
  const int64_t elems = a.n_rows * a.d;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= elems) return;
  float v[8] = {};
  for (int s = 0; s < slices; ++s) {
    float p[8];
    load_run(sums + s * elems + i, p);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += p[k];
  }
  if constexpr (F == kHalves) {
    const int64_t n = i / a.d;
    const bool given = has_target(a.targets, a.index_bytes, a.vocab, n);
    const float g = given ? dlogp[n] * a.scale : 0.f;
    const float f = power_of_two(-kDlExponent - exponent_for(*amax));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = given ? v[k] * f * g : 0.f;
  }
  if constexpr (sizeof(E) == 2) {
    put_run<kBf16>(reinterpret_cast<uint16_t*>(dx) + i, 0, 0, v);
  } else {
    *reinterpret_cast<float4*>(dx + i) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(dx + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__global__ __launch_bounds__(256) void head_zero_kernel(uint4* p, int64_t count) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- sizes
// Columns of the vocabulary taken at a time: all where the forward pass reads w in
// place, else as many as keep what is made per column within `budget`, in equal
// pieces.
int piece_of(int vocab, size_t per_column, size_t budget) {
  const int64_t most = std::max<int64_t>(budget / per_column / 256 * 256, 1024);
  const int64_t pieces = blocks(vocab, static_cast<int>(std::min<int64_t>(most, vocab)));
  return static_cast<int>(std::min<int64_t>(blocks(blocks(vocab, static_cast<int>(pieces)), 256) * 256, vocab));
}

constexpr size_t kFewPiece = size_t{96} << 20;  // bytes of w
constexpr int kAmax = 2;  // largest magnitudes: of w, of scale * dlogp * x

// The form of the operands; and the stages of a product over k.
Form form_of(int elem_bytes, int64_t n) {
  return elem_bytes == 2 ? kBf16 : n <= kFewColumns ? kRaw : kHalves;
}
int stages(Form f, int64_t k) { return static_cast<int>(blocks(k, f == kRaw ? 32 : 64)); }
int dl_parts(Form f, int64_t n) { return f == kBf16 && n <= kFewColumns ? 2 : parts_of(f); }

struct ForwardPlan {
  int piece, tiles;
  Tile tile;
  uint16_t *xp, *wp;
  float *amax, *undo;
  float2* parts;
  float* target_z;
  size_t bytes;
};
ForwardPlan forward_plan(const HeadArgs& a, int elem_bytes, void* ws) {
  ForwardPlan p{};
  const Form f = form_of(elem_bytes, a.n_rows);
  const size_t ld = up64(a.d), part_bytes = 2 * parts_of(f) * ld;
  // pieces but the last are whole tiles
  p.piece = f == kHalves ? piece_of(a.vocab, part_bytes, size_t{128} << 20) : a.vocab;
  const int64_t steps = stages(f, a.d) * products_of(f);
  p.tile = a.n_rows <= kFewColumns ? few_cut(p.piece, a.n_rows, steps, 1).tile
                                   : wide_cut(p.piece, a.n_rows, steps, 1, false).tile;
  p.tiles = static_cast<int>(blocks(a.vocab, tile_rows(p.tile)));
  Carve c{static_cast<char*>(ws)};
  p.parts = c.take<float2>(static_cast<size_t>(p.tiles) * a.n_rows);
  p.target_z = c.take<float>(a.n_rows);
  if (f == kHalves) {
    p.amax = c.take<float>(kAmax);
    p.undo = c.take<float>(a.n_rows);
    p.xp = c.take<uint16_t>(part_bytes / 2 * a.n_rows);
    p.wp = c.take<uint16_t>(part_bytes / 2 * p.piece);
  }
  p.bytes = c.used;
  return p;
}

struct BackwardPlan {
  int piece;
  Tile dl_tile;
  Cut dx_cut;
  uint16_t *xp, *wp, *gx, *dl;
  float *amax, *undo, *sums;
  size_t bytes;
};
BackwardPlan backward_plan(const HeadArgs& a, int elem_bytes, void* ws) {
  BackwardPlan p{};
  const Form f = form_of(elem_bytes, a.n_rows);
  const bool few = a.n_rows <= kFewColumns;
  const size_t ld = up64(a.d), n = a.n_rows;
  const size_t element = f == kRaw ? 4 : 2 * dl_parts(f, n);  // bytes of a place of dl
  // few rows: a piece of w that the Infinity Cache still holds when dx reads it
  const size_t per_column = few ? static_cast<size_t>(a.d) * elem_bytes
                                : n * element + (f == kHalves ? 4 * ld : 0);
  p.piece = piece_of(a.vocab, per_column, few ? kFewPiece : size_t{192} << 20);
  const size_t ldv = up64(p.piece);
  // dx: K is a piece of the vocabulary; split until the tiles fill the CUs
  if (few) {
    p.dl_tile = few_cut(p.piece, n, 1, 1).tile;
    p.dx_cut = few_cut(a.d, n, stages(f, ldv) * (f == kBf16 ? 2 : 1), 32);
  } else {
    p.dl_tile = wide_cut(p.piece, n, stages(f, a.d) * products_of(f), 1, false).tile;
    p.dx_cut = wide_cut(a.d, n, stages(f, ldv) * products_of(f), 32, false);
  }
  Carve c{static_cast<char*>(ws)};
  p.gx = c.take<uint16_t>((f == kBf16 ? 1 : 2) * n * a.d);
  p.dl = c.take<uint16_t>(element / 2 * n * ldv);
  p.sums = c.take<float>(p.dx_cut.slices * n * a.d);
  if (f == kHalves) {
    p.amax = c.take<float>(kAmax);
    p.undo = c.take<float>(n);
    p.xp = c.take<uint16_t>(2 * ld * n);
    p.wp = c.take<uint16_t>(2 * ld * p.piece);
  }
  p.bytes = c.used;
  return p;
}

// ---------------------------------------------------------------- launches
// The operand x, in place or as parts in xp; halves: amax of w (and of the gradient's x)
// on the way.
template <Form F>
Operand x_operand(const HeadArgs& a, const float* dlogp, float* amax, float* undo, uint16_t* xp,
                  hipStream_t s) {
  const int n = static_cast<int>(a.n_rows), units = F == kRaw ? 2 * a.d : a.d;
  if (F != kHalves) return Operand{static_cast<const uint16_t*>(a.x), 0, units, n, units};
  const int ld = static_cast<int>(up64(a.d));
  head_clear_kernel<<<1, kAmax, 0, s>>>(amax);
  const int64_t runs = static_cast<int64_t>(a.vocab) * a.d / 8;
  head_amax_kernel<<<static_cast<uint32_t>(blocks(runs, kAmaxRuns)), 256, 0, s>>>(
      static_cast<const float*>(a.w), runs, amax);
  head_x_kernel<<<static_cast<uint32_t>(blocks(n, 4)), 256, 0, s>>>(a, ld, dlogp, undo, amax + 1,
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

// f(tile) with the tiles for few rows or for many; raw: few.
template <Form F, class Call>
hipError_t with_tile(bool few, Tile t, const Call& f) {
  if constexpr (F == kRaw) return with_few_tile(t, f);
  else if constexpr (F == kHalves) return with_wide_tile(t, f);
  else return few ? with_few_tile(t, f) : with_wide_tile(t, f);
}

template <Form F>
hipError_t forward(const HeadArgs& a, void* ws, float* logp, float* lse, float* stats,
                   hipStream_t s) {
  const ForwardPlan p = forward_plan(a, F == kBf16 ? 2 : 4, ws);
  const int n = static_cast<int>(a.n_rows);
  const Operand x = x_operand<F>(a, nullptr, p.amax, p.undo, p.xp, s);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const Operand w = w_operand<F>(a, v0, rows, p.amax, p.wp, s);
    const StatsArgs k{w, x, static_cast<int>(v0), a.vocab, stages(F, a.d), a.scale, p.amax,
                      p.undo, a.targets, a.index_bytes,
                      p.parts + v0 / tile_rows(p.tile) * a.n_rows, p.target_z};
    const hipError_t e = with_tile<F>(n <= kFewColumns, p.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(rows, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      head_stats_kernel<CF, F><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(k, mb, nb);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  head_join_kernel<<<static_cast<uint32_t>(blocks(n, 16)), 256, 0, s>>>(
      p.parts, p.tiles, a.n_rows, a.targets, a.index_bytes, a.vocab, p.target_z, logp, lse,
      reinterpret_cast<float2*>(stats));
  return hipGetLastError();
}

// FEW: at most kFewColumns rows.
template <Form F, bool FEW>
hipError_t backward(const HeadArgs& a, const float* stats, const float* dlogp, void* ws, void* dx,
                    void* dw, hipStream_t s) {
  typedef std::conditional_t<F == kBf16, uint16_t, float> E;
  constexpr int PARTS = F == kBf16 && FEW ? 2 : parts_of(F);  // dl_parts
  constexpr Form PRODUCT = F == kBf16 && FEW ? kBf16Two : F;
  const BackwardPlan p = backward_plan(a, sizeof(E), ws);
  const int n = static_cast<int>(a.n_rows);
  const float* const amax_w = F == kHalves ? p.amax : nullptr;
  const float* const amax_x = F == kHalves ? p.amax + 1 : nullptr;
  const int per = F == kRaw ? 2 : 1;  // 16-bit units of an element
  const Operand x = x_operand<F>(a, dlogp, p.amax, p.undo, p.xp, s);
  head_gx_kernel<F><<<static_cast<uint32_t>(blocks(n, 4)), 256, 0, s>>>(a, dlogp, amax_x, p.gx);
  const Operand gx{p.gx, a.n_rows * a.d, static_cast<int64_t>(per) * a.d, a.d, n};
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const int ldv = static_cast<int>(up64(rows));
    const Operand w = w_operand<F>(a, v0, rows, amax_w, p.wp, s);
    const DlArgs k{w, x, static_cast<int>(v0), a.vocab, stages(F, a.d), a.scale, amax_w, p.undo,
                   a.targets, a.index_bytes, reinterpret_cast<const float2*>(stats), dlogp, p.dl,
                   ldv};
    hipError_t e = with_tile<F>(FEW, p.dl_tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(rows, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      if constexpr ((CF::BN <= kFewColumns) == FEW)
        head_dl_kernel<CF, F, PARTS><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(k, mb, nb);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    // dx: K is the vocabulary, along w's columns; dw: K is the rows, along dl's and gx's
    const int64_t dl_part = a.n_rows * ldv;
    const Operand wt{w.p, w.part, w.ld, a.d, rows};
    const Operand dl{p.dl, dl_part, static_cast<int64_t>(per) * ldv, n, per * ldv};
    const Operand dlt{p.dl, dl_part, static_cast<int64_t>(per) * ldv, ldv, n};
    e = with_tile<F>(FEW, p.dx_cut.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      if constexpr ((CF::BN <= kFewColumns) == FEW)
        product_kernel<CF, PRODUCT, true, false, float, true>
            <<<dim3(static_cast<uint32_t>(mb) * nb, p.dx_cut.slices), CF::NT, 0, s>>>(
                wt, dl, stages(F, ldv), mb, nb, n, v0 > 0, a.d, nullptr, 0, p.sums);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    const auto dw_product = [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM));
      const int nb = static_cast<int>(blocks(rows, CF::BN));
      product_kernel<CF, PRODUCT, true, true, E, false>
          <<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(
              gx, dlt, stages(F, n), mb, nb, rows, false, a.d, amax_x, -kDlExponent,
              static_cast<E*>(dw) + v0 * a.d);
      return hipGetLastError();
    };
    if constexpr (FEW)
      e = dw_product(Mid());
    else
      e = with_wide_tile(wide_cut(a.d, rows, stages(F, n) * products_of(F), 1, false).tile,
                         dw_product);
    if (e != hipSuccess) return e;
  }
  head_dx_kernel<E, F><<<static_cast<uint32_t>(blocks(a.n_rows * a.d / 8, 256)), 256, 0, s>>>(
      a, p.sums, p.dx_cut.slices, dlogp, amax_w, static_cast<E*>(dx));
  return hipGetLastError();
}

}  // namespace

size_t head_forward_bytes(const HeadArgs& a, int elem_bytes) {
  return a.n_rows == 0 ? 0 : forward_plan(a, elem_bytes, nullptr).bytes;
}
size_t head_backward_bytes(const HeadArgs& a, int elem_bytes) {
  return a.n_rows == 0 ? 0 : backward_plan(a, elem_bytes, nullptr).bytes;
}

hipError_t launch_head_forward(const HeadArgs& a, int elem_bytes, void* ws, float* logp,
                               float* lse, float* stats, hipStream_t s) {
  if (a.n_rows == 0) return hipSuccess;
  switch (form_of(elem_bytes, a.n_rows)) {
    case kBf16: return forward<kBf16>(a, ws, logp, lse, stats, s);
    case kRaw: return forward<kRaw>(a, ws, logp, lse, stats, s);
    default: return forward<kHalves>(a, ws, logp, lse, stats, s);
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
  switch (form_of(elem_bytes, a.n_rows)) {
    case kRaw: return backward<kRaw, true>(a, stats, dlogp, ws, dx, dw, s);
    case kHalves: return backward<kHalves, false>(a, stats, dlogp, ws, dx, dw, s);
    default:
      return a.n_rows <= kFewColumns ? backward<kBf16, true>(a, stats, dlogp, ws, dx, dw, s)
                                     : backward<kBf16, false>(a, stats, dlogp, ws, dx, dw, s);
  }
}

}  // namespace twell
