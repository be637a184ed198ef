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
// is of the size of dx's and dw's own.  With float32 ones every operand is two
// half-precision parts (nt_gemm.h), w scaled by its largest element, x by each row's;
// dl / g lies in [-1, 1] and is scaled by 2^14, with g taken into dx at the end and
// into the x of dw.  Both products read w, x and dl as they lie, turning fragments with
// LDS transpose reads where K runs along a column.
#include <algorithm>

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

// The form of operands of elements E.
template <typename E>
constexpr Form form_of() {
  return sizeof(E) == 2 ? kBf16 : kHalves;
}
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

// parts [rows][ld] of a piece of w, src [rows][d], scaled by *amax (halves); columns
// past d are zeros.
template <typename E>
__global__ __launch_bounds__(256) void head_w_kernel(const E* __restrict__ src, int64_t rows,
                                                     int d, int ld, const float* amax,
                                                     uint16_t* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = i / (ld / 8);
  const int c = static_cast<int>(i % (ld / 8)) * 8;
  if (row >= rows) return;
  float v[8] = {};
  if (c < d) load_run(src + row * d + c, v);
  if constexpr (form_of<E>() == kHalves) {
    const float f = power_of_two(exponent_for(*amax));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
  }
  put_run<form_of<E>()>(out + row * ld, rows * ld, c, v);
}

// parts [rows][ld] of x, a wave a row.  Halves: scaled by the row's largest element,
// what undoes it in undo[row]; and, for the gradient (dlogp not null), *amax = the
// largest of |scale dlogp x| over rows with a target.
template <typename E>
__global__ __launch_bounds__(256) void head_x_kernel(HeadArgs a, int ld,
                                                     const float* __restrict__ dlogp,
                                                     float* __restrict__ undo, float* amax,
                                                     uint16_t* __restrict__ out) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  if (row >= a.n_rows) return;
  const E* src = static_cast<const E*>(a.x) + row * a.d;
  float f = 1.f;
  if constexpr (form_of<E>() == kHalves) {
    float m = 0.f;
    for (int c = lane_id() * 8; c < a.d; c += kWave * 8) {
      float v[8];
      load_run(src + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max_finite(m, v[k]);
    }
    m = wave_max(m);
    const int e = exponent_for(m);
    f = power_of_two(e);
    if (lane_id() == 0) {
      undo[row] = power_of_two(-e);
      if (dlogp != nullptr && has_target(a.targets, a.index_bytes, a.vocab, row))
        atomicMax(reinterpret_cast<int*>(amax),
                  __float_as_int(max_finite(0.f, dlogp[row] * a.scale * m)));
    }
  }
  for (int c = lane_id() * 8; c < ld; c += kWave * 8) {
    float v[8] = {};
    if (c < a.d) load_run(src + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
    put_run<form_of<E>()>(out + row * ld, a.n_rows * ld, c, v);
  }
}

// parts [lines][ld] of dw's x, a wave a row: rows without a target, and past the end, are
// zeros (whatever x holds there meets gradients of zero, and a NaN must not spread).
// Halves: scale * dlogp * x, scaled by *amax.
template <typename E>
__global__ __launch_bounds__(256) void head_gx_kernel(HeadArgs a, int64_t lines, int ld,
                                                      const float* __restrict__ dlogp,
                                                      const float* amax,
                                                      uint16_t* __restrict__ out) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / kWave;
  if (row >= lines) return;
  const bool live = row < a.n_rows && has_target(a.targets, a.index_bytes, a.vocab, row);
  const E* src = static_cast<const E*>(a.x) + row * a.d;
  float f = 1.f, g = 1.f;
  if constexpr (form_of<E>() == kHalves) {
    f = power_of_two(exponent_for(*amax));
    if (live) g = dlogp[row] * a.scale;
  }
  for (int c = lane_id() * 8; c < ld; c += kWave * 8) {
    float v[8] = {};
    if (live && c < a.d) load_run(src + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * g * f;
    put_run<form_of<E>()>(out + row * ld, lines * ld, c, v);
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
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
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
        g = F == kBf16 ? a.dlogp[n] * a.scale : power_of_two(kDlExponent);
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

// dx = the sum of the slices, rounded; 8 elements a lane.  Halves: times scale * dlogp
// of the row and the powers of two undone.
template <typename E>
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
  if constexpr (form_of<E>() == kHalves) {
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
int part_count(int elem_bytes) { return elem_bytes == 2 ? 1 : 2; }

// Whether x and w serve as operands where they are.
bool direct(int elem_bytes, int d) { return elem_bytes == 2 && d % 64 == 0; }

// Columns of the vocabulary taken at a time: all where the forward pass reads w in
// place, else as many as keep what is made per column within `budget`, in equal
// pieces.
int piece_of(int vocab, size_t per_column, size_t budget) {
  const int64_t most = std::max<int64_t>(budget / per_column / 256 * 256, 1024);
  const int64_t pieces = blocks(vocab, static_cast<int>(std::min<int64_t>(most, vocab)));
  return static_cast<int>(std::min<int64_t>(blocks(blocks(vocab, static_cast<int>(pieces)), 256) * 256, vocab));
}

constexpr int kAmax = 2;  // largest magnitudes: of w, of scale * dlogp * x

// Stages of a contraction over d columns.
int64_t stages(const HeadArgs& a, int elem_bytes) {
  return up64(a.d) / 64 * (elem_bytes == 2 ? 1 : products_of(kHalves));
}

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
  const size_t ld = up64(a.d), part_bytes = 2 * part_count(elem_bytes) * ld;
  const bool in_place = direct(elem_bytes, a.d);
  p.piece = in_place ? a.vocab : piece_of(a.vocab, part_bytes, size_t{128} << 20);
  // tiles of a piece start at its first column: pieces but the last are whole tiles
  p.tile = cut_for(p.piece, a.n_rows, stages(a, elem_bytes), 1, false).tile;
  p.tiles = static_cast<int>(blocks(a.vocab, tile_rows(p.tile)));
  Carve c{static_cast<char*>(ws)};
  p.parts = c.take<float2>(static_cast<size_t>(p.tiles) * a.n_rows);
  p.target_z = c.take<float>(a.n_rows);
  if (!in_place) {
    p.amax = c.take<float>(kAmax);
    p.undo = c.take<float>(a.n_rows);
    p.xp = c.take<uint16_t>(part_bytes / 2 * a.n_rows);
    p.wp = c.take<uint16_t>(part_bytes / 2 * p.piece);
  }
  p.bytes = c.used;
  return p;
}

struct BackwardPlan {
  int piece, ldn;
  Tile dl_tile;
  Cut dx_cut;
  uint16_t *xp, *wp, *gx, *dl;
  float *amax, *undo, *sums;
  size_t bytes;
};
BackwardPlan backward_plan(const HeadArgs& a, int elem_bytes, void* ws) {
  BackwardPlan p{};
  const size_t P = part_count(elem_bytes), ld = up64(a.d), n = a.n_rows;
  const bool in_place = direct(elem_bytes, a.d);
  p.ldn = static_cast<int>(up64(n));
  const size_t per_column = 2 * P * (n + (in_place ? 0 : ld));
  p.piece = piece_of(a.vocab, per_column, size_t{192} << 20);
  const size_t ldv = up64(p.piece);
  // dx: K is a piece of the vocabulary; split until the tiles fill the CUs
  const int products = elem_bytes == 2 ? 1 : products_of(kHalves);
  p.dx_cut = cut_for(a.d, n, ldv / 64 * products, 32, false);
  p.dl_tile = cut_for(p.piece, n, stages(a, elem_bytes), 1, false).tile;
  Carve c{static_cast<char*>(ws)};
  p.gx = c.take<uint16_t>(P * p.ldn * ld);
  p.dl = c.take<uint16_t>(P * n * ldv);
  p.sums = c.take<float>(p.dx_cut.slices * n * a.d);
  if (!in_place) {
    p.amax = c.take<float>(kAmax);
    p.undo = c.take<float>(n);
    p.xp = c.take<uint16_t>(P * ld * n);
    p.wp = c.take<uint16_t>(P * ld * p.piece);
  }
  p.bytes = c.used;
  return p;
}

// ---------------------------------------------------------------- launches
int columns(const HeadArgs& a) { return static_cast<int>(up64(a.d)); }

// The operand x, in place or as parts in xp; halves: amax of w (and of the gradient's x)
// on the way.
template <typename E>
Operand x_operand(const HeadArgs& a, const float* dlogp, float* amax, float* undo, uint16_t* xp,
                  hipStream_t s) {
  const int n = static_cast<int>(a.n_rows), ld = columns(a);
  if (direct(sizeof(E), a.d)) return Operand{static_cast<const uint16_t*>(a.x), 0, a.d, n, 0};
  if constexpr (form_of<E>() == kHalves) {
    head_clear_kernel<<<1, kAmax, 0, s>>>(amax);
    const int64_t runs = static_cast<int64_t>(a.vocab) * a.d / 8;
    head_amax_kernel<<<static_cast<uint32_t>(blocks(runs, kAmaxRuns)), 256, 0, s>>>(
        static_cast<const float*>(a.w), runs, amax);
  }
  head_x_kernel<E><<<static_cast<uint32_t>(blocks(n, 4)), 256, 0, s>>>(a, ld, dlogp, undo,
                                                                      amax + 1, xp);
  return Operand{xp, a.n_rows * ld, ld, n, 0};
}

// The operand of columns [v0, v0 + rows) of the vocabulary.
template <typename E>
Operand w_operand(const HeadArgs& a, int64_t v0, int rows, const float* amax, uint16_t* wp,
                  hipStream_t s) {
  const E* src = static_cast<const E*>(a.w) + v0 * a.d;
  const int ld = columns(a);
  if (direct(sizeof(E), a.d)) return Operand{reinterpret_cast<const uint16_t*>(src), 0, a.d, rows, 0};
  head_w_kernel<E><<<static_cast<uint32_t>(blocks(static_cast<int64_t>(rows) * (ld / 8), 256)), 256,
                     0, s>>>(src, rows, a.d, ld, amax, wp);
  return Operand{wp, static_cast<int64_t>(rows) * ld, ld, rows, 0};
}

template <typename E>
hipError_t forward(const HeadArgs& a, void* ws, float* logp, float* lse, float* stats,
                   hipStream_t s) {
  constexpr Form F = form_of<E>();
  const ForwardPlan p = forward_plan(a, sizeof(E), ws);
  const int n = static_cast<int>(a.n_rows);
  const Operand x = x_operand<E>(a, nullptr, p.amax, p.undo, p.xp, s);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const Operand w = w_operand<E>(a, v0, rows, p.amax, p.wp, s);
    const StatsArgs k{w, x, static_cast<int>(v0), a.vocab, columns(a) / 64, a.scale, p.amax,
                      p.undo, a.targets, a.index_bytes,
                      p.parts + v0 / tile_rows(p.tile) * a.n_rows, p.target_z};
    const hipError_t e = with_tile(p.tile, [&](auto cf) {
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

template <typename E>
hipError_t backward(const HeadArgs& a, const float* stats, const float* dlogp, void* ws, void* dx,
                    void* dw, hipStream_t s) {
  constexpr Form F = form_of<E>();
  if (a.n_rows == 0) {
    const int64_t count = static_cast<int64_t>(a.vocab) * a.d * sizeof(E) / 16;
    head_zero_kernel<<<static_cast<uint32_t>(std::min<int64_t>(blocks(count, 256), 1 << 20)), 256,
                       0, s>>>(static_cast<uint4*>(dw), count);
    return hipGetLastError();
  }
  const BackwardPlan p = backward_plan(a, sizeof(E), ws);
  const int n = static_cast<int>(a.n_rows);
  const float* const amax_w = F == kHalves ? p.amax : nullptr;
  const float* const amax_x = F == kHalves ? p.amax + 1 : nullptr;
  const Operand x = x_operand<E>(a, dlogp, p.amax, p.undo, p.xp, s);
  const int ld = columns(a);
  head_gx_kernel<E><<<static_cast<uint32_t>(blocks(p.ldn, 4)), 256, 0, s>>>(a, p.ldn, ld, dlogp,
                                                                           amax_x, p.gx);
  const Operand gx{p.gx, static_cast<int64_t>(p.ldn) * ld, ld, a.d, p.ldn};
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
    const int rows = static_cast<int>(std::min<int64_t>(p.piece, a.vocab - v0));
    const int ldv = static_cast<int>(up64(rows));
    const Operand w = w_operand<E>(a, v0, rows, amax_w, p.wp, s);
    const DlArgs k{w, x, static_cast<int>(v0), a.vocab, columns(a) / 64, a.scale, amax_w, p.undo,
                   a.targets, a.index_bytes, reinterpret_cast<const float2*>(stats), dlogp, p.dl, ldv};
    hipError_t e = with_tile(p.dl_tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(rows, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      head_dl_kernel<CF, F><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(k, mb, nb);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    // dx: K is the vocabulary, along w's columns; dw: K is the rows, along dl's and gx's
    const Operand wt{w.p, w.part, w.ld, a.d, rows};
    const Operand dl{p.dl, static_cast<int64_t>(n) * ldv, ldv, n, 0};
    const Operand dlt{p.dl, static_cast<int64_t>(n) * ldv, ldv, ldv, n};
    e = with_tile(p.dx_cut.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM)), nb = static_cast<int>(blocks(n, CF::BN));
      product_kernel<CF, F, true, false, float, true>
          <<<dim3(static_cast<uint32_t>(mb) * nb, p.dx_cut.slices), CF::NT, 0, s>>>(
              wt, dl, ldv / 64, mb, nb, n, v0 > 0, a.d, nullptr, 0, p.sums);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    const Cut dw_cut = cut_for(a.d, rows, p.ldn / 64 * products_of(F), 1, false);
    e = with_tile(dw_cut.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      const int mb = static_cast<int>(blocks(a.d, CF::BM));
      const int nb = static_cast<int>(blocks(rows, CF::BN));
      product_kernel<CF, F, true, true, E, false><<<static_cast<uint32_t>(mb) * nb, CF::NT, 0, s>>>(
          gx, dlt, p.ldn / 64, mb, nb, rows, false, a.d, amax_x, -kDlExponent,
          static_cast<E*>(dw) + v0 * a.d);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  head_dx_kernel<E><<<static_cast<uint32_t>(blocks(a.n_rows * a.d / 8, 256)), 256, 0, s>>>(
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
  return elem_bytes == 2 ? forward<uint16_t>(a, ws, logp, lse, stats, s)
                         : forward<float>(a, ws, logp, lse, stats, s);
}

hipError_t launch_head_backward(const HeadArgs& a, int elem_bytes, const float* stats,
                                const float* dlogp, void* ws, void* dx, void* dw, hipStream_t s) {
  return elem_bytes == 2 ? backward<uint16_t>(a, stats, dlogp, ws, dx, dw, s)
                         : backward<float>(a, stats, dlogp, ws, dx, dw, s);
}

}  // namespace twell
