// The orthogonalised update of a weight matrix M by Newton-Schulz products: with
// X = M / (|M|_F + eps), its shorter side m along the rows,
//   G = X X^T,   B = b G + c G G,   X <- a X + B X        (steps times)
// every singular value s of X becomes a s + b s^3 + c s^5, which the usual
// coefficients drive towards 1.
//
// All products run on MFMA over half-precision parts of float32 values (nt_gemm.h).
// X, G and B are held in two parts.  For a bfloat16 M the X of X X^T and of B X enters
// by its first part alone, an eighth of the rounding that M itself carries, in 1, 3 and
// 2 products instead of 3, 3 and 3; a X keeps both parts, so the rounding of one step is
// not handed to the next (14336 x 4096: 0.0005 beside the output's own 0.0017; with a X
// rounded too 0.0016).  G and B stay in two parts: a diagonal G of one value would be
// off by one common factor.
// |X| <= 1 at the start, and max |a s + b s^3 + c s^5| bounds it after each step, so the
// powers of two that the parts are scaled by are known on the host.  A product leaves
// float32 partial sums, slices of K where its tiles are few; a pass over them adds the
// slices, forms G, B or the next X in float32 and writes its parts.  Where B X takes one
// slice, its epilogue does that.  G contracts X's rows and B X its columns, which it reads
// turned (nt_gemm.h).
#include <algorithm>
#include <cmath>

#include "nt_gemm.h"
#include "train_kernels.h"

namespace twell {
namespace {

using namespace nt;

constexpr int kNormBlocks = 512;

// Partial sums of squares in double: no float32 value squared leaves its range.  A lane
// reads 16 bytes at a time, four in flight (14336 x 4096 bf16 29 us, 103 an element at a time).
template <typename E>
__global__ __launch_bounds__(256) void orth_norm_kernel(const E* __restrict__ m, int64_t elems,
                                                        double* __restrict__ parts) {
  __shared__ double lds[256];
  constexpr int RUN = 16 / sizeof(E);
  const int64_t runs = elems / RUN, stride = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  double s = 0;
#pragma unroll 4
  for (int64_t i = first; i < runs; i += stride) {
    const uint4 q = reinterpret_cast<const uint4*>(m)[i];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(E) == 2) {
        const double lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
        s = fma(lo, lo, fma(hi, hi, s));
      } else {
        const double v = __uint_as_float(w[k]);
        s = fma(v, v, s);
      }
    }
  }
  for (int64_t i = runs * RUN + first; i < elems; i += stride) {
    const double v = ElemTraits<E>::to_f32(m[i]);
    s = fma(v, v, s);
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  for (int h = 128; h > 0; h /= 2) {
    if (static_cast<int>(threadIdx.x) < h) lds[threadIdx.x] += lds[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) parts[blockIdx.x] = lds[0];
}

// The factor 1 / (|M|_F + eps), from the parts in a fixed order, by every wave.
__device__ __forceinline__ double inverse_norm(const double* __restrict__ parts, int count,
                                               float eps) {
  double s = 0;
#pragma unroll 8
  for (int i = lane_id(); i < count; i += kWave) s += parts[i];
#pragma unroll
  for (int h = 1; h < kWave; h *= 2) s += __shfl_xor(s, h);
  return 1.0 / (sqrt(s) + static_cast<double>(eps));
}

struct Matrix {  // two parts of [rows][cols], columns up to ld zeros
  uint16_t* p;
  int rows, cols, ld;
};

// The parts of two values, packed: split<kHalves> but for infinities and NaN, which both
// parts carry (NaN is what M's infinities and NaN make of every result).
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&part)[2]) {
  typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
  const f16x2_t hi = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
  const f16x2_t lo = {static_cast<_Float16>(a - static_cast<float>(hi[0])),
                      static_cast<_Float16>(b - static_cast<float>(hi[1]))};
  part[0] = __builtin_bit_cast(uint32_t, hi);
  part[1] = __builtin_bit_cast(uint32_t, lo);
}

// 8 scaled values of row i, from column j on, as parts.
__device__ __forceinline__ void put_row(const Matrix& x, int i, int j, const float (&v)[8]) {
  uint32_t w[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) split_pair(v[2 * k], v[2 * k + 1], w[k]);
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<uint4*>(x.p + (static_cast<int64_t>(p) * x.rows + i) * x.ld + j) =
        make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
}
// The values of them.
__device__ __forceinline__ void get_row(const Matrix& x, int i, int j, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll
  for (int p = 1; p >= 0; --p) {
    const uint4 w = *reinterpret_cast<const uint4*>(
        x.p + (static_cast<int64_t>(p) * x.rows + i) * x.ld + j);
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
      const f16x2_t h = __builtin_bit_cast(f16x2_t, d[k]);
      v[2 * k] += static_cast<float>(h[0]);
      v[2 * k + 1] += static_cast<float>(h[1]);
    }
  }
}

// The epilogue of B X in one slice: X' = keep X + take (B X).
struct UpdateStore {
  Matrix old, out;
  float keep, take;
  __device__ __forceinline__ void operator()(int, int i, int j, float (&v)[8]) const {
    float o[8];
    get_row(old, i, j, o);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = j + k < out.cols ? fmaf(keep, o[k], take * v[k]) : 0.f;
    put_row(out, i, j, v);
  }
};

// X = 2^exponent M / (|M|_F + eps): one 64 x 64 tile a workgroup (14336 x 4096 bf16 97 us,
// 3.6 TB/s, of 7950 in all).  `tall`: M is
// [cols][rows].
template <typename E>
__global__ __launch_bounds__(256) void orth_start_kernel(const E* __restrict__ m, bool tall,
                                                         const double* __restrict__ parts,
                                                         int count, float eps, int exponent,
                                                         Matrix x) {
  __shared__ float tile[64][65];
  const double inv = ldexp(inverse_norm(parts, count, eps), exponent);
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  for (int e = threadIdx.x; e < 64 * 64; e += 256) {
    const int slow = e / 64, fast = e % 64;
    const int i = tall ? fast : slow, j = tall ? slow : fast;
    float v = 0.f;
    if (i0 + i < x.rows && j0 + j < x.cols) {
      const int64_t at = tall ? static_cast<int64_t>(j0 + j) * x.rows + i0 + i
                              : static_cast<int64_t>(i0 + i) * x.cols + j0 + j;
      v = static_cast<float>(static_cast<double>(ElemTraits<E>::to_f32(m[at])) * inv);
    }
    tile[i][j] = v;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int run = threadIdx.x + 256 * u;
    const int i = run / 8, j = run % 8 * 8;
    if (i0 + i >= x.rows) continue;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = tile[i][j + k];
    put_row(x, i0 + i, j0 + j, v);
  }
}

// Bound by memory: G of 2048 x 2048 in 7 slices 13 us, the last X of 14336 x 4096 115 us
// (5.1 TB/s).
// v = keep * (old's value) + take * (the sum of the slices), to out's parts, or to `last`
// [rows][cols] as E, transposed where `tall`.  sums [slices][rows][pitch]; `block`: out is
// symmetric and sums holds its tiles of that size with columns up to the rows', the rest is
// their mirror image.
template <typename E>
__global__ __launch_bounds__(256) void orth_finish_kernel(const float* __restrict__ sums,
                                                          int slices, int block, int pitch,
                                                          float keep, float take, Matrix old,
                                                          Matrix out, E* __restrict__ last,
                                                          bool tall) {
  __shared__ float tile[64][65];
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const bool mirror = block != 0 && i0 / block != j0 / block;
  if (mirror && j0 > i0) return;
  const int64_t plane = static_cast<int64_t>(out.rows) * pitch;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int run = threadIdx.x + 256 * u;
    const int i = run / 8, j = run % 8 * 8;
    float v[8] = {};
    if (i0 + i < out.rows) {
      const float* s = sums + static_cast<int64_t>(i0 + i) * pitch + j0 + j;
#pragma unroll 4
      for (int q = 0; q < slices; ++q) {
        const float4 a = *reinterpret_cast<const float4*>(s + q * plane);
        const float4 b = *reinterpret_cast<const float4*>(s + q * plane + 4);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
      float o[8] = {};
      if (old.p != nullptr) get_row(old, i0 + i, j0 + j, o);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = j0 + j + k < out.cols ? fmaf(keep, o[k], take * v[k]) : 0.f;
      }
      if (last == nullptr) put_row(out, i0 + i, j0 + j, v);
    }
    if (mirror || last != nullptr) {
#pragma unroll
      for (int k = 0; k < 8; ++k) tile[i][j + k] = v[k];
    }
  }
  if (last == nullptr && !mirror) return;
  __syncthreads();
  if (last == nullptr) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int run = threadIdx.x + 256 * u;
      const int j = run / 8, i = run % 8 * 8;
      if (j0 + j >= out.rows) continue;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = tile[i + k][j];
      put_row(out, j0 + j, i0 + i, v);
    }
    return;
  }
  for (int e = threadIdx.x; e < 64 * 64; e += 256) {
    const int slow = e / 64, fast = e % 64;
    const int i = tall ? fast : slow, j = tall ? slow : fast;
    if (i0 + i >= out.rows || j0 + j >= out.cols) continue;
    last[tall ? static_cast<int64_t>(j0 + j) * out.rows + i0 + i
              : static_cast<int64_t>(i0 + i) * out.cols + j0 + j] =
        ElemTraits<E>::from_f32(tile[i][j]);
  }
}

// ---------------------------------------------------------------- short sides up to 128
// One launch a step: a workgroup holds G and B, 128 x 128 with zeros past m, in LDS, forms
// B for itself, and takes 128 columns of X: X' = a X + B X and their part of the next G =
// X' X'^T, which the next launch adds up.  X stays float32 [m][ld] in memory.  512 x 128
// float32 takes 90 us in all, with a launch a product and pass as below 185; 128 x 65536
// 265, and 596.  A step's 15 us are spent between barriers: 3 us on loads that wait for the
// launch before, 5 on splitting G, B and X into parts, 4 on MFMA.
constexpr int kSmallSide = 128, kSmallColumns = 128, kSmallLanes = 1024;
constexpr int kSmallGram = kSmallSide * kSmallSide;
// More workgroups' sums of G are added up by a launch of its own (128 x 768: 97 us, 98 so;
// 128 x 1024: 104, 97 so).
constexpr int kSmallSums = 6;

struct SmallArgs {
  int m, n, ld;
  bool tall;
  const void* in;       // first step: M; X = M / (|M| + eps), and only its G
  const double* norm;
  int norm_count;
  float eps;
  float* x;             // [m][ld]
  const float* gram;    // [grams][128][128], times 2^(2 ex)
  int grams;
  float g_factor;       // 2^(eg - 2 ex)
  float b_keep, b_take; // B 2^eb = b_keep * (G 2^eg) + b_take * (G G 2^(2 eg))
  float x_factor;       // 2^ex
  float keep, take;     // X' = keep X + take (B 2^eb)(X 2^ex)
  float next_factor;    // of X' for its G
  float* next_gram;     // [workgroups][128][128]; null at the last step
  void* out;            // last step: times scale
  float scale;
};

// An operand tile in LDS: rows of K in panels of 64, as a stage's (nt_gemm.h).
__device__ __forceinline__ int panel_offset(int rows, int r, int k) {
  return (k >> 6) * rows * kStep + tile_offset(r, (k >> 3) & 7) + (k & 7);
}
// 8 and 4 values side by side, as parts; and what the parts hold.
__device__ __forceinline__ void put8(uint16_t* tile, int part, int at, const float (&v)[8]) {
  uint32_t w[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) split_pair(v[2 * k], v[2 * k + 1], w[k]);
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<uint4*>(tile + p * part + at) =
        make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
}
__device__ __forceinline__ void put4(uint16_t* tile, int part, int at, const float (&v)[4]) {
  uint32_t a[2], b[2];
  split_pair(v[0], v[1], a);
  split_pair(v[2], v[3], b);
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<uint2*>(tile + p * part + at) = make_uint2(a[p], b[p]);
}
__device__ __forceinline__ void get4(const uint16_t* tile, int part, int at, float (&v)[4]) {
  typedef __attribute__((ext_vector_type(4))) _Float16 f16x4_t;
  const f16x4_t hi = __builtin_bit_cast(f16x4_t, *reinterpret_cast<const uint2*>(tile + at));
  const f16x4_t lo = __builtin_bit_cast(f16x4_t, *reinterpret_cast<const uint2*>(tile + part + at));
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = static_cast<float>(lo[k]) + static_cast<float>(hi[k]);
}

// acc = A B^T of 32 rows of A from ra and 32 of B from rb, K of KS 16s, the small products
// of the parts over the whole of K first.
template <int KS>
__device__ __forceinline__ f32x16_t small_block(const uint16_t* a, int ra, const uint16_t* b,
                                                int rb) {
  constexpr int N = kSmallSide, PART = kSmallSide * kSmallSide;
  const int l = lane_id() & 31, half = lane_id() >> 5;
  f32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
#pragma unroll 1
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int k = ks * 16 + half * 8;
      acc = mfma<kHalves>(*reinterpret_cast<const i32x4_t*>(a + (q == 0 ? PART : 0) +
                                                            panel_offset(N, ra + l, k)),
                          *reinterpret_cast<const i32x4_t*>(b + (q == 1 ? PART : 0) +
                                                            panel_offset(N, rb + l, k)),
                          acc);
    }
  return acc;
}
// The same with K the matrix's shorter side.
__device__ __forceinline__ f32x16_t small_product(const uint16_t* a, int ra, const uint16_t* b,
                                                  int rb, int m) {
  return m > 64 ? small_block<8>(a, ra, b, rb) : small_block<4>(a, ra, b, rb);
}

// Element i of column c of a block of X', K along the columns: lines of a column each, to be
// read turned (nt_gemm.h), 64 of them after another.
__device__ __forceinline__ int turned_place(int c, int i) {
  return (c >> 6) * kStep * kSmallSide + turned_offset<kSmallSide>(c & 63, i);
}
// acc = A A^T of rows ra and rb, the small products first.
__device__ __forceinline__ f32x16_t small_turned(const uint16_t* tile, int ra, int rb) {
  constexpr int N = kSmallSide, PART = kSmallSide * kSmallColumns;
  f32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
#pragma unroll 1
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int k0 = 0; k0 < kSmallColumns; k0 += kStep) {
      i32x4_t f[4], h[4];
      read_turned<N>(lds_address(tile + (q == 0 ? PART : 0) + k0 * N) + turned_at<N>(ra), f);
      read_turned<N>(lds_address(tile + (q == 1 ? PART : 0) + k0 * N) + turned_at<N>(rb), h);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) acc = mfma<kHalves>(f[ks], h[ks], acc);
    }
  return acc;
}

template <typename E>
__global__ __launch_bounds__(kSmallLanes) void orth_small_kernel(SmallArgs a) {
  constexpr int N = kSmallSide, C = kSmallColumns, PART = N * N;
  static_assert(C == N && kSmallLanes == N * C / 1024 * kWave, "a 32 x 32 block a wave");
  // G, then B: two parts [N][N]; X's block, then X': two parts [C][N]
  __shared__ __attribute__((aligned(16))) uint16_t g[2 * PART];
  __shared__ __attribute__((aligned(16))) uint16_t xb[2 * PART];
  const int wave = threadIdx.x / kWave, wm = wave / 4 * 32, wn = wave % 4 * 32;
  const int l = lane_id() & 31, half = lane_id() >> 5;
  const int j0 = blockIdx.x * C;
  const int c = wn + l, j = j0 + c;  // this lane's column, and row 4 q of its block
  const auto row = [&](int q) { return wm + 4 * half + row_of(0, 4 * q); };
  if (a.in == nullptr) {
    float x[4][4];  // its elements of X, which stay as they are until X'
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[q][k] = row(q) + k < a.m && j < a.n
                      ? a.x[static_cast<int64_t>(row(q) + k) * a.ld + j] : 0.f;
    constexpr int RUNS = N * N / 8 / kSmallLanes;  // of 8, a lane
    float v[RUNS][8] = {};
#pragma unroll 2
    for (int s = 0; s < a.grams; ++s)
#pragma unroll
      for (int u = 0; u < RUNS; ++u) {
        const float4* p = reinterpret_cast<const float4*>(a.gram + s * kSmallGram +
                                                          (threadIdx.x + u * kSmallLanes) * 8);
        const float4 q = p[0], r = p[1];
        v[u][0] += q.x, v[u][1] += q.y, v[u][2] += q.z, v[u][3] += q.w;
        v[u][4] += r.x, v[u][5] += r.y, v[u][6] += r.z, v[u][7] += r.w;
      }
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      const int e = threadIdx.x + u * kSmallLanes;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][k] *= a.g_factor;
      put8(g, PART, panel_offset(N, e / (N / 8), e % (N / 8) * 8), v[u]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f[4] = {x[q][0] * a.x_factor, x[q][1] * a.x_factor, x[q][2] * a.x_factor,
                          x[q][3] * a.x_factor};
      put4(xb, PART, panel_offset(C, c, row(q)), f);
    }
    __syncthreads();
    const f32x16_t square = small_product(g, wm, g, wn, a.m);
    // G and B are symmetric: a lane's 4 rows are 4 columns of its own row
    float b[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      get4(g, PART, panel_offset(N, c, row(q)), b[q]);
#pragma unroll
      for (int k = 0; k < 4; ++k) b[q][k] = fmaf(a.b_keep, b[q][k], a.b_take * square[4 * q + k]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) put4(g, PART, panel_offset(N, c, row(q)), b[q]);
    __syncthreads();
    const f32x16_t up = small_product(g, wm, xb, wn, a.m);
    __syncthreads();  // xb becomes X'
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = fmaf(a.keep, x[q][k], a.take * up[4 * q + k]);
        f[k] = v * a.next_factor;
        const int i = row(q) + k;
        if (i >= a.m || j >= a.n) continue;
        if (a.next_gram != nullptr)
          a.x[static_cast<int64_t>(i) * a.ld + j] = v;
        else
          static_cast<E*>(a.out)[a.tall ? static_cast<int64_t>(j) * a.m + i
                                        : static_cast<int64_t>(i) * a.n + j] =
              ElemTraits<E>::from_f32(v * a.scale);
      }
      if (a.next_gram != nullptr) put4(xb, PART, turned_place(c, row(q)), f);
    }
    if (a.next_gram == nullptr) return;
  } else {
    const double inv = inverse_norm(a.norm, a.norm_count, a.eps);
    for (int e = threadIdx.x; e < N * C; e += kSmallLanes) {
      const int i = a.tall ? e % N : e / C, c = a.tall ? e / N : e % C, j = j0 + c;
      float v = 0.f;
      if (i < a.m && j < a.n) {
        const E* in = static_cast<const E*>(a.in);
        const int64_t at = a.tall ? static_cast<int64_t>(j) * a.m + i
                                  : static_cast<int64_t>(i) * a.n + j;
        v = static_cast<float>(static_cast<double>(ElemTraits<E>::to_f32(in[at])) * inv);
        a.x[static_cast<int64_t>(i) * a.ld + j] = v;
      }
      uint32_t part[2];
      split_pair(v * a.next_factor, 0.f, part);
      xb[turned_place(c, i)] = static_cast<uint16_t>(part[0]);
      xb[PART + turned_place(c, i)] = static_cast<uint16_t>(part[1]);
    }
  }
  __syncthreads();
  const f32x16_t next = small_turned(xb, wm, wn);
  float* to = a.next_gram + static_cast<int64_t>(blockIdx.x) * kSmallGram;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<float4*>(to + (wn + l) * N + wm + 4 * half + row_of(0, 4 * q)) =
        make_float4(next[4 * q], next[4 * q + 1], next[4 * q + 2], next[4 * q + 3]);
}

// The sum of the workgroups' grams, in 4 streams.
__global__ __launch_bounds__(256) void orth_gram_kernel(const float* __restrict__ grams, int count,
                                                        float* __restrict__ out) {
  __shared__ float joint[4][64];
  const int at = threadIdx.x % 64, stream = threadIdx.x / 64;
  const int e = blockIdx.x * 64 + at;
  float s = 0.f;
#pragma unroll 8
  for (int i = stream; i < count; i += 4) s += grams[i * kSmallGram + e];
  joint[stream][at] = s;
  __syncthreads();
  if (stream == 0) out[e] = joint[0][at] + joint[1][at] + joint[2][at] + joint[3][at];
}

struct Plan {
  int m, n, ldm, ldn;
  Cut gram, square, update;
  double* norm;
  uint16_t *x[2], *g, *b;  // X before and after a step
  float *sums, *small_gram;
  bool small;
  size_t bytes;
};
constexpr Form x_form(int elem_bytes) { return elem_bytes == 2 ? kHalf : kHalves; }
Plan plan_of(const OrthArgs& a, int elem_bytes, void* ws) {
  Plan p{};
  const size_t P = parts_of(kHalves), PX = parts_of(x_form(elem_bytes));
  p.m = std::min(a.rows, a.cols);
  p.n = std::max(a.rows, a.cols);
  p.ldm = static_cast<int>(up64(p.m));
  p.ldn = static_cast<int>(up64(p.n));
  const int gram = PX == 2 ? 3 : 1, update = PX == 2 ? 3 : 2;  // products
  p.small = p.m <= kSmallSide;
  if (p.small) {
    Carve c{static_cast<char*>(ws)};
    p.norm = c.take<double>(kNormBlocks);
    p.sums = c.take<float>(static_cast<size_t>(p.m) * p.ldn);
    // G's sums of the workgroups: two sets taken in turn, or one and their sum in front
    const size_t groups = blocks(p.n, kSmallColumns);
    p.small_gram =
        c.take<float>((groups <= kSmallSums ? 2 * groups : groups + 1) * size_t{kSmallGram});
    p.bytes = c.used;
    return p;
  }
  p.gram = wide_cut(p.m, p.m, p.ldn / 64 * gram, 32, true, false);
  p.square = wide_cut(p.m, p.m, p.ldm / 64 * 3, 32, true, false);
  p.update = wide_cut(p.n, p.m, p.ldm / 64 * update, 32, false, true);
  const size_t square = static_cast<size_t>(p.m) * p.ldm, whole = static_cast<size_t>(p.m) * p.ldn;
  Carve c{static_cast<char*>(ws)};
  p.norm = c.take<double>(kNormBlocks);
  for (uint16_t*& x : p.x) x = c.take<uint16_t>(P * whole);
  p.g = c.take<uint16_t>(P * square);
  p.b = c.take<uint16_t>(P * square);
  p.sums = c.take<float>(std::max(std::max(p.gram.slices, p.square.slices) * square,
                                  p.update.slices * whole));
  p.bytes = c.used;
  return p;
}

// sums = A A^T, by its triangle of tiles.
template <Form F>
hipError_t square_of(const Operand& A, int ksteps, const Cut& cut, int pitch, float* sums,
                     hipStream_t s) {
  return with_wide_tile(cut.tile, [&](auto cf) {
    typedef decltype(cf) CF;
    const int mb = static_cast<int>(blocks(A.rows, CF::BM));
    product_kernel<CF, F, false, false>
        <<<dim3(static_cast<uint32_t>(mb) * (mb + 1) / 2, cut.slices), CF::NT, 0, s>>>(
            A, A, ksteps, mb, 0, A.rows, pitch, SumStore{sums, pitch, A.rows, false});
    return hipGetLastError();
  });
}

// The exponent by which values up to `bound` are scaled: below 2^15 (of halves, whose
// largest is 2^16 - 2^5), with room for roundings; past 2^115 they become infinities.
int exponent_below(double bound) {
  if (!std::isfinite(bound)) return -100;
  int e;
  std::frexp(std::max(bound * 1.0625, 1e-30), &e);  // bound * 1.0625 < 2^e
  return std::max(15 - e, -100);
}

// max |a s + b s^3 + c s^5| over 0 <= s <= top: at the end or where the derivative
// a + 3 b t + 5 c t^2, t = s^2, is 0.
double step_bound(const OrthArgs& p, double top) {
  const double a = p.a, b = p.b, c = p.c;
  const auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
  double most = f(top);
  const auto at = [&](double t) {
    if (t > 0 && t < top * top) most = std::max(most, f(std::sqrt(t)));
  };
  if (c != 0) {
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      at((-3 * b + std::sqrt(d)) / (10 * c));
      at((-3 * b - std::sqrt(d)) / (10 * c));
    }
  } else if (b != 0) {
    at(-a / (3 * b));
  }
  return most;
}

template <typename E>
hipError_t orthogonalize_small(const OrthArgs& a, const Plan& p, int count, hipStream_t s) {
  const uint32_t groups = static_cast<uint32_t>(blocks(p.n, kSmallColumns));
  const auto factor = [](double v, int e) { return static_cast<float>(std::ldexp(v, e)); };
  double bound = 1.0;
  int ex = exponent_below(bound);
  SmallArgs k{};
  k.m = p.m;
  k.n = p.n;
  k.ld = p.ldn;
  k.tall = a.rows > a.cols;
  k.in = a.in;
  k.norm = p.norm;
  k.norm_count = count;
  k.eps = a.eps;
  k.x = p.sums;
  k.next_factor = factor(1, ex);
  const bool few = groups <= kSmallSums;
  float* const sets[2] = {p.small_gram + (few ? 0 : kSmallGram),
                          p.small_gram + (few ? groups : 1) * kSmallGram};
  k.next_gram = sets[0];
  k.out = a.out;
  k.scale = a.scale;
  orth_small_kernel<E><<<groups, kSmallLanes, 0, s>>>(k);
  k.in = nullptr;
  for (int i = 0; i < a.steps; ++i) {
    k.gram = k.next_gram;
    k.grams = static_cast<int>(groups);
    if (few) {
      k.next_gram = sets[(i + 1) % 2];
    } else {
      orth_gram_kernel<<<kSmallGram / 64, 256, 0, s>>>(k.gram, k.grams, p.small_gram);
      k.gram = p.small_gram;
      k.grams = 1;
    }
    const double t = bound * bound;
    const int eg = exponent_below(t);
    const int eb = exponent_below(std::fabs(a.b) * t + std::fabs(a.c) * t * t);
    bound = step_bound(a, bound);
    const int next = exponent_below(bound);
    k.g_factor = factor(1, eg - 2 * ex);
    k.b_keep = factor(a.b, eb - eg);
    k.b_take = factor(a.c, eb - 2 * eg);
    k.x_factor = factor(1, ex);
    k.keep = a.a;
    k.take = factor(1, -eb - ex);
    k.next_factor = factor(1, next);
    if (i + 1 == a.steps) k.next_gram = nullptr;
    orth_small_kernel<E><<<groups, kSmallLanes, 0, s>>>(k);
    ex = next;
  }
  return hipGetLastError();
}

template <typename E>
hipError_t orthogonalize(const OrthArgs& a, void* ws, hipStream_t s) {
  constexpr Form X = x_form(sizeof(E));
  const Plan p = plan_of(a, sizeof(E), ws);
  const bool tall = a.rows > a.cols;
  const int64_t elems = static_cast<int64_t>(a.rows) * a.cols;
  const int count = static_cast<int>(std::min<int64_t>(blocks(elems, 2048), kNormBlocks));
  const E* in = static_cast<const E*>(a.in);
  orth_norm_kernel<E><<<count, 256, 0, s>>>(in, elems, p.norm);
  if (p.small) return orthogonalize_small<E>(a, p, count, s);
  const Matrix g{p.g, p.m, p.m, p.ldm}, b{p.b, p.m, p.m, p.ldm};
  const Matrix none{};
  const dim3 whole(p.ldn / 64, p.ldm / 64), square(p.ldm / 64, p.ldm / 64);
  double bound = 1.0;  // of X's singular values
  int ex = exponent_below(bound);
  orth_start_kernel<E><<<whole, 256, 0, s>>>(in, tall, p.norm, count, a.eps, ex,
                                             Matrix{p.x[0], p.m, p.n, p.ldn});
  const int64_t part = static_cast<int64_t>(p.m) * p.ldn, square_part = int64_t{p.m} * p.ldm;
  const Operand go{p.g, square_part, p.ldm, p.m, p.ldm};
  const Operand bo{p.b, square_part, p.ldm, p.m, p.ldm};
  E* no_output = nullptr;
  for (int i = 0; i < a.steps; ++i) {
    const bool end = i + 1 == a.steps;
    const Matrix x{p.x[i % 2], p.m, p.n, p.ldn}, after{p.x[(i + 1) % 2], p.m, p.n, p.ldn};
    const Operand xo{x.p, part, p.ldn, p.m, p.ldn};
    const Operand xt{x.p, part, p.ldn, p.ldn, p.m};  // turned
    const double t = bound * bound;
    const int eg = exponent_below(t);
    const int eb = exponent_below(std::fabs(a.b) * t + std::fabs(a.c) * t * t);
    bound = step_bound(a, bound);
    const int next = exponent_below(bound);
    // factors with the powers of two of what goes in undone and of what comes out applied
    const auto factor = [](double v, int e) { return static_cast<float>(std::ldexp(v, e)); };
    hipError_t e = square_of<X>(xo, p.ldn / 64, p.gram, p.ldm, p.sums, s);
    if (e != hipSuccess) return e;
    orth_finish_kernel<E><<<square, 256, 0, s>>>(p.sums, p.gram.slices, tile_rows(p.gram.tile),
                                                 p.ldm, 0.f, factor(1, eg - 2 * ex), none, g,
                                                 no_output, false);
    if ((e = square_of<kHalves>(go, p.ldm / 64, p.square, p.ldm, p.sums, s)) != hipSuccess)
      return e;
    orth_finish_kernel<E><<<square, 256, 0, s>>>(p.sums, p.square.slices,
                                                 tile_rows(p.square.tile), p.ldm,
                                                 factor(a.b, eb - eg), factor(a.c, eb - 2 * eg), g,
                                                 b, no_output, false);
    const double scale = end ? a.scale : 1.0;
    const int out = end ? 0 : next;
    const float keep = factor(scale * a.a, out - ex), take = factor(scale, out - eb - ex);
    const bool fused = p.update.slices == 1 && !end;
    e = with_wide_tile(p.update.tile, [&](auto cf) {
      typedef decltype(cf) CF;
      constexpr Form F = X == kHalf ? kMixed : kHalves;
      const int mb = static_cast<int>(blocks(p.n, CF::BM)), nb = static_cast<int>(blocks(p.m, CF::BN));
      const dim3 grid(static_cast<uint32_t>(mb) * nb, p.update.slices);
      if (fused)
        product_kernel<CF, F, true, false><<<grid, CF::NT, 0, s>>>(
            xt, bo, p.ldm / 64, mb, nb, p.m, p.ldn, UpdateStore{x, after, keep, take});
      else
        product_kernel<CF, F, true, false><<<grid, CF::NT, 0, s>>>(
            xt, bo, p.ldm / 64, mb, nb, p.m, p.ldn, SumStore{p.sums, p.ldn, p.m, false});
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    if (!fused)
      orth_finish_kernel<E><<<whole, 256, 0, s>>>(p.sums, p.update.slices, 0, p.ldn, keep, take, x,
                                                  after,
                                                  end ? static_cast<E*>(a.out) : no_output, tall);
    ex = next;
  }
  return hipGetLastError();
}

}  // namespace

size_t orth_bytes(const OrthArgs& a, int elem_bytes) { return plan_of(a, elem_bytes, nullptr).bytes; }

hipError_t launch_orthogonalize(const OrthArgs& a, int elem_bytes, void* ws, hipStream_t s) {
  return elem_bytes == 2 ? orthogonalize<uint16_t>(a, ws, s) : orthogonalize<float>(a, ws, s);
}

}  // namespace twell
