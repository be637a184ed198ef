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

constexpr int kNormBlocks = 1024;

// Partial sums of squares in double: no float32 value squared leaves its range.
template <typename E>
__global__ __launch_bounds__(256) void orth_norm_kernel(const E* __restrict__ m, int64_t elems,
                                                        double* __restrict__ parts) {
  __shared__ double lds[256];
  double s = 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < elems;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const double v = ElemTraits<E>::to_f32(m[i]);
    s += v * v;
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  for (int h = 128; h > 0; h /= 2) {
    if (static_cast<int>(threadIdx.x) < h) lds[threadIdx.x] += lds[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) parts[blockIdx.x] = lds[0];
}

// The factor 1 / (|M|_F + eps), from the parts in a fixed order, by every workgroup.
__device__ __forceinline__ double inverse_norm(const double* __restrict__ parts, int count,
                                               float eps, double* lds) {
  double s = 0;
  for (int i = threadIdx.x; i < count; i += 256) s += parts[i];
  lds[threadIdx.x] = s;
  __syncthreads();
  for (int h = 128; h > 0; h /= 2) {
    if (static_cast<int>(threadIdx.x) < h) lds[threadIdx.x] += lds[threadIdx.x + h];
    __syncthreads();
  }
  const double total = lds[0];
  __syncthreads();
  return 1.0 / (sqrt(total) + static_cast<double>(eps));
}

struct Matrix {  // two parts of [rows][cols], columns up to ld zeros
  uint16_t* p;
  int rows, cols, ld;
};

// 8 scaled values of row i, from column j on, as parts.
__device__ __forceinline__ void put_row(const Matrix& x, int i, int j, const float (&v)[8]) {
  uint32_t w[2][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t lo[2], hi[2];
    split<kHalves>(v[2 * k], lo);
    split<kHalves>(v[2 * k + 1], hi);
#pragma unroll
    for (int p = 0; p < 2; ++p) w[p][k] = lo[p] | static_cast<uint32_t>(hi[p]) << 16;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<uint4*>(x.p + (static_cast<int64_t>(p) * x.rows + i) * x.ld + j) =
        make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
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

// X = 2^exponent M / (|M|_F + eps): one 64 x 64 tile a workgroup.  `tall`: M is
// [cols][rows].
template <typename E>
__global__ __launch_bounds__(256) void orth_start_kernel(const E* __restrict__ m, bool tall,
                                                         const double* __restrict__ parts,
                                                         int count, float eps, int exponent,
                                                         Matrix x) {
  __shared__ double sum[256];
  __shared__ float tile[64][65];
  const double inv = ldexp(inverse_norm(parts, count, eps, sum), exponent);
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
// B for itself, and takes 64 columns of X: X' = a X + B X and their part of the next G =
// X' X'^T, which the next launch adds up.  X stays float32 [m][ld] in memory.  What a step
// cost before was its six launches (512 x 128: 38 us a step).
constexpr int kSmallSide = 128, kSmallColumns = 64;
constexpr int kSmallGram = kSmallSide * kSmallSide;
constexpr int kSmallSums = 16;  // more workgroups' sums of G are added up by a launch of its own

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
__device__ __forceinline__ void put8(uint16_t* tile, int rows, int r, int k, const float (&v)[8],
                                     int part) {
  uint32_t w[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t lo[2], hi[2];
    split<kHalves>(v[2 * i], lo);
    split<kHalves>(v[2 * i + 1], hi);
#pragma unroll
    for (int p = 0; p < 2; ++p) w[p][i] = lo[p] | static_cast<uint32_t>(hi[p]) << 16;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<uint4*>(tile + p * part + panel_offset(rows, r, k)) =
        make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}
__device__ __forceinline__ float value_of(const uint16_t* tile, int part, int at) {
  return static_cast<float>(__builtin_bit_cast(_Float16, tile[part + at])) +
         static_cast<float>(__builtin_bit_cast(_Float16, tile[at]));
}

// acc = A B^T of 32 rows of A from ra and 32 FN of B from rb, K in 16s, the small products
// of the parts over the whole of K first.
template <int FN>
__device__ __forceinline__ void small_product(const uint16_t* a, int rows_a, int part_a, int ra,
                                              const uint16_t* b, int rows_b, int part_b, int rb,
                                              int k16, f32x16_t (&acc)[FN]) {
  const int l = lane_id() & 31, half = lane_id() >> 5;
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const uint16_t* ap = a + (q == 0 ? part_a : 0);
    const uint16_t* bp = b + (q == 1 ? part_b : 0);
    for (int ks = 0; ks < k16; ++ks) {
      const int k = ks * 16 + half * 8;
      const i32x4_t f = *reinterpret_cast<const i32x4_t*>(ap + panel_offset(rows_a, ra + l, k));
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[j] = mfma<kHalves>(f,
                               *reinterpret_cast<const i32x4_t*>(
                                   bp + panel_offset(rows_b, rb + 32 * j + l, k)),
                               acc[j]);
    }
  }
}

template <typename E>
__global__ __launch_bounds__(512) void orth_small_kernel(SmallArgs a) {
  constexpr int N = kSmallSide, C = kSmallColumns;
  // G, then B: two parts [N][N]; X's block: two parts [C][N], then [N][C]
  __shared__ __attribute__((aligned(16))) uint16_t g[2 * N * N];
  __shared__ __attribute__((aligned(16))) uint16_t xb[2 * C * N];
  __shared__ double sum[512];
  const int wave = threadIdx.x / kWave, wm = wave / 2 * 32, wn = wave % 2;
  const int l = lane_id() & 31, half = lane_id() >> 5;
  const int j0 = blockIdx.x * C;
  if (a.in == nullptr) {
#pragma unroll
    for (int u = 0; u < N * N / 8 / 512; ++u) {
      const int e = threadIdx.x + u * 512;
      float v[8] = {};
#pragma unroll 4
      for (int s = 0; s < a.grams; ++s) {
        const float4* p = reinterpret_cast<const float4*>(a.gram + s * kSmallGram + e * 8);
        const float4 q = p[0], r = p[1];
        v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
        v[4] += r.x, v[5] += r.y, v[6] += r.z, v[7] += r.w;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= a.g_factor;
      put8(g, N, e / (N / 8), e % (N / 8) * 8, v, N * N);
    }
    // columns of X: 8 rows a lane, lanes along the columns
#pragma unroll
    for (int u = 0; u < C * N / 8 / 512; ++u) {
      const int e = threadIdx.x + u * 512;
      const int c = e % C, i = e / C * 8;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = i + k < a.m && j0 + c < a.n
                   ? a.x[static_cast<int64_t>(i + k) * a.ld + j0 + c] * a.x_factor
                   : 0.f;
      put8(xb, C, c, i, v, C * N);
    }
    __syncthreads();
    f32x16_t acc[2];
    const int k16 = (a.m + 15) / 16;
    small_product<2>(g, N, N * N, wm, g, N, N * N, wn * 64, k16, acc);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int at = panel_offset(N, wn * 64 + j * 32 + l, wm + 4 * half + row_of(0, r));
        acc[j][r] = fmaf(a.b_keep, value_of(g, N * N, at), a.b_take * acc[j][r]);
      }
    __syncthreads();
    // B is symmetric: a lane's 4 rows are 4 columns of its own row
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = panel_offset(N, wn * 64 + j * 32 + l, wm + 4 * half + row_of(0, 4 * q));
        uint16_t part[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) split<kHalves>(acc[j][4 * q + k], part[k]);
#pragma unroll
        for (int p = 0; p < 2; ++p)
          *reinterpret_cast<uint2*>(g + p * N * N + at) =
              make_uint2(part[0][p] | static_cast<uint32_t>(part[1][p]) << 16,
                         part[2][p] | static_cast<uint32_t>(part[3][p]) << 16);
      }
    __syncthreads();
    f32x16_t up[1];
    small_product<1>(g, N, N * N, wm, xb, C, C * N, wn * 32, k16, up);
    __syncthreads();  // xb becomes [N][C]
    const int c = wn * 32 + l, j = j0 + c;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = wm + 4 * half + row_of(0, r);
      float v = 0.f;
      if (i < a.m && j < a.n) {
        float* x = a.x + static_cast<int64_t>(i) * a.ld + j;
        v = fmaf(a.keep, *x, a.take * up[0][r]);
        if (a.next_gram != nullptr)
          *x = v;
        else
          static_cast<E*>(a.out)[a.tall ? static_cast<int64_t>(j) * a.m + i
                                        : static_cast<int64_t>(i) * a.n + j] =
              ElemTraits<E>::from_f32(v * a.scale);
      }
      if (a.next_gram != nullptr) {
        uint16_t part[2];
        split<kHalves>(v * a.next_factor, part);
        xb[panel_offset(N, i, c)] = part[0];
        xb[C * N + panel_offset(N, i, c)] = part[1];
      }
    }
    if (a.next_gram == nullptr) return;
  } else {
    double t = 0;
    for (int i = threadIdx.x; i < a.norm_count; i += 512) t += a.norm[i];
    sum[threadIdx.x] = t;
    __syncthreads();
    for (int h = 256; h > 0; h /= 2) {
      if (static_cast<int>(threadIdx.x) < h) sum[threadIdx.x] += sum[threadIdx.x + h];
      __syncthreads();
    }
    const double inv = 1.0 / (sqrt(sum[0]) + static_cast<double>(a.eps));
    for (int e = threadIdx.x; e < N * C; e += 512) {
      const int i = a.tall ? e % N : e / C, c = a.tall ? e / N : e % C, j = j0 + c;
      float v = 0.f;
      if (i < a.m && j < a.n) {
        const E* in = static_cast<const E*>(a.in);
        const int64_t at = a.tall ? static_cast<int64_t>(j) * a.m + i
                                  : static_cast<int64_t>(i) * a.n + j;
        v = static_cast<float>(static_cast<double>(ElemTraits<E>::to_f32(in[at])) * inv);
        a.x[static_cast<int64_t>(i) * a.ld + j] = v;
      }
      uint16_t part[2];
      split<kHalves>(v * a.next_factor, part);
      xb[panel_offset(N, i, c)] = part[0];
      xb[C * N + panel_offset(N, i, c)] = part[1];
    }
  }
  __syncthreads();
  f32x16_t acc[2];
  small_product<2>(xb, N, C * N, wm, xb, N, C * N, wn * 64, C / 16, acc);
  float* to = a.next_gram + static_cast<int64_t>(blockIdx.x) * kSmallGram;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(to + (wn * 64 + j * 32 + l) * N + wm + 4 * half +
                                 row_of(0, 4 * q)) =
          make_float4(acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]);
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
constexpr int kSmallMost = 8192;
constexpr Form x_form(int elem_bytes) { return elem_bytes == 2 ? kHalf : kHalves; }
Plan plan_of(const OrthArgs& a, int elem_bytes, void* ws) {
  Plan p{};
  const size_t P = parts_of(kHalves), PX = parts_of(x_form(elem_bytes));
  p.m = std::min(a.rows, a.cols);
  p.n = std::max(a.rows, a.cols);
  p.ldm = static_cast<int>(up64(p.m));
  p.ldn = static_cast<int>(up64(p.n));
  const int gram = PX == 2 ? 3 : 1, update = PX == 2 ? 3 : 2;  // products
  p.small = p.m <= kSmallSide && p.n <= kSmallMost;
  if (p.small) {
    Carve c{static_cast<char*>(ws)};
    p.norm = c.take<double>(kNormBlocks);
    p.sums = c.take<float>(static_cast<size_t>(p.m) * p.ldn);
    // G's sums of the workgroups: two sets taken in turn, or one and their sum in front
    const size_t groups = p.ldn / kSmallColumns;
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
  const uint32_t groups = static_cast<uint32_t>(p.ldn / kSmallColumns);
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
  orth_small_kernel<E><<<groups, 512, 0, s>>>(k);
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
    orth_small_kernel<E><<<groups, 512, 0, s>>>(k);
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
