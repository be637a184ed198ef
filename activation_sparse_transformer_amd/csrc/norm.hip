// Norms around the layer, fused with its gate and residual scale, and their
// gradient.  Per row, with r the residual stream and y the layer's output:
//   u  = y * ystd * w_post,   ystd = 1 / sqrt(mean y^2 + eps)   (or u = y)
//   r' = alpha r + gate * u
//   x  = r' * rstd * w_pre,   rstd = 1 / sqrt(mean r'^2 + eps)
// and, with p = dx * w_pre and G the whole gradient of r':
//   G  = dr' + rstd (p - r' rstd^2 mean(p r'))
//   dr = alpha G,   q = G * gate * w_post
//   dy = ystd (q - y ystd^2 mean(q y))
//   S  = sum over the rows of G * y * ystd;  dw_post = gate S, dgate = w_post S
//   dw_pre = sum over the rows of dx * r' * rstd
// A row is a group of G lanes, each with V runs of 8 columns in registers: every
// element is read once and written once, so the kernels stream.
#include <algorithm>
#include <type_traits>

#include "stream_ops.h"
#include "train_kernels.h"
#include "vec_ops.h"

namespace twell {
namespace {

constexpr int kRun = 8;  // columns of a lane's run
// Workgroups of the gradient: two a CU, one of 1024 lanes.  More only make more column sums
// to add up (4096 x 2048 bf16: 34 us in all with 512, 37 with 1024; 6374 x 5264: 123 with
// 256, 131 with 512), and loading a row ahead gains nothing.
constexpr int kNormGroups = 512;

// 8 elements as loaded.  Loads go through the caches: y and the residual come from the
// call before (gradient of 8192 x 4096 float32 166 us, 176 past the caches); stores do not.
template <typename E>
struct Run;
template <>
struct Run<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void floats(float (&f)[kRun]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[kRun]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = ElemTraits<uint16_t>::from_f32(f[2 * i]) |
             static_cast<uint32_t>(ElemTraits<uint16_t>::from_f32(f[2 * i + 1])) << 16;
    store_once(p, make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct Run<float> {
  uint4 q[2];
  __device__ __forceinline__ void load(const float* p) {
    q[0] = *reinterpret_cast<const uint4*>(p);
    q[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { q[0] = q[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void floats(float (&f)[kRun]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(q[i].x);
      f[4 * i + 1] = __uint_as_float(q[i].y);
      f[4 * i + 2] = __uint_as_float(q[i].z);
      f[4 * i + 3] = __uint_as_float(q[i].w);
    }
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[kRun]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      store_once(p + 4 * i, make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                       __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])));
  }
};

// The sums of v over a row's G lanes, in every lane, in a fixed order.  `lds`:
// 16 * U floats that no lane still reads from an earlier call (callers alternate
// between two halves; the barrier of one call ends the reads of the one before).
template <int G, int U>
__device__ __forceinline__ void row_sums(float (&v)[U], float* lds) {
  group_totals<64, U>(v);
#pragma unroll
  for (int u = 0; u < U; ++u)
    v[u] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[u]), 63));
  if constexpr (G > kWave) {
    const int wave = threadIdx.x / kWave;
    if (lane_id() == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) lds[wave * U + u] = v[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < G / kWave; ++w) s += lds[w * U + u];
      v[u] = s;
    }
  }
}

__device__ __forceinline__ void load_weights(const float* w, int c, float (&f)[kRun]) {
  const float4 a = *reinterpret_cast<const float4*>(w + c);
  const float4 b = *reinterpret_cast<const float4*>(w + c + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// gate * w_post of 8 columns, either of them 1 where absent
__device__ __forceinline__ void post_weights(const NormArgs& a, int c, float (&f)[kRun]) {
#pragma unroll
  for (int k = 0; k < kRun; ++k) f[k] = 1.f;
  if (a.w_post != nullptr) load_weights(a.w_post, c, f);
  if (a.gate != nullptr) {
    float g[kRun];
    load_weights(a.gate, c, g);
#pragma unroll
    for (int k = 0; k < kRun; ++k) f[k] *= g[k];
  }
}

// One workgroup: max(G, 256) lanes, a row per group of G.  Bound by memory: 16384 x 8192
// bf16 198 us, 5.4 TB/s of the 6.2 that a copy reaches; 16 rows are 4 us and the launch.
template <typename E, int G, int V>
__global__ __launch_bounds__(G < 256 ? 256 : G) void norm_forward_kernel(NormArgs a,
                                                                         const E* residual,
                                                                         const E* y, E* residual_out,
                                                                         E* x) {
  constexpr int ROWS = G < 256 ? 256 / G : 1;
  __shared__ float lds[2][16];
  const int t = G < 256 ? threadIdx.x % G : threadIdx.x;
  const int runs = a.d / kRun;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float post[V][kRun], pre[V][kRun];  // weights
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * G + t;
    if (c >= runs) continue;
    if (y != nullptr) post_weights(a, c * kRun, post[i]);
    if (a.w_pre != nullptr) load_weights(a.w_pre, c * kRun, pre[i]);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (G < 256 ? threadIdx.x / G : 0);
       row < a.n_rows; row += static_cast<int64_t>(gridDim.x) * ROWS) {
    const int64_t base = row * a.d;
    Run<E> rr[V], yr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * G + t;
      if (c < runs) {
        rr[i].load(residual + base + c * kRun);
        if (y != nullptr) yr[i].load(y + base + c * kRun);
      }
    }
    float v[V][kRun];
    float ystd = 1.f;
    if (a.w_post != nullptr) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i * G + t >= runs) continue;
        float f[kRun];
        yr[i].floats(f);
#pragma unroll
        for (int k = 0; k < kRun; ++k) s[0] = fmaf(f[k], f[k], s[0]);
      }
      row_sums<G, 1>(s, lds[0]);
      ystd = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * G + t;
      if (c >= runs) continue;
      rr[i].floats(v[i]);
      if (y != nullptr) {
        float f[kRun];
        yr[i].floats(f);
#pragma unroll
        for (int k = 0; k < kRun; ++k) v[i][k] = fmaf(f[k] * ystd, post[i][k], a.alpha * v[i][k]);
        Run<E>::store(residual_out + base + c * kRun, v[i]);
      }
#pragma unroll
      for (int k = 0; k < kRun; ++k) s[0] = fmaf(v[i][k], v[i][k], s[0]);
    }
    if (a.w_pre == nullptr) {
      if (G > kWave) __syncthreads();  // the reads of lds[0], before the next row's writes
      continue;
    }
    row_sums<G, 1>(s, lds[1]);
    const float rstd = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * G + t;
      if (c >= runs) continue;
#pragma unroll
      for (int k = 0; k < kRun; ++k) v[i][k] = v[i][k] * rstd * pre[i][k];
      Run<E>::store(x + base + c * kRun, v[i]);
    }
    // without w_post only lds[1] is used: its reads end before the next row's writes
    if (G > kWave && a.w_post == nullptr) __syncthreads();
  }
}

// A group walks rows group, group + groups, ... and keeps its columns' sums in
// registers; a workgroup b's sums[b][d] (S) and sums[gridDim.x + b][d] (dw_pre) are added
// up by norm_sums_kernel.  8192 x 4096 float32 157 us, 5.1 TB/s; 4096 x 2048 bf16 27 us,
// 3.7 TB/s: with eight rows a workgroup the latency of a row's loads and sums shows.  Past
// 8192 columns two runs a lane spill (bf16 13 registers, 56 bytes a lane; float32 112, 260
// bytes): 1024 x 16384 bf16 79 us, float32 205, 2.6 and 2.0 TB/s.
template <typename E, int G, int V>
__global__ __launch_bounds__(G < 256 ? 256 : G) void norm_backward_kernel(NormArgs a,
                                                                          NormGradPtrs<E> p,
                                                                          float* sums) {
  constexpr int ROWS = G < 256 ? 256 / G : 1;
  __shared__ float lds[2][48];
  const int t = G < 256 ? threadIdx.x % G : threadIdx.x;
  const int group = blockIdx.x * ROWS + (G < 256 ? threadIdx.x / G : 0);
  const int groups = gridDim.x * ROWS;
  const int runs = a.d / kRun;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float post[V][kRun], pre[V][kRun];  // column sums
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < kRun; ++k) post[i][k] = pre[i][k] = 0.f;
  for (int64_t row = group; row < a.n_rows; row += groups) {
    const int64_t base = row * a.d;
    Run<E> rr[V], yr[V], gr[V], xr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * G + t;
      if (c >= runs) continue;
      gr[i].clear();
      if (p.d_residual_out != nullptr) gr[i].load(p.d_residual_out + base + c * kRun);
      if (a.w_pre != nullptr) {
        rr[i].load(p.residual_out + base + c * kRun);
        xr[i].load(p.dx + base + c * kRun);
      }
      if (p.y != nullptr) yr[i].load(p.y + base + c * kRun);
    }
    float s[3] = {0.f, 0.f, 0.f};  // r'^2, p r', y^2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * G + t;
      if (c >= runs) continue;
      float f[kRun], d[kRun], w[kRun];
      if (a.w_pre != nullptr) {
        rr[i].floats(f);
        xr[i].floats(d);
        load_weights(a.w_pre, c * kRun, w);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          s[0] = fmaf(f[k], f[k], s[0]);
          s[1] = fmaf(d[k] * w[k], f[k], s[1]);
        }
      }
      if (a.w_post != nullptr) {
        yr[i].floats(f);
#pragma unroll
        for (int k = 0; k < kRun; ++k) s[2] = fmaf(f[k], f[k], s[2]);
      }
    }
    row_sums<G, 3>(s, lds[0]);
    const float rstd = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
    const float along = s[1] * inv_d * rstd * rstd;  // of r'
    const float ystd = a.w_post != nullptr ? 1.f / sqrtf(fmaf(s[2], inv_d, a.eps)) : 1.f;
    float g[V][kRun];
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * G + t;
      if (c >= runs) continue;
      gr[i].floats(g[i]);
      float f[kRun], d[kRun], w[kRun];
      if (a.w_pre != nullptr) {
        rr[i].floats(f);
        xr[i].floats(d);
        load_weights(a.w_pre, c * kRun, w);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          g[i][k] = fmaf(rstd, fmaf(-along, f[k], d[k] * w[k]), g[i][k]);
          pre[i][k] = fmaf(d[k], f[k] * rstd, pre[i][k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kRun; ++k) d[k] = a.alpha * g[i][k];
      Run<E>::store(p.d_residual + base + c * kRun, d);
      if (p.y != nullptr) {
        yr[i].floats(f);
        post_weights(a, c * kRun, w);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          post[i][k] = fmaf(g[i][k], f[k] * ystd, post[i][k]);
          g[i][k] *= w[k];
          q[0] = fmaf(g[i][k], f[k], q[0]);
        }
      }
    }
    if (p.y != nullptr) {
      float across = 0.f;  // of y
      if (a.w_post != nullptr) {
        row_sums<G, 1>(q, lds[1]);
        across = q[0] * inv_d * ystd * ystd;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * G + t;
        if (c >= runs) continue;
        if (a.w_post != nullptr) {
          float f[kRun];
          yr[i].floats(f);
#pragma unroll
          for (int k = 0; k < kRun; ++k) g[i][k] = ystd * fmaf(-across, f[k], g[i][k]);
        }
        Run<E>::store(p.dy + base + c * kRun, g[i]);
      }
    }
    // without w_post only lds[0] is used: its reads end before the next row's writes
    if (G > kWave && a.w_post == nullptr) __syncthreads();
  }
  if constexpr (ROWS > 1) {  // the workgroup's groups, as one
    __shared__ float joint[ROWS - 1][2][V * G * kRun];
    const int g = threadIdx.x / G;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < kRun; ++k)
        if (g > 0) {
          joint[g - 1][0][(i * kRun + k) * G + t] = post[i][k];
          joint[g - 1][1][(i * kRun + k) * G + t] = pre[i][k];
        }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < kRun; ++k)
#pragma unroll
        for (int o = 0; o < ROWS - 1; ++o) {
          post[i][k] += joint[o][0][(i * kRun + k) * G + t];
          pre[i][k] += joint[o][1][(i * kRun + k) * G + t];
        }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * G + t;
    if (c >= runs) continue;
    float* out = sums + static_cast<int64_t>(blockIdx.x) * a.d + c * kRun;
    if (p.y != nullptr) Run<float>::store(out, post[i]);
    if (a.w_pre != nullptr)
      Run<float>::store(out + static_cast<int64_t>(gridDim.x) * a.d, pre[i]);
  }
}

// Column sums over the workgroups' rows of `sums`, in 64 streams and then over those: 16
// columns a workgroup, 4 to a lane.  4096 x 2048: 6 us, mostly the launch and one latency.
constexpr int kSumCols = 16, kSumStreams = 64;
__global__ __launch_bounds__(256) void norm_sums_kernel(NormArgs a, const float* sums, int groups,
                                                        float* dw_post, float* dgate,
                                                        float* dw_pre) {
  __shared__ float4 lds[kSumStreams][kSumCols / 4];
  const int col = threadIdx.x % 4, stream = threadIdx.x / 4;
  const int c = blockIdx.x * kSumCols + col * 4;
  const bool is_pre = blockIdx.y == 1;
  if (is_pre ? dw_pre == nullptr : dw_post == nullptr && dgate == nullptr) return;
  const auto add = [](float4 p, float4 q) {
    return make_float4(p.x + q.x, p.y + q.y, p.z + q.z, p.w + q.w);
  };
  float4 s = make_float4(0, 0, 0, 0);
  if (c < a.d) {
    const float* in = sums + (is_pre ? static_cast<int64_t>(groups) * a.d : 0) + c;
#pragma unroll 8
    for (int g = stream; g < groups; g += kSumStreams)
      s = add(s, *reinterpret_cast<const float4*>(in + static_cast<int64_t>(g) * a.d));
  }
  lds[stream][col] = s;
  __syncthreads();
  if (stream >= 4 || c >= a.d) return;
  // 16 streams' sums to a lane, and the four lanes' of a column
#pragma unroll
  for (int w = 1; w < kSumStreams / 4; ++w) s = add(s, lds[stream + 4 * w][col]);
#pragma unroll
  for (int h = 4; h < 16; h *= 2)
    s = add(s, make_float4(__shfl_xor(s.x, h), __shfl_xor(s.y, h), __shfl_xor(s.z, h),
                           __shfl_xor(s.w, h)));
  if (stream != 0) return;
  const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (is_pre) {
      dw_pre[c + k] = v[k];
    } else {
      // without rows zero, also beside a weight that is infinite or NaN
      const bool some = groups > 0;
      if (dw_post != nullptr)
        dw_post[c + k] = some && a.gate != nullptr ? v[k] * a.gate[c + k] : v[k];
      if (dgate != nullptr)
        dgate[c + k] = some && a.w_post != nullptr ? v[k] * a.w_post[c + k] : v[k];
    }
  }
}

// The lanes G of a row and runs V of a lane: one run while a workgroup holds enough
// lanes (16384 x 8192 bf16 forward 204 us; 210 with 512 lanes of two runs, 299 with 256
// of four).
template <class F>
hipError_t with_group(int d, const F& f) {
  const int runs = d / kRun;
  if (runs <= 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  if (runs <= 128) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (runs <= 256) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
  if (runs <= 512) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 1>());
  if (runs <= 1024) return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 1>());
  return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

template <typename E>
hipError_t forward(const NormArgs& a, const void* residual, const void* y, void* residual_out,
                   void* x, hipStream_t s) {
  return with_group(a.d, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    constexpr int ROWS = G < 256 ? 256 / G : 1, NT = G < 256 ? 256 : G;
    // two rows a group where that leaves 2048 workgroups: the weights are read once for
    // both (16384 x 8192 bf16 204 us, 228 with one; fewer rows gain nothing).  A launch
    // holds fewer than 2^32 lanes.
    const int64_t steps = (a.n_rows + ROWS - 1) / ROWS;
    const int64_t blocks = std::min<int64_t>(steps >= 4096 ? (steps + 1) / 2 : steps, 1 << 20);
    norm_forward_kernel<E, G, V><<<static_cast<uint32_t>(blocks), NT, 0, s>>>(
        a, static_cast<const E*>(residual), static_cast<const E*>(y),
        static_cast<E*>(residual_out), static_cast<E*>(x));
    return hipGetLastError();
  });
}

template <typename E>
hipError_t backward(const NormArgs& a, const NormGradArgs& p, hipStream_t s) {
  const int groups = norm_grad_groups(a.n_rows, a.d);
  return with_group(a.d, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    constexpr int NT = G < 256 ? 256 : G;
    if (groups > 0) {
      const NormGradPtrs<E> q{static_cast<const E*>(p.residual_out), static_cast<const E*>(p.y),
                              static_cast<const E*>(p.d_residual_out),
                              static_cast<const E*>(p.dx), static_cast<E*>(p.d_residual),
                              static_cast<E*>(p.dy)};
      norm_backward_kernel<E, G, V><<<groups, NT, 0, s>>>(a, q, p.sums);
    }
    if (p.dw_post != nullptr || p.dgate != nullptr || p.dw_pre != nullptr)
      norm_sums_kernel<<<dim3((a.d + kSumCols - 1) / kSumCols, 2), 256, 0, s>>>(
          a, p.sums, groups, p.dw_post, p.dgate, p.dw_pre);
    return hipGetLastError();
  });
}

}  // namespace

int norm_grad_groups(int64_t n_rows, int d) {
  const int runs = d / kRun;
  const int64_t rows = runs <= 128 ? (n_rows + 3) / 4 : n_rows;  // steps of a workgroup in all
  const int most = runs <= 512 ? kNormGroups : kNormGroups / 2;
  return static_cast<int>(std::min<int64_t>(rows, most));
}

hipError_t launch_norm_forward(const NormArgs& a, int elem_bytes, const void* residual,
                               const void* y, void* residual_out, void* x, hipStream_t s) {
  if (a.n_rows == 0) return hipSuccess;
  return elem_bytes == 2 ? forward<uint16_t>(a, residual, y, residual_out, x, s)
                         : forward<float>(a, residual, y, residual_out, x, s);
}

hipError_t launch_norm_backward(const NormArgs& a, int elem_bytes, const NormGradArgs& p,
                                hipStream_t s) {
  return elem_bytes == 2 ? backward<uint16_t>(a, p, s) : backward<float>(a, p, s);
}

}  // namespace twell
