// 8-bit activation checkpoints: a layer's input kept between the forward and
// the backward pass as int8 codes with one float32 scale per row and block of
// kAct8Block columns.  For a block of largest magnitude a,
//   scale = a / 127,   code = rint(x * 127 / a)  (half to even),
//   x^ = code * scale,
// so |x - x^| <= a / 254 up to float32 rounding.  x * 127 is exact for bf16
// and the division is correctly rounded, so a bf16 code is the rounding of the
// real quotient, ties included.  A block of zeros has scale 0; a block that
// holds a NaN or an infinity has scale NaN and codes 0, so that it reads back
// as NaN instead of losing it.
#include <type_traits>

#include "common.h"
#include "stream_ops.h"
#include "train_kernels.h"

namespace twell {
namespace {

constexpr int kActThreads = 256;
constexpr int kPackUnits = 2;

// A lane takes one 16-byte vector of x: 8 (bf16) or 4 (float32) columns.
template <typename E>
struct ActLane {
  static constexpr int kCols = 16 / sizeof(E);
  static constexpr int kLanes = kAct8Block / kCols;  // per block of columns
  static constexpr int kWords = kCols / 4;           // 32-bit words of codes
};

template <typename E>
__device__ __forceinline__ void widen(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 2) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}

template <typename E>
__device__ __forceinline__ uint4 narrow(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 2)
      w[i] = ElemTraits<E>::from_f32(f[2 * i]) |
             static_cast<uint32_t>(ElemTraits<E>::from_f32(f[2 * i + 1])) << 16;
    else
      w[i] = __float_as_uint(f[i]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Unit (row, k) of the workgroup's units u0 + i: one 64-bit division per
// workgroup, a 32-bit one per lane.
__device__ __forceinline__ void unit_of(int64_t u0, int i, int per_row, int64_t& row, int& k) {
  const int64_t r0 = u0 / per_row;
  const uint32_t q = static_cast<uint32_t>(u0 - r0 * per_row) + static_cast<uint32_t>(i);
  row = r0 + q / static_cast<uint32_t>(per_row);
  k = static_cast<int>(q % static_cast<uint32_t>(per_row));
}

// The largest v of the group of P lanes (P = 16 or 32), in every lane of it:
// quads, half rows and rows by DPP, the other row of a pair by a swap.
template <int P>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  auto up = [&](auto ctrl) {
    const int t = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), decltype(ctrl)::value, 0xf,
                                              0xf, false);
    v = max(v, static_cast<uint32_t>(t));
  };
  up(std::integral_constant<int, 0xb1>{});   // quad_perm [1, 0, 3, 2]
  up(std::integral_constant<int, 0x4e>{});   // quad_perm [2, 3, 0, 1]
  up(std::integral_constant<int, 0x141>{});  // row_half_mirror
  up(std::integral_constant<int, 0x140>{});  // row_mirror
  if constexpr (P == 32)
    v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16, kWave)));
  return v;
}

// kLanes lanes take one (row, block) at a time: the largest magnitude as an
// integer (NaN bits exceed infinity's), then each lane's codes.  kPackUnits
// blocks per lane, read together, keep enough bytes in flight behind the
// reductions (1: 79 us, 2: 71, 4: 79 at 16384 x 8192 bf16, 5.7 TB/s).  Bound by
// HBM.
template <typename E>
__global__ __launch_bounds__(kActThreads) void act8_pack_kernel(
    const E* __restrict__ x, int64_t n_units, int d, int nb, int pitch,
    int8_t* __restrict__ codes, float* __restrict__ scales) {
  typedef ActLane<E> A;
  constexpr int kUnits = kActThreads / A::kLanes;
  const int l = threadIdx.x % A::kLanes;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kUnits * kPackUnits);
  int64_t row[kPackUnits];
  int b[kPackUnits];
  uint4 v[kPackUnits];
#pragma unroll
  for (int n = 0; n < kPackUnits; ++n) {
    const int i = n * kUnits + threadIdx.x / A::kLanes;
    unit_of(u0, i, nb, row[n], b[n]);
    const int c = b[n] * kAct8Block + l * A::kCols;
    v[n] = u0 + i < n_units && c < d ? load_once(reinterpret_cast<const uint4*>(x + row[n] * d + c))
                                     : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int n = 0; n < kPackUnits; ++n) {
    if (u0 + n * kUnits + threadIdx.x / A::kLanes >= n_units) return;
    const int c = b[n] * kAct8Block + l * A::kCols;
    float f[A::kCols];
    widen<E>(v[n], f);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < A::kCols; ++k) top = max(top, __float_as_uint(f[k]) & 0x7fffffffu);
    top = group_max<A::kLanes>(top);
    const float a = __uint_as_float(top);
    const bool finite = top < 0x7f800000u;
    if (l == 0) {
      float scale = a / 127.f;
      // near the largest float the product 127 * scale may round past it
      if (scale * 127.f > 3.402823466e38f) scale = __uint_as_float(__float_as_uint(scale) - 1u);
      scales[row[n] * nb + b[n]] = finite ? scale : __uint_as_float(0x7fc00000u);
    }
    // a power of two that keeps x * 127 and the quotient in the normal range
    const float up = a > 0x1p100f ? 0x1p-32f : a < 0x1p-90f ? 0x1p60f : 1.f;
    const float den = a * up, r = 1.f / den, k127 = 127.f * up;
    uint32_t w[A::kWords];
#pragma unroll
    for (int j = 0; j < A::kWords; ++j) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // the quotient from the rounded reciprocal and one exact remainder: a
        // product, a fused remainder and a correction instead of a division
        const float t = f[4 * j + k] * k127;
        const float q0 = t * r;
        const float q = fmaf(fmaf(-q0, den, t), r, q0);
        // 1.5 * 2^23 + q: the sum's last byte is q rounded to even
        u[k] = __float_as_uint(q + 0x1.8p23f);
      }
      const uint32_t lo = perm_b32(u[1], u[0], 0x0c0c0400u);
      const uint32_t hi = perm_b32(u[3], u[2], 0x0c0c0400u);
      w[j] = finite && top != 0 ? lo | hi << 16 : 0u;
    }
    if (c >= pitch) continue;
    int8_t* to = codes + row[n] * pitch + c;
    if constexpr (A::kWords == 2) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(to) = w[0];
  }
}

// One lane makes one 16-byte vector of x.  Bound by HBM: 16384 x 8192 bf16 73
// us, 5.6 TB/s; 8192 x 4096 float32 25 us, 6.8 TB/s.
template <typename E>
__global__ __launch_bounds__(kActThreads) void act8_unpack_kernel(
    const int8_t* __restrict__ codes, const float* __restrict__ scales, int64_t n_units, int d,
    int nb, int pitch, E* __restrict__ x) {
  typedef ActLane<E> A;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kActThreads;
  if (u0 + threadIdx.x >= n_units) return;
  int64_t row;
  int q;
  unit_of(u0, threadIdx.x, d / A::kCols, row, q);
  const int c = q * A::kCols;
  const int8_t* src = codes + row * pitch + c;
  uint32_t w[2] = {};
  if constexpr (A::kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
  const float s = scales[row * nb + c / kAct8Block];
  float f[A::kCols];
#pragma unroll
  for (int k = 0; k < A::kCols; ++k)
    f[k] = static_cast<float>(static_cast<int8_t>(w[k / 4] >> (8 * (k % 4)))) * s;
  store_once(x + row * d + c, narrow<E>(f));
}

template <typename E>
hipError_t pack(int64_t n_rows, int d, const void* x, int8_t* codes, float* scales,
                hipStream_t s) {
  const int64_t units = n_rows * act8_blocks(d);
  const int per = kActThreads / ActLane<E>::kLanes * kPackUnits;
  act8_pack_kernel<E><<<static_cast<unsigned>((units + per - 1) / per), kActThreads, 0, s>>>(
      static_cast<const E*>(x), units, d, act8_blocks(d), act8_pitch(d), codes, scales);
  return hipGetLastError();
}

template <typename E>
hipError_t unpack(int64_t n_rows, int d, const int8_t* codes, const float* scales, void* x,
                  hipStream_t s) {
  const int64_t units = n_rows * (d / ActLane<E>::kCols);
  act8_unpack_kernel<E>
      <<<static_cast<unsigned>((units + kActThreads - 1) / kActThreads), kActThreads, 0, s>>>(
          codes, scales, units, d, act8_blocks(d), act8_pitch(d), static_cast<E*>(x));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act8_pack(int64_t n_rows, int d, int elem_bytes, const void* x, int8_t* codes,
                            float* scales, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  return elem_bytes == 2 ? pack<uint16_t>(n_rows, d, x, codes, scales, s)
                         : pack<float>(n_rows, d, x, codes, scales, s);
}

hipError_t launch_act8_unpack(int64_t n_rows, int d, int elem_bytes, const int8_t* codes,
                              const float* scales, void* x, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  return elem_bytes == 2 ? unpack<uint16_t>(n_rows, d, codes, scales, x, s)
                         : unpack<float>(n_rows, d, codes, scales, x, s);
}

}  // namespace twell
