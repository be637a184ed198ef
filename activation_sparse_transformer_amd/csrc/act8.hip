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
#include "common.h"
#include "kernels.h"

namespace twell {
namespace {

constexpr int kActThreads = 256;
constexpr int kActCols = 16;                         // columns per lane
constexpr int kActLanes = kAct8Block / kActCols;     // lanes per block of columns
constexpr int kActUnits = kActThreads / kActLanes;   // blocks of columns per workgroup

// Elements c .. c + 7 of a row as float32.
template <typename E>
__device__ __forceinline__ void load8(const E* p, float* f);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float* f) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
  }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, const float* f);
template <>
__device__ __forceinline__ void store8<uint16_t>(uint16_t* p, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = ElemTraits<uint16_t>::from_f32(f[2 * i]) |
           static_cast<uint32_t>(ElemTraits<uint16_t>::from_f32(f[2 * i + 1])) << 16;
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Unit (row, k) of the workgroup's units u0 + i: one 64-bit division per
// workgroup, a 32-bit one per lane.
__device__ __forceinline__ void unit_of(int64_t u0, int i, int per_row, int64_t& row, int& k) {
  const int64_t r0 = u0 / per_row;
  const uint32_t q = static_cast<uint32_t>(u0 - r0 * per_row) + static_cast<uint32_t>(i);
  row = r0 + q / static_cast<uint32_t>(per_row);
  k = static_cast<int>(q % static_cast<uint32_t>(per_row));
}

// kActLanes lanes take one (row, block): the largest magnitude as an integer
// (NaN bits exceed infinity's), then each lane's 16 codes.
template <typename E>
__global__ __launch_bounds__(kActThreads) void act8_pack_kernel(
    const E* __restrict__ x, int64_t n_units, int d, int nb, int pitch,
    int8_t* __restrict__ codes, float* __restrict__ scales) {
  const int l = threadIdx.x % kActLanes;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kActUnits;
  const int i = threadIdx.x / kActLanes;
  if (u0 + i >= n_units) return;
  int64_t row;
  int b;
  unit_of(u0, i, nb, row, b);
  const int c = b * kAct8Block + l * kActCols;
  const E* src = x + row * d + c;
  float f[kActCols];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (c + 8 * h < d) {
      load8<E>(src + 8 * h, f + 8 * h);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[8 * h + k] = 0.f;
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kActCols; ++k) top = max(top, __float_as_uint(f[k]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < kActLanes; o <<= 1)
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o, kWave)));
  const float a = __uint_as_float(top);
  const bool finite = top < 0x7f800000u;
  if (l == 0) {
    float scale = a / 127.f;
    // near the largest float the product 127 * scale may round past it
    if (scale * 127.f > 3.402823466e38f) scale = __uint_as_float(__float_as_uint(scale) - 1u);
    scales[row * nb + b] = finite ? scale : __uint_as_float(0x7fc00000u);
  }
  // a power of two that keeps x * 127 and the quotient in the normal range
  const float up = a > 0x1p100f ? 0x1p-32f : a < 0x1p-90f ? 0x1p60f : 1.f;
  const float den = a * up, r = 1.f / den, k127 = 127.f * up;
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
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
    const uint32_t lo = perm_b32(u[1], u[0], 0x0c0c0400u), hi = perm_b32(u[3], u[2], 0x0c0c0400u);
    w[j] = finite && top != 0 ? lo | hi << 16 : 0u;
  }
  if (c < pitch)
    *reinterpret_cast<uint4*>(codes + row * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One lane takes 16 codes of one row.
template <typename E>
__global__ __launch_bounds__(kActThreads) void act8_unpack_kernel(
    const int8_t* __restrict__ codes, const float* __restrict__ scales, int64_t n_units, int d,
    int nb, int pitch, E* __restrict__ x) {
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kActThreads;
  if (u0 + threadIdx.x >= n_units) return;
  int64_t row;
  int q;
  unit_of(u0, threadIdx.x, pitch / kActCols, row, q);
  const int c = q * kActCols;
  const uint4 v = *reinterpret_cast<const uint4*>(codes + row * pitch + c);
  const float s = scales[row * nb + c / kAct8Block];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[kActCols];
#pragma unroll
  for (int k = 0; k < kActCols; ++k)
    f[k] = static_cast<float>(static_cast<int8_t>(w[k / 4] >> (8 * (k % 4)))) * s;
  E* dst = x + row * d + c;
  store8<E>(dst, f);
  if (c + 8 < d) store8<E>(dst + 8, f + 8);
}

}  // namespace

hipError_t launch_act8_pack(int64_t n_rows, int d, int elem_bytes, const void* x, int8_t* codes,
                            float* scales, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  const int nb = act8_blocks(d), pitch = act8_pitch(d);
  const int64_t units = n_rows * nb;
  const unsigned grid = static_cast<unsigned>((units + kActUnits - 1) / kActUnits);
  if (elem_bytes == 2)
    act8_pack_kernel<uint16_t><<<grid, kActThreads, 0, s>>>(static_cast<const uint16_t*>(x), units,
                                                            d, nb, pitch, codes, scales);
  else
    act8_pack_kernel<float><<<grid, kActThreads, 0, s>>>(static_cast<const float*>(x), units, d,
                                                         nb, pitch, codes, scales);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(int64_t n_rows, int d, int elem_bytes, const int8_t* codes,
                              const float* scales, void* x, hipStream_t s) {
  if (n_rows == 0) return hipSuccess;
  const int nb = act8_blocks(d), pitch = act8_pitch(d);
  const int64_t units = n_rows * (pitch / kActCols);
  const unsigned grid = static_cast<unsigned>((units + kActThreads - 1) / kActThreads);
  if (elem_bytes == 2)
    act8_unpack_kernel<uint16_t><<<grid, kActThreads, 0, s>>>(codes, scales, units, d, nb, pitch,
                                                              static_cast<uint16_t*>(x));
  else
    act8_unpack_kernel<float><<<grid, kActThreads, 0, s>>>(codes, scales, units, d, nb, pitch,
                                                           static_cast<float*>(x));
  return hipGetLastError();
}

}  // namespace twell
