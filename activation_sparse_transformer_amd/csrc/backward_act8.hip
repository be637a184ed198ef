// The layer's backward pass from an 8-bit checkpoint of its input.  Same
// gradients as the plain backward (dz = dy W_down^T where h is non-zero,
// dW_down = h^T dy, dW_up^T = dz^T x, db = column sums of dz, dx = dz W_up),
// with x = code * scale formed on the way and dz kept in float32 throughout.
//
// The non-zeros of h become one list in two orders: by row and then neuron
// (cols; h is stored there, later dz), and by neuron and then row (ents: row, h,
// and the place p in the other order).  A row has room for all that it can hold,
// so its entries go there without a count of the others; a bitmap over (row,
// neuron) gives the neuron-major places, so every sum below runs in a fixed
// order.  At the 1B layer this takes 48 us (rows 16, bits 7, their sums 11, the
// neuron order 15), chains of dependent reads each.  Three passes gather rows
// of dy, x and W_up:
//   down: per entry the dot of dy[row] with W_down[j], dW_down[j] += h dy[row];
//   up:   dz; dW_up^T[j] += dz x[row], db[j] += dz;
//   dx:   dx[row] += dz W_up[j], for TwELL and dense rows alike.
// Each gathers 335 k x 2048 columns at the 1B layer, from the L2 of the XCD
// that a column slice is dealt to: down 90 us and dx 70 us for 1.37 GB, up 77
// us for 0.69 GB of codes.  They are bound by the path that returns loaded data
// to the registers: it is busy for 82% (down), 76% (up) and 76% (dx) of their
// cycles, with 85-90% of the reads hitting the L2 at 170-225 cycles and the
// vector units busy for 19%.  Up reads half the bytes in 1.3 times dx's loads:
// beside a row's codes it loads their scale, and per entry eight partial dots.
// With a fifth fewer instructions (entries handed out by DPP broadcasts,
// unrolled) the passes took as long or longer.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "stream_ops.h"
#include "train_kernels.h"
#include "vec_ops.h"

namespace twell {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kCols = 16;  // columns of a gathered row per lane and vector group
constexpr int kScanThreads = 1024;
constexpr int kScanPer = 16;
constexpr int64_t kDenseBlocks = 1024;
constexpr int kBitCols = 2048;
constexpr int kSliceCols = 2 * kWave * kCols;  // of the widest slice
constexpr int kMaxCols = 8 * kSliceCols;

// A non-zero in the neuron order.  Twelve bytes: with one per place that h could
// fill, a fourth word would be 134 MB of workspace at the 1B layer.
struct Entry {
  int32_t row;
  uint32_t h;     // as float32 bits
  int32_t place;  // in the row order
};

__device__ __forceinline__ int64_t wave_index() {
  return static_cast<int64_t>(blockIdx.x) * kWaves + threadIdx.x / kWave;
}

__device__ __forceinline__ int64_t stored_rows(const BwdHybrid& hy, int64_t n_rows) {
  return hy.cap <= 0 ? 0 : min(static_cast<int64_t>(max(*hy.n_dense, 0)), min(hy.cap, n_rows));
}

__global__ __launch_bounds__(kThreads) void a8_zero_kernel(uint4* __restrict__ p, int64_t n) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride)
    p[i] = make_uint4(0, 0, 0, 0);
}

// m + 1 for the stored dense row m of token row n (0: none): a search of the
// ascending list by all lanes of the wave, 64 places a step.
__device__ __forceinline__ int dense_slot(const BwdHybrid& hy, int64_t n_rows, int64_t n) {
  const int lane = lane_id();
  int lo = 0, hi = static_cast<int>(stored_rows(hy, n_rows));
  while (hi - lo > kWave) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int i = lo + lane * step;
    const int under = popc64(wave_ballot(i < hi && hy.dense_rows[i] <= n));
    if (under == 0) return 0;
    lo += (under - 1) * step;
    hi = min(hi, lo + step);
  }
  const uint64_t at =
      wave_ballot(lo + lane < hi && hy.dense_rows[lo + lane] == n);
  return at != 0 ? lo + __builtin_ctzll(at) + 1 : 0;
}

// Where row n's part of the row order starts: a row has room for all of its
// slots (`slot` - 1 < 0) or, as stored dense row slot - 1, for d_ff entries.
__device__ __forceinline__ int64_t row_start(int64_t n_rows, int64_t n, int slot, int dff,
                                             int nslots) {
  return slot > 0 ? n_rows * nslots + static_cast<int64_t>(slot - 1) * dff : n * nslots;
}

// The row order: every non-zero's neuron and value, ascending in a row, whose
// {start, count} is row_at[n].  The first row_blocks workgroups take a TwELL row
// per wave, the others a dense row each.
template <typename E>
__global__ __launch_bounds__(kThreads) void a8_rows_kernel(
    BwdHybrid hy, int64_t n_rows, int dff, int T, int C, int nt, unsigned row_blocks,
    int2* __restrict__ row_at, int32_t* __restrict__ cols, float* __restrict__ vals) {
  typedef ElemTraits<E> Tr;
  constexpr int V = 16 / sizeof(E);
  constexpr int U = 4;  // vectors, or slots, of a lane in flight
  constexpr int kWaveCols = U * kWave * V, kChunk = kWaves * kWaveCols;
  __shared__ uint16_t found[kChunk];  // columns of the chunk's non-zeros, ascending
  __shared__ int wave_found[kWaves];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int nslots = nt * C;
  if (blockIdx.x < row_blocks) {
    const int64_t n = wave_index();
    if (n >= n_rows || dense_slot(hy, n_rows, n) > 0) return;
    const int64_t start = row_start(n_rows, n, 0, dff, nslots);
    const E* vrow = static_cast<const E*>(hy.vals) + n * nslots;
    const uint8_t* irow = hy.idx + n * nslots;
    int held = 0;
    for (int s0 = 0; s0 < nslots; s0 += U * kWave) {
      int local[U], tile[U];
      E v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * kWave + lane;
        tile[u] = s / C;
        local[u] = T;
        if (s < nslots && s - tile[u] * C < static_cast<int>(hy.cnt[n * nt + tile[u]]))
          local[u] = irow[s];
        v[u] = s < nslots ? vrow[s] : E(0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint64_t m = wave_ballot(local[u] < T);
        if (local[u] < T) {
          const int64_t p = start + held + popc_below(m);
          cols[p] = tile[u] * T + local[u];
          vals[p] = Tr::to_f32(v[u]);
        }
        held += popc64(m);
      }
    }
    if (lane == 0) row_at[n] = make_int2(static_cast<int>(start), held);
    return;
  }
  const int64_t stored = stored_rows(hy, n_rows);
  for (int64_t m = blockIdx.x - row_blocks; m < stored; m += gridDim.x - row_blocks) {
    const int64_t n = hy.dense_rows[m];
    if (n < 0 || n >= n_rows) continue;
    const int64_t start = row_start(n_rows, n, static_cast<int>(m) + 1, dff, nslots);
    const E* row = static_cast<const E*>(hy.dense_values) + m * dff;
    int held = 0;
    for (int c0 = 0; c0 < dff; c0 += kChunk) {
      uint4 q[U];
      const int first = wave * kWaveCols + lane * V;  // of the lane's, in the chunk
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + first + u * kWave * V;
        q[u] = c < dff ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
      }
      // the lane's non-zeros per vector, then those of the lanes up to it: two
      // counts (at most 64 V) in a register
      uint32_t mine[U / 2], upto[U / 2];
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        uint32_t c = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          E v[V];
          *reinterpret_cast<uint4*>(v) = q[u + k];
#pragma unroll
          for (int e = 0; e < V; ++e) c += (Tr::abs_bits(v[e]) != 0u ? 1u : 0u) << (16 * k);
        }
        mine[u / 2] = upto[u / 2] = c;
      }
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1)
#pragma unroll
        for (int h = 0; h < U / 2; ++h) {
          const uint32_t got = __shfl_up(upto[h], o, kWave);
          if (lane >= o) upto[h] += got;
        }
      int before[U], total = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        before[u] = total + static_cast<int>((upto[u / 2] - mine[u / 2]) >> (16 * (u % 2)) & 0xffff);
        total += static_cast<int>(__shfl(upto[u / 2], kWave - 1, kWave) >> (16 * (u % 2)) & 0xffff);
      }
      if (lane == 0) wave_found[wave] = total;
      __syncthreads();
      int base = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        base += w < wave ? wave_found[w] : 0;
        all += wave_found[w];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        E v[V];
        *reinterpret_cast<uint4*>(v) = q[u];
        int p = base + before[u];
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (Tr::abs_bits(v[e]) != 0u)
            found[p++] = static_cast<uint16_t>(first + u * kWave * V + e);
      }
      __syncthreads();
      for (int i = tid; i < all; i += kThreads) {
        const int j = c0 + found[i];
        cols[start + held + i] = j;
        vals[start + held + i] = Tr::to_f32(row[j]);
      }
      held += all;
      __syncthreads();  // found and wave_found are rewritten by the next chunk
    }
    if (tid == 0) row_at[n] = make_int2(static_cast<int>(start), held);
  }
}

// bits[w][j]: bit r is set where row 64 w + r has a non-zero at neuron j.  A
// workgroup per word and kBitCols neurons collects its bits in LDS (integer
// ors: no order) from the lists of the 64 rows, which needs no cleared memory:
// 7 us at the 1B layer.  Or-ing its 335 k bits into memory as the rows are read
// took 5 us more, with the clearing.
__global__ __launch_bounds__(kScanThreads) void a8_bits_kernel(
    const int2* __restrict__ row_at, const int32_t* __restrict__ cols, int64_t n_rows, int dff,
    int n_slices, unsigned long long* __restrict__ bits) {
  __shared__ unsigned long long word[kBitCols];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int64_t w = blockIdx.x / n_slices;
  const int j0 = static_cast<int>(blockIdx.x % n_slices) * kBitCols;
  for (int i = tid; i < kBitCols; i += kScanThreads) word[i] = 0;
  __syncthreads();
  constexpr int kRows = kWave / (kScanThreads / kWave);  // of a wave
  constexpr int U = 2;  // entries of a row in flight, of all the wave's rows together
  int2 at[kRows];
  int longest = 0;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t n = w * kWave + wave * kRows + k;
    at[k] = n < n_rows ? row_at[n] : make_int2(0, 0);
    longest = max(longest, at[k].y);
  }
  for (int i0 = lane; i0 < longest; i0 += U * kWave) {
    int j[kRows][U];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kWave;
        j[k][u] = i < at[k].y ? cols[static_cast<int64_t>(at[k].x) + i] - j0 : -1;
      }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (static_cast<unsigned>(j[k][u]) < kBitCols)
          atomicOr(word + j[k][u], 1ull << (wave * kRows + k));
  }
  __syncthreads();
  for (int i = tid; i < min(kBitCols, dff - j0); i += kScanThreads) bits[w * dff + j0 + i] = word[i];
}

// Per neuron (a lane of every wave; the words in runs, one a wave): lpre[b][j] =
// set bits of its words below b; neuron_count[j] = all.
__global__ __launch_bounds__(kScanThreads) void a8_prefix_kernel(
    const unsigned long long* __restrict__ bits, int64_t n_words, int dff,
    int32_t* __restrict__ lpre, int32_t* __restrict__ neuron_count) {
  constexpr int kRuns = kScanThreads / kWave;
  constexpr int U = 4;
  __shared__ int run_total[kRuns][kWave];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kWave + lane;
  const int64_t jr = j < dff ? j : dff - 1;
  const int64_t per = (n_words + kRuns - 1) / kRuns;
  const int64_t b0 = min(wave * per, n_words), b1 = min(b0 + per, n_words);
  int total = 0;
  for (int64_t b = b0; b < b1; b += U)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = __popcll(bits[min(b + u, n_words - 1) * dff + jr]);
      total += b + u < b1 ? c : 0;
    }
  run_total[wave][lane] = total;
  __syncthreads();
  int run = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    run += k < wave ? run_total[k][lane] : 0;
    all += run_total[k][lane];
  }
  if (j >= dff) return;
  for (int64_t b = b0; b < b1; b += U) {
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = __popcll(bits[min(b + u, n_words - 1) * dff + j]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u < b1) {
        lpre[(b + u) * dff + j] = run;
        run += c[u];
      }
  }
  if (wave == 0) neuron_count[j] = all;
}

// Exclusive sums of the neurons' counts.
__global__ __launch_bounds__(kScanThreads) void a8_scan_kernel(const int32_t* __restrict__ in,
                                                               int64_t n,
                                                               int32_t* __restrict__ out) {
  __shared__ int wave_tot[kScanThreads / kWave];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  int carry = 0;
  for (int64_t r0 = 0; r0 < n; r0 += kScanThreads * kScanPer) {
    const int64_t i0 = r0 + static_cast<int64_t>(tid) * kScanPer;
    int v[kScanPer], local = 0;
#pragma unroll
    for (int k = 0; k < kScanPer; k += 4) {
      if (i0 + k + 4 <= n) {
        const int4 q = *reinterpret_cast<const int4*>(in + i0 + k);
        v[k] = q.x, v[k + 1] = q.y, v[k + 2] = q.z, v[k + 3] = q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k + e] = i0 + k + e < n ? in[i0 + k + e] : 0;
      }
    }
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) local += v[k];
    int sc = local;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int u = __shfl_up(sc, o, kWave);
      if (lane >= o) sc += u;
    }
    if (lane == kWave - 1) wave_tot[wave] = sc;
    __syncthreads();
    int run = carry + sc - local, total = 0;
    for (int w = 0; w < kScanThreads / kWave; ++w) {
      run += w < wave ? wave_tot[w] : 0;
      total += wave_tot[w];
    }
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) {
      if (i0 + k < n) out[i0 + k] = run;
      run += v[k];
    }
    carry += total;
    __syncthreads();  // wave_tot is rewritten by the next round
  }
  if (tid == 0) out[n] = carry;
}

// Every non-zero into the neuron order, from its place in the row order:
// workgroups as for those.
__global__ __launch_bounds__(kThreads) void a8_fill_kernel(
    BwdHybrid hy, int64_t n_rows, int64_t dense_from, int dff, unsigned row_blocks,
    const unsigned long long* __restrict__ bits, const int32_t* __restrict__ lpre,
    const int32_t* __restrict__ neuron_off, const int2* __restrict__ row_at,
    const int32_t* __restrict__ cols, const float* __restrict__ vals, Entry* __restrict__ ents) {
  constexpr int U = 2;  // entries of a lane whose dependent reads overlap
  auto place = [&](int64_t n, int2 at, int first, int stride) {
    const unsigned long long below = (1ull << (n & 63)) - 1;
    for (int i0 = first; i0 < at.y; i0 += U * stride) {
      int j[U], to[U];
      uint32_t h[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t p = at.x + min(i0 + u * stride, at.y - 1);
        j[u] = cols[p];
        h[u] = __float_as_uint(vals[p]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t w = (n >> 6) * dff + j[u];
        to[u] = neuron_off[j[u]] + lpre[w] + __popcll(bits[w] & below);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * stride < at.y)
          ents[to[u]] = Entry{static_cast<int>(n), h[u], at.x + i0 + u * stride};
    }
  };
  if (blockIdx.x < row_blocks) {
    const int64_t n = wave_index();
    if (n >= n_rows) return;
    const int2 at = row_at[n];
    if (at.x < dense_from) place(n, at, lane_id(), kWave);
    return;
  }
  const int64_t stored = stored_rows(hy, n_rows);
  for (int64_t m = blockIdx.x - row_blocks; m < stored; m += gridDim.x - row_blocks) {
    const int64_t n = hy.dense_rows[m];
    if (n < 0 || n >= n_rows) continue;
    place(n, row_at[n], threadIdx.x, kThreads);
  }
}

// ---- The gathering passes.  A slice of sw columns is covered by P lanes, 64 / P
// rows at a time; block b takes slice b % S, so that a slice's rows stay in the
// L2 of the XCDs it is dealt to.  A lane holds kAcc = 16 NV columns as chunks
// of V columns (16 bytes of the gathered type): chunk k of lane l is columns
// (k P + l) V ..., so that one load of the group is one run of bytes.
// FULL: the group covers the slice exactly.
template <int V, int P, int NV, bool FULL, int FLIGHT = 8>
struct Slice {
  static constexpr int kAcc = NV * kCols, kChunks = kAcc / V;
  static constexpr int kGroups = kWave / P;
  // rows per step, in flight together: FLIGHT groups of columns
  static constexpr int kSteps = kGroups * NV >= FLIGHT ? 1 : FLIGHT / (kGroups * NV);
  static constexpr int kEntries = kGroups * kSteps;
  int first;  // column of the lane's chunk 0
  int lim;    // columns of the slice past `first`; the last slice may be shorter
  __device__ __forceinline__ Slice(int s, int sw, int dm) {
    const int l = lane_id() % P;
    first = s * sw + l * V;
    lim = min(sw, dm - s * sw) - l * V;
  }
  __device__ __forceinline__ bool ok(int k) const { return FULL || k * P * V < lim; }
  // a chunk past the slice reads the slice's first columns instead
  __device__ __forceinline__ int col(int k) const {
    return ok(k) ? first + k * P * V : first - lane_id() % P * V;
  }
  // the column of accumulator i
  __device__ __forceinline__ int col_of(int i) const { return first + i / V * (P * V) + i % V; }
  // how many columns the lane's row may be written at, from accumulator i's on
  __device__ __forceinline__ bool may_write(int i) const {
    return FULL || i / V * (P * V) + i % V < lim;
  }
};

// A lane's chunks of one row of E.
template <typename E, typename Sl>
struct Row {
  static constexpr int V = 16 / sizeof(E), K = Sl::kChunks;
  uint4 q[K];
  __device__ __forceinline__ void load(const E* row, const Sl& sl) {
#pragma unroll
    for (int k = 0; k < K; ++k) q[k] = *reinterpret_cast<const uint4*>(row + sl.col(k));
  }
  // a row that is read once
  __device__ __forceinline__ void load_past(const E* row, const Sl& sl) {
#pragma unroll
    for (int k = 0; k < K; ++k) q[k] = load_once(reinterpret_cast<const uint4*>(row + sl.col(k)));
  }
  // zero where `keep` is false or the chunk is past the slice
  __device__ __forceinline__ void keep(bool keep, const Sl& sl) {
#pragma unroll
    for (int k = 0; k < K; ++k) q[k] = keep_if(keep && sl.ok(k), q[k]);
  }
  __device__ __forceinline__ float dot(const Row& o) const {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) s += dot16<E>(q[k], o.q[k]);
    return s;
  }
  __device__ __forceinline__ void axpy(float* acc, uint32_t sbits) const {
#pragma unroll
    for (int k = 0; k < K; ++k) axpy16<E>(acc + k * V, sbits, q[k]);
  }
  // acc += f * q with f in float32
  __device__ __forceinline__ void fma32(float* acc, float f) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(E) == 2) {
          float* a = acc + k * V + 2 * i;
          a[0] = fmaf(f, __uint_as_float(w[i] << 16), a[0]);
          a[1] = fmaf(f, __uint_as_float(w[i] & 0xffff0000u), a[1]);
        } else {
          acc[k * V + i] = fmaf(f, __uint_as_float(w[i]), acc[k * V + i]);
        }
      }
    }
  }
};

typedef uint32_t swap_pair_t __attribute__((ext_vector_type(2)));

// The groups' sums added, in a fixed order, and spread: afterwards a lane of
// group g holds the kAcc / kGroups columns from g * kAcc / kGroups of its kAcc
// in acc[0 ..].  Each step swaps half a wave (or alternate rows of 16) of two
// accumulators and adds, which halves their number.
template <int P, int N>
__device__ __forceinline__ void join_groups(float (&acc)[N]) {
  if constexpr (P <= 32) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const swap_pair_t r = __builtin_bit_cast(
          swap_pair_t, __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i]),
                                                        __float_as_uint(acc[i + N / 2]), false,
                                                        false));
      acc[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
  }
  if constexpr (P <= 16) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const swap_pair_t r = __builtin_bit_cast(
          swap_pair_t, __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i]),
                                                        __float_as_uint(acc[i + N / 4]), false,
                                                        false));
      acc[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
  }
}

// The first column, in the lane's kAcc, that join_groups leaves with it.
template <int P, int N>
__device__ __forceinline__ int joined_first() {
  const int lane = lane_id();
  int c = 0;
  if constexpr (P <= 32) c += lane / 32 * (N / 2);
  if constexpr (P <= 16) c += lane / 16 % 2 * (N / 4);
  return c;
}

// The joined sums to the lane's columns of a row.
template <int P, typename O, typename Sl>
__device__ __forceinline__ void store_joined(O* row, const Sl& sl, const float* acc) {
  constexpr int kEach = Sl::kAcc / Sl::kGroups;
  const int first = joined_first<P, Sl::kAcc>();
#pragma unroll
  for (int i = 0; i < kEach; i += 4) {
    if (!sl.may_write(first + i)) continue;
    O* to = row + sl.col_of(first + i);
    if constexpr (sizeof(O) == 4) {
      store_once(to, make_uint4(__float_as_uint(acc[i]), __float_as_uint(acc[i + 1]),
                                __float_as_uint(acc[i + 2]), __float_as_uint(acc[i + 3])));
    } else {
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[k] = ElemTraits<O>::from_f32(acc[i + 2 * k]) |
               static_cast<uint32_t>(ElemTraits<O>::from_f32(acc[i + 2 * k + 1])) << 16;
      *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    }
  }
}

// The neuron or row group and the slice of a workgroup: S is a power of two.
struct Place {
  int slice;
  int64_t item;  // this wave's
  __device__ __forceinline__ explicit Place(int log_s) {
    slice = static_cast<int>(blockIdx.x) & ((1 << log_s) - 1);
    // in a scalar register, as are its offsets and counts then
    item = static_cast<int64_t>(blockIdx.x >> log_s) * kWaves +
           __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  }
};

// Down: a wave per (neuron, slice).  part[s * pstride + entry] = the slice's
// dot of dy[row] with W_down[j]; dW_down[j][slice] = sum of h dy[row].
template <typename E, int P, int NV, bool FULL>
__global__ __launch_bounds__(kThreads) void a8_down_kernel(
    const int32_t* __restrict__ neuron_off, const Entry* __restrict__ ents,
    const E* __restrict__ dy, const E* __restrict__ w_down, int dff, int dm, int log_s, int sw,
    float* __restrict__ part, int64_t pstride, float* __restrict__ dw_down) {
  typedef Slice<16 / sizeof(E), P, NV, FULL> Sl;
  typedef Row<E, Sl> R;
  const int lane = lane_id(), grp = lane / P;
  const Place at(log_s);
  if (at.item >= dff) return;
  const int j = static_cast<int>(at.item);
  const Sl sl(at.slice, sw, dm);
  const int b = neuron_off[j], L = neuron_off[j + 1] - b;
  float acc[Sl::kAcc];
#pragma unroll
  for (int i = 0; i < Sl::kAcc; ++i) acc[i] = 0.f;
  R w;
  w.load_past(w_down + static_cast<int64_t>(j) * dm, sl);
  if (!FULL) w.keep(true, sl);
  for (int base = 0; base < L; base += kWave) {
    const int cnt = min(kWave, L - base);
    const Entry mine = ents[b + base + min(lane, cnt - 1)];
    float mypd = 0.f;  // lane t: the chunk's entry t
    auto step = [&](int e0, auto check) {
      constexpr bool CHECK = decltype(check)::value;
      R y[Sl::kSteps];
      uint32_t hb[Sl::kSteps];
      float pd[Sl::kSteps];
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        const int e = e0 + u * Sl::kGroups + grp;
        const int64_t row = __shfl(mine.row, e, kWave);
        hb[u] = store_bits<E>(__shfl(mine.h, e, kWave));
        y[u].load(dy + row * dm, sl);
      }
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        if (CHECK) y[u].keep(e0 + u * Sl::kGroups + grp < cnt, sl);
        pd[u] = y[u].dot(w);
      }
      group_totals<P, Sl::kSteps>(pd);
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        // entry e's partial is in the last lane of its group; lane e takes it
        const int e_u = e0 + u * Sl::kGroups;
        const float got = __shfl(pd[u], (lane - e_u) * P + P - 1, kWave);
        if (lane >= e_u && lane < e_u + Sl::kGroups) mypd = got;
      }
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) y[u].axpy(acc, hb[u]);
    };
    int e0 = 0;
    for (; e0 + Sl::kEntries <= cnt; e0 += Sl::kEntries) step(e0, std::false_type{});
    if (e0 < cnt) step(e0, std::true_type{});
    if (lane < cnt) part[at.slice * pstride + b + base + lane] = mypd;
  }
  join_groups<P>(acc);
  store_joined<P>(dw_down + static_cast<int64_t>(j) * dm, sl, acc);
}

// Up: a wave per (neuron, slice).  dz = the n_part partial dots added in slice
// order; slice 0 stores it at its place in the row order and adds db[j];
// dW_up^T[j][slice] = sum of (dz * scale) * code.  A chunk's 16 columns lie in
// one block of scales.  Four rows in flight, not eight: the registers saved are
// worth more as waves (76 against 91 us at the 1B layer).
template <int P, int NV, bool FULL>
__global__ __launch_bounds__(kThreads) void a8_up_kernel(
    const int32_t* __restrict__ neuron_off, const Entry* __restrict__ ents,
    const int8_t* __restrict__ codes, const float* __restrict__ scales, int pitch, int nb,
    const float* __restrict__ part, int64_t pstride, int n_part, int dff, int dm, int log_s, int sw,
    float* __restrict__ dz, float* __restrict__ dw_up_t, float* __restrict__ db) {
  typedef Slice<kCols, P, NV, FULL, 4> Sl;
  const int lane = lane_id(), grp = lane / P;
  const Place at(log_s);
  if (at.item >= dff) return;
  const int j = static_cast<int>(at.item);
  const Sl sl(at.slice, sw, dm);
  const int b = neuron_off[j], L = neuron_off[j + 1] - b;
  float acc[Sl::kAcc];
#pragma unroll
  for (int i = 0; i < Sl::kAcc; ++i) acc[i] = 0.f;
  float sum = 0.f;
  for (int base = 0; base < L; base += kWave) {
    const int cnt = min(kWave, L - base);
    const int64_t me = b + base + min(lane, cnt - 1);
    const Entry mine = ents[me];
    float d = part[me];
    // eight loads together (1B layer 270 us; one after another 293); two or four
    // of them, of narrower layers, are within 1% either way and take the loop
    if (n_part == 8) {
      float p[7];
#pragma unroll
      for (int t = 0; t < 7; ++t) p[t] = part[(t + 1) * pstride + me];
#pragma unroll
      for (int t = 0; t < 7; ++t) d += p[t];
    } else {
      for (int t = 1; t < n_part; ++t) d += part[t * pstride + me];
    }
    // a lane past the entries repeats the last one with a factor of zero: its
    // row's scale is NaN only where the neuron's sum is NaN already
    if (lane >= cnt) d = 0.f;
    for (int e0 = 0; e0 < cnt; e0 += Sl::kEntries) {
      uint4 q[Sl::kSteps][NV];
      float f[Sl::kSteps][NV];
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        const int64_t row = __shfl(mine.row, e0 + u * Sl::kGroups + grp, kWave);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          q[u][v] = *reinterpret_cast<const uint4*>(codes + row * pitch + sl.col(v));
          f[u][v] = scales[row * nb + sl.col(v) / kAct8Block];
        }
      }
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        const float dzu = __shfl(d, e0 + u * Sl::kGroups + grp, kWave);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float z = dzu * f[u][v];
          const uint32_t w[4] = {q[u][v].x, q[u][v].y, q[u][v].z, q[u][v].w};
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            acc[v * kCols + i] =
                fmaf(z, static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)))),
                     acc[v * kCols + i]);
        }
      }
    }
    if (at.slice == 0 && lane < cnt) {
      dz[mine.place] = d;
      sum += d;
    }
  }
  join_groups<P>(acc);
  store_joined<P>(dw_up_t + static_cast<int64_t>(j) * dm, sl, acc);
  if (at.slice == 0) {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o, kWave);
    if (lane == 0) db[j] = sum;
  }
}

// dx: a wave per (token row, slice): dx[n][slice] = sum of dz W_up^T[j], in
// float32, rounded once.
template <typename E, int P, int NV, bool FULL>
__global__ __launch_bounds__(kThreads) void a8_dx_kernel(
    const int2* __restrict__ row_at, const int32_t* __restrict__ cols,
    const float* __restrict__ dz, const E* __restrict__ w_up_t, int64_t n_rows, int dm, int log_s,
    int sw, E* __restrict__ dx) {
  typedef Slice<16 / sizeof(E), P, NV, FULL> Sl;
  typedef Row<E, Sl> R;
  const int lane = lane_id(), grp = lane / P;
  const Place at(log_s);
  const int64_t n = at.item;
  if (n >= n_rows) return;
  const Sl sl(at.slice, sw, dm);
  const int b = row_at[n].x, L = row_at[n].y;
  float acc[Sl::kAcc];
#pragma unroll
  for (int i = 0; i < Sl::kAcc; ++i) acc[i] = 0.f;
  for (int base = 0; base < L; base += kWave) {
    const int cnt = min(kWave, L - base);
    const int my_col = cols[b + base + min(lane, cnt - 1)];
    const float my_dz = dz[b + base + min(lane, cnt - 1)];
    auto step = [&](int e0, auto check) {
      constexpr bool CHECK = decltype(check)::value;
      R w[Sl::kSteps];
      float f[Sl::kSteps];
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        const int e = e0 + u * Sl::kGroups + grp;
        const int64_t j = __shfl(my_col, e, kWave);
        f[u] = __shfl(my_dz, e, kWave);
        w[u].load(w_up_t + j * dm, sl);
      }
#pragma unroll
      for (int u = 0; u < Sl::kSteps; ++u) {
        const bool live = !CHECK || e0 + u * Sl::kGroups + grp < cnt;
        if (CHECK) w[u].keep(live, sl);
        w[u].fma32(acc, live ? f[u] : 0.f);
      }
    };
    int e0 = 0;
    for (; e0 + Sl::kEntries <= cnt; e0 += Sl::kEntries) step(e0, std::false_type{});
    if (e0 < cnt) step(e0, std::true_type{});
  }
  join_groups<P>(acc);
  store_joined<P>(dx + n * dm, sl, acc);
}

// Column slices: S of sw columns, S up to 8 (one per XCD) as long as a slice
// keeps 256 columns and whole chunks of every pass; P lanes of 16 nv columns
// cover one (nv = 0: too wide).  A width that divides only into slices too wide
// for a wave takes eight of whole chunks, the last one shorter (not empty: the
// other seven hold at most 7 (dm / 8 + 16) columns, under dm from 897 on).
SlicePlan slice_plan(int dm) {
  SlicePlan p{};
  if (dm > kMaxCols) return p;
  p.S = 8;
  while (p.S > 1 && (dm % (p.S * kCols) != 0 || dm / p.S < 256)) p.S /= 2;
  if (dm > p.S * kSliceCols) p.S = 8;
  p.sw = p.S == 1 ? dm : (dm + p.S * kCols - 1) / (p.S * kCols) * kCols;
  const int groups = (p.sw + kCols - 1) / kCols;
  p.P = groups <= 16 ? 16 : groups <= 32 ? 32 : kWave;
  p.nvl = groups <= kWave ? 1 : 2;
  return p;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct Space {
  unsigned long long* bits;  // [words][d_ff] (row, neuron) bitmap
  int2* row_at;              // {start, count} of each row's entries in the row order
  int32_t *lpre, *neuron_count, *neuron_off, *cols;
  Entry* ents;  // by neuron then row
  float* dz;    // by row then neuron: h until the neuron order is filled, then dz
  float* part;  // [S][entries] partial dots
  int64_t entries;
  size_t bytes;
};

Space carve(const Geometry& g, int64_t cap, void* ws) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t off = 0;
  auto take = [&](size_t bytes) -> void* {
    void* q = p == nullptr ? nullptr : p + off;
    off += align256(bytes);
    return q;
  };
  const size_t n = static_cast<size_t>(g.n_rows), dff = static_cast<size_t>(g.d_ff);
  const size_t words = dff * ((n + 63) / 64);
  Space w{};
  w.entries = bwd_max_entries(g, cap);
  const size_t ents = static_cast<size_t>(w.entries);
  w.bits = static_cast<unsigned long long*>(take(words * 8));
  w.row_at = static_cast<int2*>(take(n * sizeof(int2)));
  w.lpre = static_cast<int32_t*>(take(words * 4));
  w.neuron_count = static_cast<int32_t*>(take(dff * 4));
  w.neuron_off = static_cast<int32_t*>(take((dff + 1) * 4));
  w.cols = static_cast<int32_t*>(take(ents * 4));
  w.ents = static_cast<Entry*>(take(ents * sizeof(Entry)));
  w.dz = static_cast<float*>(take(ents * 4));
  w.part = static_cast<float*>(take(static_cast<size_t>(slice_plan(g.d_model).S) * ents * 4));
  w.bytes = off;
  return w;
}

unsigned blocks(int64_t items, int per) { return static_cast<unsigned>((items + per - 1) / per); }

// fn(P, NV, FULL) as types for the plan's widths.
template <typename Fn>
hipError_t with_plan(const SlicePlan& sp, int dm, Fn fn) {
  auto go = [&](auto p, auto nv) {
    return sp.sw == decltype(p)::value * decltype(nv)::value * kCols && sp.S * sp.sw == dm
               ? fn(p, nv, std::true_type{})
               : fn(p, nv, std::false_type{});
  };
  typedef std::integral_constant<int, 1> One;
  if (sp.nvl == 2)
    return go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (sp.nvl != 1) return hipErrorInvalidValue;
  if (sp.P == 16) return go(std::integral_constant<int, 16>{}, One{});
  if (sp.P == 32) return go(std::integral_constant<int, 32>{}, One{});
  return go(std::integral_constant<int, 64>{}, One{});
}

template <typename E>
hipError_t gather_passes(const Geometry& g, const Space& w, const BwdAct8& x8, const void* w_up_t,
                         const void* w_down, const void* dy, void* dx, float* dw_up_t, float* db,
                         float* dw_down, hipStream_t s) {
  const SlicePlan sp = slice_plan(g.d_model);
  const unsigned neurons = blocks(g.d_ff, kWaves), rows = blocks(g.n_rows, kWaves);
  auto log2 = [](int v) { return __builtin_ctz(static_cast<unsigned>(v)); };
  hipError_t e = with_plan(sp, g.d_model, [&](auto p, auto nv, auto full) {
    a8_down_kernel<E, decltype(p)::value, decltype(nv)::value, decltype(full)::value>
        <<<neurons * static_cast<unsigned>(sp.S), kThreads, 0, s>>>(
            w.neuron_off, w.ents, static_cast<const E*>(dy), static_cast<const E*>(w_down), g.d_ff,
            g.d_model, log2(sp.S), sp.sw, w.part, w.entries, dw_down);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  e = with_plan(sp, g.d_model, [&](auto p, auto nv, auto full) {
    a8_up_kernel<decltype(p)::value, decltype(nv)::value, decltype(full)::value>
        <<<neurons * static_cast<unsigned>(sp.S), kThreads, 0, s>>>(
            w.neuron_off, w.ents, x8.codes, x8.scales, act8_pitch(g.d_model),
            act8_blocks(g.d_model), w.part, w.entries, sp.S, g.d_ff, g.d_model, log2(sp.S), sp.sw,
            w.dz, dw_up_t, db);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return with_plan(sp, g.d_model, [&](auto p, auto nv, auto full) {
    a8_dx_kernel<E, decltype(p)::value, decltype(nv)::value, decltype(full)::value>
        <<<rows * static_cast<unsigned>(sp.S), kThreads, 0, s>>>(
            w.row_at, w.cols, w.dz, static_cast<const E*>(w_up_t), g.n_rows, g.d_model, log2(sp.S),
            sp.sw, static_cast<E*>(dx));
    return hipGetLastError();
  });
}

template <typename E>
hipError_t backward(const Geometry& g, const BwdHybrid& hy, const BwdAct8& x8, const void* w_up_t,
                    const void* w_down, const void* dy, const Space& w, void* dx, float* dw_up_t,
                    float* db, float* dw_down, hipStream_t s) {
  const int64_t n_words = (g.n_rows + 63) / 64;
  hipError_t e;
  auto zero = [&](void* p, int64_t vecs) {
    const int64_t most = int64_t{1} << 23;  // a launch holds fewer than 2^32 lanes
    a8_zero_kernel<<<blocks(std::min(vecs, most * kThreads), kThreads), kThreads, 0, s>>>(
        static_cast<uint4*>(p), vecs);
    return hipGetLastError();
  };
  if (g.n_rows == 0) {  // zero weight and bias gradients
    const int64_t weights = static_cast<int64_t>(g.d_ff) * g.d_model / 4;
    if ((e = zero(dw_up_t, weights)) != hipSuccess) return e;
    if ((e = zero(dw_down, weights)) != hipSuccess) return e;
    return zero(db, g.d_ff / 4);
  }
  // past the rows' workgroups, up to kDenseBlocks for the dense rows
  const unsigned row_blocks = blocks(g.n_rows, kWaves);
  const unsigned all_blocks =
      row_blocks + static_cast<unsigned>(std::clamp<int64_t>(hy.cap, 0, kDenseBlocks));
  a8_rows_kernel<E><<<all_blocks, kThreads, 0, s>>>(hy, g.n_rows, g.d_ff, g.tile, g.capacity,
                                                    g.n_tiles, row_blocks, w.row_at, w.cols, w.dz);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned slices = blocks(g.d_ff, kBitCols);
  a8_bits_kernel<<<static_cast<unsigned>(n_words) * slices, kScanThreads, 0, s>>>(
      w.row_at, w.cols, g.n_rows, g.d_ff, static_cast<int>(slices), w.bits);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  a8_prefix_kernel<<<blocks(g.d_ff, kWave), kScanThreads, 0, s>>>(w.bits, n_words, g.d_ff, w.lpre,
                                                                 w.neuron_count);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  a8_scan_kernel<<<1, kScanThreads, 0, s>>>(w.neuron_count, g.d_ff, w.neuron_off);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  a8_fill_kernel<<<all_blocks, kThreads, 0, s>>>(
      hy, g.n_rows, g.n_rows * g.n_tiles * g.capacity, g.d_ff, row_blocks, w.bits, w.lpre,
      w.neuron_off, w.row_at, w.cols, w.dz, w.ents);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return gather_passes<E>(g, w, x8, w_up_t, w_down, dy, dx, dw_up_t, db, dw_down, s);
}

}  // namespace

bool bwd_act8_supported(const Geometry& g) {
  // a launch holds fewer than 2^32 lanes: 64 per row or neuron and slice, one
  // per 128 bits of the bitmap
  const int64_t most = (int64_t{1} << 23) - 8;
  return slice_plan(g.d_model).nvl != 0 && g.n_rows < most && g.d_ff < most &&
         g.n_rows * g.d_ff < int64_t{1} << 38;
}

size_t bwd_act8_bytes(const Geometry& g, int64_t cap) { return carve(g, cap, nullptr).bytes; }

hipError_t launch_backward_act8(const Geometry& g, int elem_bytes, const BwdHybrid& hy,
                                const BwdAct8& x8, const void* w_up_t, const void* w_down,
                                const void* dy, void* ws, void* dx, float* dw_up_t, float* db,
                                float* dw_down, hipStream_t s) {
  const Space w = carve(g, hy.cap, ws);
  return elem_bytes == 2
             ? backward<uint16_t>(g, hy, x8, w_up_t, w_down, dy, w, dx, dw_up_t, db, dw_down, s)
             : backward<float>(g, hy, x8, w_up_t, w_down, dy, w, dx, dw_up_t, db, dw_down, s);
}

}  // namespace twell
