// The token embedding and its gradient.
//   out[n] = scale * table[tokens[n]]            (zeros where the id is outside)
//   dtable[v] = scale * sum over {n : tokens[n] = v}, n ascending, of dout[n]
// The lookup is one gather.  The gradient groups the tokens by id on the
// device: integer atomics count each id and give every token a place in its
// id's segment (in any order), and the kernel that sums a segment first puts
// its token numbers in ascending order.  Sums therefore run in a fixed order
// and repeat bit for bit, and no floating-point atomic is used.
#include "common.h"
#include "kernels.h"

namespace twell {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kEmbWaves = kEmbThreads / kWave;
constexpr int kEmbLoads = 4;  // 16-byte vectors per lane of a lookup item
constexpr unsigned kEmbMaxBlocks = 1u << 23;  // below 2^32 lanes

constexpr int kGradThreads = 1024;
constexpr int kGradWaves = kGradThreads / kWave;
constexpr int kAllocPer = 4;                         // ids per thread of the allocation
constexpr int kAllocIds = kGradThreads * kAllocPer;  // ids per workgroup
constexpr int kShort = kWave;                        // longest segment a wave takes
constexpr int kWindow = 16384;                       // token numbers per bitmap
constexpr int kLongLanes = 8;                        // lanes per row of a long segment
constexpr int kLongStreams = kGradThreads / kLongLanes;

// The id of token n, or -1 where it is outside [0, vocab).
template <typename I>
__device__ __forceinline__ int token_id(const I* __restrict__ tokens, int64_t n, int vocab) {
  const int64_t t = static_cast<int64_t>(tokens[n]);
  return t >= 0 && t < vocab ? static_cast<int>(t) : -1;
}

template <typename E>
__device__ __forceinline__ void unpack16(const uint4& v, float* f);
template <>
__device__ __forceinline__ void unpack16<uint16_t>(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack16<float>(const uint4& v, float* f) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}

template <typename E>
__device__ __forceinline__ uint4 scaled16(const uint4& v, float scale) {
  constexpr int V = 16 / sizeof(E);
  float f[V];
  unpack16<E>(v, f);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 2)
      w[i] = ElemTraits<E>::from_f32(f[2 * i] * scale) |
             static_cast<uint32_t>(ElemTraits<E>::from_f32(f[2 * i + 1] * scale)) << 16;
    else
      w[i] = __float_as_uint(f[i] * scale);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One wave per (token, chunk of kEmbLoads * 64 vectors).  Bound by HBM: rows
// that repeat come from the caches, the output is stored past them.
template <typename E, typename I>
__global__ __launch_bounds__(kEmbThreads) void embed_forward_kernel(
    const E* __restrict__ table, const I* __restrict__ tokens, int64_t n_items, int chunks, int d,
    int vocab, float scale, E* __restrict__ out) {
  constexpr int V = 16 / sizeof(E);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kEmbWaves;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kEmbWaves + threadIdx.x / kWave; i < n_items;
       i += stride) {
    const int64_t n = i / chunks;
    const int c0 = (static_cast<int>(i - n * chunks) * (kEmbLoads * kWave) + lane_id()) * V;
    const int id = token_id(tokens, n, vocab);
    const E* src = table + static_cast<int64_t>(max(id, 0)) * d;
    uint4 v[kEmbLoads];
#pragma unroll
    for (int k = 0; k < kEmbLoads; ++k) {
      const int c = c0 + k * kWave * V;
      v[k] = id >= 0 && c < d ? *reinterpret_cast<const uint4*>(src + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kEmbLoads; ++k) {
      const int c = c0 + k * kWave * V;
      if (c < d)
        store_once(out + n * d + c, id >= 0 ? scaled16<E>(v[k], scale) : make_uint4(0, 0, 0, 0));
    }
  }
}

__global__ __launch_bounds__(kEmbThreads) void embed_clear_kernel(int32_t* __restrict__ p,
                                                                  int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kEmbThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kEmbThreads)
    p[i] = 0;
}

// count[id] = tokens of that id; pos[n] = a place of its own within the id.
template <typename I>
__global__ __launch_bounds__(kEmbThreads) void embed_count_kernel(const I* __restrict__ tokens,
                                                                  int64_t n_tokens, int vocab,
                                                                  int32_t* __restrict__ count,
                                                                  int32_t* __restrict__ pos) {
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * kEmbThreads + threadIdx.x; n < n_tokens;
       n += static_cast<int64_t>(gridDim.x) * kEmbThreads) {
    const int id = token_id(tokens, n, vocab);
    if (id >= 0) pos[n] = atomicAdd(count + id, 1);
  }
}

// Zero vector v (4 floats) of dtable unless its row's id has a token: one
// vector per lane and workgroups in the order of memory.
__device__ __forceinline__ void zero_unused(const int32_t* __restrict__ count, int64_t v,
                                            int64_t end, int d, float* __restrict__ dtable) {
  if (v >= end || count[v / (d / 4)] != 0) return;
  store_once(dtable + v * 4, make_uint4(0, 0, 0, 0));
}

// Workgroups below n_alloc: each id's first place (base), and the lists of the
// ids with at most kShort tokens and of those with more, from the counts.
// Segments and list entries are handed out with one atomic per workgroup, so
// their order varies; no result depends on it.  The others zero the unused
// rows' vectors below `half` meanwhile.
__global__ __launch_bounds__(kGradThreads) void embed_alloc_kernel(
    const EmbedGradBufs b, int vocab, int n_alloc, int d, int64_t half,
    float* __restrict__ dtable) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  if (static_cast<int>(blockIdx.x) >= n_alloc) {
    zero_unused(b.count, static_cast<int64_t>(blockIdx.x - n_alloc) * kGradThreads + tid, half, d,
                dtable);
    return;
  }
  __shared__ int tot[3][kGradWaves];
  __shared__ int first[3];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kAllocIds + tid * kAllocPer;
  int c[kAllocPer], mine[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < kAllocPer; ++k) {
    c[k] = v0 + k < vocab ? b.count[v0 + k] : 0;
    mine[0] += c[k];
    mine[1] += c[k] > 0 && c[k] <= kShort;
    mine[2] += c[k] > kShort;
  }
  int at[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    int sc = mine[q];
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int u = __shfl_up(sc, o, kWave);
      if (lane >= o) sc += u;
    }
    if (lane == kWave - 1) tot[q][wave] = sc;
    at[q] = sc - mine[q];
  }
  __syncthreads();
  if (tid < 3) {
    int all = 0;
    for (int w = 0; w < kGradWaves; ++w) all += tot[tid][w];
    first[tid] = all > 0 ? atomicAdd(b.counters + tid, all) : 0;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    at[q] += first[q];
    for (int w = 0; w < wave; ++w) at[q] += tot[q][w];
  }
#pragma unroll
  for (int k = 0; k < kAllocPer; ++k) {
    if (c[k] == 0) continue;
    b.base[v0 + k] = at[0];
    at[0] += c[k];
    if (c[k] <= kShort) b.short_ids[at[1]++] = static_cast<int32_t>(v0 + k);
    else b.long_ids[at[2]++] = static_cast<int32_t>(v0 + k);
  }
}

// Workgroups below n_place put the token numbers in their segments; the others
// zero the unused rows' vectors from `half` on.
template <typename I>
__global__ __launch_bounds__(kGradThreads) void embed_place_kernel(
    const EmbedGradBufs b, const I* __restrict__ tokens, int64_t n_tokens, int vocab, int n_place,
    int d, int64_t half, float* __restrict__ dtable) {
  if (static_cast<int>(blockIdx.x) >= n_place) {
    zero_unused(b.count,
                half + static_cast<int64_t>(blockIdx.x - n_place) * kGradThreads + threadIdx.x,
                static_cast<int64_t>(vocab) * (d / 4), d, dtable);
    return;
  }
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * kGradThreads + threadIdx.x; n < n_tokens;
       n += static_cast<int64_t>(n_place) * kGradThreads) {
    const int id = token_id(tokens, n, vocab);
    if (id >= 0) b.perm[b.base[id] + b.pos[n]] = static_cast<int32_t>(n);
  }
}

// acc += rows ranks r, r + step, ... below cnt of the list, columns c..c + V.
template <typename E, typename Row>
__device__ __forceinline__ void add_rows(const E* __restrict__ dout, int d, int c, int r, int step,
                                         int cnt, Row row, float* acc) {
  constexpr int V = 16 / sizeof(E);
  constexpr int U = 4;
  for (; r < cnt; r += U * step) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = row(min(r + u * step, cnt - 1));
      v[u] = *reinterpret_cast<const uint4*>(dout + n * d + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r + u * step >= cnt) break;
      float f[V];
      unpack16<E>(v[u], f);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += f[i];
    }
  }
}

// The rows of the used ids.  Items [0, n_long * long_slices): a workgroup sums
// one slice of kLongLanes * V columns of a long segment: per window of kWindow
// token numbers it sets the segment's tokens in a bitmap (order-free), numbers
// its bits by a scan, lists them in ascending order, and stream q of
// kLongStreams adds the listed rows q, q + kLongStreams, ...; the streams'
// sums are added in a fixed tree.  Then items of the short segments: a wave
// sums one slice of 64 * V columns, its token numbers ranked in registers.
template <typename E>
__global__ __launch_bounds__(kGradThreads) void embed_rows_kernel(
    const EmbedGradBufs b, const E* __restrict__ dout, int64_t n_tokens, int d, float scale,
    float* __restrict__ dtable) {
  constexpr int V = 16 / sizeof(E);
  __shared__ uint32_t bits[kWindow / 32];
  __shared__ uint16_t list[kWindow];
  __shared__ int wave_tot[kGradWaves];
  __shared__ float part[kGradWaves][kLongLanes * V];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int long_slices = (d + kLongLanes * V - 1) / (kLongLanes * V);
  const int64_t n_long = static_cast<int64_t>(b.counters[2]) * long_slices;
  for (int64_t item = blockIdx.x; item < n_long; item += gridDim.x) {
    const int id = b.long_ids[item / long_slices];
    const int c = (static_cast<int>(item % long_slices) * kLongLanes + tid % kLongLanes) * V;
    const int cc = min(c, d - V);
    const int L = b.count[id];
    const int32_t* seg = b.perm + b.base[id];
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int64_t w0 = 0; w0 < n_tokens; w0 += kWindow) {
      if (tid < kWindow / 32) bits[tid] = 0;
      __syncthreads();
      for (int k = tid; k < L; k += kGradThreads) {
        const int64_t o = seg[k] - w0;
        if (o >= 0 && o < kWindow) atomicOr(bits + o / 32, 1u << (o % 32));
      }
      __syncthreads();
      uint32_t m = tid < kWindow / 32 ? bits[tid] : 0;
      const int pc = __popc(m);
      int sc = pc;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(sc, o, kWave);
        if (lane >= o) sc += u;
      }
      if (lane == kWave - 1) wave_tot[wave] = sc;
      __syncthreads();
      int at = sc - pc, cnt = 0;
      for (int w = 0; w < kGradWaves; ++w) {
        at += w < wave ? wave_tot[w] : 0;
        cnt += wave_tot[w];
      }
      for (; m != 0; m &= m - 1) list[at++] = static_cast<uint16_t>(tid * 32 + __ffs(m) - 1);
      __syncthreads();
      add_rows<E>(dout, d, cc, tid / kLongLanes, kLongStreams, cnt,
                  [&](int r) { return w0 + list[r]; }, acc);
      __syncthreads();  // the next window rewrites bits and list
    }
#pragma unroll
    for (int o = kLongLanes; o < kWave; o <<= 1)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
    if (lane < kLongLanes)
#pragma unroll
      for (int i = 0; i < V; ++i) part[wave][lane * V + i] = acc[i];
    __syncthreads();
    const int col = static_cast<int>(item % long_slices) * kLongLanes * V + tid;
    if (tid < kLongLanes * V && col < d) {
      float s = 0.f;
      for (int w = 0; w < kGradWaves; ++w) s += part[w][tid];
      dtable[static_cast<int64_t>(id) * d + col] = s * scale;
    }
    __syncthreads();
  }
  const int slices = (d + kWave * V - 1) / (kWave * V);
  const int64_t n_short = static_cast<int64_t>(b.counters[1]) * slices;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kGradWaves + wave; item < n_short;
       item += static_cast<int64_t>(gridDim.x) * kGradWaves) {
    const int id = b.short_ids[item / slices];
    const int c = (static_cast<int>(item % slices) * kWave + lane) * V;
    const int cc = min(c, d - V);
    const int cnt = b.count[id];
    const int32_t* seg = b.perm + b.base[id];
    const int mine = seg[min(lane, cnt - 1)];
    int rank = 0;
    for (int k = 0; k < cnt; ++k) rank += __shfl(mine, k, kWave) < mine;
    // lane r takes the token number of rank r (lanes past the segment push to
    // lanes past it)
    const int sorted = __builtin_amdgcn_ds_permute((lane < cnt ? rank : lane) * 4, mine);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    add_rows<E>(dout, d, cc, 0, 1, cnt,
                [&](int r) { return static_cast<int64_t>(__shfl(sorted, r, kWave)); }, acc);
    if (c < d) {
      float* row = dtable + static_cast<int64_t>(id) * d + c;
#pragma unroll
      for (int i = 0; i < V; i += 4)
        *reinterpret_cast<float4*>(row + i) = make_float4(
            acc[i] * scale, acc[i + 1] * scale, acc[i + 2] * scale, acc[i + 3] * scale);
    }
  }
}

unsigned blocks_for(int64_t items, int per, unsigned most) {
  const int64_t b = (items + per - 1) / per;
  return static_cast<unsigned>(b < 1 ? 1 : b < most ? b : most);
}

}  // namespace

EmbedGradBufs embed_grad_carve(int64_t n_tokens, int vocab, void* ws) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t off = 0;
  auto take = [&](int64_t ints) {
    int32_t* q = p == nullptr ? nullptr : reinterpret_cast<int32_t*>(p + off);
    off += (static_cast<size_t>(ints) * 4 + 255) / 256 * 256;
    return q;
  };
  EmbedGradBufs b{};
  b.counters = take(4);
  b.count = take(vocab);
  b.clear_ints = static_cast<int64_t>(off / 4);
  b.base = take(vocab);
  b.pos = take(n_tokens);
  b.perm = take(n_tokens);
  b.short_ids = take(n_tokens < vocab ? n_tokens : vocab);
  b.long_ids = take(n_tokens / (kShort + 1) + 1);
  b.bytes = off;
  return b;
}

hipError_t launch_embed_forward(int64_t n, int vocab, int d, int elem_bytes, int index_bytes,
                                float scale, const void* table, const void* tokens, void* out,
                                hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int per = kEmbLoads * kWave * 16 / elem_bytes;
  const int chunks = (d + per - 1) / per;
  const int64_t items = n * chunks;
  const unsigned grid = blocks_for(items, kEmbWaves, kEmbMaxBlocks);
  auto go = [&](auto e, auto i) {
    typedef decltype(e) E;
    typedef decltype(i) I;
    embed_forward_kernel<E, I><<<grid, kEmbThreads, 0, s>>>(
        static_cast<const E*>(table), static_cast<const I*>(tokens), items, chunks, d, vocab,
        scale, static_cast<E*>(out));
    return hipGetLastError();
  };
  if (elem_bytes == 2)
    return index_bytes == 8 ? go(uint16_t{}, int64_t{}) : go(uint16_t{}, int32_t{});
  return index_bytes == 8 ? go(float{}, int64_t{}) : go(float{}, int32_t{});
}

hipError_t launch_embed_backward(int64_t n, int vocab, int d, int elem_bytes, int index_bytes,
                                 float scale, const void* dout, const void* tokens,
                                 const EmbedGradBufs& b, float* dtable, hipStream_t s) {
  hipError_t e;
  embed_clear_kernel<<<blocks_for(b.clear_ints, kEmbThreads, 2048), kEmbThreads, 0, s>>>(
      b.counters, b.clear_ints);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned cgrid = blocks_for(n, kEmbThreads, 4096);
  if (index_bytes == 8)
    embed_count_kernel<<<cgrid, kEmbThreads, 0, s>>>(static_cast<const int64_t*>(tokens), n, vocab,
                                                     b.count, b.pos);
  else
    embed_count_kernel<<<cgrid, kEmbThreads, 0, s>>>(static_cast<const int32_t*>(tokens), n, vocab,
                                                     b.count, b.pos);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t vectors = static_cast<int64_t>(vocab) * (d / 4), half = vectors / 2;
  const unsigned fill = static_cast<unsigned>((vectors - half + kGradThreads - 1) / kGradThreads);
  const unsigned n_alloc = blocks_for(vocab, kAllocIds, 1u << 30);
  embed_alloc_kernel<<<n_alloc + fill, kGradThreads, 0, s>>>(b, vocab, static_cast<int>(n_alloc),
                                                             d, half, dtable);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const unsigned n_place = blocks_for(n, kGradThreads, 1024);
  if (index_bytes == 8)
    embed_place_kernel<<<n_place + fill, kGradThreads, 0, s>>>(
        b, static_cast<const int64_t*>(tokens), n, vocab, static_cast<int>(n_place), d, half,
        dtable);
  else
    embed_place_kernel<<<n_place + fill, kGradThreads, 0, s>>>(
        b, static_cast<const int32_t*>(tokens), n, vocab, static_cast<int>(n_place), d, half,
        dtable);
  if ((e = hipGetLastError()) != hipSuccess || n == 0) return e;
  const int V = 16 / elem_bytes;
  const int64_t items = (n < vocab ? n : vocab) * ((d + kWave * V - 1) / (kWave * V));
  const unsigned grid = blocks_for(items, kGradWaves, 2048);
  if (elem_bytes == 2)
    embed_rows_kernel<<<grid, kGradThreads, 0, s>>>(b, static_cast<const uint16_t*>(dout), n, d,
                                                    scale, dtable);
  else
    embed_rows_kernel<<<grid, kGradThreads, 0, s>>>(b, static_cast<const float*>(dout), n, d,
                                                    scale, dtable);
  return hipGetLastError();
}

}  // namespace twell
