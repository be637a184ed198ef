// The token embedding and its gradient.
//   out[n] = scale * table[tokens[n]]            (zeros where the id is outside)
//   dtable[v] = scale * sum over {n : tokens[n] = v}, n ascending, of dout[n]
// The lookup is one gather.  The gradient groups the tokens by id on the
// device: integer atomics count each id and give every token a place in its
// id's segment (in any order), and the kernel that sums a segment first puts
// its token numbers in ascending order.  Sums therefore run in a fixed order
// and repeat bit for bit, and no floating-point atomic is used.
#include "common.h"
#include "stream_ops.h"
#include "train_kernels.h"

namespace twell {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kEmbWaves = kEmbThreads / kWave;
constexpr int kEmbLoads = 4;  // 16-byte vectors per lane of a lookup item
constexpr unsigned kEmbMaxBlocks = 1u << 23;  // below 2^32 lanes

constexpr int kGradThreads = 256;
constexpr int kGradWaves = kGradThreads / kWave;
constexpr int kAllocPer = 16;                        // ids per thread of the allocation
constexpr int kAllocIds = kGradThreads * kAllocPer;  // ids per workgroup
constexpr int kOrderThreads = 1024;
constexpr int kOrderWaves = kOrderThreads / kWave;
// The one-workgroup sort: at most kSortMax tokens, a token's number below its
// id in one 32-bit key, kSortBits bits of it per pass.
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortNBits = 13;
constexpr int kSortMax = 1 << kSortNBits;
constexpr int kSortPer = kSortMax / kSortThreads;    // keys per lane
constexpr int kSortBits = 6;
constexpr int kSortBins = 1 << kSortBits;
static_assert(kSortBins * kSortWaves == kSortThreads, "a thread per (bin, wave)");
static_assert(kOrderThreads <= kEmbedGradStep, "the widest step over an id's tokens");
constexpr int kWindow = 1 << 19;                     // token numbers per bitmap (64 KB)
// Segments by length: a wave takes one of at most kShort tokens row after row,
// one of at most kMedium as 8 streams of rows (8 lanes a row), and a workgroup
// any longer one as kLongStreams streams.
constexpr int kShort = 8;
constexpr int kMedium = kWave;
constexpr int kStreamLanes = 8;
constexpr int kWaveStreams = kWave / kStreamLanes;
constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / kWave;
constexpr int kLongStreams = kRowThreads / kStreamLanes;
constexpr int kRowBlocks = 8192;  // at most, of the rows' launch (2048: 50 us, 4096: 45, 8192: 43
                                 // for 8192 tokens of 4096 float32)

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
// that repeat come from the caches, the output is stored past them.  16384
// tokens of 8192 bf16: 70 us, 5.4 TB/s (one vector per lane: 95 us, the id's
// read then stands before each; 2: 78, 8: 74).
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

// The table's gradient is mostly rows of zeros (ids no token has), and
// zeroing them is most of the time: the launches that group the tokens carry
// it, in workgroups past their own n_own, one 16-byte vector per lane in the
// order of memory (a 32768 x 2048 table in 42 us, 6.3 TB/s; workgroups of 1024
// lanes 47 us).  Before the counts are known (`count` null) a share also
// zeroes used rows, which the last launch then overwrites.
struct ZeroShare {
  int64_t begin, end;    // vectors of dtable
  const int32_t* count;  // skip the rows of used ids, or null
};
__device__ __forceinline__ void zero_share(const ZeroShare& z, int64_t block, int d,
                                           float* __restrict__ dtable) {
  const int64_t v = z.begin + block * blockDim.x + threadIdx.x;
  if (v >= z.end || (z.count != nullptr && z.count[v / (d / 4)] != 0)) return;
  store_once(dtable + v * 4, make_uint4(0, 0, 0, 0));
}

__global__ __launch_bounds__(kGradThreads) void embed_clear_kernel(int32_t* __restrict__ p,
                                                                   int64_t n, int n_own,
                                                                   ZeroShare z, int d,
                                                                   float* __restrict__ dtable) {
  if (static_cast<int>(blockIdx.x) >= n_own) {
    zero_share(z, blockIdx.x - n_own, d, dtable);
    return;
  }
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kGradThreads + threadIdx.x;
  if (i < n) p[i] = 0;
}

// count[id] = tokens of that id; pos[n] = a place of its own within the id.
template <typename I>
__global__ __launch_bounds__(kGradThreads) void embed_count_kernel(
    const I* __restrict__ tokens, int64_t n_tokens, int vocab, int32_t* __restrict__ count,
    int32_t* __restrict__ pos, int n_own, ZeroShare z, int d, float* __restrict__ dtable) {
  if (static_cast<int>(blockIdx.x) >= n_own) {
    zero_share(z, blockIdx.x - n_own, d, dtable);
    return;
  }
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kGradThreads + threadIdx.x;
  if (n >= n_tokens) return;
  const int id = token_id(tokens, n, vocab);
  if (id >= 0) pos[n] = atomicAdd(count + id, 1);
}

// Each id's first place (base) and the lists of the short, medium and long
// ids, from the counts.  Segments and list entries are handed out with one
// atomic per workgroup, so their order varies; no result depends on it.
__global__ __launch_bounds__(kGradThreads) void embed_alloc_kernel(
    const EmbedGradBufs b, int vocab, int n_own, ZeroShare z, int d, float* __restrict__ dtable) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  if (static_cast<int>(blockIdx.x) >= n_own) {
    zero_share(z, blockIdx.x - n_own, d, dtable);
    return;
  }
  __shared__ int tot[4][kGradWaves];
  __shared__ int first[4];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kAllocIds + tid * kAllocPer;
  int c[kAllocPer], mine[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kAllocPer; ++k) {
    c[k] = v0 + k < vocab ? b.count[v0 + k] : 0;
    mine[0] += c[k];
    mine[1] += c[k] > 0 && c[k] <= kShort;
    mine[2] += c[k] > kShort && c[k] <= kMedium;
    mine[3] += c[k] > kMedium;
  }
  int at[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
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
  if (tid < 4) {
    int all = 0;
    for (int w = 0; w < kGradWaves; ++w) all += tot[tid][w];
    first[tid] = all > 0 ? atomicAdd(b.counters + tid, all) : 0;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    at[q] += first[q];
    for (int w = 0; w < wave; ++w) at[q] += tot[q][w];
  }
#pragma unroll
  for (int k = 0; k < kAllocPer; ++k) {
    if (c[k] == 0) continue;
    const int32_t id = static_cast<int32_t>(v0 + k);
    b.base[id] = at[0];
    const int4 seg = make_int4(id, at[0], c[k], 0);
    at[0] += c[k];
    if (c[k] <= kShort) b.short_segs[at[1]++] = seg;
    else if (c[k] <= kMedium) b.medium_segs[at[2]++] = seg;
    else b.long_segs[at[3]++] = seg;
  }
}

// The token numbers into their segments.
template <typename I>
__global__ __launch_bounds__(kGradThreads) void embed_place_kernel(
    const EmbedGradBufs b, const I* __restrict__ tokens, int64_t n_tokens, int vocab, int n_own,
    ZeroShare z, int d, float* __restrict__ dtable) {
  if (static_cast<int>(blockIdx.x) >= n_own) {
    zero_share(z, blockIdx.x - n_own, d, dtable);
    return;
  }
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kGradThreads + threadIdx.x;
  if (n >= n_tokens) return;
  const int id = token_id(tokens, n, vocab);
  if (id >= 0) b.perm[b.base[id] + b.pos[n]] = static_cast<int32_t>(n);
}

// The token numbers of each long segment in ascending order, into `sorted`
// (where the places were): a workgroup sets them in a bitmap of kWindow token
// numbers (order-free), numbers its bits by a scan and lists them.
__global__ __launch_bounds__(kOrderThreads) void embed_order_kernel(
    const EmbedGradBufs b, int64_t n_tokens) {
  __shared__ uint32_t bits[kWindow / 32];
  __shared__ int wave_tot[kOrderWaves];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int n_long = b.counters[3];
  for (int i = blockIdx.x; i < n_long; i += gridDim.x) {
    const int4 seg = b.long_segs[i];
    int32_t* out = b.pos + seg.y;
    for (int64_t w0 = 0; w0 < n_tokens; w0 += kWindow) {
      const int words = static_cast<int>((min(n_tokens - w0, int64_t{kWindow}) + 31) / 32);
      const int per = (words + kOrderThreads - 1) / kOrderThreads;  // words per thread
      for (int k = tid; k < words; k += kOrderThreads) bits[k] = 0;
      __syncthreads();
      for (int k = tid; k < seg.z; k += kOrderThreads) {
        const int64_t o = b.perm[seg.y + k] - w0;
        if (o >= 0 && o < kWindow) atomicOr(bits + o / 32, 1u << (o % 32));
      }
      __syncthreads();
      int pc = 0;
      for (int k = tid * per; k < min((tid + 1) * per, words); ++k) pc += __popc(bits[k]);
      int sc = pc;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(sc, o, kWave);
        if (lane >= o) sc += u;
      }
      if (lane == kWave - 1) wave_tot[wave] = sc;
      __syncthreads();
      int at = sc - pc, all = 0;
      for (int w = 0; w < kOrderWaves; ++w) {
        at += w < wave ? wave_tot[w] : 0;
        all += wave_tot[w];
      }
      for (int k = tid * per; k < min((tid + 1) * per, words); ++k)
        for (uint32_t m = bits[k]; m != 0; m &= m - 1)
          out[at++] = static_cast<int32_t>(w0 + k * 32 + __builtin_ctz(m));
      out += all;
      __syncthreads();  // the next window rewrites bits and wave_tot
    }
  }
}

// Up to kSortMax tokens are grouped by one workgroup, in one launch that zeroes
// the whole table meanwhile (32768 x 2048: 44 us, 6.1 TB/s of zeros): a stable
// radix sort of the keys (id, token number) by id, then the segments between
// changes of id.  Key i = wave * chunk +
// round * 64 + lane keeps the tokens' order; a pass ranks a wave's keys of equal
// digit by ballots and a running count, numbers (digit, wave) by a scan, and
// moves the keys through LDS.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(
    const EmbedGradBufs b, const I* __restrict__ tokens, int n_tokens, int vocab, int id_bits,
    ZeroShare z, int d, float* __restrict__ dtable) {
  __shared__ uint32_t keys[kSortMax];
  __shared__ int cnt[kSortWaves][kSortBins];
  __shared__ int wave_tot[kSortWaves];
  __shared__ int lists[4];
  if (blockIdx.x > 0) {
    zero_share(z, blockIdx.x - 1, d, dtable);
    return;
  }
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int rounds = (n_tokens + kSortThreads - 1) / kSortThreads;
  const int chunk = rounds * kWave, total = rounds * kSortThreads;
  // exclusive sum over the workgroup's threads
  auto block_scan = [&](int v) {
    int sc = v;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int u = __shfl_up(sc, o, kWave);
      if (lane >= o) sc += u;
    }
    if (lane == kWave - 1) wave_tot[wave] = sc;
    __syncthreads();
    int at = sc - v;
    for (int w = 0; w < wave; ++w) at += wave_tot[w];
    __syncthreads();
    return at;
  };
  uint32_t key[kSortPer];
#pragma unroll
  for (int r = 0; r < kSortPer; ++r) {
    if (r >= rounds) break;
    const int n = wave * chunk + r * kWave + lane;
    const int id = n < n_tokens ? token_id(tokens, n, vocab) : -1;
    // padding sorts behind the last id
    key[r] = static_cast<uint32_t>(id >= 0 ? id : vocab) << kSortNBits |
             static_cast<uint32_t>(n & (kSortMax - 1));
  }
  for (int bit = 0; bit < id_bits; bit += kSortBits) {
    const int shift = kSortNBits + bit;
    cnt[wave][lane] = 0;
    __builtin_amdgcn_wave_barrier();
    int rank[kSortPer];
#pragma unroll
    for (int r = 0; r < kSortPer; ++r) {
      if (r >= rounds) break;
      const int bin = key[r] >> shift & (kSortBins - 1);
      uint64_t same = ~0ull;
#pragma unroll
      for (int k = 0; k < kSortBits; ++k) {
        const bool set = (bin >> k & 1) != 0;
        const uint64_t m = wave_ballot(set);
        same &= set ? m : ~m;
      }
      const int before = cnt[wave][bin], below = popc_below(same);
      rank[r] = before + below;
      __builtin_amdgcn_wave_barrier();
      if (below == 0) cnt[wave][bin] = before + popc64(same);
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    const int mine = cnt[tid % kSortWaves][tid / kSortWaves];
    const int first = block_scan(mine);
    cnt[tid % kSortWaves][tid / kSortWaves] = first;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortPer; ++r) {
      if (r >= rounds) break;
      keys[cnt[wave][key[r] >> shift & (kSortBins - 1)] + rank[r]] = key[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortPer; ++r) {
      if (r >= rounds) break;
      key[r] = keys[wave * chunk + r * kWave + lane];
    }
    __syncthreads();
  }
  // the sorted keys, and in them the segments: a wave numbers the changes of id
  // in its own chunk by ballots, after those of the waves before it
#pragma unroll
  for (int r = 0; r < kSortPer; ++r) {
    if (r >= rounds) break;
    const int i = wave * chunk + r * kWave + lane;
    keys[i] = key[r];
    if (i < n_tokens) b.perm[i] = static_cast<int32_t>(key[r] & (kSortMax - 1));
  }
  if (tid < 4) lists[tid] = 0;
  __syncthreads();
  uint32_t heads = 0;  // bit r: this lane's key of round r starts a segment
  int n_heads = 0;     // the wave's
#pragma unroll
  for (int r = 0; r < kSortPer; ++r) {
    if (r >= rounds) break;
    const int i = wave * chunk + r * kWave + lane;
    const bool head = i == 0 || key[r] >> kSortNBits != keys[i - 1] >> kSortNBits;
    heads |= head ? 1u << r : 0u;
    n_heads += popc64(wave_ballot(head));
  }
  if (lane == 0) wave_tot[wave] = n_heads;
  __syncthreads();
  int at = 0, n_segs = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    at += w < wave ? wave_tot[w] : 0;
    n_segs += wave_tot[w];
  }
  // b.pos: where each segment starts, and the end
  for (int r = 0; r < rounds; ++r) {
    const bool head = (heads >> r & 1) != 0;
    const uint64_t m = wave_ballot(head);
    if (head) b.pos[at + popc_below(m)] = wave * chunk + r * kWave + lane;
    at += popc64(m);
  }
  if (tid == 0) b.pos[n_segs] = total;
  __threadfence_block();
  __syncthreads();
  for (int k = tid; k < n_segs; k += kSortThreads) {
    const int i = b.pos[k], c = b.pos[k + 1] - i;
    const int id = static_cast<int>(keys[i] >> kSortNBits);
    if (id >= vocab) continue;  // padding
    const int4 seg = make_int4(id, i, c, 0);
    if (c <= kShort) b.short_segs[atomicAdd(lists + 1, 1)] = seg;
    else if (c <= kMedium) b.medium_segs[atomicAdd(lists + 2, 1)] = seg;
    else b.long_segs[atomicAdd(lists + 3, 1)] = seg;
  }
  __syncthreads();
  if (tid > 0 && tid < 4) b.counters[tid] = lists[tid];
}

// acc += the rows of ranks r, r + step, ... below cnt, columns c .. c + V:
// U rows in flight, added in rank order.
template <typename E, int U, typename Row>
__device__ __forceinline__ void add_rows(const E* __restrict__ dout, int d, int c, int r, int step,
                                         int cnt, Row row, float* acc) {
  constexpr int V = 16 / sizeof(E);
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

// scale * acc to V columns of a row.
template <int V>
__device__ __forceinline__ void put_row(float* to, const float* acc, float scale) {
#pragma unroll
  for (int i = 0; i < V; i += 4)
    *reinterpret_cast<float4*>(to + i) = make_float4(acc[i] * scale, acc[i + 1] * scale,
                                                     acc[i + 2] * scale, acc[i + 3] * scale);
}

// Token numbers of a segment of cnt <= 64, one per lane and in the order they
// came, to ascending order: lane r gets the r-th smallest.
__device__ __forceinline__ int sorted_segment(int mine, int cnt) {
  const int lane = lane_id();
  int rank = 0;
  for (int k = 0; k < cnt; ++k) rank += __builtin_amdgcn_readlane(mine, k) < mine;
  // lanes past the segment push to lanes past it
  return __builtin_amdgcn_ds_permute((lane < cnt ? rank : lane) * 4, mine);
}

// The streams' sums, added over the lanes of a wave in a fixed order.
template <int V>
__device__ __forceinline__ void join_streams(float* acc) {
#pragma unroll
  for (int o = kStreamLanes; o < kWave; o <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += __shfl_xor(acc[i], o, kWave);
}

// The rows of the used ids, as items (segment, slice of columns): a
// workgroup's for long segments, whose streams' sums meet in LDS; a wave's for
// medium and short ones, whose token numbers are ranked in registers.
// Bound by the latency of dout's rows for few tokens and by HBM for many: 4096
// tokens of 2048 bf16 14 us, 8192 of 4096 float32 43 us (4.4 TB/s).
template <typename E>
__global__ __launch_bounds__(kRowThreads) void embed_rows_kernel(
    const EmbedGradBufs b, const int32_t* __restrict__ long_order, const E* __restrict__ dout,
    int d, float scale, float* __restrict__ dtable) {
  constexpr int V = 16 / sizeof(E);
  constexpr int kStreamCols = kStreamLanes * V, kShortCols = kWave * V;
  __shared__ float part[kRowWaves][kStreamCols];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  float acc[V];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
  };
  const int stream_slices = (d - 1) / kStreamCols + 1;
  const int64_t n_long = static_cast<int64_t>(b.counters[3]) * stream_slices;
  for (int64_t item = blockIdx.x; item < n_long; item += gridDim.x) {
    const int4 seg = b.long_segs[item / stream_slices];
    const int c0 = static_cast<int>(item % stream_slices) * kStreamCols;
    const int32_t* sorted = long_order + seg.y;
    clear();
    add_rows<E, 8>(dout, d, min(c0 + tid % kStreamLanes * V, d - V), tid / kStreamLanes,
                   kLongStreams, seg.z, [&](int r) { return static_cast<int64_t>(sorted[r]); },
                   acc);
    join_streams<V>(acc);
    if (lane < kStreamLanes)
#pragma unroll
      for (int i = 0; i < V; ++i) part[wave][lane * V + i] = acc[i];
    __syncthreads();
    if (tid < kStreamCols && c0 + tid < d) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kRowWaves; ++w) s += part[w][tid];
      dtable[static_cast<int64_t>(seg.x) * d + c0 + tid] = s * scale;
    }
    __syncthreads();
  }
  // a wave's items: (medium segment, slice), then (short segment, slice).  The
  // next item's token numbers and the one after's segment are read while an
  // item is summed, so the three dependent reads of an item do not add up.
  const int64_t waves = static_cast<int64_t>(gridDim.x) * kRowWaves;
  const int short_slices = (d - 1) / kShortCols + 1;
  const int64_t n_medium = static_cast<int64_t>(b.counters[2]) * stream_slices;
  const int64_t n_items = n_medium + static_cast<int64_t>(b.counters[1]) * short_slices;
  struct Item {
    int4 seg = make_int4(0, 0, 0, 0);
    int slice = 0;
  };
  auto item_at = [&](int64_t i) {
    Item t;
    if (i >= n_items) return t;
    const bool medium = i < n_medium;
    const int64_t k = medium ? i : i - n_medium;
    const int slices = medium ? stream_slices : short_slices;
    const int64_t q = k >> 32 ? k / slices : static_cast<uint32_t>(k) / static_cast<uint32_t>(slices);
    t.seg = (medium ? b.medium_segs : b.short_segs)[q];
    t.slice = static_cast<int>(k - q * slices);
    return t;
  };
  auto tokens_of = [&](const Item& t) {
    return t.seg.z > 0 ? b.perm[t.seg.y + min(lane, t.seg.z - 1)] : 0;
  };
  int64_t i = static_cast<int64_t>(blockIdx.x) * kRowWaves + wave;
  Item now = item_at(i), next = item_at(i + waves);
  int tokens = tokens_of(now);
  for (; i < n_items; i += waves) {
    const int after = tokens_of(next);
    const Item third = item_at(i + 2 * waves);
    const int cnt = __builtin_amdgcn_readfirstlane(now.seg.z);
    const int sorted = sorted_segment(tokens, cnt);
    float* row = dtable + static_cast<int64_t>(now.seg.x) * d;
    clear();
    if (i < n_medium) {
      const int c = (now.slice * kStreamLanes + lane % kStreamLanes) * V;
      // every lane runs the same number of steps, for the shuffles
      constexpr int U = 4;
      for (int r0 = 0; r0 < cnt; r0 += U * kWaveStreams) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * kWaveStreams + lane / kStreamLanes;
          const int64_t n = __shfl(sorted, min(r, cnt - 1), kWave);
          v[u] = *reinterpret_cast<const uint4*>(dout + n * d + min(c, d - V));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (r0 + u * kWaveStreams + lane / kStreamLanes >= cnt) continue;
          float f[V];
          unpack16<E>(v[u], f);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += f[e];
        }
      }
      join_streams<V>(acc);
      if (lane < kStreamLanes && c < d) put_row<V>(row + c, acc, scale);
    } else {
      const int c = (now.slice * kWave + lane) * V;
      add_rows<E, kShort>(dout, d, min(c, d - V), 0, 1, cnt, [&](int r) {
        return static_cast<int64_t>(__builtin_amdgcn_readlane(sorted, r));
      }, acc);
      if (c < d) put_row<V>(row + c, acc, scale);
    }
    now = next, next = third, tokens = after;
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
  b.pos = take(n_tokens + kSortThreads);  // the sort rounds its keys up
  b.perm = take(n_tokens);
  auto segs = [&](int64_t n) { return reinterpret_cast<int4*>(take(4 * n)); };
  b.short_segs = segs(n_tokens < vocab ? n_tokens : vocab);
  b.medium_segs = segs(n_tokens / (kShort + 1) + 1);
  b.long_segs = segs(n_tokens / (kMedium + 1) + 1);
  b.bytes = off;
  return b;
}

hipError_t launch_embed_forward(int64_t n, int vocab, int d, int elem_bytes, int index_bytes,
                                float scale, const void* table, const void* tokens, void* out,
                                hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int per = kEmbLoads * kWave * 16 / elem_bytes;
  const int chunks = (d - 1) / per + 1;
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

namespace {

// The segments of the tokens and the zeroing, by the general sequence: the
// counts, segments for the used ids, the tokens into them, the long segments
// in order.  16384 tokens of 2048 bf16: 116 us for 32768 ids (the zeros about 65,
// the rows 48), 89 us for 8000; of 4096 float32 and 49999 ids 239 us (157, 78).
// The count launch alone takes 22 us of the second: an id's tokens all count on
// one address.
template <typename I>
hipError_t group_tokens(int64_t n, int vocab, int d, const I* ids, const EmbedGradBufs& b,
                        float* dtable, hipStream_t s) {
  // Shares of the zeroing per launch, about as long as each launch's own work
  // takes.  With more tokens than ids most rows are used, and zeroing them
  // early would be lost work.
  const int64_t vectors = static_cast<int64_t>(vocab) * (d / 4);
  const double early = n < vocab ? 1.0 : 0.0;
  const double upto[4] = {0.2 * early, 0.5 * early, 0.75, 1.0};
  ZeroShare z[4];
  unsigned fill[4];
  for (int k = 0; k < 4; ++k) {
    z[k].begin = k == 0 ? 0 : z[k - 1].end;
    z[k].end = k == 3 ? vectors : static_cast<int64_t>(upto[k] * static_cast<double>(vectors));
    z[k].count = k < 2 ? nullptr : b.count;
    fill[k] = static_cast<unsigned>((z[k].end - z[k].begin + kGradThreads - 1) / kGradThreads);
  }
  auto own = [](int64_t items, int per) { return static_cast<int>((items + per - 1) / per); };
  hipError_t e;
  const int clear = own(b.clear_ints, kGradThreads), each = own(n, kGradThreads),
            alloc = own(vocab, kAllocIds);
  embed_clear_kernel<<<clear + fill[0], kGradThreads, 0, s>>>(b.counters, b.clear_ints, clear, z[0],
                                                              d, dtable);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (each + fill[1] > 0)
    embed_count_kernel<<<each + fill[1], kGradThreads, 0, s>>>(ids, n, vocab, b.count, b.pos, each,
                                                               z[1], d, dtable);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  embed_alloc_kernel<<<alloc + fill[2], kGradThreads, 0, s>>>(b, vocab, alloc, z[2], d, dtable);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (each + fill[3] > 0)
    embed_place_kernel<<<each + fill[3], kGradThreads, 0, s>>>(b, ids, n, vocab, each, z[3], d,
                                                               dtable);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (n > kMedium)
    embed_order_kernel<<<blocks_for(n / (kMedium + 1), 1, 256), kOrderThreads, 0, s>>>(b, n);
  return hipGetLastError();
}

// The same by one workgroup beside the zeroing of the whole table.
template <typename I>
hipError_t sort_tokens(int64_t n, int vocab, int d, const I* ids, const EmbedGradBufs& b,
                       float* dtable, hipStream_t s) {
  const int64_t vectors = static_cast<int64_t>(vocab) * (d / 4);
  const ZeroShare z{0, vectors, nullptr};
  const unsigned fill = static_cast<unsigned>((vectors + kSortThreads - 1) / kSortThreads);
  int id_bits = 0;
  while (vocab >> id_bits != 0) ++id_bits;  // ids 0 .. vocab (padding)
  embed_sort_kernel<<<1 + fill, kSortThreads, 0, s>>>(b, ids, static_cast<int>(n), vocab, id_bits,
                                                      z, d, dtable);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_backward(int64_t n, int vocab, int d, int elem_bytes, int index_bytes,
                                 float scale, const void* dout, const void* tokens,
                                 const EmbedGradBufs& b, float* dtable, hipStream_t s) {
  // One workgroup sorts while the others zero the table, two launches in all,
  // unless the tokens or ids exceed its keys or most rows are used anyway
  // (zeroing them first would be lost work).  It is ahead of the general
  // sequence up to the most tokens its keys hold: 53 against 60 us for 1024
  // tokens, 59 against 69 for 4096, 65 against 80 for 8192 (32768 x 2048 bf16),
  // 179 against 195 for 8192 of 49999 x 4096 float32.
  const bool sort = n <= kSortMax && n < vocab && vocab < 1 << (32 - kSortNBits);
  auto group = [&](const auto* ids) {
    return sort ? sort_tokens(n, vocab, d, ids, b, dtable, s)
                : group_tokens(n, vocab, d, ids, b, dtable, s);
  };
  const hipError_t e = index_bytes == 8 ? group(static_cast<const int64_t*>(tokens))
                                        : group(static_cast<const int32_t*>(tokens));
  if (e != hipSuccess) return e;
  const int32_t* long_order = sort ? b.perm : b.pos;
  const int V = 16 / elem_bytes;
  const int64_t items = (n < vocab ? n : vocab) * ((d - 1) / (kWave * V) + 1);
  const unsigned grid = blocks_for(items, kRowWaves, kRowBlocks);
  if (elem_bytes == 2)
    embed_rows_kernel<<<grid, kRowThreads, 0, s>>>(b, long_order, static_cast<const uint16_t*>(dout),
                                                   d, scale, dtable);
  else
    embed_rows_kernel<<<grid, kRowThreads, 0, s>>>(b, long_order, static_cast<const float*>(dout),
                                                   d, scale, dtable);
  return hipGetLastError();
}

}  // namespace twell
