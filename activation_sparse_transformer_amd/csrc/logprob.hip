// Log probabilities of given tokens, with the entropy and the top
// alternatives of each row, and their gradient.  With z = scale * x,
//   lse = log sum_j exp z_j,  logp = z_t - lse,  p_j = exp(z_j - lse),
//   entropy = -sum_j p_j log p_j.
// The forward pass reads the logits once.  A lane keeps the running maximum m
// of its x and, with d = (x - m) * scale * log2(e),
//   s = sum 2^d,   t = sum d 2^d
// (rescaled when m grows), so that lse = scale m + ln s and
// entropy = ln s - ln2 * t / s: both terms are non-negative, nothing cancels.
// A masked place (x = -inf) adds nothing to either sum.
#include <type_traits>

#include "common.h"
#include "stream_ops.h"
#include "train_kernels.h"

namespace twell {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / kWave;
constexpr int kLpLoads = 4;             // 16-byte vectors per lane and batch (forward)
constexpr int kLpGradLoads = 4;         // 16-byte vectors per lane and chunk (backward; 1: 118 us, 2: 104,
                                        // 4: 102 for 4096 x 32768 bf16)
constexpr int kLpWantWaves = 4096;      // waves that keep 256 CUs busy (1024 .. 16384 measured:
                                        // within 5% at 1000 and 2000 rows, 64 rows 40% slower at 1024)
constexpr int kLpMinVectors = 128;      // vectors of a row that are worth a wave
constexpr int kLpMaxSplits = kWave;     // parts of a row: one lane each when joined
constexpr int kLpCand = 4 * kWave;      // candidates packed at a time
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kFarLse = 128.f;        // past it float32 lse moves p by over 2^-17
constexpr float kFloorExp = -200.f;     // 2^d is 0 from here down, so d * 2^d is too

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float exp2_hw(float d) { return __builtin_amdgcn_exp2f(d); }

template <typename E>
__device__ __forceinline__ float elem(const uint4& v, int e);
template <>
__device__ __forceinline__ float elem<uint16_t>(const uint4& v, int e) {
  const uint32_t w = e / 2 == 0 ? v.x : e / 2 == 1 ? v.y : e / 2 == 2 ? v.z : v.w;
  return __uint_as_float(e % 2 == 0 ? w << 16 : w & 0xffff0000u);
}
template <>
__device__ __forceinline__ float elem<float>(const uint4& v, int e) {
  return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
}

// Sixteen bytes of -inf.
template <typename E>
__device__ __forceinline__ uint4 masked16() {
  const uint32_t w = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;
  return make_uint4(w, w, w, w);
}

struct SoftStat {
  float m = kLowest, s = 0.f, t = 0.f;
  // a larger maximum: 2^d shrinks by f = 2^delta and every d moves by delta
  __device__ __forceinline__ void raise(float to, float c) {
    const float delta = fmaxf((m - to) * c, kFloorExp);
    const float f = exp2_hw(delta);
    t = f * (t + s * delta);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void term(float x, float c, float& ps, float& pt) const {
    const float d = (x - m) * c;
    const float e = exp2_hw(d);
    ps += e;
    pt = fmaf(fmaxf(d, kFloorExp), e, pt);
  }
  __device__ __forceinline__ void add(float x, float c) { term(x, c, s, t); }
};

// The lanes' statistics joined, the same in every lane.
__device__ __forceinline__ SoftStat join_lanes(SoftStat a, float c) {
  float m = a.m;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
  a.raise(m, c);
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    a.s += __shfl_xor(a.s, o, kWave);
    a.t += __shfl_xor(a.t, o, kWave);
  }
  return a;
}

__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// The best `top` (value, column) pairs seen by a wave, best first (larger
// value, then lower column), lane i holding the i-th.  A value at or below
// `floor` cannot enter from a later column.
struct TopList {
  float v = neg_inf();
  int id = -1;
  float floor = neg_inf();
};

// Scratch of the list: packed candidates, and entries on their way to their
// places.
struct TopScratch {
  float v[kWave];
  int id[kWave];
  float cand[kLpCand];
  int cand_id[kLpCand];
};

// Joins the candidates (x, col) of lanes [0, n) into the list; a lane without
// one holds x = -inf.  Per candidate, one comparison against the other
// candidates and (unless the list is empty, as for a wave's first batch) one
// against the list give every entry its new place, four candidates a step so
// that their latencies overlap; the entries then pass through LDS to their
// lanes.
__device__ __forceinline__ void merge_top(int n, float x, int col, int top, TopList& list,
                                          TopScratch& sc) {
  const int lane = lane_id();
  if (lane >= n) x = neg_inf();
  int place = lane, rank = 0;  // of this lane's list entry, of this lane's candidate
  auto ahead_of = [](float ax, int ac, float bx, int bc) {
    return ax > bx || (ax == bx && ac < bc);
  };
  const bool empty = __builtin_amdgcn_readlane(list.id, 0) < 0;
  if (empty) {
    for (int l0 = 0; l0 < n; l0 += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        rank += ahead_of(lane_value(x, l0 + k), __builtin_amdgcn_readlane(col, l0 + k), x, col);
    }
  } else {
    for (int l0 = 0; l0 < n; l0 += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float cx = lane_value(x, l0 + k);
        const int cc = __builtin_amdgcn_readlane(col, l0 + k);
        rank += ahead_of(cx, cc, x, col);
        const bool ahead = ahead_of(cx, cc, list.v, list.id);
        place += ahead;
        // the list entries this candidate is not ahead of come before it
        const int before = popc64(wave_ballot(!ahead));
        rank += lane == l0 + k ? before : 0;
      }
    }
  }
  const bool cand = x > neg_inf();
  if (empty) sc.v[lane] = neg_inf(), sc.id[lane] = -1;
  else if (place < kWave) sc.v[place] = list.v, sc.id[place] = list.id;
  __builtin_amdgcn_wave_barrier();
  if (cand && rank < kWave) sc.v[rank] = x, sc.id[rank] = col;
  __builtin_amdgcn_wave_barrier();
  list.v = sc.v[lane], list.id = sc.id[lane];
  __builtin_amdgcn_wave_barrier();
  list.floor = fmaxf(list.floor, lane_value(list.v, top - 1));
}

// The largest float below x (of an x that is not NaN).
__device__ __forceinline__ float below(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x == neg_inf()) return x;
  if (x == 0.f) return __uint_as_float(0x80000001u);
  return __uint_as_float(x > 0.f ? u - 1u : u + 1u);
}

// A float that orders as the whole number it comes from, and back.
__device__ __forceinline__ int order_of(float x) {
  const int u = __float_as_int(x);
  return u ^ ((u >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_order(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// A floor that leaves few of a set of which the lanes hold one element each:
// just below a value that at least `top` of them reach, the largest such one
// to within 2^-12 of their spread (-inf where fewer lanes hold one at all).
__device__ __forceinline__ float floor_of(float x, int top) {
  float hi = x, lo = x == neg_inf() ? -neg_inf() : x;
  if (popc64(wave_ballot(x > neg_inf())) < top) return neg_inf();
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor(hi, o, kWave));
    lo = fminf(lo, __shfl_xor(lo, o, kWave));
  }
  // [a, b): at least `top` lanes are at or above a
  int64_t a = order_of(lo), b = static_cast<int64_t>(order_of(hi)) + 1;
  const int key = order_of(x);
#pragma unroll 1
  for (int k = 0; k < 12 && b - a > 1; ++k) {
    const int64_t mid = (a + b) >> 1;
    if (popc64(wave_ballot(key >= static_cast<int>(mid) && x > neg_inf())) >= top) a = mid;
    else b = mid;
  }
  return below(of_order(static_cast<int>(a)));
}

// Merges n packed candidates (n <= kLpCand), 64 at a time.
__device__ __forceinline__ void merge_packed(int n, int top, TopList& list, TopScratch& sc) {
  __builtin_amdgcn_wave_barrier();
#pragma unroll 1
  for (int i = 0; i < n; i += kWave)
    merge_top(min(n - i, kWave), sc.cand[i + lane_id()], sc.cand_id[i + lane_id()], top, list, sc);
}

// Inclusive sum over the lanes, by DPP.
__device__ __forceinline__ int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast15, rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast31, rows 2 and 3
  return v;
}

// Takes the batch's elements above the list's floor into the list; lane l's
// vector u holds columns col0 + (u * 64 + l) * V.  Each lane marks its own, a
// scan gives it their places, and it picks them from a copy of the batch in
// LDS (registers cannot be indexed).  They are few once the list is warm
// (about top * ln of the batches seen, in all).  Where they are many (the
// first batch, a rising row) the floor is raised first, by the lanes' maxima.
// Many equal values may still pass it; those go in 64 columns at a time.
template <typename E, int U>
__device__ __forceinline__ void take_top(const uint4 (&q)[U], float bmax, int col0, int top,
                                         TopList& list, TopScratch& sc, E* stage) {
  constexpr int V = 16 / sizeof(E);
  if (wave_ballot(bmax > list.floor) == 0) return;
  const int lane = lane_id();
#pragma unroll
  for (int u = 0; u < U; ++u) reinterpret_cast<uint4*>(stage)[u * kWave + lane] = q[u];
  bool raised = list.floor == neg_inf();
  if (raised) list.floor = floor_of(bmax, top);
  for (;;) {
    const float floor = list.floor;
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) mine |= elem<E>(q[u], e) > floor ? 1u << (u * V + e) : 0u;
    const int end = lane_scan(__popc(mine));
    const int n = __builtin_amdgcn_readlane(end, kWave - 1);
    if (n <= (raised ? kLpCand : kWave)) {
      int at = end - __popc(mine);
      __builtin_amdgcn_wave_barrier();
      for (; mine != 0; mine &= mine - 1, ++at) {
        const int b = __builtin_ctz(mine);
        const int i = (b / V * kWave + lane) * V + b % V;
        sc.cand[at] = ElemTraits<E>::to_f32(stage[i]);
        sc.cand_id[at] = col0 + i;
      }
      merge_packed(n, top, list, sc);
      return;
    }
    if (raised) break;
    raised = true;
    list.floor = fmaxf(floor, floor_of(bmax, top));
  }
  const float floor = list.floor;
  __builtin_amdgcn_wave_barrier();
#pragma unroll 1
  for (int i = 0; i < U * V; ++i) {
    const float x = ElemTraits<E>::to_f32(stage[i * kWave + lane]);
    if (wave_ballot(x > floor && x >= lane_value(list.v, top - 1)) != 0)
      merge_top(kWave, x > floor ? x : neg_inf(), col0 + i * kWave + lane, top, list, sc);
  }
}

template <typename E, int U, bool TOP>
__device__ __forceinline__ void take_batch(const uint4 (&q)[U], float c, int col0, int top,
                                           SoftStat& a, TopList& list, TopScratch* sc, E* stage) {
  constexpr int V = 16 / sizeof(E);
  float bmax = neg_inf();
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < V; ++e) bmax = fmaxf(bmax, elem<E>(q[u], e));
  if (bmax > a.m) a.raise(bmax, c);
  // the batch's own sums first, one per vector: a lane's chain of additions to
  // s and t is then one per batch, not one per element (error of the entropy
  // over 131072 columns: 7e-8 against 9e-7, the same time)
  float ps[U], pt[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    ps[u] = pt[u] = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) a.term(elem<E>(q[u], e), c, ps[u], pt[u]);
  }
#pragma unroll
  for (int u = 1; u < U; ++u) {
    ps[0] += ps[u];
    pt[0] += pt[u];
  }
  a.s += ps[0];
  a.t += pt[0];
  if constexpr (TOP) take_top<E, U>(q, bmax, col0, top, list, *sc, stage);
}

// A row's target, read before the row's reductions: whether there is one, and
// its logit (lane 0's; the others do without).
struct Target {
  bool given = false;
  float x = 0.f;
  template <typename E, typename I>
  __device__ __forceinline__ void load(const LogprobArgs& a, int64_t row) {
    if (lane_id() != 0) return;
    const int64_t t = static_cast<int64_t>(static_cast<const I*>(a.targets)[row]);
    given = t >= 0 && t < a.vocab;
    if (given) x = ElemTraits<E>::to_f32(static_cast<const E*>(a.logits)[row * a.stride + t]);
  }
};

// The row's outputs from its joined statistics.
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const Target& t,
                                          const SoftStat& st, const TopList& list) {
  const int lane = lane_id();
  const float ln_s = logf(st.s);
  const bool empty = st.s == 0.f;  // every place masked
  if (lane == 0) {
    a.logp[row] = !t.given ? 0.f : empty ? neg_inf() : fmaf(t.x - st.m, a.scale, -ln_s);
    a.entropy[row] = empty ? 0.f : ln_s - kLn2 * (st.t / st.s);
    // below float32's range its lowest value: -inf is a masked row's alone
    const float lse = fmaf(st.m, a.scale, ln_s);
    a.lse[row] = empty ? neg_inf() : lse == neg_inf() ? kLowest : lse;
  }
  if (lane < a.top) {
    a.top_ids[row * a.top + lane] = list.id;
    a.top_logp[row * a.top + lane] =
        list.id < 0 ? neg_inf() : fmaf(list.v - st.m, a.scale, -ln_s);
  }
}

// One pass over the logits, a wave per row (or part of one) so that nothing
// waits on a barrier.  4096 x 131072 bf16 with 5 alternatives: 194-210 us over
// runs and cards, 5.1-5.5 TB/s, without alternatives 184-190; float32 6.0 TB/s.  Bound by HBM and, in bf16,
// as much by the ten or so instruction slots per element (the exponential is
// four): a batch prefetched ahead, or one fused multiply-add for d, change
// nothing.  Wave i of the grid takes part i % splits of row i / splits: the row's whole
// 16-byte vectors [part * per, (part + 1) * per), the first part also the
// elements before the first vector and the last one those after the last.
template <typename E, typename I, bool TOP>
__global__ __launch_bounds__(kLpThreads) void logprob_forward_kernel(const LogprobArgs a,
                                                                    int splits, int per,
                                                                    int64_t n_items) {
  constexpr int V = 16 / sizeof(E);
  const int lane = lane_id();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kLpWaves + threadIdx.x / kWave;
  if (item >= n_items) return;
  const int64_t row = item / splits;
  const int part = static_cast<int>(item - row * splits);
  const E* x = static_cast<const E*>(a.logits) + row * a.stride;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(E) % V);
  const int head = min((V - off) % V, a.vocab);
  const int nv = (a.vocab - head) / V;
  const uint4* body = reinterpret_cast<const uint4*>(x + head);
  const float c = a.scale * kLog2e;
  __shared__ TopScratch scratch[TOP ? kLpWaves : 1];
  __shared__ uint4 staged[TOP ? kLpWaves : 1][kLpLoads * kWave];
  const int wave = TOP ? threadIdx.x / kWave : 0;
  TopScratch* sc = scratch + wave;
  SoftStat st;
  TopList list;
  // at most V - 1 elements from column col0, one per lane
  auto take_edge = [&](int col0, int n) {
    const float v = lane < n ? ElemTraits<E>::to_f32(x[col0 + lane]) : neg_inf();
    if (v > st.m) st.raise(v, c);
    st.add(v, c);
    if constexpr (TOP) {
      if (wave_ballot(v > list.floor) != 0)
        merge_top(n, v > list.floor ? v : neg_inf(), col0 + lane, a.top, list, *sc);
    }
  };
  if (part == 0 && head > 0) take_edge(0, head);
  const int end = min(nv, (part + 1) * per);
  for (int v0 = part * per; v0 < end; v0 += kLpLoads * kWave) {
    uint4 q[kLpLoads];
#pragma unroll
    for (int u = 0; u < kLpLoads; ++u) {
      const int v = v0 + u * kWave + lane;
      q[u] = v < end ? load_once(body + v) : masked16<E>();
    }
    take_batch<E, kLpLoads, TOP>(q, c, head + v0 * V, a.top, st, list, sc,
                                  reinterpret_cast<E*>(staged[wave]));
  }
  const int tail0 = head + nv * V;
  if (part == splits - 1 && tail0 < a.vocab) take_edge(tail0, a.vocab - tail0);
  Target target;
  if (splits == 1) target.load<E, I>(a, row);
  st = join_lanes(st, c);
  if (splits == 1) {
    write_row(a, row, target, st, list);
    return;
  }
  if (lane == 0) a.parts[item] = make_float4(st.m, st.s, st.t, 0.f);
  if (TOP && lane < a.top) {
    a.part_top[item * a.top + lane] = list.v;
    a.part_ids[item * a.top + lane] = list.id;
  }
}

// One workgroup per row joins its parts: lane l takes part l's statistics.  The
// parts' lists (best first) are cut at the floor that their best values give,
// packed in any order, and merged by the first wave.  16 rows of 64 parts with
// 20 alternatives: 6.6 us after the parts' own 7.6, all of it latency.
template <typename E, typename I>
__global__ __launch_bounds__(kLpThreads) void logprob_join_kernel(const LogprobArgs a,
                                                                 int splits) {
  __shared__ TopScratch sc;
  __shared__ int n;
  constexpr int kPer = kLpMaxSplits * kLogprobMaxTop / kLpThreads;
  const int lane = lane_id(), tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float c = a.scale * kLog2e;
  const float* vals = a.part_top + row * splits * a.top;
  const int32_t* ids = a.part_ids + row * splits * a.top;
  const int total = splits * a.top;
  SoftStat st;
  TopList list;
  Target target;
  if (lane < splits) {
    const float4 p = a.parts[row * splits + lane];
    st.m = p.x, st.s = p.y, st.t = p.z;
  }
  if (tid < kWave) target.load<E, I>(a, row);
  float floor = neg_inf();
  if (total > 0) {
    float x[kPer];
    int col[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = k * kLpThreads + tid;
      x[k] = i < total ? vals[i] : neg_inf();
      col[k] = i < total ? ids[i] : -1;
    }
    // one element per lane: the first places of every part's list
    const int place = lane / splits;
    floor = floor_of(lane < total && place < a.top ? vals[lane % splits * a.top + place]
                                                   : neg_inf(), a.top);
    if (tid == 0) n = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (!(x[k] > floor)) continue;
      const int at = atomicAdd(&n, 1);
      if (at < kLpCand) sc.cand[at] = x[k], sc.cand_id[at] = col[k];
    }
    __syncthreads();
  }
  if (tid >= kWave) return;
  if (total > 0) {
    const int count = n;
    if (count <= kLpCand) {
      merge_packed(count, a.top, list, sc);
    } else {  // many equal values
#pragma unroll 1
      for (int i0 = 0; i0 < total; i0 += kWave) {
        const int i = i0 + lane;
        const float x = i < total ? vals[i] : neg_inf();
        const int col = i < total ? ids[i] : -1;
        if (wave_ballot(x > floor && x >= lane_value(list.v, a.top - 1)) != 0)
          merge_top(kWave, x > floor ? x : neg_inf(), col, a.top, list, sc);
      }
    }
  }
  write_row(a, row, target, join_lanes(st, c), list);
}

// dlogits of one element: scale * (g * [j is the target] - p * (g + w * (log p + H))).
// log p = (x - m) * scale - ln_s: m = 0 and ln_s = lse, or a row's own maximum
// and sum (FAR) where lse alone would not hold them.
struct RowGrad {
  float m, ln_s, scale, g, w, h;
  template <bool ENT, bool FAR>
  __device__ __forceinline__ float at(float x, bool target) const {
    const float lp = fmaf(FAR ? x - m : x, scale, -ln_s);
    const float p = exp2_hw(lp * kLog2e);
    // a masked place has p = 0 and log p = -inf: its product is 0
    const float k = ENT ? fmaf(w, fmaxf(lp, kFloorExp) + h, g) : g;
    const float d = fmaf(-p, k, target ? g : 0.f);
    return d * scale;
  }
};

// The workgroup's statistics of a whole row (every lane gets them).
template <typename E>
__device__ SoftStat block_stat(const E* x, int vocab, float c) {
  __shared__ float3 waves[kLpWaves];
  SoftStat st;
  for (int j = threadIdx.x; j < vocab; j += kLpThreads) {
    const float v = ElemTraits<E>::to_f32(x[j]);
    if (v > st.m) st.raise(v, c);
    st.add(v, c);
  }
  st = join_lanes(st, c);
  __syncthreads();
  if (lane_id() == 0) waves[threadIdx.x / kWave] = make_float3(st.m, st.s, st.t);
  __syncthreads();
  SoftStat w;
  if (lane_id() < kLpWaves) {
    const float3 p = waves[lane_id()];
    w.m = p.x, w.s = p.y, w.t = p.z;
  }
  return join_lanes(w, c);
}

template <typename E>
__device__ __forceinline__ uint4 pack16(const float* f) {
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

// One chunk of a row: kLpThreads * kLpGradLoads vectors, for the row's first
// chunk also the elements before its first vector and for the last one those
// after its last.  VEC: input and output rows share their alignment.
template <typename E, bool VEC>
struct GradChunk {
  static constexpr int V = VEC ? 16 / sizeof(E) : 1;
  typedef ElemTraits<E> Tr;
  const E* x;
  E* out;
  int vocab, chunk, chunks, head, nv;
  uint4 q[kLpGradLoads];
  __device__ __forceinline__ GradChunk(const E* x_, E* out_, int vocab_, int chunk_, int chunks_)
      : x(x_), out(out_), vocab(vocab_), chunk(chunk_), chunks(chunks_) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(E) % V);
    head = min((V - off) % V, vocab);
    nv = (vocab - head) / V;
  }
  __device__ __forceinline__ int at(int u) const {
    return (chunk * kLpGradLoads + u) * kLpThreads + static_cast<int>(threadIdx.x);
  }
  __device__ __forceinline__ void load() {
    if constexpr (VEC) {
#pragma unroll
      for (int u = 0; u < kLpGradLoads; ++u)
        if (at(u) < nv) q[u] = load_once(reinterpret_cast<const uint4*>(x + head) + at(u));
    }
  }
  template <bool ENT, bool FAR>
  __device__ __forceinline__ void finish(const RowGrad& r, int t) const {
    auto one = [&](int j) {
      out[j] = Tr::from_f32(r.template at<ENT, FAR>(Tr::to_f32(x[j]), j == t));
    };
    if (chunk == 0 && static_cast<int>(threadIdx.x) < head) one(threadIdx.x);
    const int tail0 = head + nv * V;
    if (chunk == chunks - 1 && static_cast<int>(threadIdx.x) < vocab - tail0)
      one(tail0 + threadIdx.x);
#pragma unroll
    for (int u = 0; u < kLpGradLoads; ++u) {
      const int v = at(u);
      if (v >= nv) continue;
      if constexpr (!VEC) {
        one(v);
      } else {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
          f[e] = r.template at<ENT, FAR>(elem<E>(q[u], e), head + v * V + e == t);
        store_once(reinterpret_cast<uint4*>(out + head) + v, pack16<E>(f));
      }
    }
  }
};

// A workgroup takes one chunk of a row; its logits are on their way before the
// row's scalars are read (102 -> 97 us).  4096 x 32768 bf16: 95 us, 5.7 TB/s;
// 2000 x 49999 float32 with the entropy's part: 139 us, 5.8 TB/s; bound by HBM.
// lse is rounded to float32, which moves every p of the row by |lse| * 2^-24 of
// itself; past kFarLse (a row of the type's lowest values, or logits far from
// zero) the row's own maximum and sum are formed again instead.  dlogits may be
// the logits, where the chunks of such a row would see each other's results:
// there one workgroup forms the sums and takes the row's chunks in turn.  That
// costs: 4096 x 32768 bf16 with 80% of such rows 986 us, 16 x 131072 with
// nearly all 224 us against 11 without.
template <typename E, typename I, bool ENT, bool VEC>
__global__ __launch_bounds__(kLpThreads) void logprob_backward_kernel(const LogprobGradArgs a,
                                                                     int chunks,
                                                                     int64_t n_items) {
  for (int64_t item = blockIdx.x; item < n_items; item += gridDim.x) {
    const int64_t row = item / chunks;
    const E* x = static_cast<const E*>(a.logits) + row * a.stride;
    E* out = static_cast<E*>(a.dlogits) + row * a.out_stride;
    GradChunk<E, VEC> c(x, out, a.vocab, static_cast<int>(item - row * chunks), chunks);
    c.load();
    const int64_t t64 = static_cast<int64_t>(static_cast<const I*>(a.targets)[row]);
    const int t = t64 >= 0 && t64 < a.vocab ? static_cast<int>(t64) : -1;
    const float lse = a.lse[row];
    RowGrad r;
    r.m = 0.f;
    r.ln_s = lse;
    r.scale = a.scale;
    r.g = a.dlogp[row];
    if (t < 0) r.g = 0.f;
    r.w = ENT ? a.dentropy[row] : 0.f;
    r.h = ENT ? a.entropy[row] : 0.f;
    if (lse == neg_inf()) {  // every place masked: no gradient
      r.ln_s = -neg_inf();
      r.g = r.w = 0.f;
    } else if (fabsf(lse) > kFarLse) {
      if (c.chunk != 0) continue;
      const SoftStat st = block_stat<E>(x, a.vocab, a.scale * kLog2e);
      r.m = st.m;
      r.ln_s = logf(st.s);
      __syncthreads();  // every read of the row before its first write
      for (int k = 0; k < chunks; ++k) {
        GradChunk<E, VEC> ck(x, out, a.vocab, k, chunks);
        ck.load();
        ck.template finish<ENT, true>(r, t);
      }
      continue;
    }
    c.template finish<ENT, false>(r, t);
  }
}

}  // namespace

// Parts a row is split in: enough waves for the whole GPU, but no part under
// kLpMinVectors vectors.
int logprob_splits(int64_t n_rows, int vocab, int elem_bytes) {
  const int nv = vocab / (16 / elem_bytes);
  const int64_t want = (kLpWantWaves + n_rows - 1) / (n_rows < 1 ? 1 : n_rows);
  int64_t most = nv / kLpMinVectors;
  if (most > kLpMaxSplits) most = kLpMaxSplits;
  const int64_t n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n);
}

size_t logprob_carve(LogprobArgs* a, int elem_bytes, void* ws) {
  const int splits = logprob_splits(a->n_rows, a->vocab, elem_bytes);
  if (splits == 1) return 0;
  const size_t parts = static_cast<size_t>(a->n_rows) * splits;
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = p == nullptr ? nullptr : p + off;
    off += (bytes + 255) / 256 * 256;
    return q;
  };
  a->parts = reinterpret_cast<float4*>(take(parts * sizeof(float4)));
  a->part_top = reinterpret_cast<float*>(take(parts * a->top * 4));
  a->part_ids = reinterpret_cast<int32_t*>(take(parts * a->top * 4));
  return off;
}

hipError_t launch_logprob_forward(const LogprobArgs& a, int elem_bytes, int index_bytes,
                                  hipStream_t s) {
  if (a.n_rows == 0) return hipSuccess;
  const int splits = logprob_splits(a.n_rows, a.vocab, elem_bytes);
  const int V = 16 / elem_bytes;
  int per = (a.vocab / V + splits - 1) / splits;
  per = (per + kWave - 1) / kWave * kWave;
  const int64_t items = a.n_rows * splits;
  const unsigned grid = static_cast<unsigned>((items + kLpWaves - 1) / kLpWaves);
  auto go = [&](auto e, auto i) {
    typedef decltype(e) E;
    typedef decltype(i) I;
    if (a.top > 0)
      logprob_forward_kernel<E, I, true><<<grid, kLpThreads, 0, s>>>(a, splits, per, items);
    else
      logprob_forward_kernel<E, I, false><<<grid, kLpThreads, 0, s>>>(a, splits, per, items);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || splits == 1) return err;
    logprob_join_kernel<E, I><<<static_cast<unsigned>(a.n_rows), kLpThreads, 0, s>>>(a, splits);
    return hipGetLastError();
  };
  if (elem_bytes == 2)
    return index_bytes == 8 ? go(uint16_t{}, int64_t{}) : go(uint16_t{}, int32_t{});
  return index_bytes == 8 ? go(float{}, int64_t{}) : go(float{}, int32_t{});
}

hipError_t launch_logprob_backward(const LogprobGradArgs& a, int elem_bytes, int index_bytes,
                                   hipStream_t s) {
  if (a.n_rows == 0) return hipSuccess;
  // rows of both arrays start at the same place within 16 bytes
  const bool vec = (a.stride - a.out_stride) * elem_bytes % 16 == 0;
  const int per = kLpThreads * kLpGradLoads;
  const int nv = vec ? a.vocab / (16 / elem_bytes) : a.vocab;
  const int chunks = nv < 1 ? 1 : (nv + per - 1) / per;
  const int64_t items = a.n_rows * chunks;
  const unsigned grid = static_cast<unsigned>(items < (1 << 23) ? items : (1 << 23));
  auto go = [&](auto e, auto i, auto ent, auto v) {
    logprob_backward_kernel<decltype(e), decltype(i), decltype(ent)::value, decltype(v)::value>
        <<<grid, kLpThreads, 0, s>>>(a, chunks, items);
    return hipGetLastError();
  };
  auto by_vec = [&](auto e, auto i, auto ent) {
    return vec ? go(e, i, ent, std::true_type{}) : go(e, i, ent, std::false_type{});
  };
  auto by_ent = [&](auto e, auto i) {
    return a.dentropy != nullptr ? by_vec(e, i, std::true_type{}) : by_vec(e, i, std::false_type{});
  };
  if (elem_bytes == 2)
    return index_bytes == 8 ? by_ent(uint16_t{}, int64_t{}) : by_ent(uint16_t{}, int32_t{});
  return index_bytes == 8 ? by_ent(float{}, int64_t{}) : by_ent(float{}, int32_t{});
}

}  // namespace twell
