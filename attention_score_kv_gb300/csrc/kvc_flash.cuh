// Attention of many query rows per KV head on the tensor cores: a prompt chunk
// over the active layer's bf16 rows, and many tokens over the 8-bit cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(x_j),  lse = log sum_j p_j
//
// One pass over the keys with a running reference r: o and the sum are kept for
// weights 2^(x - r), and r follows the maximum only when a score passes it by
// 2^kSlack, so the output is hardly ever rescaled.
//
// A CTA has two streams of 128 query rows against tiles of 128 keys (tcgen05, fp32
// accumulators in tensor memory: S and O of both streams are its 512 columns):
//   S = Q K^T   (both in shared memory);   O += P V   (P in tensor memory, over S)
// A warp per stream issues the last tile's P V and the next tile's Q K^T, 1024 cycles
// of products at D = 128, while eight warps make the other stream's weights, two
// threads a row.  S is overwritten by P and P by the next S: the products of a
// warp run in order, and the two threads of a row, one of which writes P where the
// other's scores were, meet at a barrier of theirs with S in registers, each time that
// they take it.
// Two ways to feed the streams:
//   row pairs    two row tiles of a head share each tile of keys and values
//   key pairs    one row tile (few rows: down to a single token); the streams take
//                tiles of keys in turn, and their outputs are joined at the end
// A row tile is nt = 128 / G tokens of all G query heads of the KV head, so a
// causal or a document's border cuts few tiles.
//
// Work split: a unit is (sequence, KV head, row tile or pair), its steps the key
// tiles (pairs of them) that some query of it sees.  A planning kernel counts them
// from the device-held masks and row counts, lays all units end to end and gives
// every SM's CTA an equal range, whatever the masks and lengths.  Units that a
// range's end cuts leave partial results, which a third kernel joins in order.
//
// Measured (D = 128, 32/8 heads): 2048 tokens over 32K behind a prefix 743 to 783 us by the
// clocks under load (1375 to 1450 TFLOP/s; the products alone, without weights, 575),
// over 8K 186, with a bias 213, with a cap 238 to 387 by how large the scores are against
// it; one token over 8K 16.5, of 16 sequences 85.9 (6.3 TB/s); 512 tokens over 4.8K rows
// of the 8-bit cache 96.5.  A tile's chain bounds it: weights 1300 to 1570 cycles,
// products 920, hand-overs 750 to 1000.
//
// e4m3 keys and values (the 8-bit cache): the products take e4m3 operands.  A query
// row is scaled by a power of two to below 2^8 and split into two e4m3 parts, four
// significant bits each, so that all of a bf16's eight are there; weights are split
// the same way: two products of twice bf16's rate each.  What is split is a weight times the
// scale of its block of values, a contribution, in a unit of the row's own, 2^unit, which
// follows the row's largest contribution as the reference follows its largest score: e4m3
// reaches 2^-10 down, so a unit that other rows' blocks decided would lose a row's own.
#pragma once

#include <algorithm>
#include <cmath>

#include "kvc_device.cuh"
#include "kvc_internal.cuh"
#include "kvc_q4.cuh"
#include "kvc_q8.cuh"
#include "kvc_scan_common.cuh"
#include "kvc_tc.cuh"

namespace kvc {
namespace flash {

constexpr int kRows = 128, kKeys = 128;
constexpr int kHalf = kKeys / 2;     // keys of a thread of the weights
constexpr int kSoftWarps = 16, kMmaWarp = 16, kLoadWarp = 18, kMetaWarp = 19;
// Five groups of four warps: the two streams' weights, and the two issuing, the
// loading and the 8-bit cache's warp, whose registers the first four groups take: 4 * 104 + 64 =
// 5 * 96, what the block is launched with.
constexpr int kThreads = 20 * 32, kSoftRegs = 104, kOtherRegs = 64;
constexpr uint32_t kCols = 512, kColS = 0, kColO = 256;    // stream x: S at kColS + 128 x, O at kColO + 128 x
constexpr float kNoRef = -1.7e38f;   // reference of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994530942f;
constexpr float kLeastUnit = 7.8886090522101181e-31f;      // 2^-100, the smallest scale
constexpr int kPasses = 3;           // times that a tile's maximum is looked at
constexpr float kExact = 8192.f;     // below it steps of fp32 are 2^-11 at most
constexpr int kMaxStages = 11;
constexpr int kMeta = 8;             // tiles whose positions and scales are in shared memory

// What a tile of the 8-bit cache's rows is.
struct alignas(16) Meta {
  int pos[kKeys];
  float rel[kKeys];                  // position less the unit's last query's
  float2 scale[kKeys / q8::kRows];   // of the blocks' keys and values
  uint32_t some[4];                  // rows that some query of the call may see
  uint32_t mixed[4];                 // some query does not see all of these 32
};

// Where a CTA's range begins: a unit, and the steps of it before the range.
struct Start { int b, h, tile, n, k0; long long off; };
struct Plan {                        // in the workspace
  long long total, L;                // all steps; steps of a range
};

struct Args {
  CUtensorMap qmap, kmap, vmap;
  const __nv_bfloat16* q;
  // chunk: query (b, t) at q_pos sees keys first .. last
  const int32_t *q_pos, *first, *last;
  // 8-bit cache
  const int32_t *pos, *rows;
  const float2* scale;
  Q4Slots s;
  const float* slopes;
  __nv_bfloat16* out;
  float* lse;
  Plan* plan;
  int2* units;                       // [B1][tiles]: first key tile, steps
  int2 *sees, *seen;                 // [B1][tiles], [B1]: what units and sequences see
  long long* before;                 // [B1 * tiles + 1] steps before, of one head
  Start* start;                      // [P + 1]
  float2* part_ml;                   // [2 P][rows of a unit]: reference, sum of the weights
  float* part_o;                     // [2 P][rows of a unit x D], see part_row; divided by the sum
  int* status;
  int B1, H1;                        // units are [B1][H1][tiles]: B, H_kv (chunk) or B * H_kv, 1 (cache)
  int T, H_q, H_kv, G, S, extra;
  int nt, tiles, P;
  int planned;                       // by a kernel of its own; else every CTA does it
  int pair_keys;                     // the streams share rows and take key tiles in turn
  // Where four dims of a row of partial results lie: row * part_row + d / 4 * part_step.
  // Row after row when a unit has less than a warp's rows, or when four CTAs and more
  // share a unit, so that a row has many parts and reading them counts; else four dims
  // of all rows side by side, as a warp (a row a lane) writes them.  Row after row, and
  // side by side: one token over 8K 16.4 and 20.2 us, 32 tokens 23.0 and 26.2; a turn
  // of 512 102.7 and 97.6, causal at D = 64 136.5 and 133.6, documents 106.4 and 104.7.
  int part_row, part_step;
  uint32_t wait_limit;
  float scale2, cap2, inv_cap2;      // log2(e) / sqrt(D); cap in log2 units, 0: none
};

// ------------------------------------------------------------------- planning
// The keys a query sees: 0 <= lo, -1 <= hi < S, so that differences to a tile's keys fit ints.
__device__ __forceinline__ bool key_range(const Args& a, int64_t bt, int& lo, int& hi) {
  const int qp = __ldg(a.q_pos + bt);
  lo = a.first ? max(__ldg(a.first + bt), 0) : 0;
  hi = qp < 0 ? -1 : max(min(a.last ? __ldg(a.last + bt) : qp, a.S - 1), -1);
  return lo <= hi;
}
__device__ __forceinline__ int rows_held(const Args& a, int bh, bool* bad) {
  const int h = bh % a.H_kv;
  const int64_t cap = a.s.off[h + 1] - a.s.off[h], n = (int64_t)__ldg(a.rows + bh) + a.extra;
  *bad = n < 0 || n > cap;
  return (int)(n < 0 ? 0 : n > cap ? cap : n);
}
// One unit, by a warp: its first key tile and steps, and what its tokens see: the first
// and last key, and whether their ranges leave holes between them or to the next
// unit's (each token's touches the next one's, and those that see nothing come last).
// 8-bit cache: the last position that a token of it may see.  Packed: the first key, -1
// with holes, and the last.
template <bool FP8>
__device__ __forceinline__ int2 unit_steps(const Args& a, int b, int tile, int2& sees) {
  const int lane = threadIdx.x & 31, per = a.nt * (a.pair_keys ? 1 : 2), t0 = tile * per, t1 = min(t0 + per, a.T);
  int k0 = 0, n = 1, lo = INT_MAX, hi = -1;
  bool holes = false;
  if constexpr (FP8) {
    bool bad;
    n = (rows_held(a, b, &bad) + kKeys - 1) / kKeys;
    if (bad && lane == 0) record_status(a.status, kStatusBadInput);
    for (int t = t0 + lane; t < t1; t += 32) hi = max(hi, __ldg(a.q_pos + (int64_t)(b / a.H_kv) * a.T + t));
    hi = __reduce_max_sync(0xffffffffu, hi);
  } else {
    for (int t = t0 + lane; t < t1; t += 32) {
      int l, h, l1 = 0, h1 = -1;
      const bool some = key_range(a, (int64_t)b * a.T + t, l, h);
      const bool next = t + 1 < a.T && key_range(a, (int64_t)b * a.T + t + 1, l1, h1);
      if (some) lo = min(lo, l), hi = max(hi, h);
      holes |= next && (!some || l1 > h + 1 || l > h1 + 1);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    holes = __any_sync(0xffffffffu, holes);
    if (lo <= hi) k0 = lo / kKeys, n = hi / kKeys - k0 + 1;
  }
  sees = make_int2(holes ? -1 : lo, hi);
  // a unit that sees nothing takes a step all the same, which writes its zeros
  if (a.pair_keys) n = (n + 1) / 2;
  return make_int2(k0, max(n, 1));
}
// The same of a whole sequence, from its units', a warp each.
__device__ __forceinline__ void join_sees(const Args& a, const int2* sees, int2* seen) {
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < a.B1; b += blockDim.x >> 5) {
    int lo = INT_MAX, hi = -1;
    for (int t = lane; t < a.tiles; t += 32) {
      const int2 x = sees[(int64_t)b * a.tiles + t];
      lo = min(lo, x.x), hi = max(hi, x.y);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) seen[b] = make_int2(lo, hi);
  }
}
// The steps of many units, a warp each (few: the next kernel counts them itself).
template <bool FP8>
__global__ void __launch_bounds__(256) count_kernel(const __grid_constant__ Args a) {
  grid_dep_wait();
  grid_dep_launch();
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= a.B1 * a.tiles) return;
  int2 sees;
  const int2 u = unit_steps<FP8>(a, i / a.tiles, i % a.tiles, sees);
  if ((threadIdx.x & 31) == 0) a.units[i] = u, a.sees[i] = sees;
}
// Where the range that begins with step f does.
__device__ __forceinline__ Start find_start(const Args& a, long long f, long long total, const long long* before,
                                            const int2* units) {
  Start st{-1, 0, 0, 0, 0, 0};
  if (f >= total) return st;
  int lo = 0, hi = a.B1;             // the sequence: before[b * tiles] * H1 <= f
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (before[(int64_t)mid * a.tiles] * a.H1 <= f) lo = mid; else hi = mid;
  }
  const int b = lo;
  const long long b0 = before[(int64_t)b * a.tiles], nb = before[(int64_t)(b + 1) * a.tiles] - b0;
  const int h = (int)((f - b0 * a.H1) / nb);
  const long long in = f - b0 * a.H1 - h * nb + b0;          // among one head's
  lo = 0, hi = a.tiles;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (before[(int64_t)b * a.tiles + mid] <= in) lo = mid; else hi = mid;
  }
  const int64_t at = (int64_t)b * a.tiles + lo;
  return {b, h, lo, units[at].y, units[at].x, in - before[at]};
}
// Lays the units end to end and finds where each CTA's range begins.  Up to kPlanned
// units its searches stay in shared memory.
constexpr int kPlanned = 2048;
template <bool FP8>
__global__ void __launch_bounds__(1024) plan_kernel(const __grid_constant__ Args a, int counted) {
  __shared__ long long s_part[32], s_run, s_before[kPlanned + 1];
  __shared__ int2 s_units[kPlanned];
  const int N = a.B1 * a.tiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool here = N <= kPlanned;
  long long* const before = here ? s_before : a.before;
  grid_dep_wait();
  grid_dep_launch();
  if (!counted) {
    for (int i = warp; i < N; i += 32) {
      int2 sees;
      const int2 u = unit_steps<FP8>(a, i / a.tiles, i % a.tiles, sees);
      if (lane == 0) a.units[i] = s_units[i] = u, a.sees[i] = sees;
    }
  } else if (here) {
    for (int i = threadIdx.x; i < N; i += 1024) s_units[i] = a.units[i];
  }
  const int2* const units = here ? s_units : a.units;
  if (threadIdx.x == 0) s_run = 0;
  __syncthreads();
  join_sees(a, a.sees, a.seen);
  for (int i0 = 0; i0 < N; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const long long n = i < N ? units[i].y : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s_part[warp] = inc;
    __syncthreads();
    long long run = s_run;
    for (int w = 0; w < warp; ++w) run += s_part[w];
    if (i < N) before[i] = run + inc - n;
    __syncthreads();
    if (threadIdx.x == 1023) s_run = run + inc;
    __syncthreads();
  }
  const long long one = s_run, total = one * a.H1;
  if (threadIdx.x == 0) before[N] = one;
  const long long L = (total + a.P - 1) / a.P;
  if (threadIdx.x == 0) a.plan->total = total, a.plan->L = L;
  __syncthreads();
  for (int c = threadIdx.x; c < a.P; c += 1024) a.start[c] = find_start(a, c * L, total, before, units);
}

// ------------------------------------------------------------------- a CTA's range
struct Seg {
  int b, h, tile;                    // the unit
  int k0, n;                         // its first key tile, its steps
  int s0, cnt;                       // steps of this range
  // The key tile that comes first, of `subs` a step.  The last keys do: with a bias by
  // distance they have the largest scores, and the reference would move at every tile
  // the other way round (2048 tokens over 8K: 315 us).
  __device__ __forceinline__ int last(int subs) const { return k0 + (n - s0) * subs - 1; }
};
// Few units: every CTA counts all of them and finds its own range, a launch less
// (8 units of a single token over 8K: 18.5 -> 17.2 us).
constexpr int kPlanHere = 34;
struct Here {
  Start start;
  Plan plan;
  int2 units[kPlanHere], seen[kPlanHere];
};
struct Scratch {                     // where the ring will be
  long long before[kPlanHere + 1];
  int2 sees[kPlanHere];
};
template <bool FP8>
__device__ __forceinline__ void plan_here(const Args& a, Here& here, Scratch& tmp) {
  const int N = a.B1 * a.tiles, lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < N; i += blockDim.x >> 5) {
    int2 sees;
    const int2 u = unit_steps<FP8>(a, i / a.tiles, i % a.tiles, sees);
    if (lane == 0) here.units[i] = u, tmp.sees[i] = sees;
  }
  __syncthreads();
  join_sees(a, tmp.sees, here.seen);
  if (threadIdx.x == 0) {
    long long run = 0;
    for (int i = 0; i < N; ++i) {
      tmp.before[i] = run;
      run += here.units[i].y;
    }
    tmp.before[N] = run;
    const long long total = run * a.H1, L = (total + a.P - 1) / a.P;
    here.plan = {total, L};
    here.start = find_start(a, blockIdx.x * L, total, tmp.before, here.units);
    a.start[blockIdx.x] = here.start;  // for the join
    if (blockIdx.x == 0) *a.plan = here.plan;
  }
  tc::fence_proxy_async();           // the copies write there next
  __syncthreads();
}

// Walks the units of a range; every role does it by itself, the next unit's place
// asked for ahead.
struct Walk {
  Seg g;
  long long left;
  int2 ahead;
  const int2 *units, *seen;
  __device__ __forceinline__ bool begin(const Args& a, const Here& here) {
    const Start st = a.planned ? a.start[blockIdx.x] : here.start;
    const Plan p = a.planned ? *a.plan : here.plan;
    units = a.planned ? a.units : here.units;
    seen = a.planned ? a.seen : here.seen;
    if (st.b < 0) return false;
    left = min(p.L, p.total - (long long)blockIdx.x * p.L);
    g.b = st.b, g.h = st.h, g.tile = st.tile;
    g.k0 = st.k0, g.n = st.n;
    g.s0 = (int)st.off;
    g.cnt = (int)min((long long)(g.n - g.s0), left);
    look(a);
    return true;
  }
  __device__ __forceinline__ void step(const Args& a, int& b, int& h, int& tile) const {
    if (++tile == a.tiles) {
      tile = 0;
      if (++h == a.H1) h = 0, ++b;
    }
  }
  __device__ __forceinline__ void look(const Args& a) {
    int b = g.b, h = g.h, tile = g.tile;
    step(a, b, h, tile);
    ahead = left > g.cnt ? units[(int64_t)b * a.tiles + tile] : make_int2(0, 0);
  }
  __device__ __forceinline__ bool next(const Args& a) {
    left -= g.cnt;
    if (left <= 0) return false;
    step(a, g.b, g.h, g.tile);
    g.k0 = ahead.x, g.n = ahead.y;
    g.s0 = 0;
    g.cnt = (int)min((long long)g.n, left);
    look(a);
    return true;
  }
};

// ------------------------------------------------------------------- pieces
template <int D, bool FP8>
struct Cfg {
  static constexpr int kStageBytes = kKeys * D * (FP8 ? 1 : 2);
  static constexpr int kQBytes = FP8 ? 2 * kRows * D : kRows * D * 2;       // of a stream: two parts, or bf16
  static constexpr int kStages = FP8 ? 9 : D == 128 ? 5 : 11;
  static constexpr int kMetaBytes = FP8 ? (int)sizeof(Meta) * kMeta : 0;
  static constexpr int kMostBytes = FP8 ? 4 * kRows * (int)sizeof(float) : 0;   // largest contributions
  static constexpr int kSmem = 2 * kQBytes + kStages * kStageBytes + kMetaBytes + kMostBytes;
  // A row's largest weight may be up to 2^kHigh, and the first tile's as small as 2^kLow:
  // bf16 and fp32 reach as far down as they have to.  e4m3's two parts end at 2^-10, so
  // the largest contribution of a row is kept between 2^kLeast and 2^kMost units (from 2^6
  // on, twice as many tiles move it).
  static constexpr float kLow = -24.f, kHigh = FP8 ? 16.f : 8.f, kLeast = 5.f, kMost = 8.f;
  static constexpr int kQSteps = FP8 ? D / 32 : D / 16, kVSteps = FP8 ? kKeys / 32 : kKeys / 16;
};

// q_full, kv_full / kv_empty (a ring over the tiles of keys and values in the order
// of their products), s_full (a stream's scores are there; at a segment's end: its
// output), p_full (a stream's weights are there, and its scores in registers).
// A wait looks at the parity of a phase alone, so none may be two phases ahead of
// a warp that still waits for the first:
//   kv_full(i + kStages)   kv_empty(i), committed behind products that waited for kv_full(i)
//   kv_empty(i + kStages)  kv_full(i + kStages), loaded after a look at kv_empty(i)
//   s_full(i + 1)          p_full(i) of all eight warps, which saw s_full(i); a segment's
//                          end likewise, and the next segment's first scores come
//                          at once: the end's barrier is another, s_end
//   s_end(i + 1)           p_full of the next segment, made after a look at s_end(i)
//   p_full(i + 1)          s_full(i + 1), issued after a look at p_full(i)
//   q_full(i + 1)          q_empty(i) (bf16), committed behind products after q_full(i); or
//                          s_end(i) (e4m3: the rows' own warps write the queries)
//   turn(i + 1)            the other stream's warp issues in between, after a look at turn(i)
//   meta_full(i + kMeta)   meta_empty(i) of every warp that reads the tile's, after meta_full(i)
//   meta_empty(i + kMeta)  meta_full(i + kMeta), written after a look at meta_empty(i)
struct Bars {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], s_full[2], s_end[2], p_full[2], q_full, q_empty, meta_full[kMeta], meta_empty[kMeta], turn[2], drain[2];
};

__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, uint32_t limit) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
      "LOOK:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra SEEN;\n"
      " add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra LOOK;\n"
      "SEEN:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(limit)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two values below 448 -> two e4m3 parts each (low byte first): x = a + b to 8
// significant bits, or to 2^-10.
__device__ __forceinline__ void split2(float lo, float hi, uint16_t& a, uint16_t& b) {
  uint32_t h, back, rest;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h) : "f"(hi), "f"(lo));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(a) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(back) : "h"(a));
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(rest) : "r"(h), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(b) : "r"(rest));
}

// One lane of the warp, the same each time.  A branch on it, unlike one on the lane's
// number, tells the compiler that a single thread is left, whose operands then stay in
// uniform registers: a product's issue costs 64 cycles less.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}

// Products from one thread.  A in shared memory (scores) or tensor memory (output).
template <bool FP8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (FP8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
template <bool FP8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (FP8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Instruction descriptor: fp32 accumulator, A K-major; B K-major (keys) or, with
// rows = contraction index, MN-major (values).
template <bool FP8>
__host__ __device__ constexpr uint32_t idesc(int N, bool b_mn) {
  return (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
// Rows of 128 or 64 bytes in swizzled atoms of 8 rows.  As a K-major operand: groups
// of 8 rows `8 * row bytes` apart (stride); as an MN-major one the same groups along
// the contraction, and `lead` bytes between panels of a row's width.
template <int ROW>
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)((8 * ROW) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(ROW == 128 ? 2 : 4) << 61;      // swizzle of 128 or 64 bytes
  return d;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// ------------------------------------------------------------------- the loads
// Tile `t` (an index of key tiles of the unit) of keys or values into a stage.
template <int D, bool FP8>
__device__ __forceinline__ void load_tile(const Args& a, const Seg& g, bool vals, int t, uint32_t dst, uint32_t bar) {
  const CUtensorMap* map = vals ? &a.vmap : &a.kmap;
  tc::mbar_arrive_expect_tx(bar, Cfg<D, FP8>::kStageBytes);
  if constexpr (FP8) {
    const int b = g.b / a.H_kv, h = g.b - b * a.H_kv;
    const int64_t row = (int64_t)b * a.s.off[a.H_kv] + a.s.off[h];
    tc::tma_load_3d(dst, map, bar, 0, 0, (int)(row / q8::kRows) + t * (kKeys / q8::kRows));
  } else {
#pragma unroll
    for (int p = 0; p < D / 64; ++p)
      tc::tma_load_3d(dst + p * (kKeys * 128), map, bar, p * 64, t * kKeys, g.b * a.H1 + g.h);
  }
}

// The warp that copies (lane 0).
template <int D, bool FP8>
__device__ bool load_warp(const Args& a, const Here& here, Bars* bars, uint32_t sQ, uint32_t ring) {
  using C = Cfg<D, FP8>;
  const int lane = threadIdx.x & 31;
  const int subs = a.pair_keys ? 2 : 1;           // key tiles of a step
  uint32_t it = 0, nq = 0;                       // tiles, queries asked for
  bool ok = true;
  Walk w;
  if (!w.begin(a, here)) return true;
  do {
    const Seg& g = w.g;
    bool wants_q = !FP8;               // the segment's queries are not asked for yet
    const auto ask_q = [&] {
      ++nq;
      wants_q = false;
      if (lane == 0) {
        const int rows = a.nt * a.G, qs = a.pair_keys ? 1 : 2;
        const uint32_t bar = smem_u32(&bars->q_full);
        tc::mbar_arrive_expect_tx(bar, (uint32_t)(qs * rows * D * 2));
        for (int x = 0; x < qs; ++x)
          for (int p = 0; p < D / 64; ++p)
            tc::tma_load_3d(sQ + x * C::kQBytes + p * (kRows * 128), &a.qmap, bar, p * 64, (g.tile * qs + x) * a.nt,
                            g.b * a.H_q + g.h * a.G);
      }
      __syncwarp();
    };
    const auto put = [&](bool vals, int t) {
      const uint32_t st = it % C::kStages;
      // keys and values run ahead of the queries, which wait for the last segment's products
      for (uint32_t n = 0; wants_q; ++n) {
        if (nq == 0 || __all_sync(0xffffffffu, tc::mbar_try_wait(smem_u32(&bars->q_empty), (nq - 1) & 1))) ask_q();
        else if (__all_sync(0xffffffffu, tc::mbar_try_wait(smem_u32(&bars->kv_empty[st]), ((it / C::kStages) & 1) ^ 1))) break;
        else if (n >= a.wait_limit) ok = false;
        if (!ok) return;
      }
      if (ok) ok = poll(smem_u32(&bars->kv_empty[st]), ((it / C::kStages) & 1) ^ 1, a.wait_limit);
      if (!ok) return;
      if (lane == 0) load_tile<D, FP8>(a, g, vals, t, ring + st * C::kStageBytes, smem_u32(&bars->kv_full[st]));
      __syncwarp();
      ++it;
    };
    // in the order of the products
    const int t1 = g.last(subs);
    for (int i = 0; i <= g.cnt && ok; ++i) {
      for (int x = 0; x < subs; ++x) {
        if (i > 0) put(true, t1 - (i - 1) * subs - x);
        if (i < g.cnt) put(false, t1 - i * subs - x);
      }
    }
    if (wants_q && ok) {
      ok = poll(smem_u32(&bars->q_empty), (nq - 1) & 1, a.wait_limit);
      if (ok) ask_q();
    }
  } while (ok && w.next(a));
  // every copy issued has landed before the CTA may leave
  const uint32_t lo = it > (uint32_t)C::kStages ? it - C::kStages : 0;
  for (uint32_t i = lo; i < it; ++i)
    scan::drain_wait(smem_u32(&bars->kv_full[i % C::kStages]), (i / C::kStages) & 1, a.status);
  if (nq > 0) scan::drain_wait(smem_u32(&bars->q_full), (nq - 1) & 1, a.status);
  return ok;
}

// 8-bit cache: the warp that brings in a tile's positions and scales, and what the
// queries see of them.  A warp of its own: beside the copies it took as long as the
// products of a pair of tiles.
template <bool BIAS>
__device__ bool meta_warp(const Args& a, const Here& here, Bars* bars, Meta* meta) {
  const int lane = threadIdx.x & 31, subs = a.pair_keys ? 2 : 1;
  uint32_t mt = 0;
  bool ok = true;
  Walk w;
  if (!w.begin(a, here)) return true;
  do {
    const Seg& g = w.g;
    bool bad;
    const int n_rows = rows_held(a, g.b, &bad), b = g.b / a.H_kv, h = g.b - b * a.H_kv;
    const int per = a.nt * (a.pair_keys ? 1 : 2), tk0 = g.tile * per, tk1 = min(tk0 + per, a.T);
    const int q_seen = w.seen[g.b].y;
    int q_hi = -1, q_lo = INT_MAX;
    for (int t = tk0 + lane; t < tk1; t += 32) {
      const int p = __ldg(a.q_pos + (int64_t)b * a.T + t);
      q_lo = min(q_lo, p), q_hi = max(q_hi, p);
    }
    q_lo = __reduce_min_sync(0xffffffffu, q_lo);
    q_hi = __reduce_max_sync(0xffffffffu, q_hi);
    // the next tiles' are on their way
    constexpr int kAhead = 3;
    struct Rows { int pos[4]; float2 scale; };
    Rows ahead[kAhead];
    const int64_t row0 = (int64_t)b * a.s.off[a.H_kv] + a.s.off[h];
    const int t1 = g.last(subs), t_end = t1 - g.cnt * subs;    // the tiles go downward
    const auto fetch = [&](int t) {
      Rows r;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = t * kKeys + x * 32 + lane;
        r.pos[x] = t > t_end && row < n_rows ? __ldg(a.pos + row0 + row) : -1;
      }
      r.scale = make_float2(1.f, kLeastUnit);
      const int block = t * (kKeys / q8::kRows) + lane;
      if (t > t_end && lane < kKeys / q8::kRows && block * q8::kRows < n_rows)
        r.scale = __ldg(a.scale + row0 / q8::kRows + block);
      return r;
    };
#pragma unroll
    for (int x = 0; x < kAhead; ++x) ahead[x] = fetch(t1 - x);
    for (int t = t1; t > t_end; --t, ++mt) {
      const Rows r = ahead[0];
#pragma unroll
      for (int x = 0; x + 1 < kAhead; ++x) ahead[x] = ahead[x + 1];
      ahead[kAhead - 1] = fetch(t - kAhead);
      ok = poll(smem_u32(&bars->meta_empty[mt % kMeta]), ((mt / kMeta) & 1) ^ 1, a.wait_limit);
      if (!ok) return false;
      Meta& m = meta[mt % kMeta];
      uint32_t seen = 0;             // lane y: of block y
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int p = r.pos[x];
        m.pos[x * 32 + lane] = p;
        if constexpr (BIAS) m.rel[x * 32 + lane] = (float)(int)((uint32_t)p - (uint32_t)q_hi);
        const uint32_t some = __ballot_sync(0xffffffffu, p >= 0 && p <= q_seen);
        const bool all = __all_sync(0xffffffffu, p >= 0 && p <= q_lo);
        if (lane == 0) m.some[x] = some, m.mixed[x] = all ? 0 : 1;
        if (lane >> 1 == x) seen = some >> (lane & 1) * 16 & 0xffffu;
      }
      if (lane < kKeys / q8::kRows)  // a block of which nothing is seen may have anything for a scale
        m.scale[lane] = seen ? r.scale : make_float2(1.f, kLeastUnit);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(smem_u32(&bars->meta_full[mt % kMeta]));
    }
  } while (w.next(a));
  return ok;
}

// ------------------------------------------------------------------- the products
// Rows of a stage whose bit is not set become zeros: what no query of the unit sees
// may hold anything, and a weight of zero times NaN would not be zero.
template <int D, bool FP8>
__device__ __forceinline__ void zero_rows(uint32_t stage, uint32_t keep, int word) {
  constexpr int kRow = FP8 && D == 64 ? 64 : 128, kPanels = FP8 || D == 64 ? 1 : 2;
  constexpr int kAtOnce = 512 / kRow;              // rows of a store of the warp
  const int lane = threadIdx.x & 31, row = lane / (kRow / 16);
#pragma unroll
  for (int y = 0; y < 32; y += kAtOnce)
    if (!(keep >> (y + row) & 1)) {
#pragma unroll
      for (int p = 0; p < kPanels; ++p)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(stage + p * (kKeys * 128) +
                                                                        (word * 32 + y) * kRow + lane * 16),
                     "r"(0)
                     : "memory");
    }
}

template <int D>
__device__ __forceinline__ uint32_t col_o(int x) { return kColO + x * D; }
// The weights over the scores; at D = 64, where the two products have different
// shapes and so no order of their own, in columns that are left.
template <int D>
__device__ __forceinline__ uint32_t col_p(int x) { return D == 64 ? kColO + 128 + x * 64 : kColS + x * 128; }

template <int D, bool FP8>
__device__ __forceinline__ void issue_scores(uint32_t tmem, int x, uint32_t q, uint32_t stage) {
  constexpr uint32_t kId = idesc<FP8>(kKeys, false);
  constexpr int kRow = FP8 ? D : 128;
  const uint64_t qd = desc_rows<kRow>(q, 16), kd = desc_rows<kRow>(stage, 16);
  const uint32_t d = tmem + kColS + x * 128;
  if constexpr (FP8) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int s = 0; s < D / 32; ++s)
        mma_ss<true>(d, qd + ((p * (kRows * D) + s * 32) >> 4), kd + (s * 32 >> 4), kId, p + s > 0);
  } else {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint32_t at = ((s >> 2) * (kRows * 128) + (s & 3) * 32) >> 4;
      mma_ss<false>(d, qd + at, kd + at, kId, s > 0);
    }
  }
}
template <int D, bool FP8>
__device__ __forceinline__ void issue_output(uint32_t tmem, int x, uint32_t stage, bool add) {
  constexpr uint32_t kId = idesc<FP8>(D, true);
  constexpr int kRow = FP8 ? D : 128;
  const uint64_t vd = desc_rows<kRow>(stage, kKeys * 128);
  const uint32_t d = tmem + col_o<D>(x), p = tmem + col_p<D>(x);
  if constexpr (FP8) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int s = 0; s < kKeys / 32; ++s)
        mma_ts<true>(d, p + y * 32 + s * 8, vd + (s * 32 * D >> 4), kId, add || y + s > 0);
  } else {
#pragma unroll
    for (int s = 0; s < kKeys / 16; ++s) mma_ts<false>(d, p + s * 8, vd + (s * 16 * 128 >> 4), kId, add || s > 0);
  }
}

// A warp per stream; it waits as a whole, lane 0 issues.  Two, as an issuer spends
// about as long on its waits and hand-overs as its products run, which the other
// stream's products cover.  They take turns: products issued at once share the
// tensor core and end together, and then both streams make weights at once, with
// the tensor core idle, and wait for it at once.
template <int D, bool FP8>
__device__ bool mma_warp(const Args& a, const Here& here, Bars* bars, int x, uint32_t sQ, uint32_t ring,
                         const Meta* meta, uint32_t tmem) {
  using C = Cfg<D, FP8>;
  const int lane = threadIdx.x & 31;
  const int subs = a.pair_keys ? 2 : 1;
  const uint32_t q_at = sQ + (a.pair_keys ? 0 : x) * C::kQBytes;
  uint32_t it = 0, mt = 0, seg = 0, steps = 0, turns = 0;
  bool ok = true;
  const auto wait = [&](uint64_t* bar, uint32_t phase) { return poll(smem_u32(bar), phase & 1, a.wait_limit); };
  Walk w;
  if (w.begin(a, here)) do {
    const Seg& g = w.g;
    const int t1 = g.last(subs);
    const int2 seen = w.seen[g.b];
    // Rows of tile `t` that no query of the call sees become zeros (both streams' warps may
    // write the same ones).  Only those may hold anything: where the sequence's queries
    // see one range between them (no holes), tiles within need no look; else what no query
    // of the unit sees does.
    const auto clean = [&](int t, uint32_t m, uint32_t stage) {
      uint32_t keep[4] = {};
      const int k = t * kKeys;
      const auto add = [&](int l, int h) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int first = max(l - k - 32 * y, 0), last = min(h - k - 32 * y, 31);
          if (first <= last) keep[y] |= (0xffffffffu >> (31 - last)) & (0xffffffffu << first);
        }
      };
      if constexpr (FP8) {
        ok = ok && wait(&bars->meta_full[m % kMeta], m / kMeta);
#pragma unroll
        for (int y = 0; y < 4; ++y) keep[y] = meta[m % kMeta].some[y];
      } else if (seen.x >= 0) {
        if (seen.x <= k && seen.y >= k + kKeys - 1) return;
        add(seen.x, seen.y);
      } else {
        const int per = a.nt * (a.pair_keys ? 1 : 2), tk0 = g.tile * per, tk1 = min(tk0 + per, a.T);
        for (int tk = tk0 + lane; tk < tk1; tk += 32) {
          int l, h;
          if (key_range(a, (int64_t)g.b * a.T + tk, l, h)) add(l, h);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) keep[y] = __reduce_or_sync(0xffffffffu, keep[y]);
      }
      if ((keep[0] & keep[1] & keep[2] & keep[3]) == 0xffffffffu) return;
#pragma unroll
      for (int y = 0; y < 4; ++y) zero_rows<D, FP8>(stage, keep[y], y);
      tc::fence_proxy_async();
      __syncwarp();
    };
    ok = ok && wait(&bars->q_full, seg);
    for (int i = 0; i <= g.cnt && ok; ++i, ++turns) {
      // places in the ring: K(0), then V(i - 1), K(i), ..; key pairs: both streams' in turn
      const uint32_t v_it = it + (a.pair_keys ? 4 * i - 2 + (i == g.cnt ? x : 2 * x) : 2 * i - 1);
      const uint32_t k_it = it + (a.pair_keys ? (i == 0 ? x : 4 * i - 1 + 2 * x) : 2 * i);
      const uint32_t v_st = v_it % C::kStages, k_st = k_it % C::kStages;
      if (i > 0) {
        ok = ok && wait(&bars->kv_full[v_st], v_it / C::kStages);
        if (!ok) break;
        const int sub = a.pair_keys ? 2 * (i - 1) + x : i - 1;
        clean(t1 - sub, mt + sub, ring + v_st * C::kStageBytes);
        if (FP8 && lane == 0) tc::mbar_arrive(smem_u32(&bars->meta_empty[(mt + sub) % kMeta]));
      }
      if (i < g.cnt) ok = ok && wait(&bars->kv_full[k_st], k_it / C::kStages);
      ok = ok && wait(&bars->turn[x], x == 0 ? turns - 1 : turns);
      if (i > 0) ok = ok && wait(&bars->p_full[x], steps + i - 1);
      if (!ok) break;
      tc::fence_after_sync();
      if (elect_one()) {
        if (i > 0) {
          issue_output<D, FP8>(tmem, x, ring + v_st * C::kStageBytes, i > 1);
          tc::mma_commit(smem_u32(&bars->kv_empty[v_st]));
          if (i == g.cnt) tc::mma_commit(smem_u32(&bars->s_end[x]));
        }
        if (i < g.cnt) {
          issue_scores<D, FP8>(tmem, x, q_at, ring + k_st * C::kStageBytes);
          tc::mma_commit(smem_u32(&bars->s_full[x]));
          tc::mma_commit(smem_u32(&bars->kv_empty[k_st]));
          if (!FP8 && i == g.cnt - 1) tc::mma_commit(smem_u32(&bars->q_empty));
        }
        tc::mbar_arrive(smem_u32(&bars->turn[x ^ 1]));
      }
      __syncwarp();
    }
    it += g.cnt * 2 * subs;
    mt += g.cnt * subs;
    steps += g.cnt;
    ++seg;
  } while (ok && w.next(a));
  if (elect_one()) scan::drain_mma(smem_u32(&bars->drain[x]), a.status);
  __syncwarp();
  return ok;
}

// ------------------------------------------------------------------- the weights
// A query row of bf16 -> two e4m3 parts in shared memory; returns the power of two
// that was taken out.
template <int D>
__device__ __forceinline__ float write_query(const __nv_bfloat16* q, bool live, uint32_t sq, int row) {
  uint4 w[D / 8];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    w[i] = live ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
    mx = __vmaxu2(__vmaxu2(mx, w[i].x & 0x7fff7fffu), __vmaxu2(w[i].y & 0x7fff7fffu, w[i].z & 0x7fff7fffu));
    mx = __vmaxu2(mx, w[i].w & 0x7fff7fffu);
  }
  mx = max(mx & 0xffffu, mx >> 16);
  // the row's largest value into [2^7, 2^8)
  const uint32_t e = mx >> 7, ee = e == 255 ? 134u : min(max(e, 8u), 254u);
  // a row that is not finite becomes NaN: the conversions would make an infinity a number
  const float down = __uint_as_float(e == 255 ? 0x7fffffffu : (261u - ee) << 23);
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t p[2][4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint4 v = w[2 * c + (y >> 1)];
      const uint32_t u0 = y & 1 ? v.z : v.x, u1 = y & 1 ? v.w : v.y;
      uint16_t a[2], b[2];
      split2(__uint_as_float(u0 << 16) * down, __uint_as_float(u0 & 0xffff0000u) * down, a[0], b[0]);
      split2(__uint_as_float(u1 << 16) * down, __uint_as_float(u1 & 0xffff0000u) * down, a[1], b[1]);
      p[0][y] = (uint32_t)a[0] | (uint32_t)a[1] << 16;
      p[1][y] = (uint32_t)b[0] | (uint32_t)b[1] << 16;
    }
    const uint32_t at = D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ (row >> 1 & 3)) << 4);
#pragma unroll
    for (int y = 0; y < 2; ++y)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(sq + y * (kRows * D) + at), "r"(p[y][0]),
                   "r"(p[y][1]), "r"(p[y][2]), "r"(p[y][3])
                   : "memory");
  }
  return __uint_as_float((ee - 7u) << 23);
}

// tanh of a pair, |x| <= kTanhNear: tanh_near.
__device__ __forceinline__ float2 tanh_near2(float2 x) {
  const auto both = [](float c) { return make_float2(c, c); };
  const float2 w = mul2(x, x);
  float2 p = fma2(w, both(0.015050944872200489f), both(-0.051821865141391754f));
  p = fma2(w, p, both(0.1330452561378479f));
  p = fma2(w, p, both(-0.3333195447921753f));
  p = fma2(w, p, both(0.9999998807907104f));
  return mul2(x, p);
}
// The same for |x| <= kTanhMid: eight terms, relative error 1.9e-7 with fp32's roundings.
constexpr float kTanhMid = 1.25f;
__device__ __forceinline__ float2 tanh_mid2(float2 x) {
  const auto both = [](float c) { return make_float2(c, c); };
  const float2 w = mul2(x, x);
  float2 p = fma2(w, both(-0.000182598116225563f), both(0.0015881144208833575f));
  p = fma2(w, p, both(-0.0067961555905640125f));
  p = fma2(w, p, both(0.02055717259645462f));
  p = fma2(w, p, both(-0.05349034070968628f));
  p = fma2(w, p, both(0.1332450658082962f));
  p = fma2(w, p, both(-0.3333269953727722f));
  p = fma2(w, p, both(0.9999999403953552f));
  return mul2(x, p);
}
// A score's product -> the cap's share of it, tanh, up to the factor returned.  Warps
// whose 32 rows have no large one take a polynomial alone: up to kTanhLow one of three
// terms (relative error 5e-7, fitted as tanh_near), which without block scales has the
// score's factor in its coefficients, then tanh_near and tanh_mid2, and only above those
// the special functions.  So a cap's cost goes by the scores: 2048 tokens behind 6K take
// 238 us where warps' largest scores are at 0.2 of the cap (260 with tanh_near for all,
// 186 without a cap), and 285, 332 and 387 at 0.7, 1.4 and 7 times the cap (336, 389, 396
// without tanh_mid2, before later steps).  Factors whose powers could leave the range
// take no coefficients of their own.
constexpr float kTanhLow = 0.25f;
template <bool BLOCKS>
__device__ __forceinline__ float cap_all(float (&x)[kHalf], const float2* f, float f1, float cap2) {
  constexpr float c0 = 0.9999995827674866f, c1 = -0.33321908116340637f, c2 = 0.12841613590717316f;
  const auto both = [](float c) { return make_float2(c, c); };
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < kHalf; k += 2) {
    if constexpr (BLOCKS) {
      const float2 v = mul2(make_float2(x[k], x[k + 1]), both(f[k / 16].x));
      x[k] = v.x, x[k + 1] = v.y;
    }
    asm("max.f32 %0, %0, %1, %2;\n" : "+f"(top) : "f"(fabsf(x[k])), "f"(fabsf(x[k + 1])));
  }
  if (!BLOCKS) top *= f1;
  if (__all_sync(0xffffffffu, top <= kTanhLow) && (BLOCKS || (f1 > 1e-6f && f1 < 1e3f))) {
    const float ff = BLOCKS ? 1.f : f1 * f1;
    const float2 d1 = both(c1 * ff), d2 = both(c2 * ff * ff);
#pragma unroll
    for (int k = 0; k < kHalf; k += 2) {
      const float2 v = make_float2(x[k], x[k + 1]), w = mul2(v, v), y = mul2(v, fma2(w, fma2(w, d2, d1), both(c0)));
      x[k] = y.x, x[k + 1] = y.y;
    }
    return BLOCKS ? cap2 : cap2 * f1;
  }
  if constexpr (!BLOCKS) {
#pragma unroll
    for (int k = 0; k < kHalf; k += 2) {
      const float2 v = mul2(make_float2(x[k], x[k + 1]), both(f1));
      x[k] = v.x, x[k + 1] = v.y;
    }
  }
  if (__all_sync(0xffffffffu, top <= kTanhNear)) {
#pragma unroll
    for (int k = 0; k < kHalf; k += 2) {
      const float2 v = tanh_near2(make_float2(x[k], x[k + 1]));
      x[k] = v.x, x[k + 1] = v.y;
    }
  } else if (__all_sync(0xffffffffu, top <= kTanhMid)) {
#pragma unroll
    for (int k = 0; k < kHalf; k += 2) {
      const float2 v = tanh_mid2(make_float2(x[k], x[k + 1]));
      x[k] = v.x, x[k + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kHalf; k += 2) {
      const float2 v = tanh_near2(make_float2(x[k], x[k + 1]));
      x[k] = fabsf(x[k]) <= kTanhNear ? v.x : tanh_far(x[k]);
      x[k + 1] = fabsf(x[k + 1]) <= kTanhNear ? v.y : tanh_far(x[k + 1]);
    }
  }
  return cap2;
}
// Four weights, fp16 pairs of 2^-8 of them, below 2^-8 * 448 and not negative -> the
// e4m3 codes of their two parts.  Times 2^-8 the exponents of e4m3 and fp16 are the
// same, subnormal numbers' too, so a code is bits 7 to 14: the first part is the weight
// cut off there, the second the rest, rounded.  The conversion instructions would
// take eight times as long as these few of the integer unit.
__device__ __forceinline__ void split4(uint32_t h0, uint32_t h1, uint32_t& a, uint32_t& b) {
  uint32_t r0, r1;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r0) : "r"(h0), "r"(h0 & 0xff80ff80u));
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r1) : "r"(h1), "r"(h1 & 0xff80ff80u));
  a = __byte_perm(h0 >> 7, h1 >> 7, 0x6420);
  b = __byte_perm((r0 + 0x00400040u) >> 7, (r1 + 0x00400040u) >> 7, 0x6420);
}

// A thread has a row's scores of half a tile; the two threads of a row tell each
// other their maxima (both need one reference: the row has one output).
template <int D, bool FP8, bool CAP, bool BIAS>
__device__ bool soft_warps(const Args& a, const Here& here, Bars* bars, float* s_max, float* s_most, uint32_t sQ,
                           const Meta* meta, uint32_t tmem, float* s_x) {
  using C = Cfg<D, FP8>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = warp >> 3, half = warp >> 2 & 1;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t s_at = tmem + lanes + kColS + x * 128 + half * kHalf, o_at = tmem + lanes;
  const uint32_t p_at = tmem + lanes + col_p<D>(x) + half * (FP8 ? 16 : 32);
  const int mine = (x * 2 + half) * kRows + row, its = (x * 2 + (half ^ 1)) * kRows + row;
  float* my_max = s_max + mine;
  const float* its_max = s_max + its;
  const int pair = 2 + x * 4 + (warp & 3);                   // the barrier of a row's two warps
  const int gq = row / a.nt, tl = row - gq * a.nt;           // query head of the group, token of the tile
  const int subs = a.pair_keys ? 2 : 1;
  const bool any_row = (warp & 3) * 32 < a.nt * a.G;         // none of the warp's rows is one: nothing reads its part
  uint32_t steps = 0, mt = 0, seg = 0;
  float ref = 0.f;
  int unit = 0;                        // 8-bit cache: outputs are in 2^unit
  bool ok = true;
  // after a wait that gave up: go on without waiting, so that no barrier is left alone
  const auto wait = [&](const uint64_t* bar, uint32_t phase) { return poll(smem_u32(bar), phase & 1, a.wait_limit); };
  Walk w;
  if (!w.begin(a, here)) return true;
  do {
    const Seg& g = w.g;
    const int bh = g.b * a.H1 + g.h, b = FP8 ? bh / a.H_kv : g.b, h = FP8 ? bh - b * a.H_kv : g.h;
    const int t = (g.tile * (a.pair_keys ? 1 : 2) + (a.pair_keys ? 0 : x)) * a.nt + tl;
    const bool live = gq < a.G && t < a.T;
    const int64_t q_row = ((int64_t)b * a.H_q + h * a.G + gq) * a.T + t;
    int lo = 0, hi = INT_MAX, qp = -1;
    float slope = 0.f, q_rel = 0.f;
    if (live) {
      qp = max(__ldg(a.q_pos + (int64_t)b * a.T + t), -1);
      if constexpr (!FP8) key_range(a, (int64_t)b * a.T + t, lo, hi);
      if constexpr (BIAS) slope = __ldg(a.slopes + h * a.G + gq) * kLog2e;
    }
    float c2 = a.scale2;
    if constexpr (FP8) {
      if constexpr (BIAS) {
        // positions in Meta are relative to the unit's last query
        const int per = a.nt * (a.pair_keys ? 1 : 2), t0 = g.tile * per, t1 = min(t0 + per, a.T);
        int last = -1;
        for (int y = t0 + lane; y < t1; y += 32) last = max(last, __ldg(a.q_pos + (int64_t)b * a.T + y));
        q_rel = (float)(__reduce_max_sync(0xffffffffu, last) - qp);
      }
      if (half == 0 && (!a.pair_keys || x == 0)) {
        c2 *= write_query<D>(a.q + (live ? q_row * D : 0), live, sQ + (a.pair_keys ? 0 : x) * C::kQBytes, row);
        tc::fence_proxy_async();
        s_max[(a.pair_keys ? 0 : x) * 2 * kRows + row] = c2;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(smem_u32(&bars->q_full));
      }
      asm volatile("bar.sync 1, 512;\n" ::: "memory");
      c2 = s_max[(a.pair_keys ? 0 : x) * 2 * kRows + row];
      asm volatile("bar.sync 1, 512;\n" ::: "memory");       // read before the first maxima are written there
    }
    // the last segment's reference, another row's, stands in until the row sees keys
    if (!(fabsf(ref) < 1e30f)) ref = 0.f;
    bool seen = false;
    float2 sum2[2] = {};
    const int t1 = g.last(subs);
    for (int i = 0; i < g.cnt; ++i, ++steps) {
      const int tile = t1 - i * subs - (a.pair_keys ? x : 0);
      const uint32_t m_at = mt + i * subs + (a.pair_keys ? x : 0);
      const Meta& me = meta[m_at % kMeta];
      if constexpr (FP8) ok = ok && wait(&bars->meta_full[m_at % kMeta], m_at / kMeta);
      ok = ok && wait(&bars->s_full[x], steps);
      tc::fence_after_sync();
      // The weights are made against the reference as it is, while the maximum is still
      // being found: it hardly ever moves.  Where it has to, the scores, which are still in
      // tensor memory, are taken again; and looked at again after a step of large numbers,
      // which are not exact where scores differ by a few.
      const bool fresh = !seen;        // nothing has been added up for the row
      for (int pass = 0; any_row; ++pass) {
        float s[kHalf];
#pragma unroll
        for (int y = 0; y < 2; ++y) tmem_ld32(s_at + 32 * y, s + 32 * y);
        float2 f[kHalf / 16] = {};     // of 16 keys: factor to log2 units (x), of the values (y)
        if constexpr (FP8) {
#pragma unroll
          for (int y = 0; y < kHalf / 16; ++y) {
            f[y] = me.scale[half * (kHalf / 16) + y];
            // a factor of 0 would make NaN of the masked scores
            f[y].x = CAP ? f[y].x * c2 * a.inv_cap2 : fmaxf(f[y].x * c2, 1.2e-38f);
          }
        }
        tc::tmem_wait_ld();
        tc::reg_fence(s, kHalf);
        if (pass) {                    // and the other's maxima of the last pass have been read
          tc::fence_before_sync();
          asm volatile("bar.sync %0, 64;\n" ::"r"(pair) : "memory");
          tc::fence_after_sync();
        }
        float cap2 = 0.f;
        if constexpr (CAP) cap2 = cap_all<FP8>(s, f, c2 * a.inv_cap2, a.cap2);
        // ---- mask
        if constexpr (FP8) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (me.mixed[2 * half + y]) {
#pragma unroll
              for (int z = 0; z < 8; ++z) {
                const int4 p = *reinterpret_cast<const int4*>(&me.pos[half * kHalf + 32 * y + 4 * z]);
                if (p.x < 0 || p.x > qp) s[32 * y + 4 * z] = -INFINITY;
                if (p.y < 0 || p.y > qp) s[32 * y + 4 * z + 1] = -INFINITY;
                if (p.z < 0 || p.z > qp) s[32 * y + 4 * z + 2] = -INFINITY;
                if (p.w < 0 || p.w > qp) s[32 * y + 4 * z + 3] = -INFINITY;
              }
            }
        } else {
          const int l = max(lo - tile * kKeys - half * kHalf, 0), r = min(hi - tile * kKeys - half * kHalf, kHalf - 1);
          if (__any_sync(0xffffffffu, r - l < kHalf - 1)) {
            unsigned long long in = l > r ? 0 : (~0ull >> (63 - (r - l))) << l;
            // as far as the compiler sees, no two rounds have the same: it would work the 64
            // bits out ahead of the loop, for every tile
            asm volatile("" : "+l"(in));
            const uint32_t in0 = (uint32_t)in, in1 = (uint32_t)(in >> 32);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (!(in0 & 1u << k)) s[k] = -INFINITY;
              if (!(in1 & 1u << k)) s[32 + k] = -INFINITY;
            }
          }
        }
        // ---- the scores less the reference: s times a factor plus `neg` and the bias.  The bias
        // of key k is `to` * (d0 + k) where the half tile lies on one side of the query
        float neg = -ref, to = 0.f;
        bool cross = false;
        int d0 = 0;
        if constexpr (BIAS && !FP8) {
          d0 = tile * kKeys + half * kHalf - qp;
          asm volatile("" : "+r"(d0));             // as l and r above
          cross = __any_sync(0xffffffffu, d0 < 0 && d0 + kHalf > 0);
          to = d0 < 0 ? slope : -slope;
          if (!cross) neg = fmaf(to, (float)d0, neg);
        }
        const auto both = [](float v) { return make_float2(v, v); };
        const auto scores = [&](int k, bool crossing) {            // of keys k and k + 1
          const float2 fk = both(CAP ? cap2 : FP8 ? f[k / 16].x : c2);
          float2 c = both(neg);
          if constexpr (BIAS && FP8) {
            const float2 rel = *reinterpret_cast<const float2*>(&me.rel[half * kHalf + k]);
            c = fma2(both(slope), add2(rel, both(q_rel)), c);
          } else if constexpr (BIAS) {
            c = crossing ? make_float2(fmaf(-slope, fabsf((float)d0 + k), neg), fmaf(-slope, fabsf((float)d0 + k + 1), neg))
                         : fma2(both(to), make_float2(k, k + 1), c);
          }
          return fma2(make_float2(s[k], s[k + 1]), fk, c);
        };
        if constexpr (BIAS && !FP8) {  // one or the other for the whole half tile
          if (cross) {
#pragma unroll
            for (int k = 0; k < kHalf; k += 2) {
              const float2 e = scores(k, true);
              s[k] = e.x, s[k + 1] = e.y;
            }
          } else {
#pragma unroll
            for (int k = 0; k < kHalf; k += 2) {
              const float2 e = scores(k, false);
              s[k] = e.x, s[k + 1] = e.y;
            }
          }
        }
        // ---- weights, and the maximum beside them: the exponentials' unit is the narrow one
        uint32_t p[kHalf / 2];         // bf16: pairs; e4m3: fours of the first part, then of the second
        float2 part[2] = {};
        float v[2] = {-INFINITY, -INFINITY}, top = -INFINITY, most = -INFINITY;
#pragma unroll
        for (int y = 0; y < kHalf / 4; ++y) {
          uint32_t h[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int k = 4 * y + 2 * z;
            float2 e = make_float2(s[k], s[k + 1]);
            if constexpr (!BIAS || FP8) e = scores(k, false);
            v[z] = max3(v[z], e.x, e.y);
            float2 u = make_float2(ex2(e.x), ex2(e.y));
            part[z] = add2(part[z], u);
            if constexpr (FP8) {
              // times the values' scale over 2^unit and 2^-8.  0 below the normal numbers; above them
              // the weight is 0, or the tile is taken again
              const int e = (int)(__float_as_uint(f[k / 16].y) >> 23) - unit - 8;
              u = mul2(u, both(__int_as_float(min(max(e, 0), 254) << 23)));
              asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h[z]) : "f"(u.y), "f"(u.x));
            } else {
              p[2 * y + z] = bf16x2_of(u.x, u.y);
            }
          }
          if constexpr (FP8) split4(h[0], h[1], p[y], p[kHalf / 4 + y]);
          if (FP8 && y % 4 == 3) {     // the end of a block
            const float b = fmaxf(v[0], v[1]);
            top = fmaxf(top, b);
            most = fmaxf(most, b + log2_of(f[y / 4].y));
            v[0] = v[1] = -INFINITY;
          }
        }
        if constexpr (!FP8) top = fmaxf(v[0], v[1]);
        // ---- did the reference and the unit hold?  (m: the row's largest score less the
        // reference, c: log2 of its largest contribution, in units)
        if (pass < kPasses) {
          *my_max = top;
          if constexpr (FP8) s_most[mine] = most;
          tc::fence_before_sync();
          asm volatile("bar.sync %0, 64;\n" ::"r"(pair) : "memory");
          tc::fence_after_sync();
          const float m = fmaxf(top, *its_max);
          float c = C::kLeast;
          if constexpr (FP8) c = fmaxf(most, s_most[its]) - (float)unit;
          // the row's first keys, and the reference and the unit, which are another row's, far from them
          const bool first =
              fresh && m > -INFINITY && !(m >= C::kLow && m <= C::kHigh && c >= C::kLeast && c <= C::kMost);
          const bool move = first || m > C::kHigh || c > C::kMost;
          seen |= m > -INFINITY;
          if (__any_sync(0xffffffffu, move)) {
            // whole steps, so that a unit can follow them: weights are 2^(x - ref), contributions
            // in 2^(ref + unit)
            const float was = ref;
            ref += first ? floorf(m) : fmaxf(0.f, floorf(m));
            const float up = ref - was;
            if (!__any_sync(0xffffffffu, fabsf(was) > kExact || fabsf(up) > kExact)) pass = kPasses;
            float fo = fresh ? 1.f : ex2(-up);
#pragma unroll
            for (int y = 0; y < 2; ++y) sum2[y].x *= fo, sum2[y].y *= fo;
            if constexpr (FP8) {
              const float more = first ? floorf(c) - C::kLeast : fmaxf(0.f, floorf(c) - C::kLeast);
              unit = max(-126, min((int)((float)unit + (more - up)), 127));
              if (!fresh) fo = ex2(-more);
            }
            if (i > 0) {               // half of the row's output
#pragma unroll
              for (int y = 0; y < D / 32; ++y) {
                float o[16];
                const uint32_t at = o_at + col_o<D>(x) + half * (D / 2) + 16 * y;
                tc::tmem_ld16(at, o);
                tc::tmem_wait_ld();
                tc::reg_fence(o, 16);
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] *= fo;
                tc::tmem_st16(at, reinterpret_cast<const uint32_t*>(o));
              }
            }
            continue;
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) sum2[y] = add2(sum2[y], part[y]);
        tc::tmem_st16(p_at, p);
        tc::tmem_st16(p_at + (FP8 ? 32 : 16), p + 16);
        tc::tmem_wait_st();
        break;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(smem_u32(&bars->p_full[x]));
      if (FP8 && lane == 0) tc::mbar_arrive(smem_u32(&bars->meta_empty[m_at % kMeta]));
    }
    // ---- the segment's end: the threads of a row tell each other their sums (and, key
    // pairs, the streams' references), and share out its dims
    ok = ok && wait(&bars->s_end[x], seg);
    float sum = (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
    const bool whole = g.s0 == 0 && g.cnt == g.n;
    const int64_t slot = 2 * blockIdx.x + (g.s0 == 0 ? 1 : 0);
    float said = seen ? ref : kNoRef;
    tc::fence_before_sync();
    *my_max = sum;
    if (a.pair_keys && half == 0) s_x[x * kRows + row] = said, s_x[(2 + x) * kRows + row] = FP8 ? q8::pow2(unit + 127) : 1.f;
    asm volatile("bar.sync 1, 512;\n" ::: "memory");
    tc::fence_after_sync();
    sum = s_max[x * 2 * kRows + row] + s_max[(x * 2 + 1) * kRows + row];
    float f0 = FP8 ? q8::pow2(unit + 127) : 1.f, f1 = 0.f;
    int from = half * (D / 2), dims = D / 2, first = x;
    if (a.pair_keys) {
      const float ra = s_x[row], rb = s_x[kRows + row], top = fmaxf(ra, rb);
      f0 = ex2(ra - top), f1 = ex2(rb - top);
      sum = (s_max[row] + s_max[kRows + row]) * f0 + (s_max[2 * kRows + row] + s_max[3 * kRows + row]) * f1;
      said = top;
      if constexpr (FP8) f0 *= s_x[2 * kRows + row], f1 *= s_x[3 * kRows + row];
      from = (2 * x + half) * (D / 4), dims = D / 4, first = 0;
    }
    if (any_row) {
      // a part of a unit is divided by its own sum, and joined by it: no larger than a value
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      f0 *= inv, f1 *= inv;
      const int64_t part = slot * ((a.pair_keys ? 1 : 2) * kRows) + (a.pair_keys ? 0 : x) * kRows + row;
      for (int d = from; d < from + dims; d += 16) {
        float o[16];
        tc::tmem_ld16(o_at + col_o<D>(first) + d, o);
        tc::tmem_wait_ld();
        tc::reg_fence(o, 16);
        if (a.pair_keys) {
          float o1[16];
          tc::tmem_ld16(o_at + col_o<D>(1) + d, o1);
          tc::tmem_wait_ld();
          tc::reg_fence(o1, 16);
#pragma unroll
          for (int z = 0; z < 16; ++z) o[z] = o[z] * f0 + o1[z] * f1;
        } else {
#pragma unroll
          for (int z = 0; z < 16; ++z) o[z] *= f0;
        }
        if (sum == 0.f) {              // a row that saw nothing
#pragma unroll
          for (int z = 0; z < 16; ++z) o[z] = 0.f;
        }
        if (!live) continue;
        if (whole) {
          uint32_t v[8];
#pragma unroll
          for (int z = 0; z < 8; ++z) v[z] = bf16x2_of(o[2 * z], o[2 * z + 1]);
          uint4* p = reinterpret_cast<uint4*>(a.out + q_row * D + d);
          p[0] = make_uint4(v[0], v[1], v[2], v[3]);
          p[1] = make_uint4(v[4], v[5], v[6], v[7]);
        } else {
          float* p = a.part_o + slot * ((a.pair_keys ? 1 : 2) * kRows * D) +
                     ((a.pair_keys ? 0 : x) * kRows + row) * a.part_row + d / 4 * a.part_step;
#pragma unroll
          for (int z = 0; z < 4; ++z)
            *reinterpret_cast<float4*>(p + z * a.part_step) = make_float4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
        }
      }
      if (live && from == 0) {
        if (!whole) a.part_ml[part] = make_float2(said, sum);
        else if (a.lse) a.lse[q_row] = sum == 0.f ? -INFINITY : (said + log2f(sum)) * kLn2;
      }
    }
    // the next segment's weights, outputs and what is told come after everybody's reads
    tc::fence_before_sync();
    asm volatile("bar.sync 1, 512;\n" ::: "memory");
    mt += g.cnt * subs;
    ++seg;
  } while (w.next(a));
  return ok;
}

// Rows of the streams' tiles that are no query, bf16: the copies of the queries never
// write them, so they are made zeros once.  Their scores take part where a warp decides for
// its rows together (does a reference move, which form of the tangent), and what an
// earlier kernel left there would decide with them.
template <int D>
__device__ __forceinline__ void clear_rows(const Args& a, uint32_t sQ) {
  const int rows = a.nt * a.G, pieces = (kRows - rows) * 8;  // of 16 bytes; a row of a panel is 128 bytes
  for (int x = 0; x < (a.pair_keys ? 1 : 2); ++x)
    for (int p = 0; p < D / 64; ++p)
      for (int i = threadIdx.x; i < pieces; i += kThreads)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(sQ + x * Cfg<D, false>::kQBytes +
                                                                        p * (kRows * 128) + rows * 128 + i * 16),
                     "r"(0)
                     : "memory");
  tc::fence_proxy_async();
}

template <int D, bool FP8, bool CAP, bool BIAS>
__device__ __forceinline__ void attend(const Args& a) {
  using C = Cfg<D, FP8>;
  static_assert(C::kStages <= kMaxStages, "barriers of the ring");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // a whole number of 1024 bytes, so that what follows is aligned without a gap: at
  // D = 128 the two fill a CTA's 227 KB
  struct alignas(1024) Small {
    Bars bars;
    uint32_t tmem;
    float max[4 * kRows];
    Here here;
  };
  static_assert(sizeof(Small) == 3 * 1024 && C::kSmem + sizeof(Small) <= 232448, "shared memory of a CTA");
  __shared__ Small small;
  Bars& bars = small.bars;
  uint32_t& s_tmem = small.tmem;
  uint8_t* const base = smem_raw;
  const uint32_t sQ = smem_u32(base), ring = sQ + 2 * C::kQBytes;
  if (sQ % 1024 != 0) {              // no placement does this; the products need it
    record_status(a.status, kStatusTimeout);
    return;
  }
  Meta* meta = reinterpret_cast<Meta*>(base + 2 * C::kQBytes + C::kStages * C::kStageBytes);
  float* s_most = reinterpret_cast<float*>(base + C::kSmem - C::kMostBytes);
  float* s_x = reinterpret_cast<float*>(base + C::kQBytes);       // key pairs: stream 1 has no queries of its own
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(smem_u32(&bars.kv_full[i]), 1);
      tc::mbar_init(smem_u32(&bars.kv_empty[i]), a.pair_keys ? 1 : 2);   // streams that multiply a tile
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(smem_u32(&bars.s_full[i]), 1);
      tc::mbar_init(smem_u32(&bars.s_end[i]), 1);
      tc::mbar_init(smem_u32(&bars.p_full[i]), 8);
    }
    for (int i = 0; i < kMeta; ++i) {
      tc::mbar_init(smem_u32(&bars.meta_full[i]), 1);
      tc::mbar_init(smem_u32(&bars.meta_empty[i]), a.pair_keys ? 9 : 18);      // eight warps of weights and an issuer a stream
    }
    tc::mbar_init(smem_u32(&bars.q_full), FP8 ? (a.pair_keys ? 4 : 8) : 1);
    tc::mbar_init(smem_u32(&bars.q_empty), 2);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(smem_u32(&bars.turn[i]), 1);
      tc::mbar_init(smem_u32(&bars.drain[i]), 1);
    }
    tc::fence_barrier_init();
    tc::tma_prefetch_desc(&a.kmap);
    tc::tma_prefetch_desc(&a.vmap);
    if (!FP8) tc::tma_prefetch_desc(&a.qmap);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_u32(&s_tmem), kCols);
    tc::tmem_relinquish();
  }
  if constexpr (!FP8) clear_rows<D>(a, sQ);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  grid_dep_wait();
  grid_dep_launch();
  Here& here = small.here;
  if (!a.planned) plan_here<FP8>(a, here, *reinterpret_cast<Scratch*>(base + 2 * C::kQBytes));
  bool ok = true;
  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    ok = soft_warps<D, FP8, CAP, BIAS>(a, here, &bars, small.max, s_most, sQ, meta, tmem, s_x);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) ok = load_warp<D, FP8>(a, here, &bars, sQ, ring);
    else if (FP8 && warp == kMetaWarp) ok = meta_warp<BIAS>(a, here, &bars, meta);
    else if (warp < kLoadWarp) ok = mma_warp<D, FP8>(a, here, &bars, warp - kMmaWarp, sQ, ring, meta, tmem);
  }
  if (!ok && (threadIdx.x & 31) == 0) record_status(a.status, kStatusTimeout);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kCols);
}

// ------------------------------------------------------------------- the join
// The CTAs of blockIdx.x = c join the unit that is cut first at the start of range
// c + 1, if one is: a warp a row, its parts in the order of the ranges.
constexpr int kJoinRows = 8;         // rows of a CTA
template <int D>
__global__ void __launch_bounds__(kJoinRows * 32) join_kernel(const __grid_constant__ Args a) {
  constexpr int V = D / 32;
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, streams = a.pair_keys ? 1 : 2, rows = a.nt * a.G;
  const int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5), x = r / rows, row = r - x * rows, gq = row / a.nt;
  grid_dep_wait();
  grid_dep_launch();
  const Start st = a.start[c];
  const long long L = a.plan->L;
  if (x >= streams || st.b < 0 || st.off == 0 || st.off > L) return;
  const int t = (st.tile * streams + x) * a.nt + row - gq * a.nt;
  if (t >= a.T) return;
  const int parts = 1 + (int)((st.n - st.off + L - 1) / L);
  const int bh = st.b * a.H1 + st.h, b = bh / a.H_kv, h = bh - b * a.H_kv;
  const int64_t q_row = ((int64_t)b * a.H_q + h * a.G + gq) * a.T + t;
  const auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + p)); };
  const int unit_rows = streams * kRows, in = x * kRows + row;
  float top = kNoRef, l = 0.f, v[V];
#pragma unroll
  for (int z = 0; z < V; ++z) v[z] = 0.f;
  for (int p0 = 0; p0 < parts; p0 += 32) {        // 32 parts at a time: a lane has one's reference and sum
    const float2 ml = p0 + lane < parts ? a.part_ml[slot(p0 + lane) * unit_rows + in] : make_float2(kNoRef, 0.f);
    float next = fmaxf(top, ml.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, o));
    const float f0 = ex2(top - next), f = ml.y * ex2(ml.x - next);
    top = next;
    float sum = f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = fmaf(l, f0, sum);
#pragma unroll
    for (int z = 0; z < V; ++z) v[z] *= f0;
    const int n = min(32, parts - p0);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float fp = __shfl_sync(0xffffffffu, f, p);
      float y[V];
      const float* o = a.part_o + slot(p0 + p) * (unit_rows * D) + in * a.part_row + lane * V / 4 * a.part_step + lane * V % 4;
      if constexpr (V == 4) *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(o);
      else *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(o);
#pragma unroll
      for (int z = 0; z < V; ++z) v[z] = fmaf(y[z], fp, v[z]);
    }
  }
  uint32_t w[V / 2];
#pragma unroll
  for (int z = 0; z < V / 2; ++z) w[z] = l == 0.f ? 0u : bf16x2_of(v[2 * z] / l, v[2 * z + 1] / l);
  __nv_bfloat16* o = a.out + q_row * D + lane * V;
  if constexpr (V == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
  if (a.lse && lane == 0) a.lse[q_row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- host side
// How a call's query rows are laid out, and its scratch.
struct Layout {
  int nt, tiles, pair_keys, P;
  size_t off_units, off_sees, off_seen, off_before, off_start, off_ml, off_o, total;
};
inline Layout layout(int64_t B1, int T, int G, int D) {
  Layout l{};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.P = std::max(num_sms(), 1);
  l.pair_keys = T <= kRows / G;
  l.nt = l.pair_keys ? T : kRows / G;
  const int per = l.nt * (l.pair_keys ? 1 : 2);
  l.tiles = (T + per - 1) / per;
  const size_t units = (size_t)B1 * l.tiles, rows = (size_t)2 * l.P * kRows * (l.pair_keys ? 1 : 2);
  l.off_units = 256;
  l.off_sees = up(l.off_units + units * sizeof(int2));
  l.off_seen = up(l.off_sees + units * sizeof(int2));
  l.off_before = up(l.off_seen + (size_t)B1 * sizeof(int2));
  l.off_start = up(l.off_before + (units + 1) * sizeof(long long));
  l.off_ml = up(l.off_start + (size_t)(l.P + 1) * sizeof(Start));
  l.off_o = up(l.off_ml + rows * sizeof(float2));
  l.total = l.off_o + rows * D * sizeof(float);
  return l;
}
inline void place(Args& a, const Layout& l, int D, void* ws) {
  char* w = static_cast<char*>(ws);
  a.plan = reinterpret_cast<Plan*>(w);
  a.units = reinterpret_cast<int2*>(w + l.off_units);
  a.sees = reinterpret_cast<int2*>(w + l.off_sees);
  a.seen = reinterpret_cast<int2*>(w + l.off_seen);
  a.before = reinterpret_cast<long long*>(w + l.off_before);
  a.start = reinterpret_cast<Start*>(w + l.off_start);
  a.part_ml = reinterpret_cast<float2*>(w + l.off_ml);
  a.part_o = reinterpret_cast<float*>(w + l.off_o);
  a.nt = l.nt, a.tiles = l.tiles, a.pair_keys = l.pair_keys, a.P = l.P;
  const bool spread = l.nt * a.G < 32 || (int64_t)a.B1 * a.H1 * l.tiles * 4 < l.P;
  a.part_row = spread ? D : 4, a.part_step = spread ? 4 : 4 * kRows * (l.pair_keys ? 1 : 2);
  a.status = status_word_ptr();
  a.wait_limit = wait_limit_polls();
}

inline bool encode3(CUtensorMap* map, CUtensorMapDataType type, const void* ptr, const cuuint64_t (&dims)[3],
                    const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
  auto enc = scan::get_encode();
  if (!enc) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Queries [heads][T][D] bf16 in boxes of nt tokens of G heads: a row tile.
inline bool map_queries(CUtensorMap* map, const void* q, int D, int T, uint64_t heads, int nt, int G) {
  return encode3(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, {(cuuint64_t)D, (cuuint64_t)T, heads},
                 {(cuuint64_t)D * 2, (cuuint64_t)T * D * 2}, {64, (cuuint32_t)nt, (cuuint32_t)G},
                 CU_TENSOR_MAP_SWIZZLE_128B);
}
// Blocks of 16 rows of D bytes, in boxes of a key tile.
inline bool map_blocks(CUtensorMap* map, const void* p, int D, uint64_t blocks) {
  return encode3(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, {(cuuint64_t)D, q8::kRows, blocks},
                 {(cuuint64_t)D, (cuuint64_t)D * q8::kRows}, {(cuuint32_t)D, q8::kRows, kKeys / q8::kRows},
                 D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Up to so many units the planning kernel counts the steps itself: one launch less.
constexpr int kCountHere = 256;
template <int D, bool FP8>
cudaError_t launch(Args& a, void (*kern)(Args), cudaStream_t st) {
  using C = Cfg<D, FP8>;
  const int64_t units = (int64_t)a.B1 * a.tiles;
  a.planned = units > kPlanHere;
  const int counted = units > kCountHere;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmem);
  if (e == cudaSuccess && counted)
    e = launch_pdl(count_kernel<FP8>, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, st, a);
  if (e == cudaSuccess && a.planned) e = launch_pdl(plan_kernel<FP8>, dim3(1), dim3(1024), 0, st, a, counted);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(a.P), dim3(kThreads), C::kSmem, st, a);
  if (e == cudaSuccess && a.P > 1)
    e = launch_pdl(join_kernel<D>,
                   dim3(a.P - 1, ((a.pair_keys ? 1 : 2) * a.nt * a.G + kJoinRows - 1) / kJoinRows),
                   dim3(kJoinRows * 32), 0, st, a);
  note_launches(2 + a.planned + counted);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace flash
}  // namespace kvc
