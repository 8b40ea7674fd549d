// Attention over a retained cache in blocks of 16 rows, few query rows per KV
// head: the decoding step.  Shared by the cache's formats (F): how a block is
// copied in, and how its codes become operands, is the format's.
//
//   o = sum_r p_r v_r / sum_r p_r,  p_r = exp(x_r) over the rows a query sees
//
// One read of the cache bounds it.  So the rows of all (sequence, KV head) pairs
// are laid end to end, in blocks of 16, and cut into equal ranges, one per CTA,
// whatever the heads' lengths: a CTA computes its range from the device-held row
// counts.  A range may end inside a head; each CTA writes per head it touches the
// running maximum, sum and unnormalised output, and a second kernel joins the
// parts in order.
//
// A warp takes one block at a time and copies blocks ahead into shared memory
// asynchronously, a ring of its own, so the copies need no barrier of the CTA (and
// none at all where every lane reads back what it copied).  The products are
//   S^T (16 rows x 8 queries) = K Q^T,   O^T (D x 8 queries) += V^T P^T,
// with up to 8 query rows as the narrow N side, so that no row of the
// matrix instruction is wasted when a KV head has 4 or 5 query heads.  P goes
// from accumulator to operand layout with movmatrix.
//
// A format F has:
//   kD; kJoinInRing: a ring stage has room for a warp's outputs; kScaled: the values of a block have one scale, a power of two; kMods: scores
//   may be capped and biased (then its scales give the keys' scale too)
//   Source, Cursor, cursor(source, row), touch(source): where a row's block is
//   kStageBytes, copy(stage, cursor, block, pos, lane): a block in a ring; kCross: lanes
//   read what others copied
//   q_at(j, i): dims of the i-th 8 of lane quarter j; q_pair(w, s, y, lo, hi)
//   positions, scales, mask, scores, outputs: a block's products
#pragma once

#include <algorithm>
#include <cmath>

#include "kvc_device.cuh"
#include "kvc_internal.cuh"
#include "kvc_q4.cuh"

namespace kvc {
namespace few {

constexpr int kBlockRows = 16;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 8;             // query rows per KV head: the narrow side of the products
constexpr int kMinBlocks = kWarps;   // blocks of 16 rows a CTA takes at least
constexpr int kCluster = 8;          // CTAs of a cluster that takes a head
constexpr int kStages = 3;           // blocks of a warp's ring
constexpr float kNoRef = -1.7e38f;   // reference of a query that has seen no row
constexpr float kShift = 4.0f;       // weights are kept as 2^(x - max + kShift)
constexpr float kSlack = 8.0f;       // the reference moves when a score passes it by more
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeastUnit = 7.8886090522101181e-31f;    // 2^-100, the smallest scale

template <class F>
struct Args {
  const __nv_bfloat16* q;
  typename F::Source src;
  const int32_t *pos, *rows, *q_pos;
  const float* slopes;               // [H_q] or null: bias by distance
  __nv_bfloat16* out;
  float* lse;
  float2* part_ml;                   // [P + B * H_kv][R] maximum, sum: part of range c and head bh at c + bh
  float* part_o;                     // [..][R][D], dims in the order of dim_of
  int* place;                        // [B * H_kv] blocks before each head, then all blocks
  int* status;
  int B, T, G, extra, P;
  uint32_t inv_h;                    // ceil(2^32 / H_kv): bh / H_kv as a product (bh < 2^24, H_kv <= 128)
  float scale;                       // log2(e) / sqrt(D)
  float cap2, inv_cap2;              // cap of the scores in log2 units, 0: none
  Q4Slots s;
};

// The heads' slots, in shared memory: lanes look up different heads at a time,
// which the constant bank would serve one after the other.
struct SlotTable { int64_t off[kMaxHkv]; int cap[kMaxHkv]; };
template <class F>
__device__ __forceinline__ void fill_slots(const Args<F>& a, SlotTable& t) {
  for (int h = threadIdx.x; h < a.s.H_kv; h += blockDim.x) {
    t.off[h] = a.s.off[h];
    t.cap[h] = (int)(a.s.off[h + 1] - a.s.off[h]);
  }
}
template <class F>
__device__ __forceinline__ int batch_of(const Args<F>& a, int bh) {
  // a divisor of 1 has no such product below 2^32
  return a.s.H_kv == 1 ? bh : (int)__umulhi((uint32_t)bh, a.inv_h);
}
// Rows that (sequence, KV head) bh counts; bad: the count does not fit the slot.
template <class F>
__device__ __forceinline__ int rows_of(const Args<F>& a, const SlotTable& t, int bh, int held, bool* bad) {
  const int cap = t.cap[bh - batch_of(a, bh) * a.s.H_kv];
  const int64_t n = (int64_t)held + a.extra;
  *bad |= n < 0 || n > cap;
  return (int)(n < 0 ? 0 : n > cap ? cap : n);
}
__device__ __forceinline__ int blocks_of(int n_rows) { return (n_rows + kBlockRows - 1) / kBlockRows; }

// Blocks of a CTA's range when N blocks are shared out.  Block numbers are
// ints: all of this GPU's memory holds less than 2^28 blocks.
__device__ __forceinline__ int range_blocks(int N, int P) {
  const int L = (int)(((uint32_t)N + P - 1) / (uint32_t)P);
  return L < kMinBlocks ? kMinBlocks : L;
}

// Where a CTA's range begins: the head that holds its first block, and the
// blocks before that head.  Each warp adds up its share of the heads; the warp
// whose share holds the place finds it.
// write: leave every head's place to the joining kernel, and record counts
// that do not fit.
struct Place { int total, L, before, bh, n_rows; };    // L: blocks of a range
template <class F>
__device__ __forceinline__ Place find_place(const Args<F>& a, const SlotTable& t, int cta, bool write) {
  __shared__ int s_sum[kWarps], s_at[3];
  const int BH = a.B * a.s.H_kv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = (BH + kThreads - 1) / kThreads * 32;
  const int i0 = min(warp * share, BH), i1 = min(i0 + share, BH);
  bool bad = false;
  int sum = 0, n0 = 0;
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    const int n = i < i1 ? rows_of(a, t, i, __ldg(a.rows + i), &bad) : 0;
    if (base == i0) n0 = n;
    sum += blocks_of(n);
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  Place p{};
  int run = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    run += w < warp ? s_sum[w] : 0;
    p.total += s_sum[w];
  }
  p.L = range_blocks(p.total, a.P);
  const int f0 = (int)min((int64_t)cta * p.L, (int64_t)p.total);
  if ((f0 >= run && f0 < run + sum) || write)
    for (int base = i0; base < i1; base += 32) {
      const int i = base + lane;
      const int n = base == i0 ? n0 : i < i1 ? rows_of(a, t, i, __ldg(a.rows + i), &bad) : 0, nb = blocks_of(n);
      int inc = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int before = run + inc - nb;
      if (write && i < i1) a.place[i] = before;
      if (f0 >= before && f0 < before + nb) s_at[0] = before, s_at[1] = i, s_at[2] = n;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  if (write && threadIdx.x == 0) a.place[BH] = p.total;
  if (write && bad) record_status(a.status, kStatusBadInput);
  __syncthreads();
  if (f0 < p.total) p.before = s_at[0], p.bh = s_at[1], p.n_rows = s_at[2];
  return p;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// The heads of a range, one after the other.
template <class F>
struct Segment {
  typename F::Cursor rec;            // first block of the segment, its rows' positions
  const int32_t* pos;
  int f, bh, cnt, s0, n_rows;        // flat block it starts at; head; blocks; first block in the head; the head's rows
};
template <class F>
__device__ __forceinline__ Segment<F> segment_of(const Args<F>& a, const SlotTable& t, int f, int f1, int bh,
                                                 int before, int n_rows) {
  const int b = batch_of(a, bh);
  Segment<F> g;
  g.f = f;
  g.bh = bh;
  g.n_rows = n_rows;
  g.s0 = f - before;
  g.cnt = min(f1 - f, blocks_of(n_rows) - g.s0);
  const int64_t row = (int64_t)b * a.s.off[a.s.H_kv] + t.off[bh - b * a.s.H_kv] + (int64_t)g.s0 * kBlockRows;
  g.rec = F::cursor(a.src, row);
  g.pos = a.pos + row;
  return g;
}
// The next one: a segment that does not end the range ends its head.
template <class F>
__device__ __forceinline__ bool next_segment(const Args<F>& a, const SlotTable& t, int f1, const Segment<F>& g,
                                             Segment<F>* next) {
  const int f = g.f + g.cnt;
  if (f >= f1) return false;
  bool bad = false;                  // recorded where the places are found
  int n, bh = g.bh + 1;
  while ((n = rows_of(a, t, bh, __ldg(a.rows + bh), &bad)) == 0) ++bh;     // f < f1 <= total: a head with rows follows
  *next = segment_of<F>(a, t, f, f1, bh, f, n);
  return true;
}

// Block `in` of a segment (if it has one) into a stage of the warp's ring.
template <class F>
__device__ __forceinline__ void fetch_block(const Segment<F>& x, int in, uint32_t stage, int lane) {
  if (in < x.cnt)
    F::copy(stage, x.rec, in, x.pos + (int64_t)in * kBlockRows, lane);
  copies_commit();
}

// Shared memory: the warps' outputs (kJoinInRing: in the stage of a warp's ring that
// is not being filled, which leaves room for a second CTA), then their rings.
// Position d' = 16 m + 2 r + e of an output row holds dim r*D/8 + 2m + e: a lane
// of the output fragments stores pairs side by side with its neighbours', and
// rows D + 4 apart keep the four columns of a store on different banks.
__host__ __device__ constexpr int o_stride(int D) { return D + 4; }
template <class F>
__host__ __device__ constexpr int o_bytes(int R) {
  return F::kJoinInRing ? 0 : kWarps * R * o_stride(F::kD) * (int)sizeof(float);
}
// Where a warp's outputs go, and its ring.
template <class F>
__device__ __forceinline__ float* outputs_of(uint8_t* dyn, int R, int warp, int stage_out) {
  static_assert(!F::kJoinInRing || F::kStageBytes >= kCols * o_stride(F::kD) * (int)sizeof(float), "a stage holds them");
  if constexpr (F::kJoinInRing)
    return reinterpret_cast<float*>(dyn + (warp * kStages + (stage_out + kStages - 1) % kStages) * F::kStageBytes);
  return reinterpret_cast<float*>(dyn) + warp * R * o_stride(F::kD);
}
template <int D>
__device__ __forceinline__ int dim_of(int at) { return (at >> 1 & 7) * (D / 8) + (at >> 4) * 2 + (at & 1); }

// What a warp has of a head: output fragments (columns 2j and 2j + 1 of dims
// dim_of), per column the reference and the sum; with kScaled formats the fragments
// are in units of 2^unit, which follow a column's largest contribution (weight times
// the scale of the block's values) as the reference follows its largest score, so
// that fp16 holds it whatever scales there are in rows of no weight to the column.
template <class F>
struct Acc {
  static constexpr int D = F::kD;
  float o[D / 16][4], ref[2], sum[2];
  int unit[2];
  __device__ __forceinline__ void clear() {
    unit[0] = unit[1] = 0;
#pragma unroll
    for (int m = 0; m < D / 16; ++m)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[m][y] = 0.f;
    ref[0] = ref[1] = kNoRef;
    sum[0] = sum[1] = 0.f;
  }
};

// The warp's share of a segment: blocks warp, warp + 8, ...  start() and fetch(g,
// i) copy blocks ahead into the warp's ring.
template <class F, typename Start, typename Fetch>
__device__ __forceinline__ void attend_segment(const Args<F>& a, const Segment<F>& g, int b, const int (&t_of)[2],
                                               const uint8_t* ring, int& stage_out, Start start, Fetch fetch,
                                               Acc<F>& acc_out) {
  constexpr int D = F::kD;
  constexpr int KS = D / 16;         // k-steps of the scores, m-tiles of the output
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, j = lane & 3;
  const int R = a.G * a.T, bh = g.bh, n_rows = g.n_rows;
  auto& o = acc_out.o;
  auto& ref = acc_out.ref;
  auto& sum = acc_out.sum;
  acc_out.clear();
  // queries: column n = lane / 4, quarter j of its dims
  uint32_t w[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) w[i] = 0;
  if (r < R) {
    const __nv_bfloat16* p = a.q + ((int64_t)bh * R + r) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + F::q_at(j, i)));
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  int qp[2];                       // positions of columns 2j and 2j + 1
#pragma unroll
  for (int y = 0; y < 2; ++y)
    qp[y] = 2 * j + y < R ? __ldg(a.q_pos + (int64_t)b * a.T + t_of[y]) : -1;
  float slope[2] = {};             // in log2 units
  if constexpr (F::kMods)
    if (a.slopes) {
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (2 * j + y < R)
          slope[y] = __ldg(a.slopes + (bh - b * a.s.H_kv) * a.G + (2 * j + y - t_of[y]) / a.T) * kLog2e;
    }
  start();                         // behind the queries' loads, which the blocks' traffic would hold up
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
  mx = max(mx & 0xffffu, mx >> 16);
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // scale by the power of two that brings the row's largest value into [1, 2)
  const uint32_t e = mx >> 7, ee = (e == 0 || e == 255) ? 127u : min(e, 253u);
  float down = __uint_as_float((254u - ee) << 23);
  if constexpr (F::kMods)            // a row that is not finite becomes NaN, capped or not, as with many rows
    if (e == 255) down = __uint_as_float(0x7fffffffu);
  const float c = __uint_as_float(ee << 23) * a.scale;
  uint32_t qf[KS][2];
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t lo, hi;
      F::q_pair(w, s, y, lo, hi);
      qf[s][y] = pack_half2(__uint_as_float(lo << 16) * down, __uint_as_float(hi << 16) * down);
    }
  float c2[2];                     // factor from accumulator to log2 units, columns 2j and 2j + 1
  int q_lo = INT32_MAX, q_hi = -1;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    c2[y] = __shfl_sync(0xffffffffu, c, (2 * j + y) * 4);
    if (2 * j + y < R) q_lo = min(q_lo, qp[y]), q_hi = max(q_hi, qp[y]);
  }
  q_lo = __reduce_min_sync(0xffffffffu, q_lo);
  q_hi = __reduce_max_sync(0xffffffffu, q_hi);

  const int mine = (g.cnt - warp + kWarps - 1) / kWarps;       // blocks of this warp (may be <= 0)
  for (int i = 0; i < mine; ++i) {
    const int blk = g.s0 + warp + i * kWarps;
    if constexpr (F::kCross) __syncwarp();         // all have read the stage that is filled now
    fetch(g, i + kStages - 1);
    copies_wait<kStages - 1>();
    if constexpr (F::kCross) __syncwarp();
    const uint8_t* st = ring + stage_out * F::kStageBytes;
    stage_out = stage_out + 1 == kStages ? 0 : stage_out + 1;
    auto sc = F::scales(st, lane);
    const int2 xp = F::positions(st, lane);        // of rows r and r + 8
    // ---- scores
    float acc[4] = {};
    F::scores(st, lane, sc, qf, acc);
    float u[2] = {c2[0], c2[1]};   // what is left from acc to log2 units
    if constexpr (F::kMods) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float x = acc[y] * (sc.k * c2[y & 1]);
        if (a.cap2 > 0.f) x = a.cap2 * tanh_of(x * a.inv_cap2);
        const int far = (int)((uint32_t)(y < 2 ? xp.x : xp.y) - (uint32_t)qp[y & 1]);
        acc[y] = fmaf(slope[y & 1], (float)far, x);
      }
      u[0] = u[1] = 1.f;
    }
    // ---- mask: acc[y], acc[2 + y] are rows r, r + 8 against column 2j + y
    const int row = blk * kBlockRows + r;
    const bool in0 = row < n_rows && xp.x >= 0, in1 = row + 8 < n_rows && xp.y >= 0;
    if (!__all_sync(0xffffffffu, in0 && xp.x <= q_lo && in1 && xp.y <= q_lo)) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (!in0 || xp.x > qp[y]) acc[y] = -INFINITY;
        if (!in1 || xp.y > qp[y]) acc[2 + y] = -INFINITY;
      }
      // a row that no query sees may hold anything: its values count as zeros
      const uint32_t see0 = __ballot_sync(0xffffffffu, in0 && xp.x <= q_hi);
      const uint32_t see1 = __ballot_sync(0xffffffffu, in1 && xp.y <= q_hi);
      uint32_t keep = 0;           // a byte each: rows 2j, 2j + 1, 2j + 8, 2j + 9; lane 4r' speaks for row r'
      if (see0 >> (8 * j) & 1) keep |= 0x000000ffu;
      if (see0 >> (8 * j + 4) & 1) keep |= 0x0000ff00u;
      if (see1 >> (8 * j) & 1) keep |= 0x00ff0000u;
      if (see1 >> (8 * j + 4) & 1) keep |= 0xff000000u;
      F::mask(sc, keep, (see0 | see1) != 0);
    }
    // ---- weights
    bool above = false;
    float lv = 0.f;
    if constexpr (F::kScaled) lv = log2_of(sc.v);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float m = fmaxf(acc[y], acc[2 + y]) * u[y];
      above |= m > ref[y] + (kSlack + kShift);
      if constexpr (F::kScaled) above |= m - ref[y] + lv > (float)acc_out.unit[y] + (kSlack + kShift);
    }
    if (__any_sync(0xffffffffu, above)) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float m = fmaxf(acc[y], acc[2 + y]) * u[y];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        // whole steps with kScaled: what the reference rises, the unit falls, and then rises to
        // where the block's largest contribution is 2^kShift of it
        const float next = fmaxf(ref[y], (F::kScaled ? floorf(m) : m) - kShift);
        float f = ex2(ref[y] - next);
        sum[y] *= f;
        if constexpr (F::kScaled) {
          const float was = (float)acc_out.unit[y] - (next - ref[y]);
          const float now = fmaxf(was, floorf((m - next) + lv) - kShift);
          acc_out.unit[y] = max(-126, min((int)now, 127));
          f = ex2(was - now);
        }
        ref[y] = next;
#pragma unroll
        for (int m2 = 0; m2 < KS; ++m2) o[m2][y] *= f, o[m2][2 + y] *= f;
      }
    }
    float p[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      p[y] = ex2(fmaf(acc[y], u[y & 1], -ref[y & 1]));
      sum[y & 1] += p[y];
    }
    if constexpr (F::kScaled) {    // contributions in the columns' units
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        // quotient of two powers of two, 0 below the normal numbers; above them the weight is 0
        const int e = (int)(__float_as_uint(sc.v) >> 23) - acc_out.unit[y];
        const float f = __int_as_float(min(max(e, 0), 254) << 23);
        p[y] *= f, p[2 + y] *= f;
      }
    }
    const uint32_t pf0 = transpose8(pack_half2(p[0], p[1])), pf1 = transpose8(pack_half2(p[2], p[3]));
    // ---- output
    F::outputs(st, lane, sc, pf0, pf1, o);
  }
}

// Joins the CTA's warps, in warp order, into sum_o [R][D] and sum_ml [R]: shared
// or global memory.
template <class F>
__device__ __forceinline__ void join_warps(const Acc<F>& x, int R, float2 (*s_ml)[kCols], float* mine, float* sum_o,
                                           float2* sum_ml) {
  __shared__ const float* s_at[kWarps];
  constexpr int D = F::kD, KS = D / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, j = lane & 3;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    float v = x.sum[y];
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (r == 0) s_ml[warp][2 * j + y] = make_float2(x.ref[y], v);
  }
  if (lane == 0) s_at[warp] = mine;
  __syncthreads();
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int col = 2 * j + y;
    if (col >= R) continue;
    float top = s_ml[0][col].x;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_ml[w][col].x);
    float f = ex2(x.ref[y] - top);
    if constexpr (F::kScaled) f *= __int_as_float((x.unit[y] + 127) << 23);
    float* to = mine + col * o_stride(D) + 2 * r;
#pragma unroll
    for (int m = 0; m < KS; ++m)
      *reinterpret_cast<float2*>(to + 16 * m) = make_float2(x.o[m][y] * f, x.o[m][2 + y] * f);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * (D / 4); i += kThreads) {
    const int col = i / (D / 4), at = i % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 z = *reinterpret_cast<const float4*>(s_at[w] + col * o_stride(D) + at);
      v.x += z.x, v.y += z.y, v.z += z.z, v.w += z.w;
    }
    *reinterpret_cast<float4*>(sum_o + col * D + at) = v;
  }
  if (threadIdx.x < R) {
    float top = kNoRef, l = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][threadIdx.x].x);
    for (int w = 0; w < kWarps; ++w) l += s_ml[w][threadIdx.x].y * ex2(s_ml[w][threadIdx.x].x - top);
    sum_ml[threadIdx.x] = make_float2(top, l);
  }
}

// What does not depend on the previous grid comes before the wait for it: the
// tokens of columns 2j and 2j + 1, and the arguments' first loads.
template <class F>
__device__ __forceinline__ void begin(const Args<F>& a, int (&t_of)[2]) {
  const int j = threadIdx.x & 3;
  t_of[0] = 2 * j % a.T, t_of[1] = (2 * j + 1) % a.T;
  F::touch(a.src);
  asm volatile("" ::"l"(a.q), "l"(a.pos), "l"(a.rows), "l"(a.q_pos), "l"(a.part_ml), "l"(a.part_o),
               "l"(a.place), "r"(a.extra), "r"(a.P), "r"(a.inv_h), "f"(a.scale));
}

template <class F>
__device__ __forceinline__ void scan_ranges(const Args<F>& a) {
  constexpr int D = F::kD;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ float2 s_ml[kWarps][kCols];
  __shared__ SlotTable slots;
  fill_slots(a, slots);
  int t_of[2];
  begin(a, t_of);
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = a.G * a.T;           // query rows, at most kCols
  uint8_t* ring = dyn + o_bytes<F>(R) + warp * kStages * F::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);

  // the CTA's range [f0, f1) of the blocks laid end to end
  const Place pl = find_place(a, slots, blockIdx.x, blockIdx.x == 0);
  const int f0 = (int)min((int64_t)blockIdx.x * pl.L, (int64_t)pl.total), f1 = min(f0 + pl.L, pl.total);
  Segment<F> g;
  bool more = f0 < f1;
  if (more) g = segment_of<F>(a, slots, f0, f1, pl.bh, pl.before, pl.n_rows);

  // block `i` (0, 1, ...) of the warp's share of a segment into its ring; a group is
  // committed whether or not there is one, so that the waits can count
  int stage_in = 0, stage_out = 0;
  const auto fetch = [&](const Segment<F>& x, int i) {
    fetch_block<F>(x, warp + i * kWarps, ring_u + stage_in * F::kStageBytes, lane);
    stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
  };
  bool started = false;
  const auto start = [&] {
    if (!started)
      for (int i = 0; i < kStages - 1; ++i) fetch(g, i);
    started = true;
  };
  while (more) {
    Acc<F> acc;
    attend_segment<F>(a, g, batch_of(a, g.bh), t_of, ring, stage_out, start, fetch, acc);
    // the next head's first blocks come in while this one is joined.  Groups that the
    // loop's tail committed empty are behind the ones it used; the ring starts afresh.
    Segment<F> next;
    more = next_segment<F>(a, slots, f1, g, &next);
    stage_in = stage_out;
    if (more)
      for (int i = 0; i < kStages - 1; ++i) fetch(next, i);
    const int64_t part = ((int64_t)blockIdx.x + g.bh) * R;
    join_warps<F>(acc, R, s_ml, outputs_of<F>(dyn, R, warp, stage_out), a.part_o + part * D, a.part_ml + part);
    __syncthreads();
    g = next;
  }
}

// Few and short heads: a cluster of CTAs per head, each with an equal share of
// its blocks, which join their parts through each other's shared memory: one
// launch, no partial results in memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t of_rank(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float remote(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
template <class F>
__device__ __forceinline__ void scan_cluster(const Args<F>& a) {
  constexpr int D = F::kD;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ float2 s_ml[kWarps][kCols];
  __shared__ __align__(16) float s_sum[kCols * D];
  __shared__ float2 s_sum_ml[kCols];
  int t_of[2];
  begin(a, t_of);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = a.G * a.T, H = a.s.H_kv;
  const int bh = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, b = bh / H, h = bh - b * H;
  const int64_t cap = a.s.off[h + 1] - a.s.off[h], row0 = (int64_t)b * a.s.off[H] + a.s.off[h];
  uint8_t* ring = dyn + o_bytes<F>(R) + warp * kStages * F::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  grid_dep_wait();
  grid_dep_launch();
  int64_t n = (int64_t)__ldg(a.rows + bh) + a.extra;
  if (n < 0 || n > cap) {
    if (rank == 0 && threadIdx.x == 0) record_status(a.status, kStatusBadInput);
    n = n < 0 ? 0 : cap;
  }
  const int nb = blocks_of((int)n), per = (nb + kCluster - 1) / kCluster;
  Segment<F> g;
  g.f = 0;
  g.bh = bh;
  g.n_rows = (int)n;
  g.s0 = min(rank * per, nb);
  g.cnt = min(per, nb - g.s0);
  g.rec = F::cursor(a.src, row0 + (int64_t)g.s0 * kBlockRows);
  g.pos = a.pos + row0 + (int64_t)g.s0 * kBlockRows;
  int stage_in = 0, stage_out = 0;
  const auto fetch = [&](const Segment<F>& x, int i) {
    fetch_block<F>(x, warp + i * kWarps, ring_u + stage_in * F::kStageBytes, lane);
    stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
  };
  const auto start = [&] {
    for (int i = 0; i < kStages - 1; ++i) fetch(g, i);
  };
  Acc<F> acc;
  attend_segment<F>(a, g, b, t_of, ring, stage_out, start, fetch, acc);
  join_warps<F>(acc, R, s_ml, outputs_of<F>(dyn, R, warp, stage_out), s_sum, s_sum_ml);
  cluster_sync();
  for (int i = rank * kThreads + threadIdx.x; i < R * D; i += kCluster * kThreads) {
    const int row = i / D, d = i % D;
    float m[kCluster], l[kCluster], v[kCluster], top = kNoRef, sum = 0.f, o = 0.f;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      const uint32_t ml = of_rank(&s_sum_ml[row], c);
      m[c] = remote(ml), l[c] = remote(ml + 4), v[c] = remote(of_rank(&s_sum[i], c));
    }
#pragma unroll
    for (int c = 0; c < kCluster; ++c) top = fmaxf(top, m[c]);
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      const float f = ex2(m[c] - top);
      sum = fmaf(l[c], f, sum);
      o = fmaf(v[c], f, o);
    }
    const int64_t at = (int64_t)bh * R + row;
    a.out[at * D + dim_of<D>(d)] = __float2bfloat16_rn(sum == 0.f ? 0.f : o / sum);
    if (a.lse && d == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
  }
  cluster_sync();                    // nobody leaves while its part is read
}

// One CTA per (sequence, KV head) and query row: joins the parts.  Warp w goes
// through parts w, w + 4, ... in range order, each lane with a vector of the
// row, against a maximum of its own (so that a part's sum and output are
// loaded together), and the four are joined in warp order.
constexpr int kJoinWarps = 4, kJoinAhead = 4;
template <class F>
__device__ __forceinline__ void join_ranges(const Args<F>& a) {
  constexpr int D = F::kD, V = D / 32;          // values of a lane
  __shared__ float s_v[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, BH = a.B * a.s.H_kv;
  const int R = a.G * a.T, bh = blockIdx.x / R, row = blockIdx.x - bh * R;
  grid_dep_wait();
  grid_dep_launch();
  const int total = a.place[BH], before = a.place[bh], after = a.place[bh + 1];   // place[BH] is the total
  const int L = range_blocks(total, a.P);
  const int c0 = before / L;
  const int n = after > before ? (after - 1) / L - c0 + 1 : 0;
  const int64_t slot0 = bh + c0;
  const float2* ml = a.part_ml + slot0 * R + row;
  const float* po = a.part_o + (slot0 * R + row) * D + lane * V;
  float top = kNoRef, l = 0.f, v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
  for (int c = warp; c < n; c += kJoinWarps * kJoinAhead) {
    float2 x[kJoinAhead];
    float y[kJoinAhead][V];
#pragma unroll
    for (int z = 0; z < kJoinAhead; ++z) {
      const int cz = c + z * kJoinWarps;
      x[z] = make_float2(kNoRef, 0.f);
#pragma unroll
      for (int i = 0; i < V; ++i) y[z][i] = 0.f;
      if (cz < n) {
        x[z] = ml[(int64_t)cz * R];
        const float* p = po + (int64_t)cz * R * D;
        if constexpr (V == 4) *reinterpret_cast<float4*>(y[z]) = *reinterpret_cast<const float4*>(p);
        else *reinterpret_cast<float2*>(y[z]) = *reinterpret_cast<const float2*>(p);
      }
    }
    float next = top;
#pragma unroll
    for (int z = 0; z < kJoinAhead; ++z) next = fmaxf(next, x[z].x);
    const float f0 = ex2(top - next);
    top = next;
    l *= f0;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= f0;
#pragma unroll
    for (int z = 0; z < kJoinAhead; ++z) {
      const float f = ex2(x[z].x - top);
      l = fmaf(x[z].y, f, l);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fmaf(y[z][i], f, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s_v[warp][lane * V + i] = v[i];
  if (lane == 0) s_ml[warp] = make_float2(top, l);
  __syncthreads();
  float f[kJoinWarps];
  top = kNoRef, l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w].x);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) f[w] = ex2(s_ml[w].x - top), l = fmaf(s_ml[w].y, f[w], l);
  const int64_t at = blockIdx.x;
  for (int d = threadIdx.x; d < D; d += kJoinWarps * 32) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) o = fmaf(s_v[w][d], f[w], o);
    a.out[at * D + dim_of<D>(d)] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  }
  if (a.lse && threadIdx.x == 0) a.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
}


// Places of a call's partial results, and its arguments from them.
template <class F>
inline void place_parts(Args<F>& a, const Q4AttendPlan& p, void* ws) {
  a.part_ml = static_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_o);
  a.place = reinterpret_cast<int*>(static_cast<char*>(ws) + p.off_place);
  a.status = status_word_ptr();
  a.P = p.P;
  a.scale = (float)(1.4426950408889634 / std::sqrt((double)F::kD));
  a.inv_h = (uint32_t)(((1ull << 32) + a.s.H_kv - 1) / a.s.H_kv);
}

// Whether clusters may take the heads: two CTAs an SM hold them all, and the
// longest slot leaves no CTA more than `most` blocks.
inline bool in_clusters(int BH, const Q4Slots& slots, int most) {
  int64_t longest = 0;
  for (int h = 0; h < slots.H_kv; ++h) longest = std::max(longest, slots.off[h + 1] - slots.off[h]);
  return (int64_t)BH * kCluster <= 2 * (int64_t)num_sms() && longest <= (int64_t)kCluster * most * kBlockRows;
}

template <class F>
cudaError_t launch(const Args<F>& a, bool clusters, void (*scan)(Args<F>), void (*cluster)(Args<F>),
                   void (*join)(Args<F>), cudaStream_t st) {
  const int H = a.s.H_kv, R = a.G * a.T;
  const size_t smem = o_bytes<F>(R) + kWarps * kStages * F::kStageBytes;
  if (clusters) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(cluster), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * H * kCluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, cluster, a);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(scan), smem);
  if (e == cudaSuccess) e = launch_pdl(scan, dim3(a.P), dim3(kThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(join, dim3((unsigned)(a.B * H * R)), dim3(kJoinWarps * 32), 0, st, a);
  note_launches(2);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace few
}  // namespace kvc
