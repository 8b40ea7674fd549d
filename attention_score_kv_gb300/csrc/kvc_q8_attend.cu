// Attention over the 8-bit retained cache (format: kvc_q8.cuh), few query rows
// per KV head: the decoding step, with capped or biased scores.
//
//   x = q.k / sqrt(D);  x <- cap tanh(x / cap);  x <- x - slope_h (q_pos - pos);
//   o = sum p v / sum p,  p = exp(x)
//
// One read of the cache bounds it: 2D + 4.5 bytes a row.  How the rows are shared
// out and the products made: kvc_few_rows.cuh.  Rows are held row after row, and
// go into shared memory 512 bytes a copy.  The order of a contraction is free, so
// keys go from a row's bytes through one conversion into mma operands, with the
// queries laid out alike; values, whose rows are the contraction's index, take a
// byte permutation first (two rows in one operand).
// Codes are exact in fp16.  A block's scale of the keys multiplies its scores,
// that of the values the block's weights, in units that follow the query's own
// largest product of the two, so that fp16 holds it.
// Measured: one token of 64 sequences over 8 heads of 4.3K rows (582 MB) 96.5 us, 6.0
// TB/s (97 with capped scores); one token over 8 heads of 4096 rows 7.5 us.  Copies
// of 16 bytes a lane in the order of the fragments (two lines of 64 bytes a row) left
// it at 4.75 TB/s; one CTA an SM, with the joins' room beside the rings, took 35
// instead of 29 us over uneven heads.
#include "kvc_few_rows.cuh"
#include "kvc_q8.cuh"

namespace kvc {
namespace {

constexpr int kClusterBlocks = 128;  // blocks a CTA of a cluster takes at most

struct Q8Source { const uint8_t *k8, *v8; const float* scale; };

template <int D>
struct Q8Rows {
  static constexpr int kD = D;
  static constexpr bool kJoinInRing = true, kCross = true, kScaled = true, kMods = true;
  using Source = Q8Source;
  using Cursor = Q8Source;
  static __device__ __forceinline__ void touch(const Source& s) {
    asm volatile("" ::"l"(s.k8), "l"(s.v8), "l"(s.scale));
  }
  static __device__ __forceinline__ Cursor cursor(const Source& s, int64_t row) {
    return {s.k8 + row * D, s.v8 + row * D, s.scale + row / q8::kRows * 2};
  }

  // A stage of a warp's ring: the keys, the values, 16 positions, the two scales.  A copy
  // of the warp takes 512 bytes in a row.  Lines of 128 bytes (a row, or two of D = 64)
  // have their eight pieces of 16 bytes swapped about, so that the eight lanes of a
  // read's phase find theirs on different banks: keys, two rows' even or odd pieces, by
  // the row; values, two pieces of every other row, by the pair of rows.
  static constexpr int kV = D / 8;                 // bytes of a slice of a value row
  static constexpr int kValuesAt = 16 * D, kPosAt = 32 * D, kScaleAt = kPosAt + 64, kStageBytes = kPosAt + 128;
  static __device__ __forceinline__ int at_line(int line, int piece, bool vals) {
    const int flip = D == 128 ? (vals ? 2 * (line >> 1 & 3) : line & 7) : (vals ? 2 * (line & 3) : 0);
    return line * 128 + ((piece ^ flip) << 4);
  }
  static __device__ __forceinline__ void copy(uint32_t dst, const Cursor& at, int in, const int32_t* pos, int lane) {
    const uint8_t* k = at.k8 + (int64_t)in * (16 * D) + lane * 16;
    const uint8_t* v = at.v8 + (int64_t)in * (16 * D) + lane * 16;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int line = 4 * i + (lane >> 3), piece = lane & 7;
      few::copy16(dst + at_line(line, piece, false), k + i * 512);
      few::copy16(dst + kValuesAt + at_line(line, piece, true), v + i * 512);
    }
    if (lane < 16) few::copy_small<4>(dst + kPosAt + lane * 4, pos + lane);
    else if (lane == 16) few::copy_small<8>(dst + kScaleAt, at.scale + (int64_t)in * 2);
  }
  static __device__ __forceinline__ int2 positions(const uint8_t* st, int lane) {
    const int* p = reinterpret_cast<const int*>(st + kPosAt);
    return make_int2(p[lane >> 2], p[(lane >> 2) + 8]);
  }

  // a lane's quarter of a row, pairs of dims side by side
  static __device__ __forceinline__ int q_at(int j, int i) { return j * (D / 4) + 8 * i; }
  static __device__ __forceinline__ void q_pair(const uint32_t* w, int s, int y, uint32_t& lo, uint32_t& hi) {
    lo = w[2 * s + y] & 0xffffu, hi = w[2 * s + y] >> 16;
  }

  struct Scales { float k, v; uint32_t keep; };
  static __device__ __forceinline__ Scales scales(const uint8_t* st, int) {
    const float2 s = *reinterpret_cast<const float2*>(st + kScaleAt);
    return {s.x, s.y, 0xffffffffu};
  }
  // keep: a byte each for rows 2j, 2j + 1, 2j + 8, 2j + 9
  static __device__ __forceinline__ void mask(Scales& sc, uint32_t keep, bool some) {
    sc.keep = keep;
    if (!some) sc.v = few::kLeastUnit;             // no row of the block: its scales may be anything
  }

  // in two chains of products, half as long
  static __device__ __forceinline__ void scores(const uint8_t* st, int lane, const Scales&,
                                                const uint32_t (&qf)[D / 16][2], float (&acc)[4]) {
    float odd[4] = {};
    const int r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {             // rows r and r + 8, 16 dims
      const int at = D == 128 ? at_line(r, 2 * j + i, false) : at_line(r >> 1, (r & 1) * 4 + j, false);
      const uint4 a4 = *reinterpret_cast<const uint4*>(st + at);
      const uint4 b4 = *reinterpret_cast<const uint4*>(st + 8 * D + at);       // the same place: rows r and r + 8 flip alike
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t ha[2], hb[2];
        q8::to_half2(a[x], ha);
        q8::to_half2(b[x], hb);
        const int s = 4 * i + x;
        few::mma_f16(x & 1 ? odd : acc, ha[0], hb[0], ha[1], hb[1], qf[s][0], qf[s][1]);
      }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) acc[y] += odd[y];
  }
  static __device__ __forceinline__ void outputs(const uint8_t* st, int lane, const Scales& sc, uint32_t pf0,
                                                 uint32_t pf1, float (&o)[D / 16][4]) {
    uint32_t v[4][kV / 4];
    const int r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; ++e) {                  // slice r of rows 2j, 2j + 1, 2j + 8, 2j + 9
      const int row = 2 * j + (e & 1) + (e >> 1) * 8;
      const uint8_t* p = st + kValuesAt + (D == 128 ? at_line(row, r, true)
                                                    : at_line(row >> 1, (row & 1) * 4 + (r >> 1), true) + (r & 1) * 8);
      if constexpr (kV == 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        v[e][0] = x.x, v[e][1] = x.y, v[e][2] = x.z, v[e][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v[e][0] = x.x, v[e][1] = x.y;
      }
    }
    if (__any_sync(0xffffffffu, sc.keep != 0xffffffffu)) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int x = 0; x < kV / 4; ++x)
          if (!(sc.keep >> (8 * e) & 1)) v[e][x] = 0;
    }
#pragma unroll
    for (int x = 0; x < kV / 4; ++x) {
      uint32_t lo[2], lo2[2], hi[2], hi2[2];       // dims 4x .. 4x + 3 of rows 2j, 2j + 1, and of 2j + 8, 2j + 9
      q8::to_half2(__byte_perm(v[0][x], v[1][x], 0x5140), lo);
      q8::to_half2(__byte_perm(v[0][x], v[1][x], 0x7362), lo2);
      q8::to_half2(__byte_perm(v[2][x], v[3][x], 0x5140), hi);
      q8::to_half2(__byte_perm(v[2][x], v[3][x], 0x7362), hi2);
      few::mma_f16(o[2 * x], lo[0], lo[1], hi[0], hi[1], pf0, pf1);
      few::mma_f16(o[2 * x + 1], lo2[0], lo2[1], hi2[0], hi2[1], pf0, pf1);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(few::kThreads, 2)
kvc_attend_q8_kernel(const __grid_constant__ few::Args<Q8Rows<D>> a) {
  few::scan_ranges(a);
}
template <int D>
__global__ void __launch_bounds__(few::kThreads, 2)
kvc_attend_q8_cluster_kernel(const __grid_constant__ few::Args<Q8Rows<D>> a) {
  few::scan_cluster(a);
}
template <int D>
__global__ void __launch_bounds__(few::kJoinWarps * 32)
kvc_attend_q8_join_kernel(const __grid_constant__ few::Args<Q8Rows<D>> a) {
  few::join_ranges(a);
}

template <int D>
cudaError_t launch_of(const Q8Attend& x, bool clusters, cudaStream_t st) {
  few::Args<Q8Rows<D>> a{};
  a.q = x.q, a.src = {x.c.k8, x.c.v8, x.c.scale}, a.pos = x.c.pos, a.rows = x.rows, a.q_pos = x.q_pos;
  a.slopes = x.slopes, a.out = x.out, a.lse = x.lse;
  a.B = x.B, a.T = x.T, a.G = x.H_q / x.slots->H_kv, a.extra = x.extra;
  a.s = *x.slots;
  a.cap2 = x.cap * few::kLog2e;
  a.inv_cap2 = x.cap > 0.f ? 1.f / a.cap2 : 0.f;
  few::place_parts(a, plan_attend_q4(x.B, x.T, x.H_q, x.slots->H_kv, D), x.ws);
  return few::launch(a, clusters, kvc_attend_q8_kernel<D>, kvc_attend_q8_cluster_kernel<D>,
                     kvc_attend_q8_join_kernel<D>, st);
}

}  // namespace

cudaError_t launch_attend_q8(const Q8Attend& x, cudaStream_t st) {
  const bool c = few::in_clusters(x.B * x.slots->H_kv, *x.slots, kClusterBlocks);
  return x.D == 128 ? launch_of<128>(x, c, st) : launch_of<64>(x, c, st);
}

}  // namespace kvc
