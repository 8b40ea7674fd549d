// Attention over the 8-bit retained cache (format: kvc_q8.cuh), few query rows
// per KV head: the decoding step, with capped or biased scores.
//
//   x = q.k / sqrt(D);  x <- cap tanh(x / cap);  x <- x - slope_h (q_pos - pos);
//   o = sum p v / sum p,  p = exp(x)
//
// One read of the cache bounds it: 2D + 4.5 bytes a row.  How the rows are shared
// out and the products made: kvc_few_rows.cuh.  Rows are held row after row; a
// lane's share of a block is 16 bytes of a row at a time, four lanes (keys) or
// eight (values) on the same 64 or 128 bytes, so whole sectors move.  The order
// of a contraction is free, so keys go from a row's bytes through one conversion
// into mma operands, with the queries laid out alike; values, whose rows are the
// contraction's index, take a byte permutation first (two rows in one operand).
// Codes are exact in fp16.  A block's scale of the keys multiplies its scores,
// that of the values the block's weights, in units of the largest scale that the
// warp has met, so that fp16 holds the weights.
#include "kvc_few_rows.cuh"
#include "kvc_q8.cuh"

namespace kvc {
namespace {

constexpr int kClusterBlocks = 128;  // blocks a CTA of a cluster takes at most

struct Q8Source { const uint8_t *k8, *v8; const float* scale; };

template <int D>
struct Q8Rows {
  static constexpr int kD = D;
  static constexpr bool kJoinInRing = true, kScaled = true, kMods = true;
  using Source = Q8Source;
  using Cursor = Q8Source;
  static __device__ __forceinline__ void touch(const Source& s) {
    asm volatile("" ::"l"(s.k8), "l"(s.v8), "l"(s.scale));
  }
  static __device__ __forceinline__ Cursor cursor(const Source& s, int64_t row) {
    return {s.k8 + row * D, s.v8 + row * D, s.scale + row / q8::kRows * 2};
  }

  // A stage of a warp's ring, in the order in which the lanes read it.  Lane
  // 4r + j has rows r and r + 8 of the keys, 16 bytes at 16 j (and 64 + 16 j); slice
  // r of rows 2j, 2j + 1, 2j + 8 and 2j + 9 of the values; the two scales; and the
  // positions of rows r and r + 8.
  static constexpr int kV = D / 8;                 // bytes of a slice
  static constexpr int kValuesAt = 16 * D, kScaleAt = 32 * D, kPosAt = kScaleAt + 32 * 8, kStageBytes = kPosAt + 32 * 8;
  static __device__ __forceinline__ void copy(uint32_t dst, const Cursor& at, int in, const int32_t* pos, int lane) {
    const int r = lane >> 2, j = lane & 3;
    const uint8_t* k = at.k8 + (int64_t)in * (16 * D) + r * D + 16 * j;
    const uint8_t* v = at.v8 + (int64_t)in * (16 * D) + 2 * j * D + r * kV;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int row = i / (D / 64) * 8, part = i % (D / 64) * 64;
      few::copy16(dst + i * 512 + lane * 16, k + row * D + part);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* p = v + ((e & 1) + (e >> 1) * 8) * D;
      const uint32_t to = dst + kValuesAt + (e * 32 + lane) * kV;
      if constexpr (kV == 16) few::copy16(to, p);
      else few::copy_small<8>(to, p);
    }
    few::copy_small<8>(dst + kScaleAt + lane * 8, at.scale + (int64_t)in * 2);
    few::copy_small<4>(dst + kPosAt + lane * 8, pos + r);
    few::copy_small<4>(dst + kPosAt + lane * 8 + 4, pos + r + 8);
  }

  static __device__ __forceinline__ int q_at(int j, int i) { return 16 * j + i / 2 * 64 + i % 2 * 8; }
  static __device__ __forceinline__ void q_pair(const uint32_t* w, int s, int y, uint32_t& lo, uint32_t& hi) {
    lo = w[2 * s + y] & 0xffffu, hi = w[2 * s + y] >> 16;
  }

  struct Scales { float k, v; uint32_t keep; };
  static __device__ __forceinline__ Scales scales(const uint8_t* st, int lane) {
    const float2 s = *reinterpret_cast<const float2*>(st + kScaleAt + lane * 8);
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
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 a4 = *reinterpret_cast<const uint4*>(st + i * 512 + lane * 16);
      const uint4 b4 = *reinterpret_cast<const uint4*>(st + (i + D / 64) * 512 + lane * 16);
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
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* p = st + kValuesAt + (e * 32 + lane) * kV;
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
