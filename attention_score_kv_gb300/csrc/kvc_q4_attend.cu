// Attention over the 4-bit retained cache (format: kvc_q4.cuh), few query rows
// per KV head: the decoding step.
//
//   o = sum_r p_r v_r / sum_r p_r,  p_r = exp(q.k_r / sqrt(D)) over the rows a query sees
//
// One read of the cache bounds it: 9D/8 + 4 bytes a row for 4*G*T*D flops.  How
// the rows are shared out and the products made: kvc_few_rows.cuh.  The codes
// come in fragment order, so they go through two conversions straight into mma
// operands.
// Measured: one token of 64 sequences over 8 heads of 4.3K rows (331 MB) takes
// 62 us, 56 of them the scan, 5.9 TB/s; reading the same bytes and nothing else
// takes 51 to 54 us.  A block is 280 instructions of a warp, 60% of the issue
// slots.  Without the copies ahead it took 87 us; 3 or more ranges an SM cost 4
// us of start each (66 to 75 us); ranges per warp, without the join in the CTA,
// leave eight times the parts to the second kernel (uneven heads 26 instead of 18
// us).
// Numerics: codes times scales are exact in fp16; q is scaled by a power of
// two per row into fp16's range (values below 2^-24 of the row's largest round
// off there); sums, maxima and outputs are fp32; p is rounded to fp16
// (2^-11 relative; the reference point leaves it below 2^12, so that steps below
// fp16's normal numbers are 2^-28 of the largest weight or less).
#include <algorithm>
#include <cmath>

#include "kvc_few_rows.cuh"
#include "kvc_q4.cuh"

namespace kvc {
namespace {

constexpr int kClusterBlocks = 128;  // blocks a CTA of a cluster takes at most

template <int N>
struct Codes { uint32_t w[N]; };
template <int kB>
__device__ __forceinline__ Codes<kB / 4> load_codes(const uint8_t* p) {
  Codes<kB / 4> c;
  if constexpr (kB == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    c.w[0] = v.x, c.w[1] = v.y, c.w[2] = v.z, c.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c.w[0] = v.x, c.w[1] = v.y;
  }
  return c;
}

template <int D>
struct Q4Rows {
  static constexpr int kD = D, kB = D / 8;
  static constexpr bool kJoinInRing = false, kCross = false, kScaled = false, kMods = false;
  using Source = const uint8_t*;
  using Cursor = const uint8_t*;
  static __device__ __forceinline__ void touch(Source s) { asm volatile("" ::"l"(s)); }
  static __device__ __forceinline__ Cursor cursor(Source s, int64_t row) {
    return s + row / q4::kRows * q4::block_bytes(D);
  }

  // A stage of a warp's ring: a block's bytes as they are in the cache, and its
  // positions.  Lane 4r + j copies the pieces it reads itself: rows r and r + 8
  // of the keys, slice r of the values' pairs j and j + 4, their scales, and the
  // positions of rows r and r + 8 (four lanes each, the same value).
  static constexpr int kPosAt = q4::block_bytes(D), kStageBytes = kPosAt + 32 * 8;
  static __device__ __forceinline__ void copy(uint32_t dst, Cursor at, int in, const int32_t* pos, int lane) {
    const uint8_t* rec = at + (int64_t)in * q4::block_bytes(D);
    const int r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {    // the keys' two halves, then the values' two halves
      if constexpr (kB == 16) few::copy16(dst + i * 4 * D + lane * kB, rec + i * 4 * D + lane * kB);
      else few::copy_small<8>(dst + i * 4 * D + lane * kB, rec + i * 4 * D + lane * kB);
    }
    if constexpr (D == 128) {
      few::copy_small<4>(dst + q4::k_scales(D) + lane * 4, rec + q4::k_scales(D) + lane * 4);
      few::copy_small<4>(dst + q4::v_scales(D) + lane * 4, rec + q4::v_scales(D) + lane * 4);
    } else {
      // two bytes of key scales a lane: the word of an even lane and the next; both copy it
      const int kw = (lane >> 1) * 4, vw = ((r >> 1) * 4 + j) * 4;
      few::copy_small<4>(dst + q4::k_scales(D) + kw, rec + q4::k_scales(D) + kw);
      few::copy_small<4>(dst + q4::v_scales(D) + vw, rec + q4::v_scales(D) + vw);
    }
    few::copy_small<4>(dst + kPosAt + lane * 8, pos + r);
    few::copy_small<4>(dst + kPosAt + lane * 8 + 4, pos + r + 8);
  }

  static __device__ __forceinline__ int2 positions(const uint8_t* st, int lane) {
    return *reinterpret_cast<const int2*>(st + kPosAt + lane * 8);
  }

  // quarter j of a row, pairs of dims D/8 apart
  static __device__ __forceinline__ int q_at(int j, int i) { return j * (D / 4) + 8 * i; }
  static __device__ __forceinline__ void q_pair(const uint32_t* w, int s, int y, uint32_t& lo, uint32_t& hi) {
    lo = q4::bf16_of(w, 2 * s + y), hi = q4::bf16_of(w, kB + 2 * s + y);
  }

  struct Scales { uint32_t k, v; };
  static __device__ __forceinline__ Scales scales(const uint8_t* st, int lane) {
    const int r = lane >> 2, j = lane & 3;
    Scales sc;
    if constexpr (D == 128) {
      sc.k = *reinterpret_cast<const uint32_t*>(st + q4::k_scales(D) + lane * 4);
      sc.v = *reinterpret_cast<const uint32_t*>(st + q4::v_scales(D) + lane * 4);
    } else {
      const uint32_t two = *reinterpret_cast<const uint16_t*>(st + q4::k_scales(D) + lane * 2);
      sc.k = (two & 0xffu) * 0x101u | (two >> 8) * 0x1010000u;
      sc.v = *reinterpret_cast<const uint32_t*>(st + q4::v_scales(D) + ((r >> 1) * 4 + j) * 4);
    }
    return sc;
  }
  static __device__ __forceinline__ void mask(Scales& sc, uint32_t keep, bool) { sc.v &= keep; }

  // in two chains of products, half as long
  static __device__ __forceinline__ void scores(const uint8_t* st, int lane, const Scales& sc,
                                                const uint32_t (&qf)[D / 16][2], float (&acc)[4]) {
    float odd[4] = {};
    const uint32_t ks[2] = {q4::scales_to_half2((uint16_t)sc.k), q4::scales_to_half2((uint16_t)(sc.k >> 16))};
    const Codes<kB / 4> kc0 = load_codes<kB>(st + q4::k_codes(D) + lane * kB);
    const Codes<kB / 4> kc1 = load_codes<kB>(st + q4::k_codes(D) + 4 * D + lane * kB);
#pragma unroll
    for (int x = 0; x < kB / 4; ++x) {
      uint32_t ka[4], kb[4];
      q4::codes_to_half2(kc0.w[x], ka);
      q4::codes_to_half2(kc1.w[x], kb);
#pragma unroll
      for (int y = 0; y < 4; ++y) ka[y] = q4::mul_half2(ka[y], ks[0]), kb[y] = q4::mul_half2(kb[y], ks[1]);
      few::mma_f16(acc, ka[0], kb[0], ka[1], kb[1], qf[2 * x][0], qf[2 * x][1]);
      few::mma_f16(odd, ka[2], kb[2], ka[3], kb[3], qf[2 * x + 1][0], qf[2 * x + 1][1]);
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) acc[y] += odd[y];
  }
  static __device__ __forceinline__ void outputs(const uint8_t* st, int lane, const Scales& sc, uint32_t pf0,
                                                 uint32_t pf1, float (&o)[D / 16][4]) {
    const Codes<kB / 4> vc0 = load_codes<kB>(st + q4::v_codes(D) + lane * kB);
    const Codes<kB / 4> vc1 = load_codes<kB>(st + q4::v_codes(D) + 4 * D + lane * kB);
    const uint32_t vs2[2] = {q4::scales_to_half2((uint16_t)sc.v), q4::scales_to_half2((uint16_t)(sc.v >> 16))};
#pragma unroll
    for (int x = 0; x < kB / 4; ++x) {
      uint32_t va[4], vb[4];
      q4::codes_to_half2(vc0.w[x], va);
      q4::codes_to_half2(vc1.w[x], vb);
#pragma unroll
      for (int y = 0; y < 4; ++y) va[y] = q4::mul_half2(va[y], vs2[0]), vb[y] = q4::mul_half2(vb[y], vs2[1]);
      few::mma_f16(o[2 * x], va[0], va[1], vb[0], vb[1], pf0, pf1);
      few::mma_f16(o[2 * x + 1], va[2], va[3], vb[2], vb[3], pf0, pf1);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(few::kThreads, 2)
kvc_attend_q4_kernel(const __grid_constant__ few::Args<Q4Rows<D>> a) {
  few::scan_ranges(a);
}
template <int D>
__global__ void __launch_bounds__(few::kThreads, 2)
kvc_attend_q4_cluster_kernel(const __grid_constant__ few::Args<Q4Rows<D>> a) {
  few::scan_cluster(a);
}
template <int D>
__global__ void __launch_bounds__(few::kJoinWarps * 32)
kvc_attend_q4_join_kernel(const __grid_constant__ few::Args<Q4Rows<D>> a) {
  few::join_ranges(a);
}

template <int D>
cudaError_t launch_of(const __nv_bfloat16* q, const uint8_t* cache, const int32_t* pos, const int32_t* rows, int extra,
                      const int32_t* q_pos, int B, int T, int H_q, const Q4Slots& slots, __nv_bfloat16* out, float* lse,
                      void* ws, bool clusters, cudaStream_t st) {
  few::Args<Q4Rows<D>> a{};
  a.q = q, a.src = cache, a.pos = pos, a.rows = rows, a.q_pos = q_pos, a.out = out, a.lse = lse;
  a.B = B, a.T = T, a.G = H_q / slots.H_kv, a.extra = extra;
  a.s = slots;
  few::place_parts(a, plan_attend_q4(B, T, H_q, slots.H_kv, D), ws);
  return few::launch(a, clusters, kvc_attend_q4_kernel<D>, kvc_attend_q4_cluster_kernel<D>,
                     kvc_attend_q4_join_kernel<D>, st);
}

}  // namespace

// More query rows go to the tensor cores' other form, whose 128 rows cost the
// same however many are used: at 8 heads of 4096 rows 20 query rows take 10.2 us
// there (16 sequences: 36.6 us) and took 24.6 us here in tiles of 32 columns (62
// us), 12 rows 9.4 us (36.6 us) and 16.4 us in tiles of 16 (38 us).
bool attend_q4_on_tc(int H_q, int H_kv, int T) { return (int64_t)(H_q / H_kv) * T > few::kCols; }

// Whether clusters take the heads: while two CTAs an SM hold them all and the
// longest slot leaves no CTA more than kClusterBlocks blocks.  One launch instead
// of two, and no partial results: 8 heads of 1024, 4096 and 13000 rows take 4.9,
// 6.3 and 10.6 us instead of 8.0, 10.2 and 14.0; 32 heads of 4096 and 9830 rows 8.7
// and 15.0 instead of 12.8 and 17.7.  Ranges are even where heads are not: 32
// unequal heads of up to 16.6K rows take 18.2 us in ranges, 19.0 in clusters, and
// 8 heads of 40000 rows 19.6 and 24.6.  Clusters of 16 were slower (8 heads of
// 4096 rows 7.0, 16 heads 11.7 against 8.0), but for one long head alone.
static bool in_clusters(int BH, const Q4Slots& slots) { return few::in_clusters(BH, slots, kClusterBlocks); }

Q4AttendPlan plan_attend_q4(int B, int T, int H_q, int H_kv, int D) {
  Q4AttendPlan p{};
  p.P = std::max(num_sms(), 1) * 2;
  const size_t rows = ((size_t)p.P + (size_t)B * H_kv) * (size_t)(H_q / H_kv * T);
  p.off_o = (rows * sizeof(float2) + 255) / 256 * 256;
  p.off_place = p.off_o + rows * D * sizeof(float);
  p.total = p.off_place + ((size_t)B * H_kv + 1) * sizeof(int);
  return p;
}

cudaError_t launch_attend_q4(const __nv_bfloat16* q, const uint8_t* cache, const int32_t* pos, const int32_t* rows,
                             int extra, const int32_t* q_pos, int B, int T, int H_q, int D, const Q4Slots& slots,
                             __nv_bfloat16* out, float* lse, void* ws, cudaStream_t st) {
  const bool c = in_clusters(B * slots.H_kv, slots);
  return D == 128 ? launch_of<128>(q, cache, pos, rows, extra, q_pos, B, T, H_q, slots, out, lse, ws, c, st)
                  : launch_of<64>(q, cache, pos, rows, extra, q_pos, B, T, H_q, slots, out, lse, ws, c, st);
}

}  // namespace kvc
