// Writers and reader of the 8-bit retained cache (format: kvc_q8.cuh).
//
//   scale = 2^ceil(log2(max |x| / 448)),  code = e4m3(x / scale)   per block of 16 rows
//
// A warp takes the keys or the values of one block of 16 rows and has them in
// registers whole (D / 2 values a lane), so the block's maximum is one warp
// reduction and every byte moves once.  D / 16 lanes share a row, 32 bytes of bf16
// and 16 bytes of codes each: loads and stores of whole sectors.
// The scattered rows of 2 D bytes bound a gather, latency an append.  Measured at 315K
// of 1M rows of 128: gather and read-back 74 us (486 MB, 6.55 TB/s, 97% of a plain
// copy); one token appended to 8 heads and read back 4.5 us, five to 512 heads 6.2.
#include <algorithm>

#include "kvc_device.cuh"
#include "kvc_internal.cuh"
#include "kvc_q4.cuh"
#include "kvc_q8.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// A lane's share of a row: 16 values from dim 16 * (lane % (D / 16)).  Step i
// takes rows i * kAtOnce + lane / kLanes.
template <int D>
struct Lay {
  static constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes, kSteps = q8::kRows / kAtOnce;
};

template <bool WIDE>
__device__ __forceinline__ void load16(const __nv_bfloat16* p, uint32_t* w) {
  if constexpr (WIDE) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint32_t* w) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::"r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Largest magnitude of 16 packed bf16, as bf16 bits.  What cannot be held is
// made so first: NaN becomes 0 and infinities the largest value, both noted, and
// magnitudes above the largest value become it.
__device__ __forceinline__ uint32_t clean_max(uint32_t* w, bool* bad) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  m = max(m & 0xffffu, m >> 16);
  if (m > q8::kTop) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int s = 0; s < 32; s += 16) {
        uint32_t x = w[i] >> s & 0x7fffu;
        const uint32_t sign = w[i] >> s & 0x8000u;
        *bad |= x >= 0x7f80u;
        x = x > 0x7f80u ? 0 : min(x, q8::kTop);
        m = max(m, x);
        w[i] = (w[i] & ~(0xffffu << s)) | (x | sign) << s;
      }
  }
  return m;
}

enum RowWhat : int { kLeave = 0, kWrite = 1, kZero = 2 };

// Writes rows of one block's keys or values.  src(row, &what): what to do with
// row 0..15 and, for kWrite, the element offset of its values in x.  held: rows
// before this one are held already; where the scale grows, their codes follow it.
template <int D, bool WIDE, typename Src>
__device__ __forceinline__ void store_block(uint8_t* codes, float* scale, const __nv_bfloat16* __restrict__ x, Src src,
                                            int held, bool* bad) {
  using L = Lay<D>;
  const int lane = threadIdx.x & 31, part = lane % L::kLanes, r0 = lane / L::kLanes;
  const uint32_t was = held > 0 ? min(__float_as_uint(*scale) >> 23 & 0xffu, q8::kMost) : 0;
  uint32_t w[L::kSteps][8];
  int what[L::kSteps];
#pragma unroll
  for (int i = 0; i < L::kSteps; ++i) {
    const int64_t at = src(i * L::kAtOnce + r0, &what[i]);
    if (what[i] == kWrite) {
      load16<WIDE>(x + at + part * 16, w[i]);
    } else {
#pragma unroll
      for (int y = 0; y < 8; ++y) w[i][y] = 0;
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < L::kSteps; ++i) m = max(m, clean_max(w[i], bad));
  m = __reduce_max_sync(0xffffffffu, m);
  const uint32_t e = max(q8::scale_exp(m), was);
  const float inv = q8::pow2(254 - e);
#pragma unroll
  for (int i = 0; i < L::kSteps; ++i) {
    const int row = i * L::kAtOnce + r0;
    uint8_t* to = codes + row * D + part * 16;
    uint4 c;
    if (what[i] == kLeave) {
      if (row >= held || e == was) continue;
      const float f = q8::pow2(127 - min(e - was, 126u));     // 2^(was - e); beyond 2^-126 all codes are 0 either way
      c = *reinterpret_cast<const uint4*>(to);
      uint32_t* v = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t h[2];
        q8::to_half2(v[y], h);
        uint16_t two[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h[z]));
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(two[z]) : "f"(g.y * f), "f"(g.x * f));
        }
        v[y] = (uint32_t)two[0] | (uint32_t)two[1] << 16;
      }
    } else {
      c.x = q8::codes_of(w[i][0], w[i][1], inv);
      c.y = q8::codes_of(w[i][2], w[i][3], inv);
      c.z = q8::codes_of(w[i][4], w[i][5], inv);
      c.w = q8::codes_of(w[i][6], w[i][7], inv);
    }
    *reinterpret_cast<uint4*>(to) = c;
  }
  // every lane has read the old scale before the reduction above
  if (lane == 0) *scale = q8::pow2(e);
}

// Which head holds item i of a list in which head h's items start at first[h].
template <typename F>
__device__ __forceinline__ int head_of(int H, int64_t i, F first) {
  int lo = 0, hi = H;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= i) lo = mid; else hi = mid;
  }
  return lo;
}

struct GatherArgs {
  const __nv_bfloat16 *k, *v;
  const int32_t* idx;
  Q8Cache c;
  int* status;
  int B, H_kv, S;
  int64_t warps, rows;               // (blocks, keys or values) to write in all; rows of a batch element
  int32_t blk0[kMaxHkv + 1];         // head h writes blocks blk0[h] .. blk0[h+1]-1 of a batch element's list
  int32_t kept[kMaxHkv];
  int64_t off[kMaxHkv];
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) kvc_gather_q8_kernel(const __grid_constant__ GatherArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.warps) return;
  const int vals = (int)(i & 1), per = a.blk0[a.H_kv];
  const int64_t b = (i >> 1) / per;
  const int in = (int)((i >> 1) - b * per);
  const int h = head_of(a.H_kv, in, [&](int x) { return a.blk0[x]; });
  const int row0 = (in - a.blk0[h]) * q8::kRows;
  const int64_t at0 = b * a.rows + a.off[h] + row0;
  const int n = min(q8::kRows, a.kept[h] - row0);
  // idx and pos may be one buffer: the values' warp of a block takes its positions
  // from it too, and what the keys' warp writes there is what it read
  int p = lane < n ? a.idx[at0 + lane] : 0;
  bool bad = p < 0 || p >= a.S;
  if (bad) p = 0;                                   // outside the contract: any row of the head, and the status
  const int64_t base = (b * a.H_kv + h) * (int64_t)a.S;
  if (lane < n && !vals) a.c.pos[at0 + lane] = p;
  auto src = [&](int row, int* what) {
    const int pr = __shfl_sync(0xffffffffu, p, row);
    *what = row < n ? kWrite : kZero;
    return (base + pr) * D;
  };
  store_block<D, WIDE>((vals ? a.c.v8 : a.c.k8) + at0 * D, a.c.scale + at0 / q8::kRows * 2 + vals, vals ? a.v : a.k,
                       src, 0, &bad);
  if (bad) record_status(a.status, kStatusBadInput);
}

struct AppendArgs {
  const __nv_bfloat16 *k, *v;
  const int32_t *pos, *rows;
  Q8Cache c;
  int* status;
  int B, T, nb;                      // nb: blocks that T rows may touch
  Q4Slots slots;
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) kvc_append_q8_kernel(const __grid_constant__ AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, H = a.slots.H_kv;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= (int64_t)a.B * H * a.nb * 2) return;
  const int vals = (int)(i & 1);
  const int64_t bh = (i >> 1) / a.nb;
  const int64_t b = bh / H;
  const int h = (int)(bh - b * H);
  const int64_t cap = a.slots.off[h + 1] - a.slots.off[h];
  const int n0 = a.rows[bh];
  if (n0 < 0 || (int64_t)n0 + a.T > cap) {          // no room: nothing of this head is written
    if (lane == 0) record_status(a.status, kStatusBadInput);
    return;
  }
  const int64_t row0 = ((int64_t)(n0 / q8::kRows) + ((i >> 1) - bh * a.nb)) * q8::kRows;
  if (row0 >= (int64_t)n0 + a.T) return;
  const int64_t at0 = b * a.slots.off[H] + a.slots.off[h] + row0;
  const int64_t t_of0 = row0 - n0;                  // token of the block's row 0 (may be negative)
  int p = -1;
  if (lane < q8::kRows && t_of0 + lane >= 0 && t_of0 + lane < a.T) {
    p = a.pos[b * a.T + t_of0 + lane];
    if (p < 0) p = -1;                              // an absent token: zeros that no query sees
    if (!vals) a.c.pos[at0 + lane] = p;
  }
  bool bad = false;
  auto src = [&](int row, int* what) {
    const int pr = __shfl_sync(0xffffffffu, p, row);
    const int64_t t = t_of0 + row;
    *what = (t < 0 || t >= a.T) ? kLeave : pr < 0 ? kZero : kWrite;
    return (bh * a.T + t) * D;
  };
  store_block<D, WIDE>((vals ? a.c.v8 : a.c.k8) + at0 * D, a.c.scale + at0 / q8::kRows * 2 + vals, vals ? a.v : a.k,
                       src, t_of0 < 0 ? (int)-t_of0 : 0, &bad);
  if (bad) record_status(a.status, kStatusBadInput);
}

struct ReadArgs {
  Q8Cache c;
  const int32_t* first;
  __nv_bfloat16 *k_out, *v_out;
  int* status;
  int64_t warps, out_rows;           // (blocks, keys or values) to look at in all; output rows of a batch element
  int32_t blk0[kMaxHkv + 1];
  int32_t n_rows[kMaxHkv];
  int64_t out_off[kMaxHkv];
  Q4Slots slots;
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) kvc_read_q8_kernel(const __grid_constant__ ReadArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using L = Lay<D>;
  const int lane = threadIdx.x & 31, part = lane % L::kLanes, r0 = lane / L::kLanes, H = a.slots.H_kv;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.warps) return;
  const int vals = (int)(i & 1), per = a.blk0[H];
  const int64_t b = (i >> 1) / per;
  const int in = (int)((i >> 1) - b * per);
  const int h = head_of(H, in, [&](int x) { return a.blk0[x]; });
  const int64_t cap = a.slots.off[h + 1] - a.slots.off[h];
  const int64_t first = a.first ? a.first[b * H + h] : 0;
  const int64_t row0 = ((first >> 4) + (in - a.blk0[h])) * q8::kRows, end = first + a.n_rows[h];
  if (row0 >= end) return;
  const bool there = row0 >= 0 && row0 < cap;
  if (!there && lane == 0) record_status(a.status, kStatusBadInput);
  const int64_t at0 = b * a.slots.off[H] + a.slots.off[h] + (there ? row0 : 0);
  const uint8_t* codes = (vals ? a.c.v8 : a.c.k8) + at0 * D + r0 * D + part * 16;
  __nv_bfloat16* out = (vals ? a.v_out : a.k_out) + (b * a.out_rows + a.out_off[h] + row0 - first + r0) * D + part * 16;
  const auto wanted = [&](int row) { return row0 + row >= first && row0 + row < end; };
  uint4 c[L::kSteps];
  float s = 0.f;
  if (there) {
    s = a.c.scale[at0 / q8::kRows * 2 + vals];
#pragma unroll
    for (int x = 0; x < L::kSteps; ++x) {
      c[x] = make_uint4(0, 0, 0, 0);
      if (wanted(x * L::kAtOnce + r0)) c[x] = *reinterpret_cast<const uint4*>(codes + x * L::kAtOnce * D);
    }
  }
#pragma unroll
  for (int x = 0; x < L::kSteps; ++x) {
    if (!wanted(x * L::kAtOnce + r0)) continue;
    uint32_t w[8];
    const uint32_t v[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      uint32_t f[2];
      q8::to_half2(there ? v[y] : 0, f);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&f[z]));
        const __nv_bfloat162 r = __floats2bfloat162_rn(g.x * s, g.y * s);   // exact
        w[2 * y + z] = *reinterpret_cast<const uint32_t*>(&r);
      }
    }
    store16<WIDE>(out + (int64_t)x * L::kAtOnce * D, w);
  }
}

bool wide(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 31) == 0;
}
dim3 grid_for(int64_t warps) { return dim3((unsigned)((warps + kWarps - 1) / kWarps)); }

}  // namespace

cudaError_t launch_gather_q8(const __nv_bfloat16* k, const __nv_bfloat16* v, const int32_t* idx, int B,
                             const SelParams& sel, int D, const Q8Cache& c, cudaStream_t st) {
  GatherArgs a{};
  a.k = k, a.v = v, a.idx = idx, a.c = c, a.status = status_word_ptr();
  a.B = B, a.H_kv = sel.H_kv, a.S = sel.S, a.rows = sel.T;
  for (int h = 0; h < sel.H_kv; ++h) {
    a.kept[h] = sel.kept[h];
    a.off[h] = sel.off[h];
    a.blk0[h + 1] = a.blk0[h] + (sel.kept[h] + q8::kRows - 1) / q8::kRows;
  }
  a.warps = (int64_t)B * a.blk0[sel.H_kv] * 2;
  if (a.warps == 0) return cudaSuccess;
  const bool w = wide(k, v);
  auto* kern = D == 128 ? (w ? kvc_gather_q8_kernel<128, true> : kvc_gather_q8_kernel<128, false>)
                        : (w ? kvc_gather_q8_kernel<64, true> : kvc_gather_q8_kernel<64, false>);
  cudaError_t e = launch_pdl(kern, grid_for(a.warps), dim3(kThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_append_q8(const __nv_bfloat16* k, const __nv_bfloat16* v, const int32_t* pos, int B, int T, int D,
                             const Q4Slots& slots, const int32_t* rows, const Q8Cache& c, cudaStream_t st) {
  AppendArgs a{};
  a.k = k, a.v = v, a.pos = pos, a.rows = rows, a.c = c, a.status = status_word_ptr();
  a.B = B, a.T = T, a.nb = (T + q8::kRows - 2) / q8::kRows + 1;
  a.slots = slots;
  const bool w = wide(k, v);
  auto* kern = D == 128 ? (w ? kvc_append_q8_kernel<128, true> : kvc_append_q8_kernel<128, false>)
                        : (w ? kvc_append_q8_kernel<64, true> : kvc_append_q8_kernel<64, false>);
  cudaError_t e = launch_pdl(kern, grid_for((int64_t)B * slots.H_kv * a.nb * 2), dim3(kThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_read_q8(const Q8Cache& c, int B, int D, const Q4Slots& slots, const int32_t* first,
                           const SelParams& out, __nv_bfloat16* k_out, __nv_bfloat16* v_out, cudaStream_t st) {
  ReadArgs a{};
  a.c = c, a.first = first, a.k_out = k_out, a.v_out = v_out, a.status = status_word_ptr();
  a.out_rows = out.T;
  a.slots = slots;
  for (int h = 0; h < slots.H_kv; ++h) {
    const int n = out.kept[h];
    a.n_rows[h] = n;
    a.out_off[h] = out.off[h];
    // an unaligned start may touch one block more
    const int blocks = first ? (n + q8::kRows - 2) / q8::kRows + 1 : (n + q8::kRows - 1) / q8::kRows;
    a.blk0[h + 1] = a.blk0[h] + (n == 0 ? 0 : blocks);
  }
  a.warps = (int64_t)B * a.blk0[slots.H_kv] * 2;
  if (a.warps == 0) return cudaSuccess;
  const bool w = wide(k_out, v_out);
  auto* kern = D == 128 ? (w ? kvc_read_q8_kernel<128, true> : kvc_read_q8_kernel<128, false>)
                        : (w ? kvc_read_q8_kernel<64, true> : kvc_read_q8_kernel<64, false>);
  cudaError_t e = launch_pdl(kern, grid_for(a.warps), dim3(kThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvc
