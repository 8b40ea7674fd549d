// Writers and reader of the 4-bit retained cache (format: kvc_q4.cuh).
//
//   scale = e4m3(max |x| / 6),  code = e2m1(x / scale)   per 16 values of a row
//
// One warp per block of 16 rows.  Its lanes load the values in the order in
// which the block holds them, 16 bytes a load, so that each lane has whole
// scale groups (D = 128) or halves of them (values at D = 64, one shuffle) in
// registers, and writes its codes and scales as vectors: no shared memory.
// A gather moves 4D + 4 bytes in and 9D/8 + 4 out per row; the scattered rows
// of 2D bytes bound it.  Measured at 315K of 1M rows of 128: gather 35.9 us (209
// MB, 5.8 TB/s), read-back 33.4 us (207 MB, 6.2 TB/s); one token appended to 8
// heads 3.5 us, five to 512 heads 4.8 us.  16-byte accesses, which touch every
// sector twice, took 42 us each; codes made one by one in fp32, 39 us.
#include <algorithm>

#include "kvc_device.cuh"
#include "kvc_internal.cuh"
#include "kvc_q4.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 4;            // blocks of rows per CTA
constexpr int kThreads = kWarps * 32;

enum RowWhat : int { kLeave = 0, kWrite = 1, kZero = 2 };

// max of |x| over 2*N packed bf16, as bf16 bits.  Values that are not finite
// are made harmless first (NaN: 0; infinities stay and saturate) and noted.
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t* w, bool* bad) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  m = max(m & 0xffffu, m >> 16);
  if (m >= 0x7f80u) {
    *bad = true;
    m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if ((w[i] & 0x7fffu) > 0x7f80u) w[i] &= 0xffff0000u;
      if (((w[i] >> 16) & 0x7fffu) > 0x7f80u) w[i] &= 0x0000ffffu;
      m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
    m = max(m & 0xffffu, m >> 16);
  }
  return m;
}

// Rows of the bf16 tensors.  WIDE: 32 bytes an access, a whole sector each, for
// tensors that start on 32 bytes (16-byte accesses move every sector twice).
template <int N, bool WIDE>
__device__ __forceinline__ void load_vecs(const __nv_bfloat16* p, uint32_t* w) {
  if constexpr (WIDE && N >= 8) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                   : "=r"(w[8 * i]), "=r"(w[8 * i + 1]), "=r"(w[8 * i + 2]), "=r"(w[8 * i + 3]), "=r"(w[8 * i + 4]),
                     "=r"(w[8 * i + 5]), "=r"(w[8 * i + 6]), "=r"(w[8 * i + 7])
                   : "l"(p + 16 * i));
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}
template <int N, bool WIDE>
__device__ __forceinline__ void store_vecs(__nv_bfloat16* p, const uint32_t* w) {
  if constexpr (WIDE && N >= 8) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::"r"(w[8 * i]), "r"(w[8 * i + 1]),
                   "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]), "r"(w[8 * i + 6]),
                   "r"(w[8 * i + 7]), "l"(p + 16 * i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

template <int N>
__device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t* w) {
  if constexpr (N == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// Write rows of one block.  src(row, &what): what to do with row 0..15 of the
// block and, for kWrite, the element offset of its values in k and v.  A warp
// owns the whole block, so the nibbles that two rows share in a value byte are
// read and written by one lane.
template <int D, bool WIDE, typename Src>
__device__ void store_block(uint8_t* rec, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                            Src src, bool* bad) {
  constexpr int kB = D / 8;                 // code bytes of a lane and row
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  // ---- keys: rows r and r + 8, dims j*D/4 .. (j+1)*D/4 - 1
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    int what;
    const int row = r + 8 * s;
    const int64_t at = src(row, &what);
    if (what == kLeave) continue;
    uint32_t w[D / 8];
    if (what == kWrite) load_vecs<D / 8, WIDE>(k + at + j * (D / 4), w);
    else
#pragma unroll
      for (int i = 0; i < D / 8; ++i) w[i] = 0;
    float inv[2];
    uint32_t sc[2];
    if constexpr (D == 128) {
      sc[0] = q4::scale_of(group_max<8>(w, bad), &inv[0]);
      sc[1] = q4::scale_of(group_max<8>(w + 8, bad), &inv[1]);
    } else {
      sc[0] = q4::scale_of(group_max<8>(w, bad), &inv[0]);
      inv[1] = inv[0];
      sc[1] = 0;
    }
    uint32_t c[kB / 4];
#pragma unroll
    for (int x = 0; x < kB / 4; ++x) c[x] = q4::code_bytes(w + 2 * x, w + kB / 2 + 2 * x, make_float2(inv[0], inv[1]));
    store_bytes<kB>(rec + q4::k_codes(D) + row * (D / 2) + j * kB, c);
    if constexpr (D == 128)
      *reinterpret_cast<uint16_t*>(rec + q4::k_scales(D) + (lane * 2 + s) * 2) = (uint16_t)(sc[0] | sc[1] << 8);
    else
      rec[q4::k_scales(D) + lane * 2 + s] = (uint8_t)sc[0];
  }
  // ---- values: slice r (dims r*D/8 ..), rows 8s + 2j and 8s + 2j + 1
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t w[2][D / 16];
    int what[2];
    uint32_t sc[2];
    float inv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t at = src(8 * s + 2 * j + e, &what[e]);
      if (what[e] == kWrite) load_vecs<D / 16, WIDE>(v + at + r * (D / 8), w[e]);
      else
#pragma unroll
        for (int i = 0; i < D / 16; ++i) w[e][i] = 0;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t m = group_max<D / 16>(w[e], bad);
      if constexpr (D == 64) m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));   // slices 2g and 2g + 1
      sc[e] = q4::scale_of(m, &inv[e]);
    }
    if (what[0] == kLeave && what[1] == kLeave) continue;
    uint8_t* pc = rec + q4::v_codes(D) + s * 4 * D + lane * kB;
    uint32_t c[kB / 4];
#pragma unroll
    for (int x = 0; x < kB / 4; ++x) c[x] = q4::code_bytes(w[0] + 2 * x, w[1] + 2 * x, make_float2(inv[0], inv[1]));
    if (what[0] == kLeave || what[1] == kLeave) {
      const uint32_t mine = what[0] == kLeave ? 0xf0f0f0f0u : 0x0f0f0f0fu;
      uint32_t old[kB / 4];
      load_bytes<kB>(pc, old);
#pragma unroll
      for (int b4 = 0; b4 < kB / 4; ++b4) c[b4] = (c[b4] & mine) | (old[b4] & ~mine);
    }
    store_bytes<kB>(pc, c);
    if (D == 128 || (r & 1) == 0) {
      uint8_t* ps = rec + q4::v_scales(D) + ((D == 128 ? r : r >> 1) * 4 + j) * 4 + s * 2;
      if (what[0] != kLeave) ps[0] = (uint8_t)sc[0];
      if (what[1] != kLeave) ps[1] = (uint8_t)sc[1];
    }
  }
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
  uint8_t* cache;
  int32_t* pos;
  int* status;
  int B, H_kv, S;
  int64_t warps, rows;               // blocks to write in all; rows of a batch element
  int32_t blk0[kMaxHkv + 1];         // head h writes blocks blk0[h] .. blk0[h+1]-1 of a batch element's list
  int32_t kept[kMaxHkv];
  int64_t off[kMaxHkv];
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) kvc_gather_q4_kernel(const __grid_constant__ GatherArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.warps) return;
  const int per = a.blk0[a.H_kv];
  const int64_t b = i / per;
  const int in = (int)(i - b * per);
  const int h = head_of(a.H_kv, in, [&](int x) { return a.blk0[x]; });
  const int row0 = (in - a.blk0[h]) * q4::kRows;
  const int64_t at0 = b * a.rows + a.off[h] + row0;
  const int n = min(q4::kRows, a.kept[h] - row0);
  int p = lane < n ? a.idx[at0 + lane] : 0;
  bool bad = p < 0 || p >= a.S;
  if (bad) p = 0;                                   // outside the contract: any row of the head, and the status
  const int64_t base = (b * a.H_kv + h) * (int64_t)a.S;
  if (lane < n) a.pos[at0 + lane] = p;
  auto src = [&](int row, int* what) {
    const int pr = __shfl_sync(0xffffffffu, p, row);
    *what = row < n ? kWrite : kZero;
    return (base + pr) * D;
  };
  store_block<D, WIDE>(a.cache + (at0 / q4::kRows) * q4::block_bytes(D), a.k, a.v, src, &bad);
  if (bad) record_status(a.status, kStatusBadInput);
}

struct AppendArgs {
  const __nv_bfloat16 *k, *v;
  const int32_t *pos, *rows;
  uint8_t* cache;
  int32_t* pos_cache;
  int* status;
  int B, T, nb;                      // nb: blocks that T rows may touch
  Q4Slots slots;
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) kvc_append_q4_kernel(const __grid_constant__ AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, H = a.slots.H_kv;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= (int64_t)a.B * H * a.nb) return;
  const int64_t bh = i / a.nb;
  const int64_t b = bh / H;
  const int h = (int)(bh - b * H);
  const int64_t cap = a.slots.off[h + 1] - a.slots.off[h];
  const int n0 = a.rows[bh];
  if (n0 < 0 || (int64_t)n0 + a.T > cap) {          // no room: nothing of this head is written
    if (lane == 0) record_status(a.status, kStatusBadInput);
    return;
  }
  const int64_t row0 = ((int64_t)(n0 / q4::kRows) + (i - bh * a.nb)) * q4::kRows;
  if (row0 >= (int64_t)n0 + a.T) return;
  const int64_t at0 = b * a.slots.off[H] + a.slots.off[h] + row0;
  const int64_t t_of0 = row0 - n0;                  // token of the block's row 0 (may be negative)
  int p = -1;
  if (lane < q4::kRows && t_of0 + lane >= 0 && t_of0 + lane < a.T) {
    p = a.pos[b * a.T + t_of0 + lane];
    if (p < 0) p = -1;                              // an absent token: zeros that no query sees
    a.pos_cache[at0 + lane] = p;
  }
  bool bad = false;
  auto src = [&](int row, int* what) {
    const int pr = __shfl_sync(0xffffffffu, p, row);
    const int64_t t = t_of0 + row;
    *what = (t < 0 || t >= a.T) ? kLeave : pr < 0 ? kZero : kWrite;
    return (bh * a.T + t) * D;
  };
  store_block<D, WIDE>(a.cache + (at0 / q4::kRows) * q4::block_bytes(D), a.k, a.v, src, &bad);
  if (bad) record_status(a.status, kStatusBadInput);
}

struct ReadArgs {
  const uint8_t* cache;
  const int32_t* first;
  __nv_bfloat16 *k_out, *v_out;
  int* status;
  int64_t warps, out_rows;           // blocks to look at in all; output rows of a batch element
  int32_t blk0[kMaxHkv + 1];
  int32_t n_rows[kMaxHkv];
  int64_t out_off[kMaxHkv];
  Q4Slots slots;
};

__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);   // exact
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads) kvc_read_q4_kernel(const __grid_constant__ ReadArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kB = D / 8;
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3, H = a.slots.H_kv;
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.warps) return;
  const int per = a.blk0[H];
  const int64_t b = i / per;
  const int in = (int)(i - b * per);
  const int h = head_of(H, in, [&](int x) { return a.blk0[x]; });
  const int64_t cap = a.slots.off[h + 1] - a.slots.off[h];
  const int64_t first = a.first ? a.first[b * H + h] : 0;
  const int64_t blk = (first >> 4) + (in - a.blk0[h]);
  const int64_t row0 = blk * q4::kRows;
  const int64_t end = first + a.n_rows[h];
  if (row0 >= end) return;
  const bool there = row0 >= 0 && row0 < cap;
  if (!there && lane == 0) record_status(a.status, kStatusBadInput);
  const uint8_t* rec = a.cache + ((b * a.slots.off[H] + a.slots.off[h]) / q4::kRows + (there ? blk : 0)) *
                                     (int64_t)q4::block_bytes(D);
  const int64_t o0 = b * a.out_rows + a.out_off[h] + row0 - first;   // output row of the block's row 0
  const auto wanted = [&](int row) { return row0 + row >= first && row0 + row < end; };
#pragma unroll
  for (int s = 0; s < 2; ++s) {                     // keys: row r + 8s, quarter j
    const int row = r + 8 * s;
    if (!wanted(row)) continue;
    uint32_t dims[kB], *lo = dims, *hi = dims + kB / 2;       // dims b and D/8 + b of the quarter, as bf16 pairs
#pragma unroll
    for (int x = 0; x < kB; ++x) dims[x] = 0;
    if (there) {
      uint32_t c[kB / 4];
      load_bytes<kB>(rec + q4::k_codes(D) + row * (D / 2) + j * kB, c);
      uint32_t sc;
      if constexpr (D == 128) {
        sc = *reinterpret_cast<const uint16_t*>(rec + q4::k_scales(D) + (lane * 2 + s) * 2);
      } else {
        sc = rec[q4::k_scales(D) + lane * 2 + s];
        sc |= sc << 8;
      }
      const uint32_t s2 = q4::scales_to_half2((uint16_t)sc);
#pragma unroll
      for (int x = 0; x < kB / 4; ++x) {
        uint32_t f[4];
        q4::codes_to_half2(c[x], f);
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] = half2_to_bf16x2(q4::mul_half2(f[y], s2));
        lo[2 * x] = __byte_perm(f[0], f[1], 0x5410), hi[2 * x] = __byte_perm(f[0], f[1], 0x7632);
        lo[2 * x + 1] = __byte_perm(f[2], f[3], 0x5410), hi[2 * x + 1] = __byte_perm(f[2], f[3], 0x7632);
      }
    }
    store_vecs<kB, WIDE>(a.k_out + (o0 + row) * D + j * (D / 4), dims);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {                     // values: slice r, rows 8s + 2j and the next
    const int row = 8 * s + 2 * j;
    uint32_t even[kB / 2], odd[kB / 2];
#pragma unroll
    for (int x = 0; x < kB / 2; ++x) even[x] = odd[x] = 0;
    if (there) {
      uint32_t c[kB / 4];
      load_bytes<kB>(rec + q4::v_codes(D) + s * 4 * D + lane * kB, c);
      const uint32_t s2 = q4::scales_to_half2(*reinterpret_cast<const uint16_t*>(
          rec + q4::v_scales(D) + ((D == 128 ? r : r >> 1) * 4 + j) * 4 + s * 2));
#pragma unroll
      for (int x = 0; x < kB / 4; ++x) {
        uint32_t f[4];
        q4::codes_to_half2(c[x], f);
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] = half2_to_bf16x2(q4::mul_half2(f[y], s2));
        even[2 * x] = __byte_perm(f[0], f[1], 0x5410), odd[2 * x] = __byte_perm(f[0], f[1], 0x7632);
        even[2 * x + 1] = __byte_perm(f[2], f[3], 0x5410), odd[2 * x + 1] = __byte_perm(f[2], f[3], 0x7632);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!wanted(row + e)) continue;
      store_vecs<kB / 2, WIDE>(a.v_out + (o0 + row + e) * D + r * (D / 8), e ? odd : even);
    }
  }
}

bool wide(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 31) == 0;
}
dim3 grid_for(int64_t warps) { return dim3((unsigned)((warps + kWarps - 1) / kWarps)); }

}  // namespace

cudaError_t launch_gather_q4(const __nv_bfloat16* k, const __nv_bfloat16* v, const int32_t* idx, int B,
                             const SelParams& sel, int D, uint8_t* cache, int32_t* pos, cudaStream_t st) {
  GatherArgs a{};
  a.k = k, a.v = v, a.idx = idx, a.cache = cache, a.pos = pos, a.status = status_word_ptr();
  a.B = B, a.H_kv = sel.H_kv, a.S = sel.S, a.rows = sel.T;
  for (int h = 0; h < sel.H_kv; ++h) {
    a.kept[h] = sel.kept[h];
    a.off[h] = sel.off[h];
    a.blk0[h + 1] = a.blk0[h] + (sel.kept[h] + q4::kRows - 1) / q4::kRows;
  }
  a.warps = (int64_t)B * a.blk0[sel.H_kv];
  if (a.warps == 0) return cudaSuccess;
  const bool w = wide(k, v);
  auto* kern = D == 128 ? (w ? kvc_gather_q4_kernel<128, true> : kvc_gather_q4_kernel<128, false>)
                        : (w ? kvc_gather_q4_kernel<64, true> : kvc_gather_q4_kernel<64, false>);
  cudaError_t e = launch_pdl(kern, grid_for(a.warps), dim3(kThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_append_q4(const __nv_bfloat16* k, const __nv_bfloat16* v, const int32_t* pos, int B, int T, int D,
                             const Q4Slots& slots, const int32_t* rows, uint8_t* cache, int32_t* pos_cache,
                             cudaStream_t st) {
  AppendArgs a{};
  a.k = k, a.v = v, a.pos = pos, a.rows = rows, a.cache = cache, a.pos_cache = pos_cache;
  a.status = status_word_ptr();
  a.B = B, a.T = T, a.nb = (T + q4::kRows - 2) / q4::kRows + 1;
  a.slots = slots;
  const bool w = wide(k, v);
  auto* kern = D == 128 ? (w ? kvc_append_q4_kernel<128, true> : kvc_append_q4_kernel<128, false>)
                        : (w ? kvc_append_q4_kernel<64, true> : kvc_append_q4_kernel<64, false>);
  cudaError_t e = launch_pdl(kern,
                             grid_for((int64_t)B * slots.H_kv * a.nb), dim3(kThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_read_q4(const uint8_t* cache, int B, int D, const Q4Slots& slots, const int32_t* first,
                           const SelParams& out, __nv_bfloat16* k_out, __nv_bfloat16* v_out, cudaStream_t st) {
  ReadArgs a{};
  a.cache = cache, a.first = first, a.k_out = k_out, a.v_out = v_out, a.status = status_word_ptr();
  a.out_rows = out.T;
  a.slots = slots;
  for (int h = 0; h < slots.H_kv; ++h) {
    const int n = out.kept[h];
    a.n_rows[h] = n;
    a.out_off[h] = out.off[h];
    // an unaligned start may touch one block more
    const int blocks = first ? (n + q4::kRows - 2) / q4::kRows + 1 : (n + q4::kRows - 1) / q4::kRows;
    a.blk0[h + 1] = a.blk0[h] + (n == 0 ? 0 : blocks);
  }
  a.warps = (int64_t)B * a.blk0[slots.H_kv];
  if (a.warps == 0) return cudaSuccess;
  const bool w = wide(k_out, v_out);
  auto* kern = D == 128 ? (w ? kvc_read_q4_kernel<128, true> : kvc_read_q4_kernel<128, false>)
                        : (w ? kvc_read_q4_kernel<64, true> : kvc_read_q4_kernel<64, false>);
  cudaError_t e = launch_pdl(kern, grid_for(a.warps), dim3(kThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvc
