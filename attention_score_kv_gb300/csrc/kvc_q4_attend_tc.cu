// Attention over the 4-bit retained cache (format: kvc_q4.cuh), many query rows
// per KV head: a follow-up prompt, long drafts.
//
// 128 query rows of a KV head (its G*T rows, head by head) against tiles of 128
// cache rows, both products on the tensor cores (tcgen05, fp16 operands, fp32
// accumulators in tensor memory):
//   S = Q K^T  (Q in tensor memory, K in shared memory)
//   O += P V   (P in tensor memory; V in shared)
// 4*128*128*D flops a tile against 128*9D/8 bytes of cache: the products bound
// it, 1024 cycles a tile at D = 128, if nothing else takes longer.  So:
//  - Q and P come from tensor memory: with both operands in shared memory its
//    128 bytes a cycle would be the limit before the products are;
//  - a warp copies tiles of codes in, and four warps turn them into fp16
//    operands (exact, as codes times scales), each 32 cache rows of a tile, in
//    double-buffered shared tiles;
//  - eight warps take the softmax: two threads a row, 64 scores each, against a
//    reference that follows the running maximum only when a score passes it by
//    2^8, so the output in tensor memory is hardly ever rescaled;
//  - S is double buffered and free again as soon as the softmax has it in
//    registers: the next scores are computed while this tile's weights are.
// Orders inside a tile are free (the contraction of S runs over dims, that of O
// over rows), so each operand is written in the order that falls out of the
// block format and keeps 16-byte stores on different banks:
//   dims    16-byte chunk c of a K row: codes 4i .. 4i+3 of quarter j (pairs with
//           the dims D/8 further), c = (D/32) j + i, i ^ 2 in the upper quarters of
//           D = 128; Q is laid out alike
//   rows    row k = r + 8s of block x of a warp's two is row 8 (r / 2) + 4x + 2s +
//           r % 2 of its 32: the four rows of a value pair j, twice, side by side
//   values  dim y of slice r is row r*D/8 + (y ^ 4 (r % 2)) of V^T
// Measured: 512 tokens of 32 heads over 8 heads of 4.9K rows, 38.7 GFLOP, take 45.0
// us (860 TFLOP/s), 1900 to 2000 cycles a tile where the products are 1024.  No one
// thing bounds them: the converters take 1400 and the softmax 1450 of them, a tile
// moves 164 KB through shared memory (1280 cycles at 128 bytes), a product beside
// the softmax's use of tensor memory takes a third longer than alone, and each
// hand-over from warp to warp 150 to 300.  On the way: one warp issuing both
// products 52.5 us, a lane polling alone 57, codes loaded ahead into registers 56
// (a proxy fence waits for loads in flight), eight converter warps with 96
// registers a thread 48.8, Q in shared memory and P twice in tensor memory 55.8.
// Pairs of CTAs that convert half of a tile each for products of 256 rows
// (cta_group::2) have the converters wait half of the time and gain nothing (45.4;
// D = 64 lost 5%): the hand-overs between the two cost what the halves save.
// A CTA takes a row tile of a head.  Few of them leave SMs idle; then the cache
// rows are split over several CTAs per row tile, whose parts a second kernel joins
// in order.  The split is the same for every head and a whole number, so SMs idle
// where row tiles do not divide them (the turn of 512 has 128 on 152 SMs; 16 x 8
// heads of 4096 rows take 36.6 us, 20 x 8, eight more than there are SMs, 70.3) or
// where heads are uneven (7800 and 900 rows by turns under the turn of 512: 69 us,
// even heads of the same sum 45).
#include <algorithm>
#include <cmath>

#include "kvc_q4.cuh"
#include "kvc_scan_common.cuh"

namespace kvc {
namespace {

constexpr int kSoftWarps = 8, kCodeWarps = 4;
constexpr int kScoreWarp = kSoftWarps + kCodeWarps, kOutWarp = kScoreWarp + 1, kLoadWarp = kOutWarp + 1;
constexpr int kThreads = (kLoadWarp + 1) * 32;
constexpr int kRowsM = 128, kKeys = 128;
constexpr int kTileBlocks = kKeys / q4::kRows;
constexpr int kRaw = 3;              // tiles of codes in flight
constexpr int kV = 3;                // stages of V: freed a product later than K's two
// What the queries see of a tile's rows, in the tile's row order.  Tile i's is
// written when the codes of tile i - 3 have been read, that is after K's stage
// was free for tile i - 3, so the scores of tile i - 5 were done; those were
// issued after the softmax of tile i - 7, the last reader, had taken its scores.
constexpr int kSeen = 8;
struct alignas(16) Seen {
  int pos[kKeys];
  uint32_t some[4];                  // rows (of two blocks, in cache order) that some query may see
  uint8_t mixed[4];                  // some query does not see all of these 32
};
__host__ __device__ constexpr int raw_bytes(int D) { return kTileBlocks * q4::block_bytes(D); }
constexpr uint32_t kCols = 512;
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kColP = 448;     // S: two buffers of 128 columns
constexpr float kNoRef = -1.7e38f, kShift = 4.0f, kSlack = 8.0f;

struct TcArgs {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t *pos, *rows, *q_pos;
  __nv_bfloat16* out;
  float* lse;
  float2* part_ml;                   // [row tiles of all heads][splits][128]
  float* part_o;                     // [..][128][D]
  int* status;
  int T, R, extra, tiles, splits;
  uint32_t wait_limit;
  float scale;                       // log2(e) / sqrt(D)
  Q4Slots s;
};

// s_full: the scores of a tile are there, and so K's stage is free.  s_free: the
// softmax has them in registers (and has read what is seen of the tile).
// p_full: the weights are there.  o_done: a tile's output is added up, and so
// V's stage and the weights' columns are free.
// A wait looks at the parity of a phase alone, so no barrier may be two phases
// ahead of a warp that still waits for the first.  What holds each back:
//   raw_full(i + kRaw)   raw_empty(i) of every converter, which saw raw_full(i)
//   raw_empty(i + kRaw)  raw_full(i + kRaw), loaded after a look at raw_empty(i)
//   k_full(i + 2)        s_full(i), issued after a look at k_full(i)
//   v_full(i + kV)       o_done(i), issued after a look at v_full(i)
//   s_full(i + 2)        s_free(i) of the softmax and k_full(i + 2) of the
//                        converters, which all saw s_full(i)
//   s_free(i + 2)        s_full(i + 2), issued after a look at s_free(i)
//   p_full(i + 1)        o_done(i), issued after a look at p_full(i)
//   o_done(i + kV)       p_full(i + 1) and v_full(i + kV), after looks at o_done(i)
// K and V have as many full barriers as stages: on a barrier of K's two, V's
// reader could be overtaken, as the converters wait for the output of kV tiles
// before and not of two.
struct Bars {
  uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[2], v_full[kV], s_full[2], s_free[2], p_full, o_done[kV], q_full,
      drain[2];
};

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Bounded waits of a whole warp, as loops of a few instructions (written out by
// the compiler, the waits made the kernel 3% slower: its warps run five programs
// at once).
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
// Three barriers: a look at one takes about as long alone as with the others.
__device__ __forceinline__ bool poll3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2,
                                      uint32_t limit) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q, r;\n .reg .u32 n;\n mov.u32 n, 0;\n"
      "LOOK:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n and.pred p, p, q;\n and.pred p, p, r;\n @p bra SEEN;\n"
      " add.u32 n, n, 1;\n setp.lt.u32 q, n, %7;\n @q bra LOOK;\n"
      "SEEN:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1), "r"(b2), "r"(p2), "r"(limit)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// Two fp32 operations in one instruction.
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The warp that brings in the cache: a tile's blocks as they are, in one copy,
// and its positions, in the tiles' row order, with what the queries see of them.
template <int D>
__device__ bool load_warp(const TcArgs& a, Bars* bars, uint8_t* raw, Seen* seen, const uint8_t* rec,
                          const int32_t* pos, int n_rows, int t0, int t1, int q_lo, int q_hi) {
  const int lane = threadIdx.x & 31;
  const int n_blocks = (n_rows + q4::kRows - 1) / q4::kRows;
  const int n = t1 - t0;
  // row k of block x of a warp's two, as a place in its 32 (header)
  const int x = lane >> 4, k = lane & 15;
  const int place = ((k & 7) >> 1) * 8 + x * 4 + (k >> 3) * 2 + (k & 1);
  const auto fetch = [&](int t, int (&p)[4]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int row = t * kKeys + w * 32 + lane;
      p[w] = row < n_rows ? __ldg(pos + row) : -1;
    }
  };
  int next[4];
  if (n > 0) fetch(t0, next);
  int i = 0;
  for (; i < n; ++i) {
    const int st = i % kRaw, t = t0 + i;
    int p[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) p[w] = next[w];
    if (i + 1 < n) fetch(t + 1, next);
    if (!poll(smem_u32(&bars->raw_empty[st]), ((i / kRaw) & 1) ^ 1, a.wait_limit)) break;
    Seen& s = seen[i % kSeen];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      s.pos[w * 32 + place] = p[w];
      const bool all = __all_sync(0xffffffffu, p[w] >= 0 && p[w] <= q_lo);
      const uint32_t some = __ballot_sync(0xffffffffu, p[w] >= 0 && p[w] <= q_hi);
      if (lane == 0) s.mixed[w] = all ? 0 : 1, s.some[w] = some;
    }
    __syncwarp();
    if (lane == 0) {
      const uint32_t bytes = min(kTileBlocks, n_blocks - t * kTileBlocks) * q4::block_bytes(D);
      const uint32_t bar = smem_u32(&bars->raw_full[st]);
      tc::mbar_arrive_expect_tx(bar, bytes);
      tc::bulk_g2s(smem_u32(raw + st * raw_bytes(D)), rec + (int64_t)t * raw_bytes(D), bytes, bar);
    }
  }
  // every copy issued has landed before the CTA may leave
  for (int y = max(0, i - kRaw); y < i; ++y)
    scan::drain_wait(smem_u32(&bars->raw_full[y % kRaw]), (y / kRaw) & 1, a.status);
  return i >= n;
}

template <int kB>
__device__ __forceinline__ void read_codes(const uint8_t* p, uint32_t (&w)[kB / 4]) {
  if constexpr (kB == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// A warp of the code converters: 32 rows (two blocks) of every tile.  No load
// from global memory may be in flight here: the proxy fences would wait for it.
template <int D>
__device__ bool code_warp(const TcArgs& a, Bars* bars, uint32_t sK, uint32_t sV, const uint8_t* raw, const Seen* seen,
                          int n) {
  constexpr int kB = D / 8;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kSoftWarps, r = lane >> 2, j = lane & 3;
  for (int i = 0; i < n; ++i) {
    const int st = i & 1, rs = i % kRaw, vst = i % kV;
    const uint32_t ph = ((i >> 1) & 1) ^ 1;
    if (!poll3(smem_u32(&bars->raw_full[rs]), (i / kRaw) & 1, smem_u32(&bars->s_full[st]), ph,
               smem_u32(&bars->o_done[vst]), ((i / kV) & 1) ^ 1, a.wait_limit))
      return false;
    const uint8_t* rec = raw + rs * raw_bytes(D) + 2 * w * q4::block_bytes(D);
    // ---- keys
    // place of (block b, half s, chunk c) for this lane: tiles are 1024-aligned, so what
    // the lane adds and what the step adds are different bits, or swizzle bits to flip
    const uint32_t k_at = (sK + st * (kKeys * D * 2) + (D == 128 ? (j >> 1) * (kKeys * 128) : 0) +
                           (w * 32 + (r >> 1) * 8 + (r & 1)) * 128) |
                          ((D == 128 ? (j & 1) * 4 ^ 2 * (j >> 1) : j * 2) ^ (r & 1)) << 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint8_t* p = rec + b * q4::block_bytes(D);
      const uint32_t ks = D == 128 ? *reinterpret_cast<const uint32_t*>(p + q4::k_scales(D) + lane * 4)
                                   : *reinterpret_cast<const uint16_t*>(p + q4::k_scales(D) + lane * 2);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t two = D == 128 ? ks >> (16 * s) : (ks >> (8 * s) & 0xffu) * 0x101u;
        const uint32_t s2 = q4::scales_to_half2((uint16_t)two);
        uint32_t code[D / 32];
        read_codes<kB>(p + q4::k_codes(D) + s * 4 * D + lane * kB, code);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t f[4];
          q4::codes_to_half2(code[c], f);
          store16(k_at ^ ((b * 4 + s * 2) * 128 | (c ^ (b * 4 + s * 2)) << 4), q4::mul_half2(f[0], s2),
                  q4::mul_half2(f[1], s2), q4::mul_half2(f[2], s2), q4::mul_half2(f[3], s2));
        }
      }
    }
    // ---- values.  A row that no query sees may hold anything: its values count as zeros
    uint32_t code[2][2][D / 32], s2[2][2];
    const uint32_t some = seen[i % kSeen].some[w];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint8_t* p = rec + b * q4::block_bytes(D);
      uint32_t vs = *reinterpret_cast<const uint32_t*>(p + q4::v_scales(D) + ((D == 128 ? r : r >> 1) * 4 + j) * 4);
      const uint32_t see = some >> (16 * b + 2 * j);         // rows 2j, 2j + 1 and 2j + 8, 2j + 9 of the block
      vs &= (see & 1 ? 0x000000ffu : 0u) | (see & 2 ? 0x0000ff00u : 0u) | (see & 0x100 ? 0x00ff0000u : 0u) |
            (see & 0x200 ? 0xff000000u : 0u);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        s2[b][s] = q4::scales_to_half2((uint16_t)(vs >> (16 * s)));
        read_codes<kB>(p + q4::v_codes(D) + s * 4 * D + lane * kB, code[b][s]);
      }
    }
    const uint32_t v_at = (sV + vst * (kKeys * D * 2) + (w >> 1) * (D * 128) + r * (D / 8) * 128) |
                          ((4 * (r & 1)) * 128 | (((w & 1) * 4 + j) ^ (4 * (r & 1))) << 4);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t f[2][2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s) q4::codes_to_half2(code[b][s][c], f[b][s]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        store16(v_at ^ ((4 * c + e) * 128 | ((4 * c + e) & 7) << 4), q4::mul_half2(f[0][0][e], s2[0][0]),
                q4::mul_half2(f[0][1][e], s2[0][1]), q4::mul_half2(f[1][0][e], s2[1][0]),
                q4::mul_half2(f[1][1][e], s2[1][1]));
      }
    }
    tc::fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      tc::mbar_arrive(smem_u32(&bars->k_full[st]));
      tc::mbar_arrive(smem_u32(&bars->v_full[vst]));
      tc::mbar_arrive(smem_u32(&bars->raw_empty[rs]));
    }
  }
  return true;
}

// A product takes the tensor core 64 cycles, and arithmetic on descriptors
// between products took twice that from the one thread that issues them: they
// are made once, and steps add constants to them.
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool first) {
  if (first)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, 0, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.eq.b32 p, 0, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc)
        : "memory");
}
// Two warps issue the products, one the scores, one the outputs: between its
// tiles an issuer spends as long on waits and instruction fetches as its
// products run, which the other's products cover.  Each waits as a whole (a
// lane that polls alone costs 300 cycles a wait, the warp together 20 to 90);
// lane 0 issues.
template <int D>
__device__ bool score_warp(const TcArgs& a, Bars* bars, uint32_t sK, uint32_t tmem, int n) {
  constexpr uint32_t kId = tc::idesc_f16(kRowsM, kKeys);
  constexpr uint64_t kStage = kKeys * D * 2 >> 4;              // descriptor units of 16 bytes
  const bool issues = (threadIdx.x & 31) == 0;
  const uint64_t k0 = tc::desc_sw128(sK);
  const auto wait = [&](uint64_t* bar, int phase) { return poll(smem_u32(bar), phase & 1, a.wait_limit); };
  bool ok = wait(&bars->q_full, 0);
  if (ok) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      ok = wait(&bars->k_full[st], i >> 1) && wait(&bars->s_free[st], (i >> 1) ^ 1);
      if (!ok) break;
      tc::fence_after_sync();
      if (issues) {
        const uint64_t kd = k0 + st * kStage;
        const uint32_t sd = tmem + kColS + st * kKeys;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_ta(sd, tmem + kColQ + s * 8, kd + (((s >> 2) * (kKeys * 128) + (s & 3) * 32) >> 4), kId, s == 0);
        tc::mma_commit(smem_u32(&bars->s_full[st]));
      }
      __syncwarp();
    }
  }
  if (issues) scan::drain_mma(smem_u32(&bars->drain[0]), a.status);
  __syncwarp();
  return ok;
}
template <int D>
__device__ bool out_warp(const TcArgs& a, Bars* bars, uint32_t sV, uint32_t tmem, int n) {
  constexpr uint32_t kId = tc::idesc_f16(kRowsM, D);
  constexpr uint64_t kStage = kKeys * D * 2 >> 4;
  const bool issues = (threadIdx.x & 31) == 0;
  const uint64_t v0 = tc::desc_sw128(sV);
  const auto wait = [&](uint64_t* bar, int phase) { return poll(smem_u32(bar), phase & 1, a.wait_limit); };
  bool ok = true;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    ok = wait(&bars->v_full[i % kV], i / kV) && wait(&bars->p_full, i);
    if (!ok) break;
    tc::fence_after_sync();
    if (issues) {
      const uint64_t vd = v0 + (i % kV) * kStage;
      const uint32_t pd = tmem + kColP, od = tmem + kColO;
      if (i == 0) mma_ta(od, pd, vd, kId, true);
      else mma_ta(od, pd, vd, kId, false);
#pragma unroll
      for (int s = 1; s < kKeys / 16; ++s)
        mma_ta(od, pd + s * 8, vd + (((s >> 2) * (D * 128) + (s & 3) * 32) >> 4), kId, false);
      tc::mma_commit(smem_u32(&bars->o_done[i % kV]));
    }
    __syncwarp();
  }
  if (issues) scan::drain_mma(smem_u32(&bars->drain[1]), a.status);
  __syncwarp();
  return ok;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kvc_attend_q4_tc_kernel(const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(16) Seen s_seen[kSeen];
  __shared__ float s_x[2][2][kRowsM];              // what the two threads of a row tell each other

  const uint32_t sK = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sV = sK + 2 * kKeys * D * 2;
  uint8_t* raw = smem_raw + (sV + kV * kKeys * D * 2 - smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.x / a.tiles, tile = blockIdx.x - bh * a.tiles;
  // warps of the softmax that have query rows; nothing reads what the products make of
  // the others' rows, whatever tensor memory holds there
  const int live_quarters = min(4, (a.R - tile * kRowsM + 31) / 32), live_warps = 2 * live_quarters;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) {
      tc::mbar_init(smem_u32(&bars.raw_full[i]), 1);
      tc::mbar_init(smem_u32(&bars.raw_empty[i]), kCodeWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(smem_u32(&bars.k_full[i]), kCodeWarps);
      tc::mbar_init(smem_u32(&bars.s_full[i]), 1);
      tc::mbar_init(smem_u32(&bars.s_free[i]), live_warps);
      tc::mbar_init(smem_u32(&bars.drain[i]), 1);
    }
    for (int i = 0; i < kV; ++i) {
      tc::mbar_init(smem_u32(&bars.v_full[i]), kCodeWarps);
      tc::mbar_init(smem_u32(&bars.o_done[i]), 1);
    }
    tc::mbar_init(smem_u32(&bars.p_full), live_warps);
    tc::mbar_init(smem_u32(&bars.q_full), live_warps);
    tc::fence_barrier_init();
  }
  if (warp == kScoreWarp) {
    tc::tmem_alloc(smem_u32(&s_tmem), kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  grid_dep_wait();
  grid_dep_launch();

  const int H = a.s.H_kv, b = bh / H, h = bh - b * H;
  const int64_t row0 = (int64_t)b * a.s.off[H] + a.s.off[h];
  const int64_t cap = a.s.off[h + 1] - a.s.off[h];
  int64_t held = (int64_t)__ldg(a.rows + bh) + a.extra;
  if (held < 0 || held > cap) {
    if (threadIdx.x == 0) record_status(a.status, kStatusBadInput);
    held = held < 0 ? 0 : cap;
  }
  const int n_rows = (int)held;
  const int key_tiles = (n_rows + kKeys - 1) / kKeys, per = (key_tiles + a.splits - 1) / a.splits;
  const int t0 = min((int)blockIdx.y * per, key_tiles), t1 = min(t0 + per, key_tiles), n = t1 - t0;

  bool ok = true;                    // false: a wait gave up
  if (warp == kLoadWarp) {
    int q_lo = INT32_MAX, q_hi = -1;
    for (int i = lane; i < kRowsM; i += 32) {
      const int row = tile * kRowsM + i;
      if (row < a.R) {
        const int p = __ldg(a.q_pos + (int64_t)b * a.T + row % a.T);
        q_lo = min(q_lo, p), q_hi = max(q_hi, p);
      }
    }
    q_lo = __reduce_min_sync(0xffffffffu, q_lo);
    q_hi = __reduce_max_sync(0xffffffffu, q_hi);
    ok = load_warp<D>(a, &bars, raw, s_seen, a.cache + row0 / q4::kRows * q4::block_bytes(D), a.pos + row0, n_rows, t0,
                      t1, q_lo, q_hi);
  } else if (warp >= kSoftWarps && warp < kScoreWarp) {
    ok = code_warp<D>(a, &bars, sK, sV, raw, s_seen, n);
  } else if (warp == kScoreWarp) {
    if (n > 0) ok = score_warp<D>(a, &bars, sK, tmem, n);
  } else if (warp == kOutWarp) {
    if (n > 0) ok = out_warp<D>(a, &bars, sV, tmem, n);
  } else if ((warp & 3) < live_quarters) {
    // ---- softmax: thread (row, half): dims and scores [half * .., ..)
    constexpr int kHalfD = D / 2;
    const int half = warp >> 2, in = (warp & 3) * 32 + lane, row = tile * kRowsM + in;
    const bool live = row < a.R;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int qp = live ? __ldg(a.q_pos + (int64_t)b * a.T + row % a.T) : -1;
    float c2;
    {
      uint32_t w[kHalfD / 2];
#pragma unroll
      for (int i = 0; i < kHalfD / 2; ++i) w[i] = 0;
      if (live) {
        const uint4* p = reinterpret_cast<const uint4*>(a.q + ((int64_t)bh * a.R + row) * D + half * kHalfD);
#pragma unroll
        for (int i = 0; i < kHalfD / 8; ++i) {
          const uint4 v = __ldg(p + i);
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
      }
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < kHalfD / 2; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
      mx = max(mx & 0xffffu, mx >> 16);
      s_x[0][half][in] = __uint_as_float(mx);
      asm volatile("bar.sync 1, %0;\n" ::"r"(live_warps * 32) : "memory");
      mx = max(mx, __float_as_uint(s_x[0][half ^ 1][in]));
      // scale by the power of two that brings the row's largest value into [1, 2)
      const uint32_t e = mx >> 7, ee = (e == 0 || e == 255) ? 127u : min(e, 253u);
      const float down = __uint_as_float((254u - ee) << 23);
      c2 = __uint_as_float(ee << 23) * a.scale;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj)               // the half's two quarters
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            v[y] = half2_of(__uint_as_float(q4::bf16_of(w, jj * (D / 4) + 4 * i + y) << 16) * down,
                            __uint_as_float(q4::bf16_of(w, jj * (D / 4) + D / 8 + 4 * i + y) << 16) * down);
          const int j = 2 * half + jj;
          const int chunk = D == 128 ? j * 4 + (i ^ (2 * half)) : j * 2 + i;
          tc::tmem_st4(tmem + lanes + kColQ + chunk * 4, v);
        }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(smem_u32(&bars.q_full));
      asm volatile("bar.sync 1, %0;\n" ::"r"(live_warps * 32) : "memory");       // s_x is free again
    }

    float ref = kNoRef;
    float2 sum2[2] = {};             // the row's sum, in four parts
    // after a wait that gave up: go on without waiting, so that no barrier is left alone
    const auto wait = [&](uint64_t* bar, int phase) { return poll(smem_u32(bar), phase & 1, a.wait_limit); };
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint32_t s_at = tmem + lanes + kColS + st * kKeys + half * 64;
      ok = ok && wait(&bars.s_full[st], i >> 1);
      tc::fence_after_sync();
      float x[64];
#pragma unroll
      for (int y = 0; y < 4; ++y) tc::tmem_ld16(s_at + 16 * y, x + 16 * y);
      const uint32_t mixed = *reinterpret_cast<const uint16_t*>(&s_seen[i % kSeen].mixed[2 * half]);
      tc::tmem_wait_ld();
      tc::reg_fence(x, 64);
      if (mixed) {
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int4 p = *reinterpret_cast<const int4*>(&s_seen[i % kSeen].pos[half * 64 + 4 * y]);
          if (p.x < 0 || p.x > qp) x[4 * y] = -INFINITY;
          if (p.y < 0 || p.y > qp) x[4 * y + 1] = -INFINITY;
          if (p.z < 0 || p.z > qp) x[4 * y + 2] = -INFINITY;
          if (p.w < 0 || p.w > qp) x[4 * y + 3] = -INFINITY;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(smem_u32(&bars.s_free[st]));
      float m = x[0], m1 = x[1];     // two chains of three-input maxima
#pragma unroll
      for (int y = 2; y < 62; y += 4) m = max3(m, x[y], x[y + 1]), m1 = max3(m1, x[y + 2], x[y + 3]);
      m = fmaxf(max3(m, x[62], x[63]), m1);
      s_x[st][half][in] = m;
      asm volatile("bar.sync %0, 64;\n" ::"r"(2 + (warp & 3)) : "memory");
      m = fmaxf(m, s_x[st][half ^ 1][in]) * c2;
      const bool move = __any_sync(0xffffffffu, m > ref + (kSlack + kShift));
      float f = 1.f;
      if (move) {
        const float to = fmaxf(ref, m - kShift);
        f = ex2(ref - to);
        ref = to;
#pragma unroll
        for (int y = 0; y < 2; ++y) sum2[y].x *= f, sum2[y].y *= f;
      }
      const float2 c22 = make_float2(c2, c2), ref2 = make_float2(-ref, -ref);
      uint32_t p[32];
#pragma unroll
      for (int z = 0; z < 32; ++z) {
        const float2 e = fma2(make_float2(x[2 * z], x[2 * z + 1]), c22, ref2);
        const float2 u = make_float2(ex2(e.x), ex2(e.y));
        sum2[z & 1] = add2(sum2[z & 1], u);
        p[z] = half2_of(u.x, u.y);
      }
      // the weights' columns, and the output for a new reference, are free when the
      // last tile's output is added up
      if (i > 0) {
        ok = ok && wait(&bars.o_done[(i - 1) % kV], (i - 1) / kV);
        tc::fence_after_sync();
        if (move) {
#pragma unroll
          for (int y = 0; y < kHalfD / 16; ++y) {
            float o[16];
            const uint32_t at = tmem + lanes + kColO + half * kHalfD + 16 * y;
            tc::tmem_ld16(at, o);
            tc::tmem_wait_ld();
            tc::reg_fence(o, 16);
#pragma unroll
            for (int z = 0; z < 16; ++z) o[z] *= f;
            tc::tmem_st16(at, reinterpret_cast<const uint32_t*>(o));
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) tc::tmem_st16(tmem + lanes + kColP + half * 32 + 16 * y, p + 16 * y);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(smem_u32(&bars.p_full));
    }
    // ---- the row: both halves' sums, and this half's dims
    float sum = (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
    asm volatile("bar.sync 1, %0;\n" ::"r"(live_warps * 32) : "memory");
    s_x[0][half][in] = sum;
    asm volatile("bar.sync 1, %0;\n" ::"r"(live_warps * 32) : "memory");
    sum = s_x[0][0][in] + s_x[0][1][in];
    if (n > 0) {
      ok = ok && wait(&bars.o_done[(n - 1) % kV], (n - 1) / kV);
      tc::fence_after_sync();
    }
    const bool whole = a.splits == 1;
    const float f = whole ? (sum == 0.f ? 0.f : 1.0f / sum) : 1.f;
    const int64_t at = (int64_t)bh * a.R + row;
    const int64_t part = ((int64_t)blockIdx.x * a.splits + blockIdx.y) * kRowsM + in;
#pragma unroll
    for (int y = 0; y < kHalfD / 16; ++y) {
      float o[16];
      if (n > 0) {
        tc::tmem_ld16(tmem + lanes + kColO + half * kHalfD + 16 * y, o);
        tc::tmem_wait_ld();
        tc::reg_fence(o, 16);
      }
      // columns are rows of V^T; the groups of four are swapped where the slice is odd
      float v[16];
#pragma unroll
      for (int z = 0; z < 16; ++z) {
        const int n_of = half * kHalfD + 16 * y + z;
        const int odd = D == 128 ? y & 1 : (n_of >> 3) & 1;
        v[z] = n > 0 && sum != 0.f ? o[z ^ (4 * odd)] * f : 0.f;
      }
      const int d0 = half * kHalfD + 16 * y;
      if (whole) {
        if (live) {
          uint32_t w[8];
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const __nv_bfloat162 c = __floats2bfloat162_rn(v[2 * z], v[2 * z + 1]);
            w[z] = *reinterpret_cast<const uint32_t*>(&c);
          }
          uint4* to = reinterpret_cast<uint4*>(a.out + at * D + d0);
          to[0] = make_uint4(w[0], w[1], w[2], w[3]);
          to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      } else if (live) {
        float4* to = reinterpret_cast<float4*>(a.part_o + part * D + d0);
#pragma unroll
        for (int z = 0; z < 4; ++z) to[z] = make_float4(v[4 * z], v[4 * z + 1], v[4 * z + 2], v[4 * z + 3]);
      }
    }
    if (half == 0 && live) {
      if (!whole) a.part_ml[part] = make_float2(ref, sum);
      else if (a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994530942f;
    }
  }
  if (!ok && lane == 0) record_status(a.status, kStatusTimeout);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kScoreWarp) tc::tmem_dealloc(tmem, kCols);
}

// Joins the parts of a query row's splits.  WPR warps share a row, each summing
// every WPR-th part in order, and their sums are added in warp order; a CTA of
// four warps holds 4 / WPR rows.
template <int D, int WPR>
__global__ void __launch_bounds__(128) kvc_attend_q4_tc_join_kernel(const __grid_constant__ TcArgs a, int64_t n_rows) {
  constexpr int V = D / 32;
  __shared__ float s_v[4][D + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = warp % WPR;
  const int64_t at = (int64_t)blockIdx.x * (4 / WPR) + warp / WPR;
  const bool on = at < n_rows;
  const int64_t bh = on ? at / a.R : 0;
  const int row = on ? (int)(at - bh * a.R) : 0;
  const int64_t first = ((bh * a.tiles + row / kRowsM) * a.splits) * kRowsM + row % kRowsM;
  float top = kNoRef;
  for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_ml[first + (int64_t)s * kRowsM].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float l = 0.f, v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int s = me; s < a.splits; s += WPR) {
    const int64_t p = first + (int64_t)s * kRowsM;
    const float2 ml = a.part_ml[p];
    const float f = ex2(ml.x - top);
    l = fmaf(ml.y, f, l);
    const float* o = a.part_o + p * D + lane * V;
    float y[V];
    if constexpr (V == 4) *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(o);
    else *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(o);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fmaf(y[i], f, v[i]);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_v[warp][lane * V + i] = v[i];
    if (lane == 0) s_v[warp][D] = l;
    __syncthreads();
    if (me > 0) return;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      l += s_v[warp + w][D];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += s_v[warp + w][lane * V + i];
    }
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = l == 0.f ? 0.f : v[i] / l;
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const __nv_bfloat162 c = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&c);
  }
  __nv_bfloat16* o = a.out + at * D + lane * V;
  if constexpr (V == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace

Q4TcPlan plan_attend_q4_tc(int B, int T, int H_q, int H_kv, int D) {
  Q4TcPlan p{};
  const int64_t R = (int64_t)(H_q / H_kv) * T;
  p.tiles = (int)((R + kRowsM - 1) / kRowsM);
  const int64_t units = (int64_t)B * H_kv * p.tiles;
  // one wave: as many CTAs as SMs, never more parts than that
  p.splits = (int)std::max<int64_t>(1, std::max(num_sms(), 1) / units);
  if (p.splits > 1) {
    const size_t rows = (size_t)units * p.splits * kRowsM;
    p.off_o = (rows * sizeof(float2) + 255) / 256 * 256;
    p.total = p.off_o + rows * D * sizeof(float);
  }
  return p;
}

cudaError_t launch_attend_q4_tc(const __nv_bfloat16* q, const uint8_t* cache, const int32_t* pos, const int32_t* rows,
                                int extra, const int32_t* q_pos, int B, int T, int H_q, int D, const Q4Slots& slots,
                                __nv_bfloat16* out, float* lse, void* ws, cudaStream_t st) {
  const int H = slots.H_kv;
  const Q4TcPlan p = plan_attend_q4_tc(B, T, H_q, H, D);
  TcArgs a{};
  a.q = q, a.cache = cache, a.pos = pos, a.rows = rows, a.q_pos = q_pos, a.out = out, a.lse = lse;
  a.part_ml = static_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_o);
  a.status = status_word_ptr();
  a.T = T, a.R = H_q / H * T, a.extra = extra, a.tiles = p.tiles;
  // no more splits than leave two tiles to each in the longest slot
  int64_t longest = 0;
  for (int h = 0; h < H; ++h) longest = std::max(longest, slots.off[h + 1] - slots.off[h]);
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(p.splits, (longest + 2 * kKeys - 1) / (2 * kKeys)));
  a.wait_limit = wait_limit_polls();
  a.scale = (float)(1.4426950408889634 / std::sqrt((double)D));
  a.s = slots;
  const size_t smem = (2 + kV) * (size_t)kKeys * D * 2 + kRaw * (size_t)raw_bytes(D) + 1024;
  auto* kern = D == 128 ? kvc_attend_q4_tc_kernel<128> : kvc_attend_q4_tc_kernel<64>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e == cudaSuccess)
    e = launch_pdl(kern, dim3((unsigned)(B * H * p.tiles), a.splits), dim3(kThreads), smem, st, a);
  note_launches(1);
  if (e != cudaSuccess) return e;
  if (a.splits > 1) {
    const int64_t n = (int64_t)B * H_q * T;
    const bool wide = a.splits > 8;                // many parts of few rows: four warps a row
    auto* join = D == 128 ? (wide ? kvc_attend_q4_tc_join_kernel<128, 4> : kvc_attend_q4_tc_join_kernel<128, 1>)
                          : (wide ? kvc_attend_q4_tc_join_kernel<64, 4> : kvc_attend_q4_tc_join_kernel<64, 1>);
    e = launch_pdl(join, dim3((unsigned)(wide ? n : (n + 3) / 4)), dim3(128), 0, st, a, n);
    note_launches(1);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvc
