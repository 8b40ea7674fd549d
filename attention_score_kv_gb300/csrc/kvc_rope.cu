// Norm of queries and keys per head, with the position rotation in the same
// pass, from the projections' output into the layouts that the scorer and the
// active layer's buffers have:
//
//   y = x / sqrt(mean(x^2) + eps) * w              (fp32; left out without w)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin),  angle = pos * inv_freq
//
// rounded once, to bf16.  Values are copied along, so one pass over a token's
// projections does what an append of the chunk needs.
//
// The angle: pos * inv_freq in fp32 is 6e-3 rad off at position 10^5.  Here a
// frequency becomes a 64-bit binary fraction of a turn; the product with the
// integer position drops whole turns by wrapping around, and its upper 32 bits
// go to the sine and cosine as a fp32 number.  The fraction comes from a product
// in fp64, 2^-52 of the frequency off at most, which the position multiplies;
// the upper bits and their rounding to fp32 leave 2^-25 of a turn: together below
// 1e-6 rad plus pos * inv_freq * 2^-52.  The fp64 steps are done for every token
// and frequency of a CTA, once for all of the token's heads.
//
// Memory bounds it: every value is read and written once.  A chunk of 2048
// tokens of 32 + 2 x 8 heads of 128 takes 12.2 us (50 MB, 4.1 TB/s), one token
// 2.8 us.  Each thread has three shares of 32 bytes on their way before the
// angles are worked out, once per token for all of its heads (one token a CTA and
// no loads ahead: 15.4 us; with the table in frequency order, four lanes on a
// bank: 14.3 us).
//
// Eight lanes hold a head of 128 (four one of 64): 16 values each, as two
// 16-byte vectors that hold both halves of the rotated pairs, so the only
// exchange between lanes is the norm's sum.
#include <algorithm>

#include "kvc_device.cuh"
#include "kvc_internal.cuh"

namespace kvc {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTok = 16;          // tokens of a CTA
constexpr int kUnits = 3;            // lane shares a thread has in flight

struct RopeArgs {
  const __nv_bfloat16 *q, *k, *v;
  const __nv_bfloat16 *qw, *kw;
  const float* inv_freq;
  const int32_t* pos;
  __nv_bfloat16 *q_out, *k_act, *v_act;
  int64_t q_ld, k_ld, v_ld, n_tok;   // n_tok = B * T
  int64_t row0, S;
  int T, H_q, H_kv, R, tok;          // tok: tokens of a CTA
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) kvc_qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int LPH = D / 16;        // lanes of a head
  __shared__ float2 turn[kMaxTok][D / 2];
  const uint32_t tok0 = blockIdx.x * (uint32_t)a.tok;
  const int n_tok = (int)min((uint32_t)a.tok, (uint32_t)a.n_tok - tok0);
  const int half = a.R / 2;
  const uint32_t heads = a.H_q + 2 * a.H_kv;
  const uint32_t units = n_tok * heads * LPH;
  const int l = threadIdx.x % LPH;   // kRopeThreads is a multiple of LPH
  const int rot = a.R / 16;          // lanes that hold rotated pairs
  // chunks of 8 values: lanes below `rot` hold l and l + rot, the others two of the rest
  const int c0 = l < rot ? l : 2 * l, c1 = l < rot ? l + rot : 2 * l + 1;

  for (uint32_t u0 = 0; u0 < units; u0 += kRopeThreads * kUnits) {
    uint4 x[kUnits][2];
    __nv_bfloat16* dst[kUnits];
    int kind[kUnits], tok[kUnits];   // 0: query, 1: key, 2: value, -1: nothing
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t u = u0 + i * kRopeThreads + threadIdx.x;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      kind[i] = -1, tok[i] = 0, dst[i] = nullptr;
      if (u >= units) continue;
      const uint32_t hd = u / LPH, t = hd / heads, h = hd - t * heads;
      const uint32_t at = tok0 + t, b = at / (uint32_t)a.T, tt = at - b * a.T;
      const __nv_bfloat16* src;
      tok[i] = t;
      if (h < (uint32_t)a.H_q) {
        kind[i] = 0;
        src = a.q + at * a.q_ld + (int64_t)h * D;
        dst[i] = a.q_out + (((int64_t)b * a.H_q + h) * a.T + tt) * D;
      } else if (h < (uint32_t)(a.H_q + a.H_kv)) {
        const uint32_t g = h - a.H_q;
        kind[i] = 1;
        src = a.k + at * a.k_ld + (int64_t)g * D;
        dst[i] = a.k_act + (((int64_t)b * a.H_kv + g) * a.S + a.row0 + tt) * D;
      } else {
        if (!a.v) continue;
        const uint32_t g = h - a.H_q - a.H_kv;
        kind[i] = 2;
        src = a.v + at * a.v_ld + (int64_t)g * D;
        dst[i] = a.v_act + (((int64_t)b * a.H_kv + g) * a.S + a.row0 + tt) * D;
      }
      x[i][0] = *reinterpret_cast<const uint4*>(src + c0 * 8);
      x[i][1] = *reinterpret_cast<const uint4*>(src + c1 * 8);
    }
    if (u0 == 0) {                   // behind the first loads
      for (int i = threadIdx.x; i < n_tok * half; i += kRopeThreads) {
        const int t = i / half, f = i - t * half;
        const double u = (double)a.inv_freq[f] * 0.15915494309189533577;       // 1 / (2 pi)
        const uint64_t frac = (uint64_t)((u - floor(u)) * 18446744073709551616.0);
        const uint64_t at = (uint64_t)(int64_t)a.pos[tok0 + t] * frac;
        float s, c;
        sincospif((float)(int32_t)(at >> 32) * (1.0f / 2147483648.0f), &s, &c);
        // where the lanes of a head read side by side
        turn[t][INTER ? (f & 3) * (2 * rot) + (f >> 2) : (f & 7) * rot + (f >> 3)] = make_float2(c, s);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (kind[i] == 0 || kind[i] == 1) {        // the lanes of a head agree
        float y[16];
        unpack8(x[i][0], y);
        unpack8(x[i][1], y + 8);
        const __nv_bfloat16* w = kind[i] == 0 ? a.qw : a.kw;
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int z = 0; z < 16; ++z) ss = fmaf(y[z], y[z], ss);
          const uint32_t head_lanes = ((1u << LPH) - 1) << ((threadIdx.x & 31) / LPH * LPH);
#pragma unroll
          for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(head_lanes, ss, o);
          const float rms = rsqrtf(ss * (1.0f / D) + a.eps);
          float g[16];
          unpack8(__ldg(reinterpret_cast<const uint4*>(w + c0 * 8)), g);
          unpack8(__ldg(reinterpret_cast<const uint4*>(w + c1 * 8)), g + 8);
#pragma unroll
          for (int z = 0; z < 16; ++z) y[z] = y[z] * rms * g[z];
        }
        if (l < rot) {
          const float2* cs = turn[tok[i]];
          if constexpr (INTER) {
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              const float2 t = cs[(z & 3) * (2 * rot) + (z < 4 ? c0 : c1)];
              const float p = y[2 * z], r = y[2 * z + 1];
              y[2 * z] = p * t.x - r * t.y;
              y[2 * z + 1] = r * t.x + p * t.y;
            }
          } else {
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              const float2 t = cs[z * rot + c0];
              const float p = y[z], r = y[8 + z];
              y[z] = p * t.x - r * t.y;
              y[8 + z] = r * t.x + p * t.y;
            }
          }
        }
        x[i][0] = pack8(y);
        x[i][1] = pack8(y + 8);
      }
      if (kind[i] >= 0) {
        *reinterpret_cast<uint4*>(dst[i] + c0 * 8) = x[i][0];
        *reinterpret_cast<uint4*>(dst[i] + c1 * 8) = x[i][1];
      }
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v, int B, int T,
                                int H_q, int H_kv, int D, int64_t q_ld, int64_t k_ld, int64_t v_ld, int R, bool inter,
                                const __nv_bfloat16* qw, const __nv_bfloat16* kw, float eps, const float* inv_freq,
                                const int32_t* pos, int S, int row0, __nv_bfloat16* q_out, __nv_bfloat16* k_act,
                                __nv_bfloat16* v_act, cudaStream_t st) {
  RopeArgs a{q, k, v, qw, kw, inv_freq, pos, q_out, k_act, v_act, q_ld, k_ld, v_ld, (int64_t)B * T,
             row0, S, T, H_q, H_kv, R, 1, eps};
  auto* kern = D == 128 ? (inter ? kvc_qk_norm_rope_kernel<128, true> : kvc_qk_norm_rope_kernel<128, false>)
                        : (inter ? kvc_qk_norm_rope_kernel<64, true> : kvc_qk_norm_rope_kernel<64, false>);
  // tokens of a CTA: what its threads can have in flight, as long as two CTAs an SM
  // are left; a token's angles are worked out once for all of its heads
  const int per_tok = (H_q + 2 * H_kv) * (D / 16);
  const int64_t full = std::max<int64_t>(1, kRopeThreads * kUnits / per_tok);
  const int64_t spread = (a.n_tok + 2 * std::max(num_sms(), 1) - 1) / (2 * std::max(num_sms(), 1));
  a.tok = (int)std::min<int64_t>({full, spread, kMaxTok});
  const int64_t grid = (a.n_tok + a.tok - 1) / a.tok;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)grid), dim3(kRopeThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvc
