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
// frequency becomes a 64-bit binary fraction of a turn, once per thread; the
// product with the integer position drops whole turns by wrapping around, and
// its upper 32 bits are the angle to 2^-32 of a turn (times 2 pi), exact for
// every int32 position.
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
constexpr int kMaxTok = 4;           // tokens of a CTA

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
  const int64_t tok0 = (int64_t)blockIdx.x * a.tok;
  const int n_tok = (int)min((int64_t)a.tok, a.n_tok - tok0);
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < n_tok * half; i += kRopeThreads) {
    const int t = i / half, f = i - t * half;
    const double u = (double)a.inv_freq[f] * 0.15915494309189533577;       // 1 / (2 pi)
    const uint64_t frac = (uint64_t)((u - floor(u)) * 18446744073709551616.0);
    const uint64_t at = (uint64_t)(int64_t)a.pos[tok0 + t] * frac;
    float s, c;
    sincospif((float)(int32_t)(at >> 32) * (1.0f / 2147483648.0f), &s, &c);
    turn[t][f] = make_float2(c, s);
  }
  __syncthreads();

  const int heads = a.H_q + 2 * a.H_kv;
  const int units = n_tok * heads * LPH;
  const int l = threadIdx.x % LPH;   // kRopeThreads is a multiple of LPH
  const int rot = a.R / 16;          // lanes that hold rotated pairs
  // chunks of 8 values: lanes below `rot` hold l and l + rot, the others two of the rest
  const int c0 = l < rot ? l : 2 * l, c1 = l < rot ? l + rot : 2 * l + 1;
  for (int u0 = 0; u0 < units; u0 += kRopeThreads) {
    const int u = u0 + threadIdx.x;
    const bool live = u < units;
    const int hd = live ? u / LPH : 0;
    const int t = hd / heads, h = hd - t * heads;
    const int64_t tok = tok0 + t;
    const int64_t b = tok / a.T, tt = tok - b * a.T;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    const __nv_bfloat16* w = nullptr;
    bool copy = false;
    if (h < a.H_q) {
      src = a.q + tok * a.q_ld + (int64_t)h * D;
      dst = a.q_out + ((b * a.H_q + h) * a.T + tt) * D;
      w = a.qw;
    } else if (h < a.H_q + a.H_kv) {
      const int g = h - a.H_q;
      src = a.k + tok * a.k_ld + (int64_t)g * D;
      dst = a.k_act + ((b * a.H_kv + g) * a.S + a.row0 + tt) * D;
      w = a.kw;
    } else {
      const int g = h - a.H_q - a.H_kv;
      copy = true;
      src = a.v ? a.v + tok * a.v_ld + (int64_t)g * D : nullptr;
      dst = a.v_act + ((b * a.H_kv + g) * a.S + a.row0 + tt) * D;
    }
    const bool on = live && src != nullptr;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (on) {
      x0 = *reinterpret_cast<const uint4*>(src + c0 * 8);
      x1 = *reinterpret_cast<const uint4*>(src + c1 * 8);
    }
    float y[16];
    unpack8(x0, y);
    unpack8(x1, y + 8);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!on) continue;
    if (!copy) {
      if (w) {
        const float rms = rsqrtf(ss * (1.0f / D) + a.eps);
        float g[16];
        unpack8(*reinterpret_cast<const uint4*>(w + c0 * 8), g);
        unpack8(*reinterpret_cast<const uint4*>(w + c1 * 8), g + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = y[i] * rms * g[i];
      }
      if (l < rot) {
        if constexpr (INTER) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = turn[t][(i < 4 ? c0 : c1) * 4 + (i & 3)];
            const float p = y[2 * i], r = y[2 * i + 1];
            y[2 * i] = p * cs.x - r * cs.y;
            y[2 * i + 1] = r * cs.x + p * cs.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = turn[t][c0 * 8 + i];
            const float p = y[i], r = y[8 + i];
            y[i] = p * cs.x - r * cs.y;
            y[8 + i] = r * cs.x + p * cs.y;
          }
        }
      }
      x0 = pack8(y);
      x1 = pack8(y + 8);
    }
    *reinterpret_cast<uint4*>(dst + c0 * 8) = x0;
    *reinterpret_cast<uint4*>(dst + c1 * 8) = x1;
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
  const int64_t grid = (a.n_tok + a.tok - 1) / a.tok;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)grid), dim3(kRopeThreads), 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvc
