// Attention of a prompt chunk over the active layer's bf16 buffers: what runs
// between kvc_qk_norm_rope and the scorer in the layer-major schedule.  The
// kernel, its split and its numerics: kvc_flash.cuh.
//
// 4 D flops a (query, key) pair bound it where a tile of keys meets many query
// rows; a single token reads 4 D bytes a key for 4 G D flops.  Products of bf16
// are exact in fp32; the weights are rounded to bf16, 2^-8 of each, as the
// products take both operands in one type.
#include "kvc_flash.cuh"

namespace kvc {
namespace {

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(flash::kThreads, 1) kvc_attend_chunk_kernel(const __grid_constant__ flash::Args a) {
  flash::attend<D, false, CAP, BIAS>(a);
}

template <int D>
cudaError_t launch_of(flash::Args& a, cudaStream_t st) {
  auto* kern = a.cap2 > 0.f ? (a.slopes ? kvc_attend_chunk_kernel<D, true, true> : kvc_attend_chunk_kernel<D, true, false>)
                            : (a.slopes ? kvc_attend_chunk_kernel<D, false, true>
                                        : kvc_attend_chunk_kernel<D, false, false>);
  return flash::launch<D, false>(a, kern, st);
}

}  // namespace

size_t attend_chunk_ws(int B, int T, int H_q, int H_kv, int D) { return flash::layout(B, T, H_q / H_kv, D).total; }

cudaError_t launch_attend_chunk(const ChunkAttend& x, cudaStream_t st) {
  const int G = x.H_q / x.H_kv;
  const flash::Layout l = flash::layout(x.B, x.T, G, x.D);
  flash::Args a{};
  a.q_pos = x.q_pos, a.first = x.first, a.last = x.last, a.slopes = x.slopes, a.out = x.out, a.lse = x.lse;
  a.B1 = x.B, a.H1 = x.H_kv, a.T = x.T, a.H_q = x.H_q, a.H_kv = x.H_kv, a.G = G, a.S = x.S;
  a.scale2 = (float)(1.4426950408889634 / std::sqrt((double)x.D));
  a.cap2 = x.cap * flash::kLog2e;
  a.inv_cap2 = x.cap > 0.f ? 1.f / a.cap2 : 0.f;
  flash::place(a, l, x.D, x.ws);
  if (!flash::map_queries(&a.qmap, x.q, x.D, x.T, (uint64_t)x.B * x.H_q, l.nt, G) ||
      !scan::make_map(&a.kmap, x.k, x.D, x.S, (uint64_t)x.B * x.H_kv, flash::kKeys) ||
      !scan::make_map(&a.vmap, x.v, x.D, x.S, (uint64_t)x.B * x.H_kv, flash::kKeys))
    return cudaErrorInvalidValue;
  return x.D == 128 ? launch_of<128>(a, st) : launch_of<64>(a, st);
}

}  // namespace kvc
