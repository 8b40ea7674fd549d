// Attention over the 8-bit retained cache (format: kvc_q8.cuh), many query rows
// per KV head: a follow-up prompt, draft tokens.  The kernel, its split and its
// numerics: kvc_flash.cuh.
//
// Codes go from the cache into the products as they are: a tile of 128 rows is
// copied by the tensor copy engine, keys and values alike.  4 D flops a (query,
// row) pair at bf16's rate bound it, as both of the query's and the weight's parts
// are multiplied.
#include "kvc_flash.cuh"

namespace kvc {
namespace {

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(flash::kThreads, 1) kvc_attend_q8_tc_kernel(const __grid_constant__ flash::Args a) {
  flash::attend<D, true, CAP, BIAS>(a);
}

template <int D>
cudaError_t launch_of(flash::Args& a, cudaStream_t st) {
  auto* kern = a.cap2 > 0.f ? (a.slopes ? kvc_attend_q8_tc_kernel<D, true, true> : kvc_attend_q8_tc_kernel<D, true, false>)
                            : (a.slopes ? kvc_attend_q8_tc_kernel<D, false, true>
                                        : kvc_attend_q8_tc_kernel<D, false, false>);
  return flash::launch<D, true>(a, kern, st);
}

}  // namespace

size_t attend_q8_tc_ws(int B, int T, int H_q, int H_kv, int D) {
  return flash::layout((int64_t)B * H_kv, T, H_q / H_kv, D).total;
}

cudaError_t launch_attend_q8_tc(const Q8Attend& x, cudaStream_t st) {
  const int H = x.slots->H_kv, G = x.H_q / H;
  const flash::Layout l = flash::layout((int64_t)x.B * H, x.T, G, x.D);
  flash::Args a{};
  a.q = x.q, a.q_pos = x.q_pos, a.pos = x.c.pos, a.rows = x.rows, a.scale = reinterpret_cast<const float2*>(x.c.scale);
  a.s = *x.slots;
  a.slopes = x.slopes, a.out = x.out, a.lse = x.lse;
  a.B1 = x.B * H, a.H1 = 1, a.T = x.T, a.H_q = x.H_q, a.H_kv = H, a.G = G, a.extra = x.extra;
  a.scale2 = (float)(1.4426950408889634 / std::sqrt((double)x.D));
  a.cap2 = x.cap * flash::kLog2e;
  a.inv_cap2 = x.cap > 0.f ? 1.f / a.cap2 : 0.f;
  flash::place(a, l, x.D, x.ws);
  const uint64_t blocks = (uint64_t)x.B * (uint64_t)(x.slots->off[H] / q8::kRows);
  // Slots without any row: there is no block to map, and a unit's one tile, of which no row is
  // looked at, comes from the queries (more than eight rows of 2 D bytes: a block).
  const void *k8 = blocks ? x.c.k8 : (const void*)x.q, *v8 = blocks ? x.c.v8 : (const void*)x.q;
  if (!flash::map_blocks(&a.kmap, k8, x.D, std::max<uint64_t>(blocks, 1)) ||
      !flash::map_blocks(&a.vmap, v8, x.D, std::max<uint64_t>(blocks, 1)))
    return cudaErrorInvalidValue;
  return x.D == 128 ? launch_of<128>(a, st) : launch_of<64>(a, st);
}

}  // namespace kvc
