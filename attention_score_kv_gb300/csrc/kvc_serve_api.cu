// C ABI of the serving operators around the retained cache: norm and rotation
// of queries and keys, the 4-bit cache and attention over it.  Every check
// runs on the host before the launch.
#include <algorithm>
#include <cmath>

#include "kvc_internal.cuh"
#include "kvc_q4.cuh"

using namespace kvc;

namespace kvc {

int check_slots(int H_kv, const int64_t* slot_off) {
  if (H_kv > kMaxHkv) return set_error(KVC_ERR_UNSUPPORTED, "H_kv=%d above %d", H_kv, kMaxHkv);
  if (!slot_off) return set_error(KVC_ERR_INVALID_ARG, "slot_off is NULL");
  int64_t lo = 0;
  for (int h = 0; h <= H_kv; ++h) {
    const int64_t o = slot_off[h];
    if (o < lo || o % q4::kRows != 0)
      return set_error(KVC_ERR_INVALID_ARG, "slot_off[%d]=%lld must be a multiple of %d, at least %lld", h,
                       (long long)o, q4::kRows, (long long)lo);
    if (o - lo > (1 << 30))
      return set_error(KVC_ERR_UNSUPPORTED, "a slot of %lld rows: above 2^30", (long long)(o - lo));
    if (o > (int64_t)INT32_MAX * q4::kRows)
      return set_error(KVC_ERR_UNSUPPORTED, "slot_off[%d]=%lld: too many rows", h, (long long)o);
    lo = o;
  }
  return KVC_OK;
}

}  // namespace kvc

namespace {

int done(cudaError_t e, const char* what) { return e == cudaSuccess ? KVC_OK : cuda_error(e, what); }

int check_heads(int B, int H_kv, int D) {
  if (B < 1 || H_kv < 1) return set_error(KVC_ERR_INVALID_ARG, "B and H_kv must be >= 1 (got B=%d H_kv=%d)", B, H_kv);
  if (D != 64 && D != 128) return set_error(KVC_ERR_UNSUPPORTED, "head dim D=%d: only 64 and 128 are supported", D);
  if ((int64_t)B * H_kv > (1LL << 24)) return set_error(KVC_ERR_UNSUPPORTED, "batch too large");
  return KVC_OK;
}

int check_attend(int B, int T, int H_q, int H_kv, int D) {
  int rc;
  if ((rc = check_heads(B, H_kv, D))) return rc;
  if (H_kv > kMaxHkv) return set_error(KVC_ERR_UNSUPPORTED, "H_kv=%d above %d", H_kv, kMaxHkv);
  if (T < 1 || H_q < 1) return set_error(KVC_ERR_INVALID_ARG, "T and H_q must be >= 1 (got T=%d H_q=%d)", T, H_q);
  if (H_q % H_kv != 0) return set_error(KVC_ERR_INVALID_ARG, "H_q (%d) must be a multiple of H_kv (%d)", H_q, H_kv);
  if ((int64_t)(H_q / H_kv) * T > (1 << 20))
    return set_error(KVC_ERR_UNSUPPORTED, "%lld query rows per KV head: above 2^20", (long long)(H_q / H_kv) * T);
  if ((int64_t)B * H_q * T > INT32_MAX) return set_error(KVC_ERR_UNSUPPORTED, "batch too large");
  return KVC_OK;
}

size_t attend_ws(int B, int T, int H_q, int H_kv, int D) {
  return attend_q4_on_tc(H_q, H_kv, T) ? plan_attend_q4_tc(B, T, H_q, H_kv, D).total
                                       : plan_attend_q4(B, T, H_q, H_kv, D).total;
}

Q4Slots make_slots(int H_kv, const int64_t* slot_off) {
  Q4Slots s{};
  s.H_kv = H_kv;
  std::copy(slot_off, slot_off + H_kv + 1, s.off);
  return s;
}

const __nv_bfloat16* bf(const kvc_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(kvc_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }
cudaStream_t cs(kvc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

int kvc_qk_norm_rope(const kvc_bf16* q, const kvc_bf16* k, const kvc_bf16* v, int B, int T, int H_q, int H_kv, int D,
                     int64_t q_ld, int64_t k_ld, int64_t v_ld, int R, int interleaved, const kvc_bf16* q_weight,
                     const kvc_bf16* k_weight, float eps, const float* inv_freq, const int32_t* pos, int S, int row0,
                     kvc_bf16* q_out, kvc_bf16* k_act, kvc_bf16* v_act, kvc_stream_t stream) {
  int rc;
  if ((rc = check_heads(B, H_kv, D))) return rc;
  if (T < 1 || H_q < 1) return set_error(KVC_ERR_INVALID_ARG, "T and H_q must be >= 1 (got T=%d H_q=%d)", T, H_q);
  if (H_q > 65535 || H_kv > 65535) return set_error(KVC_ERR_UNSUPPORTED, "H_q and H_kv must be <= 65535");
  if ((int64_t)B * T > INT32_MAX) return set_error(KVC_ERR_UNSUPPORTED, "B*T above 2^31 - 1");
  if (R < 0 || R > D || R % 16 != 0)
    return set_error(KVC_ERR_INVALID_ARG, "R=%d rotated dims must be a multiple of 16 in [0, D=%d]", R, D);
  if (interleaved != 0 && interleaved != 1) return set_error(KVC_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (row0 < 0 || (int64_t)row0 + T > S)
    return set_error(KVC_ERR_INVALID_ARG, "rows %d .. %lld do not fit a buffer of S=%d positions", row0,
                     (long long)row0 + T - 1, S);
  if (!(eps >= 0.0f) || std::isinf(eps)) return set_error(KVC_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(k, 16, "k")) || (rc = check_ptr(q_out, 16, "q_out")) ||
      (rc = check_ptr(k_act, 16, "k_act")))
    return rc;
  if ((v == nullptr) != (v_act == nullptr)) return set_error(KVC_ERR_INVALID_ARG, "v and v_act go together");
  if (v && ((rc = check_ptr(v, 16, "v")) || (rc = check_ptr(v_act, 16, "v_act")))) return rc;
  if (q_weight && (rc = check_ptr(q_weight, 16, "q_weight"))) return rc;
  if (k_weight && (rc = check_ptr(k_weight, 16, "k_weight"))) return rc;
  if (R > 0 && ((rc = check_ptr(inv_freq, 4, "inv_freq")) || (rc = check_ptr(pos, 4, "pos")))) return rc;
  if (q_ld < (int64_t)H_q * D || k_ld < (int64_t)H_kv * D || (v && v_ld < (int64_t)H_kv * D) || q_ld % 8 || k_ld % 8 ||
      (v && v_ld % 8))
    return set_error(KVC_ERR_INVALID_ARG,
                     "token strides %lld, %lld, %lld must cover the heads (%lld, %lld) and be multiples of 8",
                     (long long)q_ld, (long long)k_ld, (long long)v_ld, (long long)H_q * D, (long long)H_kv * D);
  return done(launch_qk_norm_rope(bf(q), bf(k), bf(v), B, T, H_q, H_kv, D, q_ld, k_ld, v_ld, R, interleaved != 0,
                                  bf(q_weight), bf(k_weight), eps, inv_freq, pos, S, row0, bf(q_out), bf(k_act),
                                  bf(v_act), cs(stream)),
              "norm and rotation launch");
}

int kvc_q4_layout(int H_kv, int S, const int32_t* K_l, int extra, int64_t* slot_off) {
  if (H_kv < 1 || S < 1) return set_error(KVC_ERR_INVALID_ARG, "H_kv and S must be >= 1");
  if (extra < 0) return set_error(KVC_ERR_INVALID_ARG, "extra must be >= 0");
  if (!K_l || !slot_off) return set_error(KVC_ERR_INVALID_ARG, "K_l and slot_off must be non-NULL");
  slot_off[0] = 0;
  for (int h = 0; h < H_kv; ++h) {
    if (K_l[h] < 0) return set_error(KVC_ERR_INVALID_ARG, "K_l[%d] is negative", h);
    const int64_t rows = (int64_t)std::min(K_l[h], S) + extra;
    slot_off[h + 1] = slot_off[h] + (rows + q4::kRows - 1) / q4::kRows * q4::kRows;
  }
  return KVC_OK;
}

int kvc_gather_q4(const kvc_bf16* k, const kvc_bf16* v, const int32_t* idx, int B, int H_kv, int S, int D,
                  const int32_t* K_l, const int64_t* slot_off, uint8_t* cache, int32_t* pos, kvc_stream_t stream) {
  int rc;
  if ((rc = check_heads(B, H_kv, D))) return rc;
  if (S < 1) return set_error(KVC_ERR_INVALID_ARG, "S must be >= 1");
  if (S > (1 << 30)) return set_error(KVC_ERR_UNSUPPORTED, "S (%d) above 2^30", S);
  if ((rc = check_slots(H_kv, slot_off))) return rc;
  if ((rc = check_ptr(k, 16, "k")) || (rc = check_ptr(v, 16, "v")) || (rc = check_ptr(idx, 4, "idx")) ||
      (rc = check_ptr(cache, 16, "cache")) || (rc = check_ptr(pos, 4, "pos")))
    return rc;
  SelParams sp{};
  sp.S = S;
  sp.H_kv = H_kv;
  if ((rc = make_layout(S, H_kv, K_l, slot_off, 0, &sp))) return rc;
  return done(launch_gather_q4(bf(k), bf(v), idx, B, sp, D, cache, pos, cs(stream)), "4-bit gather launch");
}

int kvc_append_q4(const kvc_bf16* k, const kvc_bf16* v, const int32_t* pos_new, int B, int H_kv, int T, int D,
                  const int64_t* slot_off, const int32_t* rows, uint8_t* cache, int32_t* pos, kvc_stream_t stream) {
  int rc;
  if ((rc = check_heads(B, H_kv, D))) return rc;
  if (T < 1) return set_error(KVC_ERR_INVALID_ARG, "T must be >= 1");
  if (T > (1 << 30)) return set_error(KVC_ERR_UNSUPPORTED, "T=%d above 2^30", T);
  if ((int64_t)B * H_kv * ((int64_t)T / q4::kRows + 2) > INT32_MAX)
    return set_error(KVC_ERR_UNSUPPORTED, "too many rows in one append");
  if ((rc = check_slots(H_kv, slot_off))) return rc;
  if ((rc = check_ptr(k, 16, "k")) || (rc = check_ptr(v, 16, "v")) || (rc = check_ptr(pos_new, 4, "pos_new")) ||
      (rc = check_ptr(rows, 4, "rows")) || (rc = check_ptr(cache, 16, "cache")) || (rc = check_ptr(pos, 4, "pos")))
    return rc;
  return done(launch_append_q4(bf(k), bf(v), pos_new, B, T, D, make_slots(H_kv, slot_off), rows, cache, pos,
                               cs(stream)),
              "4-bit append launch");
}

int kvc_read_q4(const uint8_t* cache, int B, int H_kv, int D, const int64_t* slot_off, const int32_t* first,
                const int32_t* n_rows, const int64_t* out_off, kvc_bf16* k_out, kvc_bf16* v_out, kvc_stream_t stream) {
  int rc;
  if ((rc = check_heads(B, H_kv, D)) || (rc = check_slots(H_kv, slot_off))) return rc;
  if (!n_rows) return set_error(KVC_ERR_INVALID_ARG, "n_rows is NULL");
  for (int h = 0; h < H_kv; ++h)
    if (n_rows[h] < 0 || n_rows[h] > slot_off[h + 1] - slot_off[h])
      return set_error(KVC_ERR_INVALID_ARG, "n_rows[%d]=%d outside [0, %lld], the rows of its slot", h, n_rows[h],
                       (long long)(slot_off[h + 1] - slot_off[h]));
  if ((rc = check_ptr(cache, 16, "cache")) || (first && (rc = check_ptr(first, 4, "first"))) ||
      (rc = check_ptr(k_out, 16, "k_out")) || (rc = check_ptr(v_out, 16, "v_out")))
    return rc;
  SelParams sp{};
  sp.H_kv = H_kv;
  if ((rc = make_layout(INT32_MAX, H_kv, n_rows, out_off, 0, &sp))) return rc;
  return done(launch_read_q4(cache, B, D, make_slots(H_kv, slot_off), first, sp, bf(k_out), bf(v_out), cs(stream)),
              "4-bit read launch");
}

size_t kvc_attention_q4_workspace_size(int B, int T, int H_q, int H_kv, int D) {
  if (check_attend(B, T, H_q, H_kv, D) != KVC_OK) return 0;
  if (num_sms() <= 0) {
    set_error(KVC_ERR_CUDA, "no CUDA device to size the workspace for");
    return 0;
  }
  return std::max<size_t>(attend_ws(B, T, H_q, H_kv, D), 256);   // 0 is the error
}

int kvc_attention_q4(const kvc_bf16* q, const uint8_t* cache, const int32_t* pos, const int32_t* rows, int extra,
                     const int32_t* q_pos, int B, int T, int H_q, int H_kv, int D, const int64_t* slot_off,
                     kvc_bf16* out, float* lse, void* ws, size_t ws_bytes, kvc_stream_t stream) {
  int rc;
  if ((rc = check_attend(B, T, H_q, H_kv, D)) || (rc = check_slots(H_kv, slot_off))) return rc;
  if (extra < 0) return set_error(KVC_ERR_INVALID_ARG, "extra must be >= 0");
  if ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(cache, 16, "cache")) || (rc = check_ptr(pos, 4, "pos")) ||
      (rc = check_ptr(rows, 4, "rows")) || (rc = check_ptr(q_pos, 4, "q_pos")) || (rc = check_ptr(out, 16, "out")) ||
      (lse && (rc = check_ptr(lse, 4, "lse"))))
    return rc;
  if (num_sms() <= 0) return set_error(KVC_ERR_CUDA, "no CUDA device");
  if ((rc = check_ws(ws, ws_bytes, attend_ws(B, T, H_q, H_kv, D)))) return rc;
  auto* launch = attend_q4_on_tc(H_q, H_kv, T) ? launch_attend_q4_tc : launch_attend_q4;
  return done(launch(bf(q), cache, pos, rows, extra, q_pos, B, T, H_q, D, make_slots(H_kv, slot_off), bf(out),
                               lse, ws, cs(stream)),
              "4-bit attention launch");
}

}  // extern "C"
