// C ABI of the quantized KV cache: host-side argument validation, then launch.
// Every check runs before any HIP call, as in abi.cpp.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/rotw4a4.h"
#include "launch.hpp"

namespace {

constexpr int64_t kMax30 = int64_t(1) << 30;

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline hipStream_t strm(void* s) { return static_cast<hipStream_t>(s); }
inline rw4_status hip_status(hipError_t e) { return e == hipSuccess ? RW4_OK : RW4_ERR_HIP; }

// log2 of a page size that the kernels take, or -1
inline int lg_page(int64_t page) {
  for (int i = 4; i <= 8; ++i)
    if (page == (int64_t(1) << i)) return i;
  return -1;
}
inline bool dh_ok(int64_t dh) { return dh == 64 || dh == 128 || dh == 256; }

// the cache's sizes; its pointers are checked by check_cache
rw4_status check_geometry(int64_t n_pages, int64_t H, int64_t page, int64_t dh, unsigned flags,
                          rw4_dtype dt) {
  if (n_pages < 1 || H < 1 || (dt != RW4_BF16 && dt != RW4_F32)) return RW4_ERR_INVALID_ARG;
  if (flags & ~static_cast<unsigned>(RW4_FWHT)) return RW4_ERR_INVALID_ARG;
  if (lg_page(page) < 0 || !dh_ok(dh) || H > 65535 || n_pages >= kMax30) return RW4_ERR_UNSUPPORTED;
  // blocks of 16 tokens and one head are counted in 31 bits
  if (n_pages * H * (page / 16) >= 2 * kMax30) return RW4_ERR_UNSUPPORTED;
  return RW4_OK;
}

rw4_status check_cache(const void* k_codes, const void* k_scale, const void* v_codes,
                       const void* v_scale) {
  if (!k_codes || !k_scale || !v_codes || !v_scale) return RW4_ERR_INVALID_ARG;
  if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return RW4_ERR_MISALIGNED;
  return RW4_OK;
}

// rows of `width` values of dt, stride ld: 16-byte aligned rows
rw4_status check_rows(const void* x, int64_t ld, int64_t width, rw4_dtype dt) {
  if (!x) return RW4_ERR_INVALID_ARG;
  if (ld < width || ld % (dt == RW4_F32 ? 4 : 8) != 0) return RW4_ERR_INVALID_ARG;
  return aligned(x, 16) ? RW4_OK : RW4_ERR_MISALIGNED;
}

// numbers that kv_attention's kernels count in 31 bits, a grid of fewer than 2^32
// threads, and at most 2^14 parts of 4096 keys
bool bounds_ok(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t max_new, int64_t max_kv) {
  return T * Hq < kMax30 && T * Hq / 128 + B * H < (int64_t(1) << 23) && max_new < kMax30 &&
         max_kv < kMax30 / 16;
}

rw4::KvCacheArgs cache_args(const int8_t* k_codes, const float* k_scale, const int8_t* v_codes,
                            const float* v_scale, int64_t n_pages, int64_t H, int64_t page,
                            int64_t dh) {
  return rw4::KvCacheArgs{const_cast<int8_t*>(k_codes), const_cast<float*>(k_scale),
                          const_cast<int8_t*>(v_codes), const_cast<float*>(v_scale), n_pages,
                          static_cast<int>(H), static_cast<int>(dh), lg_page(page)};
}

// both entries of the plan; without ctx_next: the one that does not write it
rw4_status plan(const int32_t* ctx_len, const int32_t* new_len, int64_t B, int32_t* page_table,
                int64_t max_pages, int64_t page, int32_t* free_pages, int64_t capacity,
                const int32_t* n_free, int32_t* n_free_out, int32_t* cu_new, int32_t* kv_len,
                int64_t* slot, int32_t* pos, int32_t* status, int64_t T, int32_t* ctx_next,
                void* stream) {
  if (B < 1 || T < 0 || max_pages < 1 || capacity < 1) return RW4_ERR_INVALID_ARG;
  const int lg = lg_page(page);
  if (lg < 0 || B > rw4::kKvMaxBatch || max_pages >= (kMax30 * 2 >> lg) || capacity >= kMax30 ||
      T >= kMax30 || B * max_pages >= kMax30)
    return RW4_ERR_UNSUPPORTED;
  if (!ctx_len || !new_len || !page_table || !free_pages || !n_free || !n_free_out || !cu_new ||
      !kv_len || !status || (T > 0 && (!slot || !pos)))
    return RW4_ERR_INVALID_ARG;
  if (n_free_out == n_free || kv_len == ctx_len || kv_len == new_len || cu_new == new_len ||
      cu_new == ctx_len || status == ctx_len || status == new_len)
    return RW4_ERR_INVALID_ARG;
  if (!aligned(ctx_len, 4) || !aligned(new_len, 4) || !aligned(page_table, 4) ||
      !aligned(free_pages, 4) || !aligned(n_free, 4) || !aligned(n_free_out, 4) ||
      !aligned(cu_new, 4) || !aligned(kv_len, 4) || !aligned(status, 4) ||
      (T > 0 && (!aligned(slot, 8) || !aligned(pos, 4))))
    return RW4_ERR_MISALIGNED;
  const rw4::KvPlanArgs a{ctx_len, new_len, B, page_table, max_pages, lg, free_pages, capacity,
                          n_free, n_free_out, cu_new, kv_len, slot, pos, status, T, ctx_next};
  return hip_status(rw4::launch_kv_plan(a, strm(stream)));
}

}  // namespace

extern "C" {

rw4_status kv_plan(const int32_t* ctx_len, const int32_t* new_len, int64_t B, int32_t* page_table,
                   int64_t max_pages, int64_t page, int32_t* free_pages, int64_t capacity,
                   const int32_t* n_free, int32_t* n_free_out, int32_t* cu_new, int32_t* kv_len,
                   int64_t* slot, int32_t* pos, int32_t* status, int64_t T, void* stream) {
  return plan(ctx_len, new_len, B, page_table, max_pages, page, free_pages, capacity, n_free,
              n_free_out, cu_new, kv_len, slot, pos, status, T, nullptr, stream);
}

rw4_status kv_plan_next(const int32_t* ctx_len, const int32_t* new_len, int64_t B,
                        int32_t* page_table, int64_t max_pages, int64_t page, int32_t* free_pages,
                        int64_t capacity, const int32_t* n_free, int32_t* n_free_out,
                        int32_t* cu_new, int32_t* kv_len, int64_t* slot, int32_t* pos,
                        int32_t* status, int64_t T, int32_t* ctx_next, void* stream) {
  if (!ctx_next || ctx_next == ctx_len || ctx_next == new_len) return RW4_ERR_INVALID_ARG;
  if (!aligned(ctx_next, 4)) return RW4_ERR_MISALIGNED;
  return plan(ctx_len, new_len, B, page_table, max_pages, page, free_pages, capacity, n_free,
              n_free_out, cu_new, kv_len, slot, pos, status, T, ctx_next, stream);
}

rw4_status kv_append(const void* k, const void* v, rw4_dtype x_dt, int64_t ldk, int64_t ldv,
                     int64_t T, int64_t B, unsigned flags, const int32_t* cu_new,
                     const int64_t* slot, int8_t* k_codes, float* k_scale, int8_t* v_codes,
                     float* v_scale, int64_t n_pages, int64_t H, int64_t page, int64_t dh,
                     void* stream) {
  if (T < 0 || B < 0) return RW4_ERR_INVALID_ARG;
  rw4_status st = check_geometry(n_pages, H, page, dh, flags, x_dt);
  if (st != RW4_OK) return st;
  if (T >= kMax30 || B >= kMax30) return RW4_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return RW4_OK;
  // workgroups in one dimension of the grid, 256 threads each: at most two for a
  // request and one for every page or 64 rows, for each head of keys and of values
  const int lg = lg_page(page) < 6 ? lg_page(page) : 6;
  if (((T >> lg) + 2 * B + 1) * 2 * H >= kMax30 / 64) return RW4_ERR_UNSUPPORTED;
  if (!cu_new || !slot) return RW4_ERR_INVALID_ARG;
  if ((st = check_rows(k, ldk, H * dh, x_dt)) != RW4_OK) return st;
  if ((st = check_rows(v, ldv, H * dh, x_dt)) != RW4_OK) return st;
  if ((st = check_cache(k_codes, k_scale, v_codes, v_scale)) != RW4_OK) return st;
  if (!aligned(cu_new, 4) || !aligned(slot, 8)) return RW4_ERR_MISALIGNED;
  const rw4::KvAppendArgs a{k, v, x_dt == RW4_F32, ldk, ldv, T, B, (flags & RW4_FWHT) != 0,
                            cu_new, slot,
                            cache_args(k_codes, k_scale, v_codes, v_scale, n_pages, H, page, dh)};
  return hip_status(rw4::launch_kv_append(a, strm(stream)));
}

size_t kv_attention_workspace_size(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t dh,
                                   int64_t max_new, int64_t max_kv) {
  if (T < 1 || T >= kMax30 || B < 1 || B > 65535 || H < 1 || Hq < 1 || Hq > 65535 || Hq % H != 0 ||
      !dh_ok(dh) || max_new < 1 || max_kv < 1 || !bounds_ok(T, B, Hq, H, max_new, max_kv))
    return 0;
  return rw4::kv_attention_workspace(T, B, Hq, H, dh, max_new, max_kv);
}

rw4_status kv_attention(const void* q, rw4_dtype q_dt, int64_t ldq, void* out, int64_t ldo,
                        int64_t T, int64_t B, int64_t Hq, float scale, unsigned flags,
                        const int32_t* cu_new, const int32_t* kv_len, const int32_t* page_table,
                        int64_t max_pages, const int8_t* k_codes, const float* k_scale,
                        const int8_t* v_codes, const float* v_scale, int64_t n_pages, int64_t H,
                        int64_t page, int64_t dh, int64_t max_new, int64_t max_kv,
                        void* workspace, size_t ws_bytes, void* stream) {
  if (T < 0 || B < 0 || Hq < 1 || max_pages < 1 || max_new < 0 || max_kv < 0 ||
      !std::isfinite(scale))
    return RW4_ERR_INVALID_ARG;
  rw4_status st = check_geometry(n_pages, H, page, dh, flags, q_dt);
  if (st != RW4_OK) return st;
  if (Hq % H != 0) return RW4_ERR_INVALID_ARG;
  if (Hq > 65535 || B > 65535 || T >= kMax30 || max_pages >= (kMax30 * 2 >> lg_page(page)))
    return RW4_ERR_UNSUPPORTED;
  if (!bounds_ok(T, B, Hq, H, max_new, max_kv)) return RW4_ERR_UNSUPPORTED;
  if (T == 0 || B == 0 || max_new == 0) return RW4_OK;
  if (!cu_new || !kv_len || !page_table) return RW4_ERR_INVALID_ARG;
  if ((st = check_rows(q, ldq, Hq * dh, q_dt)) != RW4_OK) return st;
  if ((st = check_rows(out, ldo, Hq * dh, RW4_BF16)) != RW4_OK) return st;
  if (out == q) return RW4_ERR_INVALID_ARG;
  if ((st = check_cache(k_codes, k_scale, v_codes, v_scale)) != RW4_OK) return st;
  if (!aligned(cu_new, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4))
    return RW4_ERR_MISALIGNED;
  const size_t need = kv_attention_workspace_size(T, B, Hq, H, dh, max_new, max_kv);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || ws_bytes < need))
    return RW4_ERR_WORKSPACE;
  const rw4::KvAttnArgs a{q, q_dt == RW4_F32, ldq, static_cast<uint16_t*>(out), ldo, T, B,
                          static_cast<int>(Hq), scale, (flags & RW4_FWHT) != 0, cu_new, kv_len,
                          page_table, max_pages,
                          cache_args(k_codes, k_scale, v_codes, v_scale, n_pages, H, page, dh),
                          max_new, max_kv};
  return hip_status(rw4::launch_kv_attention(a, workspace, strm(stream)));
}

}  // extern "C"
