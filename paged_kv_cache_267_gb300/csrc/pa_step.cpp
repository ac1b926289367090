// C-ABI entry points of a serving step around the attention: growing and
// releasing block tables on the GPU (pool_ops.cu), and the per-head norm with
// rotation and cache write (norm_cache.cu). Argument checks come before any
// CUDA call, as in pa_api.cpp.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>
#include <utility>

#include "pa.h"
#include "pa_host.h"
#include "pa_internal.h"
#include "step_ops.h"

namespace {

using namespace pa;

constexpr double k2p31 = 2147483648.0;

bool misaligned(const pa_tensor* t, uintptr_t n) {
  return numel(t) > 0 && reinterpret_cast<uintptr_t>(t->data) % n;
}

// A contiguous int32 vector of n elements (n < 0: any length).
pa_status check_vec(const pa_tensor* t, const char* name, int32_t dtype, int64_t n) {
  pa_status s = check_tensor(t, name, 1);
  if (s) return s;
  if (t->dtype != dtype)
    return fail(PA_ERR_INVALID_ARG, "%s must be %s", name, dtype == PA_I64 ? "int64" : "int32");
  if (n >= 0 && t->shape[0] != n)
    return fail(PA_ERR_INVALID_ARG, "%s: expected %lld elements, got %lld", name, (long long)n,
                (long long)t->shape[0]);
  if (!is_contiguous(t)) return fail(PA_ERR_LAYOUT, "%s must be contiguous", name);
  if (misaligned(t, static_cast<uintptr_t>(elem_size(dtype))))
    return fail(PA_ERR_LAYOUT, "%s is not aligned to its elements", name);
  return PA_OK;
}

// What pa_pool_extend and pa_pool_release have in common.
pa_status check_pool(const pa_tensor* tables, const pa_tensor* lens, const pa_tensor* free_list,
                     const pa_tensor* state, const pa_tensor* lens_out, const pa_tensor* state_out,
                     int32_t block_size) {
  pa_status s;
  if ((s = check_tensor(tables, "block_tables", 2))) return s;
  if (tables->dtype != PA_I32) return fail(PA_ERR_INVALID_ARG, "block_tables must be int32");
  if (!is_contiguous(tables)) return fail(PA_ERR_LAYOUT, "block_tables must be contiguous");
  if (misaligned(tables, 4)) return fail(PA_ERR_LAYOUT, "block_tables is not aligned to its elements");
  const int64_t B = tables->shape[0], MB = tables->shape[1];
  if ((s = check_vec(lens, "seq_lens", PA_I32, B)) ||
      (s = check_vec(free_list, "free_list", PA_I32, -1)) ||
      (s = check_vec(state, "pool_state", PA_I32, 2)) ||
      (s = check_vec(lens_out, "seq_lens_out", PA_I32, B)) ||
      (s = check_vec(state_out, "pool_state_out", PA_I32, 2)))
    return s;
  if (block_size <= 0 || block_size % 16 || block_size > 1024)
    return fail(PA_ERR_UNSUPPORTED, "block_size must be a multiple of 16 in [16, 1024]");
  if (B > kMaxBatch)
    return fail(PA_ERR_UNSUPPORTED, "batch %lld > %lld", (long long)B, (long long)kMaxBatch);
  if (B > 0 && MB == 0) return fail(PA_ERR_INVALID_ARG, "block_tables has no columns");
  // lengths, block counts and ids are 32-bit; the room above is for round-ups
  if (dprod({double(MB), double(block_size)}) >= k2p31 - 2048 ||
      dprod({double(B), double(MB)}) >= k2p31 || double(free_list->shape[0]) >= k2p31 - 2048)
    return fail(PA_ERR_UNSUPPORTED, "pool or tables exceed 32-bit indexing");
  return PA_OK;
}

// No tensor that is written may overlap another one; lens_out and state_out
// may be lens and state themselves.
pa_status check_apart(std::initializer_list<const pa_tensor*> written,
                      std::initializer_list<const pa_tensor*> read, const pa_tensor* lens,
                      const pa_tensor* lens_out, const pa_tensor* state,
                      const pa_tensor* state_out) {
  for (const pa_tensor* w : written) {
    if (!w) continue;
    for (const pa_tensor* o : read) {
      if (!o) continue;
      const bool same = (w == lens_out && o == lens) || (w == state_out && o == state);
      if (same && w->data == o->data) continue;
      if (overlaps(w, o)) return fail(PA_ERR_INVALID_ARG, "an output overlaps another tensor");
    }
    for (const pa_tensor* o : written) {
      if (o == w) break;  // each pair once
      if (o && overlaps(w, o)) return fail(PA_ERR_INVALID_ARG, "two outputs overlap");
    }
  }
  return PA_OK;
}

template <typename T>
T* ptr(const pa_tensor* t) {
  return static_cast<T*>(t->data);
}

}  // namespace

extern "C" {

pa_status pa_pool_extend(const pa_tensor* block_tables, const pa_tensor* seq_lens,
                         const pa_tensor* new_tokens, const pa_tensor* free_list,
                         const pa_tensor* pool_state, const pa_tensor* seq_lens_out,
                         const pa_tensor* pool_state_out, const pa_tensor* query_start,
                         const pa_tensor* slot_mapping, const pa_tensor* positions,
                         int32_t block_size, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    pa_status s = check_pool(block_tables, seq_lens, free_list, pool_state, seq_lens_out,
                             pool_state_out, block_size);
    if (s) return s;
    const int64_t B = block_tables->shape[0];
    if ((s = check_vec(new_tokens, "new_tokens", PA_I32, B)) ||
        (s = check_vec(query_start, "query_start", PA_I32, B + 1)) ||
        (s = check_vec(slot_mapping, "slot_mapping", PA_I64, -1)) ||
        (s = check_vec(positions, "positions", PA_I32, slot_mapping->shape[0])))
      return s;
    const int64_t T = slot_mapping->shape[0];
    if (T > (int64_t(1) << 30)) return fail(PA_ERR_UNSUPPORTED, "slot_mapping has more than 2^30 rows");
    if ((s = check_apart({block_tables, seq_lens_out, pool_state_out, query_start, slot_mapping, positions},
                         {seq_lens, new_tokens, free_list, pool_state}, seq_lens, seq_lens_out,
                         pool_state, pool_state_out)))
      return s;
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{block_tables, "block_tables"},
                            {seq_lens, "seq_lens"}, {new_tokens, "new_tokens"},
                            {free_list, "free_list"}, {pool_state, "pool_state"},
                            {seq_lens_out, "seq_lens_out"}, {pool_state_out, "pool_state_out"},
                            {query_start, "query_start"}, {slot_mapping, "slot_mapping"},
                            {positions, "positions"}})
      if ((s = check_accessible(t, name))) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev))) return s;
    PoolExtendArgs a;
    a.tables = ptr<int32_t>(block_tables);
    a.lens = ptr<int32_t>(seq_lens);
    a.fresh = ptr<int32_t>(new_tokens);
    a.free_list = ptr<int32_t>(free_list);
    a.state = ptr<int32_t>(pool_state);
    a.lens_out = ptr<int32_t>(seq_lens_out);
    a.state_out = ptr<int32_t>(pool_state_out);
    a.query_start = ptr<int32_t>(query_start);
    a.slots = ptr<int64_t>(slot_mapping);
    a.positions = ptr<int32_t>(positions);
    a.err = dev.err_word;
    a.B = static_cast<int>(B);
    a.MB = static_cast<int>(block_tables->shape[1]);
    a.bs = block_size;
    a.div = fast_div(static_cast<uint32_t>(block_size));
    a.NF = static_cast<int>(free_list->shape[0]);
    a.T = static_cast<int>(T);
    a.in_place = a.lens_out == a.lens || a.state_out == a.state;
    a.wide = !misaligned(slot_mapping, 16) && !misaligned(positions, 16);
    const cudaError_t e = pool_extend_launch(a, dev.num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "pool_extend launch");
    count_launches(1);
    return ok();
  });
}

pa_status pa_pool_release(const pa_tensor* block_tables, const pa_tensor* seq_lens,
                          const pa_tensor* released, const pa_tensor* shared_tokens,
                          const pa_tensor* free_list, const pa_tensor* pool_state,
                          const pa_tensor* seq_lens_out, const pa_tensor* pool_state_out,
                          int32_t block_size, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    pa_status s = check_pool(block_tables, seq_lens, free_list, pool_state, seq_lens_out,
                             pool_state_out, block_size);
    if (s) return s;
    const int64_t B = block_tables->shape[0];
    if ((s = check_vec(released, "released", PA_I32, B)) ||
        (shared_tokens && (s = check_vec(shared_tokens, "shared_tokens", PA_I32, B))))
      return s;
    if ((s = check_apart({free_list, seq_lens_out, pool_state_out},
                         {block_tables, seq_lens, released, shared_tokens, pool_state}, seq_lens,
                         seq_lens_out, pool_state, pool_state_out)))
      return s;
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{block_tables, "block_tables"},
                            {seq_lens, "seq_lens"}, {released, "released"},
                            {shared_tokens, "shared_tokens"}, {free_list, "free_list"},
                            {pool_state, "pool_state"}, {seq_lens_out, "seq_lens_out"},
                            {pool_state_out, "pool_state_out"}})
      if ((s = check_accessible(t, name))) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev))) return s;
    PoolReleaseArgs a;
    a.tables = ptr<int32_t>(block_tables);
    a.lens = ptr<int32_t>(seq_lens);
    a.released = ptr<int32_t>(released);
    a.shared = shared_tokens ? ptr<int32_t>(shared_tokens) : nullptr;
    a.free_list = ptr<int32_t>(free_list);
    a.state = ptr<int32_t>(pool_state);
    a.lens_out = ptr<int32_t>(seq_lens_out);
    a.state_out = ptr<int32_t>(pool_state_out);
    a.err = dev.err_word;
    a.B = static_cast<int>(B);
    a.MB = static_cast<int>(block_tables->shape[1]);
    a.bs = block_size;
    a.div = fast_div(static_cast<uint32_t>(block_size));
    a.NF = static_cast<int>(free_list->shape[0]);
    a.in_place = a.lens_out == a.lens || a.state_out == a.state;
    const cudaError_t e = pool_release_launch(a, dev.num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "pool_release launch");
    count_launches(1);
    return ok();
  });
}

pa_status pa_norm_rope_and_cache(const pa_tensor* q_out, const pa_tensor* q, const pa_tensor* k,
                                 const pa_tensor* v, const pa_tensor* key_cache,
                                 const pa_tensor* value_cache, const pa_tensor* slot_mapping,
                                 const pa_tensor* positions, const pa_tensor* cos_sin,
                                 const pa_tensor* q_weight, const pa_tensor* k_weight, float eps,
                                 int32_t interleaved, int32_t kv_dtype, float k_scale,
                                 float v_scale, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    pa_status s;
    if ((s = check_tensor(q_out, "q_out", 3)) || (s = check_tensor(q, "q", 3)) ||
        (s = check_tensor(k, "k", 3)) || (s = check_tensor(v, "v", 3)) ||
        (s = check_tensor(key_cache, "key_cache", 4)) ||
        (s = check_tensor(value_cache, "value_cache", 4)) ||
        (s = check_tensor(cos_sin, "cos_sin", 2)))
      return s;
    if (q->dtype != PA_F16 && q->dtype != PA_BF16)
      return fail(PA_ERR_UNSUPPORTED, "q must be f16 or bf16");
    if (k->dtype != q->dtype || v->dtype != q->dtype || q_out->dtype != q->dtype)
      return fail(PA_ERR_INVALID_ARG, "q, k, v and q_out dtypes differ");
    const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hkv = k->shape[1];
    for (int i = 0; i < 3; ++i) {
      if (q_out->shape[i] != q->shape[i]) return fail(PA_ERR_INVALID_ARG, "q_out shape != q shape");
      if (k->shape[i] != v->shape[i]) return fail(PA_ERR_INVALID_ARG, "k and v shapes differ");
    }
    if (k->shape[0] != T || k->shape[2] != D)
      return fail(PA_ERR_INVALID_ARG, "q [T, Hq, D] does not match k [T, Hkv, D]");
    if (kv_dtype != PA_KV_AUTO && kv_dtype != PA_KV_FP8_E4M3)
      return fail(PA_ERR_INVALID_ARG, "bad kv_dtype %d", kv_dtype);
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    const int32_t cdt = fp8 ? PA_FP8_E4M3 : q->dtype;
    if (key_cache->dtype != cdt || value_cache->dtype != cdt)
      return fail(PA_ERR_INVALID_ARG, "cache dtype does not match kv_dtype");
    for (int i = 0; i < 4; ++i)
      if (key_cache->shape[i] != value_cache->shape[i])
        return fail(PA_ERR_INVALID_ARG, "key and value cache shapes differ");
    if (key_cache->shape[1] != Hkv || key_cache->shape[3] != D)
      return fail(PA_ERR_INVALID_ARG, "cache [NB, Hkv, bs, D] does not match k [T, Hkv, D]");
    if (D <= 0 || D % 16 || D > 256)
      return fail(PA_ERR_UNSUPPORTED, "head_dim %lld: a multiple of 16, at most 256", (long long)D);
    if (Hq > 65535 || Hkv > 65535 || T > (int64_t(1) << 30))
      return fail(PA_ERR_UNSUPPORTED, "too many tokens/heads");
    const int64_t R = cos_sin->shape[1], NP = cos_sin->shape[0];
    if (cos_sin->dtype != PA_F32) return fail(PA_ERR_INVALID_ARG, "cos_sin must be f32");
    if (R > D || R % 16) return fail(PA_ERR_UNSUPPORTED, "cos_sin: R = %lld must be a multiple of 16, at most head_dim", (long long)R);
    if (NP > (int64_t(1) << 30)) return fail(PA_ERR_UNSUPPORTED, "cos_sin has more than 2^30 rows");
    if ((s = check_vec(slot_mapping, "slot_mapping", PA_I64, T)) ||
        (s = check_vec(positions, "positions", PA_I32, T)))
      return s;
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{q_weight, "q_weight"},
                            {k_weight, "k_weight"}}) {
      if (!t) continue;
      if ((s = check_tensor(t, name, 1))) return s;
      if (t->dtype != q->dtype || t->shape[0] != D)
        return fail(PA_ERR_INVALID_ARG, "%s must be [head_dim] of q's dtype", name);
      if (!is_contiguous(t) || misaligned(t, 16))
        return fail(PA_ERR_LAYOUT, "%s must be contiguous and 16-byte aligned", name);
    }
    if (!(std::isfinite(eps) && eps >= 0)) return fail(PA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0 && v_scale > 0))
      return fail(PA_ERR_INVALID_ARG, "fp8 scales must be finite and positive");
    if (!is_contiguous(key_cache) || !is_contiguous(value_cache) || !is_contiguous(cos_sin))
      return fail(PA_ERR_LAYOUT, "caches and cos_sin must be contiguous");
    if (misaligned(key_cache, 16) || misaligned(value_cache, 16) || misaligned(cos_sin, 16))
      return fail(PA_ERR_LAYOUT, "caches and cos_sin must be 16-byte aligned");
    if (T == 0) return ok();
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{q, "q"}, {k, "k"}, {v, "v"},
                            {q_out, "q_out"}}) {
      if (numel(t) == 0) continue;
      if (t->strides[2] != 1 || (t->shape[1] > 1 && t->strides[1] != D))
        return fail(PA_ERR_LAYOUT, "%s rows [heads, D] must be contiguous", name);
      if (misaligned(t, 16) || (T > 1 && t->strides[0] % 8))
        return fail(PA_ERR_LAYOUT, "%s rows must be 16-byte aligned", name);
    }
    if (T > 1 && Hq > 0 && q_out->strides[0] < Hq * D)
      return fail(PA_ERR_LAYOUT, "q_out rows overlap");
    if (R > 0 && NP == 0) return fail(PA_ERR_INVALID_ARG, "cos_sin has no rows");
    if (numel(key_cache) > 0 && overlaps(key_cache, value_cache))
      return fail(PA_ERR_INVALID_ARG, "key and value caches overlap");
    const bool in_place = q_out->data == q->data && q_out->strides[0] == q->strides[0];
    // Rows of x between rows of q_out: of one row stride, and in every row
    // behind q_out's heads and before its next row.
    auto between_rows = [&](const pa_tensor* x) {
      const int64_t row = q_out->strides[0] * 2;  // bytes
      if (T < 2 || x->strides[0] != q_out->strides[0]) return false;
      int64_t at = (static_cast<const char*>(x->data) - static_cast<const char*>(q_out->data)) % row;
      if (at < 0) at += row;
      return at >= Hq * D * 2 && at + Hkv * D * 2 <= row;
    };
    for (const pa_tensor* x : {q, k, v, slot_mapping, positions, cos_sin, q_weight, k_weight}) {
      if (!x) continue;
      if (overlaps(key_cache, x) || overlaps(value_cache, x))
        return fail(PA_ERR_INVALID_ARG, "a cache overlaps an input");
      // q_out in q's place: packed rows of k and v lie between its rows
      if (!(in_place && (x == q || ((x == k || x == v) && between_rows(x)))) && overlaps(q_out, x))
        return fail(PA_ERR_INVALID_ARG, "q_out overlaps an input");
    }
    if (overlaps(q_out, key_cache) || overlaps(q_out, value_cache))
      return fail(PA_ERR_INVALID_ARG, "q_out overlaps a cache");
    if (Hq + Hkv == 0) return ok();
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{q_out, "q_out"}, {q, "q"},
                            {k, "k"}, {v, "v"}, {key_cache, "key_cache"},
                            {value_cache, "value_cache"}, {slot_mapping, "slot_mapping"},
                            {positions, "positions"}, {cos_sin, "cos_sin"},
                            {q_weight, "q_weight"}, {k_weight, "k_weight"}})
      if ((s = check_accessible(t, name))) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev))) return s;
    NormCacheArgs a;
    a.q = q->data;
    a.k = k->data;
    a.v = v->data;
    a.q_out = q_out->data;
    a.kc = key_cache->data;
    a.vc = value_cache->data;
    a.slots = ptr<int64_t>(slot_mapping);
    a.positions = ptr<int32_t>(positions);
    a.cos_sin = ptr<float>(cos_sin);
    a.q_weight = q_weight ? q_weight->data : nullptr;
    a.k_weight = k_weight ? k_weight->data : nullptr;
    a.err = dev.err_word;
    a.q_stride = q->strides[0];
    a.k_stride = k->strides[0];
    a.v_stride = v->strides[0];
    a.out_stride = q_out->strides[0];
    a.NB = key_cache->shape[0];
    a.T = static_cast<int>(T);
    a.Hq = static_cast<int>(Hq);
    a.Hkv = static_cast<int>(Hkv);
    a.D = static_cast<int>(D);
    a.R = static_cast<int>(R);
    a.NP = static_cast<int>(NP);
    a.bs = static_cast<int>(key_cache->shape[2]);
    a.eps = eps;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.interleaved = interleaved != 0;
    const cudaError_t e =
        norm_cache_launch(q->dtype, fp8, a, dev.num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "norm_rope_and_cache launch");
    count_launches(1);
    return ok();
  });
}

}  // extern "C"
