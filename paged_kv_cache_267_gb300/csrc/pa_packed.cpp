// C-ABI entry points of the ragged steps: attention of packed prompts and of drafted
// trees over the paged cache (packed_plan.cu, packed_tc.cu, packed_merge.cu), and the
// moves of cached rows (cache_moves.cu). Argument checks come before any CUDA call, as
// in pa_api.cpp.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "pa.h"
#include "pa_host.h"
#include "pa_internal.h"
#include "packed_ops.h"

namespace {

using namespace pa;

constexpr double k2p31 = 2147483648.0;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxRowStride = int64_t(1) << 23;
// Costs of a step in places (packed_plan.cuh): least share of a CTA in split mode, the
// partial results of a split and their join.
constexpr int kMinPlaces = 8;
constexpr int kSplitPlaces = 16;
constexpr int kSmallPairs = 3;  // a CTA, of a step that is planned without a kernel
// Tiles of a pair of such a step, at most, where pairs are not cut, which saves the join: one
// token each of 4 requests on 800 takes 11.7 us instead of 13.0, but on 1,800 18.3 instead of
// 14.1.
constexpr int kWholeTiles = 10;
// What a cut costs a CTA of such a step, and what a tile of one or of two row tiles takes
// there, in places of 0.38 us: whole pairs take whole rounds, cut ones an even share and this.
// (152 CTAs, 8 KV heads, 48 tokens on 1,000: whole against cut, 20 requests, in two rounds,
// 47.9 and 38.9 us, 24 49.2 and 44.2, 28 49.6 and 50.9; 4 requests 25.7 and 22.7, 16 26.8 and
// 34.5. 16 tokens on 1,000: 20 requests 25.7 and 25.6, 32 32.9 and 38.7.)
constexpr int kCutPlaces = 32;
constexpr int kTileWhole = 3, kTileWhole2 = 5;

bool misaligned(const pa_tensor* t, uintptr_t n) {
  return numel(t) > 0 && reinterpret_cast<uintptr_t>(t->data) % n;
}

// A contiguous vector of n integers of `dtype`.
pa_status check_ints(const pa_tensor* t, const char* name, int32_t dtype, int64_t n) {
  pa_status s = check_tensor(t, name, 1);
  if (s) return s;
  if (t->dtype != dtype)
    return fail(PA_ERR_INVALID_ARG, "%s must be %s", name, dtype == PA_I64 ? "int64" : "int32");
  if (t->shape[0] != n)
    return fail(PA_ERR_INVALID_ARG, "%s: expected %lld elements, got %lld", name, (long long)n,
                (long long)t->shape[0]);
  if (!is_contiguous(t)) return fail(PA_ERR_LAYOUT, "%s must be contiguous", name);
  if (misaligned(t, static_cast<uintptr_t>(elem_size(dtype))))
    return fail(PA_ERR_LAYOUT, "%s is not aligned to its elements", name);
  return PA_OK;
}

pa_status check_tables(const pa_tensor* t) {
  pa_status s = check_tensor(t, "block_tables", 2);
  if (s) return s;
  if (t->dtype != PA_I32) return fail(PA_ERR_INVALID_ARG, "block_tables must be int32");
  if (!is_contiguous(t)) return fail(PA_ERR_LAYOUT, "block_tables must be contiguous");
  if (misaligned(t, 4)) return fail(PA_ERR_LAYOUT, "block_tables is not aligned to its elements");
  if (t->shape[0] > kMaxBatch)
    return fail(PA_ERR_UNSUPPORTED, "batch %lld > %lld", (long long)t->shape[0], (long long)kMaxBatch);
  return PA_OK;
}

// Rows [T, H, D] whose heads and elements are contiguous, 16-byte aligned.
pa_status check_rows(const pa_tensor* t, const char* name) {
  const int64_t T = t->shape[0], H = t->shape[1], D = t->shape[2];
  if (numel(t) == 0) return PA_OK;
  if (t->strides[2] != 1 || (H > 1 && t->strides[1] != D))
    return fail(PA_ERR_LAYOUT, "%s: heads and elements must be contiguous", name);
  if (misaligned(t, 16) || (T > 1 && t->strides[0] % 8))
    return fail(PA_ERR_LAYOUT, "%s: rows must be 16-byte aligned", name);
  return PA_OK;
}

// What a ragged step launches, from its host-known sizes.
struct PackedSizes {
  int tpg, tpu, kv, slot_rows, ctas;
  bool small;  // each CTA plans by itself
  bool whole;  // and works on whole pairs: no join
  size_t plan_words, part_at, bytes;
};

PackedSizes packed_sizes(int64_t T, int64_t B, int64_t span, int G, int64_t Hkv, int D, int num_sms) {
  const PackedShape shape = packed_shape(D);
  PackedSizes z;
  z.tpg = 128 / G;
  z.tpu = z.tpg * shape.rows;
  z.kv = shape.kv;
  z.slot_rows = shape.rows == 2 && T > z.tpg ? 256 : 128;
  const int64_t units = T / z.tpu + std::min(B, T);  // at most
  // lane b of a warp plans sequence b; with more pairs than a few a CTA, whole ones, sorted,
  // are better (a batch of 16 prompts takes 240 us cut, 197 whole)
  z.small = B <= 32 && units * Hkv <= kSmallPairs * num_sms &&
            dprod({double(units), double(Hkv), 4.0 * double(span / z.kv + 2) + kOutPlaces}) < k2p31 - 65536;
  const double tiles = dprod({double(units), double(Hkv), double(span / z.kv + 2)});
  z.ctas = static_cast<int>(std::min<double>(num_sms, std::max(1.0, std::ceil(tiles * 4 / kMinPlaces))));
  // (lengths and how the rows are spread are not known here: full tables, even shares)
  const int64_t seqs = std::max<int64_t>(std::min(B, T), 1), each = (T + seqs * z.tpu - 1) / (seqs * z.tpu);
  const double pairs = dprod({double(seqs), double(each), double(Hkv)});
  const double cost = kOutPlaces + double((span + z.kv - 1) / z.kv) *
                                       (shape.rows == 2 && T > seqs * z.tpg ? kTileWhole2 : kTileWhole);
  z.whole = z.small && span / z.kv + 2 <= kWholeTiles &&
            std::ceil(pairs / num_sms) * cost <= pairs * cost / num_sms + kCutPlaces;
  if (z.whole) z.ctas = static_cast<int>(std::min<int64_t>(num_sms, std::max<int64_t>(units * Hkv, 1)));
  z.plan_words = packed_plan_words(z.ctas, static_cast<size_t>(units));
  // behind the decode workspace's counters, which stay zero
  z.part_at = (256 + z.plan_words * 4 + 255) / 256 * 256;
  z.bytes = z.part_at + 2 * static_cast<size_t>(z.ctas) * packed_slot_floats(z.slot_rows, D) * sizeof(float);
  return z;
}

pa_status check_heads(int64_t Hq, int64_t Hkv, int64_t D) {
  if (Hkv <= 0 || Hq <= 0) return fail(PA_ERR_INVALID_ARG, "head counts must be positive");
  if (Hq % Hkv) return fail(PA_ERR_INVALID_ARG, "num_q_heads %% num_kv_heads != 0");
  if (Hq / Hkv > 16) return fail(PA_ERR_UNSUPPORTED, "GQA group %lld > 16", (long long)(Hq / Hkv));
  if (D != 64 && D != 128 && D != 256) return fail(PA_ERR_UNSUPPORTED, "head_dim %lld", (long long)D);
  return PA_OK;
}

pa_status packed_attention(const pa_tensor* out, const pa_tensor* q, const pa_tensor* key_cache,
                           const pa_tensor* value_cache, const pa_tensor* block_tables,
                           const pa_tensor* seq_lens, const pa_tensor* query_start,
                           const pa_tensor* tree_mask, bool tree, int32_t num_kv_heads, float scale,
                           int32_t block_size, int32_t window, int32_t kv_dtype, float k_scale,
                           float v_scale, pa_stream stream) {
  pa_status s;
  if ((s = check_tensor(out, "out", 3)) || (s = check_tensor(q, "q", 3)) ||
      (s = check_tensor(key_cache, "key_cache", 4)) || (s = check_tensor(value_cache, "value_cache", 4)) ||
      (s = check_tables(block_tables)))
    return s;
  if (q->dtype != PA_F16 && q->dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "q must be f16 or bf16");
  if (out->dtype != q->dtype) return fail(PA_ERR_INVALID_ARG, "out dtype must equal q dtype");
  for (int i = 0; i < 3; ++i)
    if (out->shape[i] != q->shape[i]) return fail(PA_ERR_INVALID_ARG, "out shape != q shape");
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t B = block_tables->shape[0], MB = block_tables->shape[1];
  if ((s = check_ints(seq_lens, "seq_lens", PA_I32, B)) ||
      (s = check_ints(query_start, "query_start", PA_I32, B + 1)) ||
      (tree && (s = check_ints(tree_mask, "tree_mask", PA_I64, T))))
    return s;
  if (kv_dtype != PA_KV_AUTO && kv_dtype != PA_KV_FP8_E4M3)
    return fail(PA_ERR_INVALID_ARG, "bad kv_dtype %d", kv_dtype);
  const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
  const int32_t cdt = fp8 ? PA_FP8_E4M3 : q->dtype;
  if (key_cache->dtype != cdt || value_cache->dtype != cdt)
    return fail(PA_ERR_INVALID_ARG, "cache dtype does not match q dtype / kv_dtype");
  for (int i = 0; i < 4; ++i)
    if (key_cache->shape[i] != value_cache->shape[i])
      return fail(PA_ERR_INVALID_ARG, "key and value cache shapes differ");
  const int64_t NB = key_cache->shape[0], Hkv = key_cache->shape[1];
  if (num_kv_heads != Hkv) return fail(PA_ERR_INVALID_ARG, "num_kv_heads != key_cache.shape[1]");
  if (block_size != key_cache->shape[2]) return fail(PA_ERR_INVALID_ARG, "block_size != key_cache.shape[2]");
  if (key_cache->shape[3] != D) return fail(PA_ERR_INVALID_ARG, "cache head_dim != q head_dim");
  if ((s = check_heads(Hq, Hkv, D))) return s;
  if (fp8 && D == 64) return fail(PA_ERR_UNSUPPORTED, "fp8 caches need head_dim 128 or 256");
  if (block_size <= 0 || block_size % 16 || block_size > 1024)
    return fail(PA_ERR_UNSUPPORTED, "block_size must be a multiple of 16 in [16, 1024]");
  if (tree && window > 0 && window < 64)
    return fail(PA_ERR_INVALID_ARG, "a window of drafted trees is none or at least 64");
  if (!is_contiguous(key_cache) || !is_contiguous(value_cache))
    return fail(PA_ERR_LAYOUT, "caches must be contiguous");
  if (misaligned(key_cache, 16) || misaligned(value_cache, 16))
    return fail(PA_ERR_LAYOUT, "caches must be 16-byte aligned");
  if ((s = check_rows(q, "q")) || (s = check_rows(out, "out"))) return s;
  for (const pa_tensor* x : {q, out})
    if (T > 1 && numel(x) > 0) {
      if (x->strides[0] < Hq * D) return fail(PA_ERR_LAYOUT, "rows of q or out overlap");
      if (x->strides[0] >= kMaxRowStride)  // (a unit's rows are counted in 32 bits)
        return fail(PA_ERR_UNSUPPORTED, "rows of q or out are 2^23 elements or more apart");
    }
  if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "scale must be finite");
  if (fp8 && !(std::isfinite(k_scale) && std::isfinite(v_scale) && k_scale > 0 && v_scale > 0))
    return fail(PA_ERR_INVALID_ARG, "fp8 scales must be finite and positive");
  const int G = static_cast<int>(Hq / Hkv);
  const double pos = dprod({double(MB), double(block_size)});
  // positions, rows of the pool and tiles are counted in 32 bits, with room for round-ups
  if (T > kMaxRows || dprod({double(NB), double(Hkv), double(block_size)}) >= k2p31 || pos >= k2p31 - 4096)
    return fail(PA_ERR_UNSUPPORTED, "pool, tables or rows exceed 32-bit indexing");
  window = window > 0 ? window : 0;
  // of a unit: a window's reach and its own tokens (drafted ones: 64), else all of a table
  const int64_t span = window > 0 ? std::min<int64_t>(MB * block_size, int64_t(window) + 256) : MB * block_size;
  for (const pa_tensor* x : {q, key_cache, value_cache, block_tables, seq_lens, query_start, tree ? tree_mask : q})
    if (overlaps(out, x)) return fail(PA_ERR_INVALID_ARG, "out overlaps an input");
  if (B == 0 || T == 0) return ok();
  if (MB == 0) return fail(PA_ERR_INVALID_ARG, "block_tables has no columns");
  if (NB == 0) return fail(PA_ERR_INVALID_ARG, "empty block pool");
  for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{out, "out"}, {q, "q"},
                          {key_cache, "key_cache"}, {value_cache, "value_cache"},
                          {block_tables, "block_tables"}, {seq_lens, "seq_lens"},
                          {query_start, "query_start"}, {tree ? tree_mask : q, "tree_mask"}})
    if ((s = check_accessible(t, name))) return s;
  DeviceInfo dev;
  if ((s = device_info(&dev))) return s;
  CUtensorMap tk, tv, tq;
  const int elt = fp8 ? 1 : 2;
  if ((s = make_cache_map(&tk, key_cache->data, NB * Hkv * block_size, static_cast<int>(D), elt)) ||
      (s = make_cache_map(&tv, value_cache->data, NB * Hkv * block_size, static_cast<int>(D), elt)))
    return s;
  const PackedSizes z = packed_sizes(T, B, span, G, Hkv, static_cast<int>(D), dev.num_sms);
  if ((s = make_query_map(&tq, q->data, T, Hq, static_cast<int>(D), T > 1 ? q->strides[0] : Hq * D, G, z.tpg)))
    return s;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return with_workspace(cs, z.bytes, [&](char* ws) -> pa_status {
    PackedPlanArgs p;
    p.query_start = static_cast<const int32_t*>(query_start->data);
    p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
    p.plan = reinterpret_cast<int32_t*>(ws + 256);
    p.err = dev.err_word;
    p.B = static_cast<int>(B);
    p.T = static_cast<int>(T);
    p.MB = static_cast<int>(MB);
    p.bs = block_size;
    p.Hkv = static_cast<int>(Hkv);
    p.window = window;
    p.tpu = z.tpu;
    p.kv = z.kv;
    p.ctas = z.ctas;
    p.tpg = z.tpg;
    p.min_places = kMinPlaces;
    p.split_places = kSplitPlaces;
    p.tree = tree;
    cudaError_t e = z.small ? cudaSuccess : packed_plan_launch(p, cs, true);
    if (e != cudaSuccess) return cuda_fail(e, "packed plan launch");
    PackedArgs a;
    a.out = out->data;
    a.block_tables = static_cast<const int32_t*>(block_tables->data);
    a.tree = tree ? static_cast<const int64_t*>(tree_mask->data) : nullptr;
    a.plan = p.plan;
    a.part = reinterpret_cast<float*>(ws + z.part_at);
    a.err = dev.err_word;
    a.query_start = p.query_start;
    a.seq_lens = p.seq_lens;
    a.B = p.B;
    a.T = p.T;
    a.tpu = z.tpu;
    a.kv = z.kv;
    a.min_places = kMinPlaces;
    a.out_stride = out->strides[0];
    a.ctas = z.ctas;
    a.Hkv = p.Hkv;
    a.G = G;
    a.bs = block_size;
    a.MB = p.MB;
    a.NB = static_cast<int>(NB);
    a.window = window;
    a.tpg = z.tpg;
    a.slot_rows = z.slot_rows;
    a.score_scale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                       (fp8 ? static_cast<double>(k_scale) : 1.0));
    a.v_scale = fp8 ? v_scale : 1.f;
    e = (z.whole ? packed_launch_whole : z.small ? packed_launch_small : packed_launch)(q->dtype, fp8, static_cast<int>(D), tk, tv, tq, a, cs, true);
    if (e != cudaSuccess) return cuda_fail(e, "packed attention launch");
    if (z.whole) {
      count_launches(1);
      return ok();
    }
    PackedMergeArgs m;
    m.out = out->data;
    m.part = a.part;
    m.plan = p.plan;
    m.out_stride = a.out_stride;
    m.ctas = z.ctas;
    m.G = G;
    m.D = static_cast<int>(D);
    m.tpg = z.tpg;
    m.slot_rows = z.slot_rows;
    m.small = z.small;
    e = packed_merge_launch(q->dtype, m, cs, true);
    if (e != cudaSuccess) return cuda_fail(e, "packed merge launch");
    count_launches(z.small ? 2 : 3);
    return ok();
  });
}

// Caches of the row moves: [NB, Hkv, bs, D], or the same of several layers, a fixed
// stride apart.
struct MovedCaches {
  int64_t layers, NB, Hkv, bs, D, k_layer, v_layer;  // layer strides in bytes
  int elt;
};
pa_status check_moved(const pa_tensor* kc, const pa_tensor* vc, MovedCaches* m) {
  pa_status s;
  if (!kc) return fail(PA_ERR_INVALID_ARG, "key_cache: null tensor");
  const int nd = kc->ndim;
  if (nd != 4 && nd != 5) return fail(PA_ERR_INVALID_ARG, "key_cache: expected 4 or 5 dims, got %d", nd);
  if ((s = check_tensor(kc, "key_cache", nd)) || (s = check_tensor(vc, "value_cache", nd))) return s;
  if (kc->dtype != PA_F16 && kc->dtype != PA_BF16 && kc->dtype != PA_FP8_E4M3)
    return fail(PA_ERR_UNSUPPORTED, "caches must be f16, bf16 or e4m3");
  if (vc->dtype != kc->dtype) return fail(PA_ERR_INVALID_ARG, "key and value cache dtypes differ");
  for (int i = 0; i < nd; ++i)
    if (kc->shape[i] != vc->shape[i]) return fail(PA_ERR_INVALID_ARG, "key and value cache shapes differ");
  const int o = nd - 4;
  m->layers = o ? kc->shape[0] : 1;
  m->NB = kc->shape[o];
  m->Hkv = kc->shape[o + 1];
  m->bs = kc->shape[o + 2];
  m->D = kc->shape[o + 3];
  m->elt = elem_size(kc->dtype);
  const int64_t want[4] = {m->Hkv * m->bs * m->D, m->bs * m->D, m->D, 1};
  for (const pa_tensor* t : {kc, vc}) {
    if (numel(t) == 0) continue;
    for (int i = 0; i < 4; ++i)
      if (t->shape[o + i] != 1 && t->strides[o + i] != want[i])
        return fail(PA_ERR_LAYOUT, "the blocks of a layer must be contiguous");
    if (o && m->layers > 1 && t->strides[0] < m->NB * want[0])
      return fail(PA_ERR_LAYOUT, "layers overlap");
    if (misaligned(t, 16) || (o && m->layers > 1 && t->strides[0] * m->elt % 16))
      return fail(PA_ERR_LAYOUT, "caches must be 16-byte aligned");
  }
  m->k_layer = o ? kc->strides[0] * m->elt : 0;
  m->v_layer = o ? vc->strides[0] * m->elt : 0;
  if (m->D * m->elt % 16) return fail(PA_ERR_UNSUPPORTED, "rows must be a multiple of 16 bytes");
  if (m->layers > 1024) return fail(PA_ERR_UNSUPPORTED, "more than 1024 layers");
  if (double(m->NB) >= k2p31 || dprod({double(m->Hkv), double(m->bs), double(m->D)}) >= k2p31 ||
      dprod({double(m->Hkv), double(m->D)}) >= 4194304)  // (256 rows of all heads in 31 bits)
    return fail(PA_ERR_UNSUPPORTED, "pool exceeds 32-bit indexing");
  if (overlaps(kc, vc)) {
    // (layers of one tensor in turn: K, V, K, V ...)
    const int64_t layer = m->NB * want[0] * m->elt, step = m->k_layer;
    const int64_t ahead = static_cast<const char*>(vc->data) - static_cast<const char*>(kc->data);
    const int64_t r = step > 0 ? (ahead % step + step) % step : 0;
    if (m->layers < 2 || m->v_layer != step || r < layer || r > step - layer)
      return fail(PA_ERR_INVALID_ARG, "key and value cache overlap");
  }
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_prefill_packed(const pa_tensor* out, const pa_tensor* q, const pa_tensor* key_cache,
                            const pa_tensor* value_cache, const pa_tensor* block_tables,
                            const pa_tensor* seq_lens, const pa_tensor* query_start,
                            int32_t num_kv_heads, float scale, int32_t block_size, int32_t window,
                            int32_t kv_dtype, float k_scale, float v_scale, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    return packed_attention(out, q, key_cache, value_cache, block_tables, seq_lens, query_start, nullptr,
                            false, num_kv_heads, scale, block_size, window, kv_dtype, k_scale, v_scale, stream);
  });
}

pa_status pa_decode_tree(const pa_tensor* out, const pa_tensor* q, const pa_tensor* key_cache,
                         const pa_tensor* value_cache, const pa_tensor* block_tables,
                         const pa_tensor* seq_lens, const pa_tensor* query_start,
                         const pa_tensor* tree_mask, int32_t num_kv_heads, float scale,
                         int32_t block_size, int32_t window, int32_t kv_dtype, float k_scale,
                         float v_scale, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    return packed_attention(out, q, key_cache, value_cache, block_tables, seq_lens, query_start, tree_mask,
                            true, num_kv_heads, scale, block_size, window, kv_dtype, k_scale, v_scale, stream);
  });
}

pa_status pa_packed_workspace_size(int64_t num_rows, int64_t batch, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim, size_t* bytes) {
  return abi_guard([&]() -> pa_status {
    if (!bytes) return fail(PA_ERR_INVALID_ARG, "bytes is null");
    if (num_rows < 0 || num_rows > kMaxRows)
      return fail(PA_ERR_UNSUPPORTED, "num_rows %lld", (long long)num_rows);
    if (batch < 0 || batch > kMaxBatch) return fail(PA_ERR_UNSUPPORTED, "batch %lld", (long long)batch);
    pa_status s = check_heads(num_q_heads, num_kv_heads, head_dim);
    if (s) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev))) return s;
    *bytes = packed_sizes(num_rows, batch, int64_t(1) << 31, num_q_heads / num_kv_heads, num_kv_heads,
                          head_dim, dev.num_sms).bytes;
    return ok();
  });
}

pa_status pa_copy_blocks(const pa_tensor* key_cache, const pa_tensor* value_cache,
                         const pa_tensor* block_pairs, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    MovedCaches m;
    pa_status s = check_moved(key_cache, value_cache, &m);
    if (s || (s = check_tensor(block_pairs, "block_pairs", 2))) return s;
    if (block_pairs->dtype != PA_I32) return fail(PA_ERR_INVALID_ARG, "block_pairs must be int32");
    if (block_pairs->shape[1] != 2) return fail(PA_ERR_INVALID_ARG, "block_pairs must be [n, 2]");
    if (!is_contiguous(block_pairs)) return fail(PA_ERR_LAYOUT, "block_pairs must be contiguous");
    if (misaligned(block_pairs, 8)) return fail(PA_ERR_LAYOUT, "block_pairs is not aligned to its pairs");
    const int64_t n = block_pairs->shape[0];
    for (const pa_tensor* t : {key_cache, value_cache})
      if (overlaps(t, block_pairs)) return fail(PA_ERR_INVALID_ARG, "a cache overlaps block_pairs");
    const int64_t units = m.Hkv * m.bs * m.D * m.elt / 16, per = copy_blocks_chunk();
    const int64_t chunks = (units + per - 1) / per;
    if (dprod({double(chunks), double(n), double(m.layers), 2.0}) >= k2p31)
      return fail(PA_ERR_UNSUPPORTED, "too many pairs");
    if (n == 0 || numel(key_cache) == 0) return ok();
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{key_cache, "key_cache"},
                            {value_cache, "value_cache"}, {block_pairs, "block_pairs"}})
      if ((s = check_accessible(t, name))) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev))) return s;
    CopyBlocksArgs a;
    a.kc = key_cache->data;
    a.vc = value_cache->data;
    a.block_pairs = static_cast<const int2*>(block_pairs->data);
    a.err = dev.err_word;
    a.k_layer = m.k_layer;
    a.v_layer = m.v_layer;
    a.layers = static_cast<int>(m.layers);
    a.NB = static_cast<int>(m.NB);
    a.pairs = static_cast<int>(n);
    a.units = static_cast<int>(units);
    a.chunks = static_cast<int>(chunks);
    const cudaError_t e = copy_blocks_launch(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
    count_launches(1);
    return ok();
  });
}

pa_status pa_compact_cache(const pa_tensor* key_cache, const pa_tensor* value_cache,
                           const pa_tensor* block_tables, const pa_tensor* seq_lens,
                           const pa_tensor* query_start, const pa_tensor* kept,
                           const pa_tensor* num_kept, const pa_tensor* seq_lens_out,
                           const pa_tensor* kept_tokens, int32_t block_size, pa_stream stream) {
  return abi_guard([&]() -> pa_status {
    MovedCaches m;
    pa_status s = check_moved(key_cache, value_cache, &m);
    if (s || (s = check_tables(block_tables))) return s;
    const int64_t B = block_tables->shape[0], MB = block_tables->shape[1];
    if ((s = check_ints(seq_lens, "seq_lens", PA_I32, B)) ||
        (s = check_ints(query_start, "query_start", PA_I32, B + 1)) || (s = check_tensor(kept, "kept", 2)) ||
        (s = check_ints(num_kept, "num_kept", PA_I32, B)) ||
        (s = check_ints(seq_lens_out, "seq_lens_out", PA_I32, B)) ||
        (kept_tokens && (s = check_ints(kept_tokens, "kept_tokens", PA_I32, B))))
      return s;
    if (kept->dtype != PA_I32) return fail(PA_ERR_INVALID_ARG, "kept must be int32");
    if (kept->shape[0] != B) return fail(PA_ERR_INVALID_ARG, "kept must have a row a sequence");
    if (!is_contiguous(kept)) return fail(PA_ERR_LAYOUT, "kept must be contiguous");
    if (misaligned(kept, 4)) return fail(PA_ERR_LAYOUT, "kept is not aligned to its elements");
    if (block_size != m.bs) return fail(PA_ERR_INVALID_ARG, "block_size is not the caches'");
    if (block_size <= 0 || block_size % 16 || block_size > 1024)
      return fail(PA_ERR_UNSUPPORTED, "block_size must be a multiple of 16 in [16, 1024]");
    if (dprod({double(MB), double(block_size)}) >= k2p31 - 2048 || double(kept->shape[1]) >= k2p31 - 2048)
      return fail(PA_ERR_UNSUPPORTED, "tables exceed 32-bit indexing");
    for (const pa_tensor* w : {key_cache, value_cache, seq_lens_out, kept_tokens}) {
      if (!w) continue;
      for (const pa_tensor* t : {block_tables, seq_lens, query_start, kept, num_kept})
        if (overlaps(w, t)) return fail(PA_ERR_INVALID_ARG, "an output overlaps an input");
    }
    for (const pa_tensor* c : {key_cache, value_cache})
      if (overlaps(c, seq_lens_out) || (kept_tokens && overlaps(c, kept_tokens)))
        return fail(PA_ERR_INVALID_ARG, "two outputs overlap");
    if (kept_tokens && overlaps(seq_lens_out, kept_tokens))
      return fail(PA_ERR_INVALID_ARG, "two outputs overlap");
    if (B == 0) return ok();
    if (MB == 0) return fail(PA_ERR_INVALID_ARG, "block_tables has no columns");
    for (auto& [t, name] : {std::pair<const pa_tensor*, const char*>{key_cache, "key_cache"},
                            {value_cache, "value_cache"}, {block_tables, "block_tables"},
                            {seq_lens, "seq_lens"}, {query_start, "query_start"}, {kept, "kept"},
                            {num_kept, "num_kept"}, {seq_lens_out, "seq_lens_out"},
                            {kept_tokens, "kept_tokens"}})
      if ((s = check_accessible(t, name))) return s;
    DeviceInfo dev;
    if ((s = device_info(&dev))) return s;
    CompactArgs a;
    a.kc = key_cache->data;
    a.vc = value_cache->data;
    a.block_tables = static_cast<const int32_t*>(block_tables->data);
    a.seq_lens = static_cast<const int32_t*>(seq_lens->data);
    a.query_start = static_cast<const int32_t*>(query_start->data);
    a.kept = static_cast<const int32_t*>(kept->data);
    a.num_kept = static_cast<const int32_t*>(num_kept->data);
    a.lens_out = static_cast<int32_t*>(seq_lens_out->data);
    a.kept_tokens = kept_tokens ? static_cast<int32_t*>(kept_tokens->data) : nullptr;
    a.err = dev.err_word;
    a.k_layer = m.k_layer;
    a.v_layer = m.v_layer;
    // (without layers, heads or elements rows have no bytes, but lists and tables are looked at)
    a.layers = static_cast<int>(m.layers);
    a.B = static_cast<int>(B);
    a.MB = static_cast<int>(MB);
    a.NB = static_cast<int>(m.NB);
    a.Hkv = numel(key_cache) ? static_cast<int>(m.Hkv) : 0;
    a.bs = block_size;
    a.M = static_cast<int>(kept->shape[1]);
    a.row_units = static_cast<int>(m.D * m.elt / 16);
    const cudaError_t e = compact_cache_launch(a, dev.num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "compact_cache launch");
    count_launches(1);
    return ok();
  });
}

}  // extern "C"
