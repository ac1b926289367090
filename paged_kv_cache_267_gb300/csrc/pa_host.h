// Host-side helpers shared by the C-ABI translation units: error messages,
// tensor checks and per-device state (defined in pa_api.cpp). None of them
// throws; none touches the device except check_accessible and device_info.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <functional>
#include <initializer_list>

#include "pa.h"

namespace pa {

constexpr int64_t kMaxBatch = 4096;
constexpr double kMaxTensorBytes = 1125899906842624.0;  // 2^50: no tensor is larger

pa_status fail(pa_status code, const char* fmt, ...);
pa_status ok();
pa_status cuda_fail(cudaError_t e, const char* what);
int elem_size(int32_t dt);
bool is_contiguous(const pa_tensor* t);
int64_t numel(const pa_tensor* t);
void span(const pa_tensor* t, uintptr_t* lo, uintptr_t* hi);
bool overlaps(const pa_tensor* a, const pa_tensor* b);
pa_status check_tensor(const pa_tensor* t, const char* name, int ndim);
double dprod(std::initializer_list<double> f);
pa_status check_accessible_ptr(const void* p, const char* name);
pa_status check_accessible(const pa_tensor* t, const char* name);

// The current device's error word and SM count.
struct DeviceInfo {
  int32_t* err_word;
  int num_sms;
};
pa_status device_info(DeviceInfo* out);
void count_launches(int n);

// 2-D view of a cache for TMA: [rows, D], boxes of 16 rows x 128 bytes, 128-byte
// swizzle.
pa_status make_cache_map(CUtensorMap* map, const void* base, int64_t rows, int D, int elt);
// 3-D view of packed query rows [T, Hq, D], rows `stride` elements apart: boxes of 64
// head dims x G heads x `tokens` rows, 128-byte swizzle.
pa_status make_query_map(CUtensorMap* map, const void* base, int64_t T, int64_t Hq, int D,
                         int64_t stride, int G, int tokens);
// Calls body with the workspace of the stream's steps (the caller's, or the stream's
// own, made large enough), which no other host thread's step gets before body returns.
// Its first 256 bytes are the decode kernels' counters and stay as they are.
pa_status with_workspace(cudaStream_t stream, size_t bytes, const std::function<pa_status(char*)>& body);

}  // namespace pa
