// Host-side helpers that the C entry points share: argument checks, TMA
// descriptors, per-device lookups and the attention launch.  Defined in
// dera_relpos.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <initializer_list>

#include "../../include/dera_train.h"
#include "common.cuh"
#include "train.cuh"

namespace dera {

// Device address of the status word on the current device (looked up once per device).
int* status_ptr(int dev);

bool is16(dera_dtype t);
bool is_float(dera_dtype t);
int fmt_of(dera_dtype t);

dera_status check_shape(int BH, int H, int W, int head_dim);
// Host-only checks: non-null and 16-byte aligned (TMA operands).
dera_status check_host(std::initializer_list<const void*> ptrs);
// Device memory of device `dev` (the launcher's same-device rule).
dera_status check_ptr(const void* p, int dev);
dera_status current_device(int* dev);
// Streaming-multiprocessor count of a device (cached; 0 if the query fails).
int sm_count(int dev);
size_t align256(size_t x);

// Every box is 64 elements (128 bytes, one swizzle atom) wide; a row of
// head_dim d is d / 64 boxes, loaded at element offsets 0 and 64.
// q / out-like tensor [BH, N, d] read in tiles of `rows` rows
bool map_rows(CUtensorMap* m, const void* p, dera_dtype t, int BH, int N, int d, int rows = 128);
// k / v viewed as [BH, H, W, d], read in tiles of KHT grid rows x WP columns
bool map_keys(CUtensorMap* m, const void* p, dera_dtype t, int BH, int H, int W, int d, int WP, int KHT);

// tokens [B, N, heads, d] by their strides (elements), read in boxes of 64 elements by `rows` tokens
bool map_tokens(CUtensorMap* m, const HeadsPtr& t, dera_dtype dt, int B, int N, int heads, int d, int rows);

// the same, any type, in boxes of 32 tokens x `cols` elements (rows of 64 or 128 bytes, swizzled as wide)
bool map_boxes(CUtensorMap* m, const HeadsPtr& t, dera_dtype dt, int B, int N, int heads, int d, int cols);

// A caller's workspace: large enough, 256-byte aligned, of device `dev`.
dera_status check_workspace(const void* ws, size_t have, size_t need, int dev);
// One tensor in token order, its strides made ready for the kernels (0 where the
// dimension has size one).  `distinct`: no two rows may share an element.
dera_status take_heads(const dera_heads* t, int B, int N, int heads, int d, bool distinct, HeadsPtr* out);

// The attention launch of every entry (compact bias, or tables when `fused`).
dera_status run_attention(const void* q, const void* k, const void* v, const void* a, const void* b, void* out,
                          int BH, int H, int W, int d, float scale, dera_dtype in_dtype, dera_dtype bias_dtype,
                          dera_dtype out_dtype, bool fused, void* workspace, size_t workspace_bytes, void* stream,
                          float* lse = nullptr);

#define DERA_TRY(expr)              \
  do {                              \
    const dera_status s_ = (expr);  \
    if (s_ != DERA_OK) return s_;   \
  } while (0)

}  // namespace dera
