// kv8_host.h -- host-side checks and conversions shared by the entry points of the 8-bit
// key/value cache.
#pragma once

#include "gqa_kv8.h"
#include "kv8_sched.cuh"

namespace moe {

// Each returns false with the status to give back.
bool kv8_cache_ok(const gqa_kv8_cache_t* c, moe_status_t* st);
bool kv8_batch_ok(const gqa_kv8_cache_t* c, const gqa_kv8_batch_t* b, moe_status_t* st);
// Rows of `width` elements, `stride` elements apart.
bool kv8_rows_ok(const void* p, long long stride, long long width, moe_status_t* st);

Kv8Cache kv8_cache(const gqa_kv8_cache_t* c);
Kv8Batch kv8_batch(const gqa_kv8_batch_t* b);

// Attention with many query rows per key/value head (kv8_prompt.cu): its workspace, and its
// launch on `grid` CTAs of device `dev` (sets p.tq_shift itself).
size_t kv8_prompt_ws_bytes(int D);
cudaError_t launch_kv8_prompt(Kv8AttnParams p, int D, int format, int grid, int dev, cudaStream_t s);

}  // namespace moe
