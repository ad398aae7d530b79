// Internal launchers of the AdamW step (adamw.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "qlora.h"

namespace qlora {

// Partial sums of the norm (doubles), and the workspace's bytes.
long adamw_norm_blocks(const qlora_adamw_item* items, int count, long* chunk);
size_t adamw_bytes(const qlora_adamw_item* items, int count);
void launch_adamw(const qlora_adamw_config& cfg, const qlora_adamw_item* items, int count, void* ws,
                  hipStream_t st);

// which: 0 the first moment, 1 the root of the second
void launch_moment_read(const uint8_t* codes, const uint8_t* scales, long n, int which, int dtype, void* x,
                        hipStream_t st);
void launch_moment_write(const void* x, long n, int which, int dtype, uint8_t* codes, uint8_t* scales,
                         hipStream_t st);

}  // namespace qlora
