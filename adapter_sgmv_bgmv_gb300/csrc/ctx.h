// The parts of a context that entry points outside api.cpp use.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/lora.h"

namespace lora {

// Start of a launching call: forget the last call's path, make the device current.
int ctx_begin(lora_ctx *ctx, cudaStream_t stream);
int ctx_cuda_fail(lora_ctx *ctx, cudaError_t e);
// Count one launch; `path` is its bit of lora_last_path.
void ctx_launched(lora_ctx *ctx, cudaStream_t stream, int path);
unsigned *ctx_status(const lora_ctx *ctx);
int ctx_device(const lora_ctx *ctx);
int ctx_sms(const lora_ctx *ctx);
// The context's attention scratch, allocated and zeroed by the first call.
int ctx_attn_scratch(lora_ctx *ctx, size_t bytes, uint8_t **out);

}  // namespace lora
