// What the translation units of the library share behind the C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {
namespace api {

constexpr size_t kErrorBytes = 512;

// The calling thread's message buffer of moe_last_error (kErrorBytes).
char* error_buffer();

// Validates a layer shape and its forward workspace; *status is the workspace
// status word.
moe_status layer_status(const moe_shape* shape, void* ws, size_t ws_bytes, uint32_t** status);

}  // namespace api
}  // namespace moe
