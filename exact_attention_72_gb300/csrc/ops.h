// State of the current device that entry points outside attn_api.cu need.
#pragma once
#include <cstdint>

namespace gb300 {

// SM count and the device status word (first failure recorded by a kernel) of the current device, and the id of its
// context (0 if that cannot be read), unless context is null. False, with nothing written, when the device cannot be
// queried.
bool device_state(int* num_sms, uint32_t** status, unsigned long long* context = nullptr);

}  // namespace gb300
