// fa_device.h -- what a host launcher needs to know about the current device,
// and the calling thread's error message (both kept in fa_api.cu).
#pragma once

namespace fa {

// A bit of the device status word beside kStatusTimeout (fa_params.h): a cache
// length or table entry was out of range, and the tokens behind it skipped.
constexpr unsigned int kStatusBadIndex = 1u << 1;

struct DeviceInfo {
  int dev;
  int num_sms;
  int max_ctas;              // fa_set_max_ctas (0: no cap)
  unsigned int* status;      // the device status word (kStatus* bits)
  long long timeout_cycles;  // bound on every wait, in SM clock cycles
};

int current_device(DeviceInfo* info);  // an fa_status; the message is set on error
void set_error(const char* fmt, ...);
void clear_error();

}  // namespace fa
