// What the host keeps for each device. The callers name the device (the current
// one), so nothing here needs CUDA.
#pragma once

namespace tfx {

constexpr int kMaxDevices = 64;

// A value found once for each device. What `find` did not find (T{}) is asked for again.
template <typename T>
struct PerDevice {
  T kept[kMaxDevices] = {};
  template <typename Find>
  T of(int device, Find find) {
    if (device < 0 || device >= kMaxDevices) return find();
    if (kept[device] == T{}) kept[device] = find();
    return kept[device];
  }
};

}  // namespace tfx
