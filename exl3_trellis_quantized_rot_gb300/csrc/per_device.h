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

// The last N settings that were made for (kernel, device): an attribute set for a
// kernel holds on the device that was current.
template <int N>
struct KernelSettings {
  const void* fn[N] = {};
  int device[N] = {};
  long long value[N] = {};
  int next = 0;
  const long long* find(const void* f, int d) const {
    for (int i = 0; i < N; i++)
      if (fn[i] == f && device[i] == d) return &value[i];
    return nullptr;
  }
  void note(const void* f, int d, long long v) {
    int at = next;
    if (const long long* p = find(f, d))
      at = (int)(p - value);
    else
      next = (next + 1) % N;
    fn[at] = f;
    device[at] = d;
    value[at] = v;
  }
};

}  // namespace tfx
