// Which of a device's bounded waits that ran out a host thread has been told
// of.  The kernels only ever count them up, so that one thread's question
// takes no other thread's answer away.
#pragma once

namespace zsm {

constexpr int kMaxDevices = 64;

// Whether `count`, the device's number of such waits, is news to the calling
// thread.  (A device past kMaxDevices: whether there has been any.)
inline bool mx_errors_are_news(int device, unsigned count) {
  thread_local unsigned told[kMaxDevices] = {};
  if (device < 0 || device >= kMaxDevices) return count != 0;
  const bool news = told[device] != count;
  told[device] = count;
  return news;
}

}  // namespace zsm
