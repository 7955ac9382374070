// launch_cache.h -- facts about (device, kernel, shape) that a process looks up
// once: they cost more than the launch that needs them.  Plain C++.
#pragma once

#include <cstddef>
#include <cstdint>
#include <functional>
#include <mutex>
#include <new>
#include <unordered_map>

namespace qamw {

struct LaunchKey {
  int dev;
  const void* fn;
  int threads;
  size_t smem;
  bool operator==(const LaunchKey& o) const {
    return dev == o.dev && fn == o.fn && threads == o.threads && smem == o.smem;
  }
};

struct LaunchKeyHash {
  size_t operator()(const LaunchKey& k) const {
    uint64_t h = reinterpret_cast<uintptr_t>(k.fn);
    h = (h ^ ((uint64_t)k.smem << 20) ^ ((uint64_t)k.threads << 8) ^ (uint64_t)k.dev) * 0x9e3779b97f4a7c15ULL;
    return (size_t)(h ^ (h >> 32));
  }
};

// As many entries as there are keys (widths x kernels: some thousands at most, of
// about 60 bytes).  Where there is no memory for one, the fact is looked up again.
class LaunchCache {
 public:
  bool get(const LaunchKey& k, int* v) {
    std::lock_guard<std::mutex> lock(mu_);
    const auto it = map_.find(k);
    if (it == map_.end()) return false;
    *v = it->second;
    return true;
  }
  void put(const LaunchKey& k, int v) {
    std::lock_guard<std::mutex> lock(mu_);
    try {
      map_.emplace(k, v);
    } catch (const std::bad_alloc&) {
    }
  }

 private:
  std::mutex mu_;
  std::unordered_map<LaunchKey, int, LaunchKeyHash> map_;
};

}  // namespace qamw
