// plan_cache.h -- what was worked out once for a size, kept for the next call.
#pragma once
#include <cstddef>
#include <map>
#include <mutex>

namespace gbn {

// At most `most` entries, then the cache starts anew.  Calls from several threads
// are safe, and none throws: without host memory for an entry it is worked out again
// next time.
template <typename Key, typename Value>
class PlanCache {
 public:
  explicit PlanCache(size_t most) : most_(most) {}

  bool find(const Key &key, Value *out) {
    std::lock_guard<std::mutex> lk(mu_);
    const auto it = map_.find(key);
    if (it == map_.end()) return false;
    *out = it->second;
    return true;
  }
  void keep(const Key &key, const Value &value) {
    std::lock_guard<std::mutex> lk(mu_);
    if (map_.size() >= most_) map_.clear();
    try {
      map_[key] = value;
    } catch (...) {  // out of host memory
    }
  }

 private:
  const size_t most_;
  std::mutex mu_;
  std::map<Key, Value> map_;
};

}  // namespace gbn
