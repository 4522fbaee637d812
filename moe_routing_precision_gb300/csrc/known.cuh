// known.cuh -- what a launcher looks up once (host code, plain C++).
#pragma once

#include <map>
#include <mutex>

namespace moe {

// Values by key, for any number of keys; safe from several threads.  The key holds
// all that the value depends on (the device too, where it does).
template <class Key, class Value>
class Known {
 public:
  bool find(const Key& key, Value* value) const {
    std::lock_guard<std::mutex> lock(mu_);
    const auto it = values_.find(key);
    if (it == values_.end()) return false;
    *value = it->second;
    return true;
  }
  void put(const Key& key, const Value& value) {
    std::lock_guard<std::mutex> lock(mu_);
    values_[key] = value;
  }

 private:
  mutable std::mutex mu_;
  std::map<Key, Value> values_;
};

}  // namespace moe
