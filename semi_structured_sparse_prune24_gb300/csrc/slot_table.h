// slot_table.h -- what has been looked up of launches: how many CTAs (or clusters) of a kernel with so many threads and so
// much shared memory a device holds. No limit on entries: there are some for each width of rows, and a kernel whose entry had
// no place would be looked up in every call. Host code.
#pragma once
#include <cstddef>
#include <cstdint>
#include <functional>
#include <unordered_map>

namespace p24 {

struct SlotKey {
  const void* kern;
  std::size_t smem;
  int dev, threads, ranks;
  bool operator==(const SlotKey& o) const {
    return kern == o.kern && smem == o.smem && dev == o.dev && threads == o.threads && ranks == o.ranks;
  }
};

struct SlotHash {
  std::size_t operator()(const SlotKey& k) const {
    std::uint64_t h = reinterpret_cast<std::uintptr_t>(k.kern);
    for (const std::uint64_t v : {static_cast<std::uint64_t>(k.smem), static_cast<std::uint64_t>(k.dev),
                                  static_cast<std::uint64_t>(k.threads), static_cast<std::uint64_t>(k.ranks)})
      h = (h ^ v) * 0x9e3779b97f4a7c15ull, h ^= h >> 29;
    return static_cast<std::size_t>(h);
  }
};

// The caller holds a lock around each call.
class SlotTable {
 public:
  // 0 if it is not known.
  int find(const SlotKey& k) const {
    const auto it = all_.find(k);
    return it == all_.end() ? 0 : it->second;
  }
  // Where there is no memory for it, it will be looked up again: the callers are C functions and let no exception out.
  void put(const SlotKey& k, int slots) noexcept {
    try {
      all_.emplace(k, slots);
    } catch (...) {
    }
  }

 private:
  std::unordered_map<SlotKey, int, SlotHash> all_;
};

}  // namespace p24
