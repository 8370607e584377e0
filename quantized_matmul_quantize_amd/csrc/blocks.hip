// blocks.hip -- entry points that take another one's arguments in one block
// of 8-byte words (host only).

#include <cstring>
#include <type_traits>
#include <utility>

#include "qmm_blocks.h"

namespace {

template <typename T>
T from_word(int64_t w) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<intptr_t>(w));
  } else if constexpr (std::is_floating_point_v<T>) {
    double d;
    std::memcpy(&d, &w, sizeof d);
    return static_cast<T>(d);
  } else {
    return static_cast<T>(w);
  }
}

template <typename... A, size_t... I>
int call(int (*f)(A...), const int64_t* w, std::index_sequence<I...>) {
  return f(from_word<A>(w[I])...);
}
template <typename... A>
int call(int (*f)(A...), const int64_t* w) {
  return w ? call(f, w, std::index_sequence_for<A...>()) : QMM_EINVAL;
}

}  // namespace

extern "C" int kv4_append_block(const void* words) { return call(kv4_append, static_cast<const int64_t*>(words)); }
extern "C" int kv4_read_block(const void* words) { return call(kv4_read, static_cast<const int64_t*>(words)); }
extern "C" int kv4_copy_pages_block(const void* words) { return call(kv4_copy_pages, static_cast<const int64_t*>(words)); }
extern "C" int kv4_attention_block(const void* words) { return call(kv4_attention, static_cast<const int64_t*>(words)); }
extern "C" int qk_norm_rope_block(const void* words) { return call(qk_norm_rope, static_cast<const int64_t*>(words)); }
