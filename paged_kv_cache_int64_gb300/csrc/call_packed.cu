// call_packed.cu - pkv_call_packed: the calls after the verify with their arguments in one array.
#include <limits.h>
#include <string.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "host_common.h"

namespace pkv {
namespace {

// The argument at `at`; false: it does not fit.
template <typename T>
bool take(const uint8_t* at, T& x) {
  if constexpr (std::is_floating_point<T>::value) {
    double v;
    memcpy(&v, at, 8);
    x = (T)v;
    return true;
  } else {
    int64_t v;
    memcpy(&v, at, 8);
    if constexpr (std::is_pointer<T>::value) {
      x = reinterpret_cast<T>((uintptr_t)v);
      return true;
    } else {
      x = (T)v;
      return (int64_t)x == v;
    }
  }
}

template <typename... A, size_t... I>
pkv_status unpack(pkv_status (*f)(A...), const void* args, int64_t bytes, std::index_sequence<I...>) {
  PKV_ARG(args && bytes == (int64_t)(8 * sizeof...(A)), "call_packed: %d arguments of 8 bytes expected (got %lld bytes)",
          (int)sizeof...(A), (long long)bytes);
  std::tuple<A...> x;
  const uint8_t* at = static_cast<const uint8_t*>(args);
  PKV_ARG((take(at + 8 * I, std::get<I>(x)) & ...), "call_packed: an integer argument is out of range");
  return f(std::get<I>(x)...);
}
template <typename... A>
pkv_status call(pkv_status (*f)(A...), const void* args, int64_t bytes) {
  return unpack(f, args, bytes, std::index_sequence_for<A...>{});
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_call_packed(int32_t call_id, const void* args, int64_t bytes) {
  using namespace pkv;
  clear_error();
  switch (call_id) {
    case PKV_CALL_SPEC_VERIFY_ACCEPT: return call(pkv_spec_verify_accept, args, bytes);
    case PKV_CALL_KV_ATTN_WEIGHTS: return call(pkv_kv_attn_weights, args, bytes);
    case PKV_CALL_KV_EVICT_SELECT: return call(pkv_kv_evict_select, args, bytes);
    case PKV_CALL_KV_CACHE_COMPACT: return call(pkv_kv_cache_compact, args, bytes);
    default: PKV_ARG(false, "call_packed: unknown call %d", call_id);
  }
}
