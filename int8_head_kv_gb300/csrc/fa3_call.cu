// The packed-row calls with their arguments in one block: host code alone.  Each of these calls takes a few
// microseconds of a GPU in a decode step, and behind a foreign-function interface every argument has a price: from
// Python, fa3_norm_rope's 32 one by one make a call of 21 us, in one block of 17; the append's 32 of 25 and 21.
#include "fa3_common.cuh"

#include <cstring>
#include <limits>
#include <tuple>
#include <type_traits>
#include <utility>

namespace fa3 {
namespace {

template <class A>
bool take(int64_t v, A* out) {
  if constexpr (std::is_pointer_v<A>) {
    *out = reinterpret_cast<A>(v);
  } else if constexpr (std::is_same_v<A, float>) {
    double d;
    std::memcpy(&d, &v, sizeof d);
    *out = (float)d;
  } else {
    if (std::is_unsigned_v<A> ? v < 0
                              : v < (int64_t)std::numeric_limits<A>::min() || v > (int64_t)std::numeric_limits<A>::max())
      return false;
    *out = (A)v;
  }
  return true;
}

template <class... A, size_t... I>
int unpack(int (*f)(A...), const int64_t* args, std::index_sequence<I...>) {
  std::tuple<A...> t;
  if (!(take(args[I], &std::get<I>(t)) && ...)) return FA3_ERANGE;
  return f(std::get<I>(t)...);
}
template <class... A>
int call(int (*f)(A...), const int64_t* args, int count) {
  if (count != (int)sizeof...(A)) return FA3_EINVAL;
  return unpack(f, args, std::index_sequence_for<A...>{});
}

}  // namespace
}  // namespace fa3

FA3_API int fa3_call(int which, const int64_t* args, int count) {
  if (!args) return FA3_EINVAL;
  switch (which) {
    case FA3_CALL_NORM_ROPE: return fa3::call(fa3_norm_rope, args, count);
    case FA3_CALL_ROPE_APPEND_GQA_PAGED: return fa3::call(fa3_rope_append_gqa_paged, args, count);
    case FA3_CALL_PREFILL_ATTN_GQA_PAGED: return fa3::call(fa3_prefill_attn_gqa_paged, args, count);
    case FA3_CALL_CROSS_ATTN_GQA: return fa3::call(fa3_cross_attn_gqa, args, count);
    default: return FA3_EINVAL;
  }
}
