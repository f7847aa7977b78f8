// ask_once.h -- what the runtime is asked for once per process (an occupancy, an entry point): the answer
// is kept, a failure is not. The caller returns the failure, and the next call asks again.
#pragma once

#include <atomic>

namespace kvc {

// query(T*) returns 0 (as its error type) and an answer other than T{}, or an error.
template <typename T, typename Query>
auto ask_once(std::atomic<T>& known, T* answer, Query query) {
  *answer = known.load(std::memory_order_acquire);
  using E = decltype(query(answer));
  if (*answer != T{}) return E{};
  const E e = query(answer);
  if (e == E{}) known.store(*answer, std::memory_order_release);
  return e;
}

}  // namespace kvc
