// Drives ask_once with a query that fails, then answers: prints one line per call.
#include <cstdio>

#include "ask_once.h"

enum Error { kOk = 0, kFailed = 2 };

int main() {
  static std::atomic<int> known;
  int asked = 0;
  auto call = [&](Error e, int value) {
    int got = -1;
    const Error r = kvc::ask_once(known, &got, [&](int* answer) {
      ++asked;
      if (e == kOk) *answer = value;
      return e;
    });
    std::printf("%d %d %d\n", (int)r, got, asked);
  };
  call(kFailed, 7);   // an error: returned, not kept
  call(kFailed, 7);
  call(kOk, 5);
  call(kFailed, 7);   // not asked again
  call(kOk, 9);
  static std::atomic<const char*> entry;
  const char* p = nullptr;
  const Error a = kvc::ask_once(entry, &p, [](const char**) { return kFailed; });
  const Error b = kvc::ask_once(entry, &p, [](const char** x) { *x = "entry"; return kOk; });
  std::printf("%d %d %s\n", (int)a, (int)b, p);
  return 0;
}
