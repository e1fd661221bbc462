// Whether two arguments of a call share memory.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gptq {

// Memory that a call reads or writes, and whether two such share a byte.
struct Span {
  const void *p;
  size_t bytes;
};
inline bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace gptq
