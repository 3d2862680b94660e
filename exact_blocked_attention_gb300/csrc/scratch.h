// How much a grow-only buffer asks for.  Host code without CUDA, so that it can
// be tested without a GPU.
#pragma once
#include <cstddef>

namespace blkattn {

// A buffer of `have` bytes that needs `need` (more): twice its size, so that
// the outgrown buffers together never exceed the current one, or `need` where
// that is more; where twice finds no memory, `need` alone.  allocate(bytes)
// returns 0, or an error; no_memory(error) tells whether a smaller request may
// do better.  *got: the bytes allocated.
template <class Allocate, class NoMemory>
auto grow_scratch(size_t have, size_t need, Allocate&& allocate, NoMemory&& no_memory, size_t* got) {
  const size_t twice = 2 * have;
  *got = need > twice ? need : twice;
  auto e = allocate(*got);
  if (*got > need && no_memory(e)) {
    *got = need;
    e = allocate(*got);
  }
  return e;
}

}  // namespace blkattn
