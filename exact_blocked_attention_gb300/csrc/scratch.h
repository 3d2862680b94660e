// How much a grow-only buffer asks for, and how a call is cut so that its part of
// one stays small.  Host code without CUDA, so that it can be tested without a
// GPU.
#pragma once
#include <cstddef>
#include <cstdint>

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

// What a call does at a time: `seqs` sequences with all their heads, or `heads` of
// one sequence.  seqs = 0: nothing.
struct Slice {
  int64_t seqs, heads;
};

// B sequences of H heads, `seq` bytes of scratch for a sequence and `head` for each
// of its heads: the most that `most` bytes hold; heads in parts of much the same
// size.
inline Slice most_of(int64_t B, int64_t H, int64_t seq, int64_t head, int64_t most) {
  if (B < 1 || H < 1 || seq + head > most) return {0, 0};
  const int64_t all = seq + H * head;
  if (all <= most) return {most / all < B ? most / all : B, H};
  const int64_t fit = (most - seq) / head, parts = (H + fit - 1) / fit;
  return {1, (H + parts - 1) / parts};
}

// A buffer of *have bytes for such slices, which never asks for more than `most`
// (a power of two): it grows to most / 2^i, so that the outgrown ones together stay
// below the current one.  Where that finds no memory it grows to what is needed,
// then the slice halves until one fits, which it may in the buffer as it is.
// allocate(bytes) returns 0, or an error, and no_memory(error) tells whether a
// smaller request may do better; another error is returned in *failed (0: none).
template <class Allocate, class NoMemory, class Error>
Slice fit_slices(int64_t B, int64_t H, int64_t seq, int64_t head, int64_t most, int64_t* have, Allocate&& allocate,
                 NoMemory&& no_memory, Error* failed) {
  *failed = Error{};
  for (Slice s = most_of(B, H, seq, head, most); s.seqs > 0;) {
    const int64_t need = s.seqs * (seq + s.heads * head);
    if (need <= *have) return s;
    int64_t ask = most;
    while (ask / 2 >= need) ask /= 2;
    for (int64_t n = ask;; n = need) {
      const Error e = allocate(n);
      if (e == Error{}) {
        *have = n;
        return s;
      }
      if (!no_memory(e)) {
        *failed = e;
        return {0, 0};
      }
      if (n == need) break;
    }
    if (s.seqs > 1) s.seqs = (s.seqs + 1) / 2;
    else if (s.heads > 1) s.heads = (s.heads + 1) / 2;
    else break;
  }
  return {0, 0};
}

}  // namespace blkattn
