// The workspace of the gradient by a token table (embed.cu) and the schedule that it
// follows from.  Host code by itself: the layout is checked without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

namespace muse {

constexpr int kTile = 256;                 // columns of a warp: a block

// Sorted positions of a chunk: as many as let all warps run at once, three CTAs an SM (16,384 positions of 1,024
// columns f16 into f32 16 49.6, 18 45.8, 24 46.6, 32 52.2 us; 8,192 of 4,096 18 92, 36 90, 64 99; 16,384 of 6,656 32 442, 117
// 437.5), from 3 (301 of 6,656 f32 3 19.0, 4 20.1, 8 22.4) to 128 (100,000 of 2,048 117 235, 256 244).
constexpr int64_t kLeastChunk = 3, kMostChunk = 128;
inline int64_t chunk_of(int64_t n, int tiles, int num_sms) {
  const int64_t warps = 24 * static_cast<int64_t>(num_sms), c = (n * tiles + warps - 1) / warps;
  return c < kLeastChunk ? kLeastChunk : c < kMostChunk ? c : kMostChunk;
}

// Parts are stored and loaded 32 bytes at a time; a caller's workspace lies on 16, so it is used from the next 32 on.
constexpr size_t kCallerAlign = 16, kSpaceAlign = 32;
inline uint8_t *space_base(void *workspace) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(workspace);
  return static_cast<uint8_t *>(workspace) + (kSpaceAlign - at % kSpaceAlign) % kSpaceAlign;
}

// From its base: count, order, sorted [n], span [n], used [v / 32], done [chunks][tiles], parts
// [chunks][2][k], each from 256 bytes on; room for as many chunks as n positions or fewer have.
// `bytes` has room for the base's distance too.
struct BackwardSpace {
  size_t order, sorted, span, used, done, part, bytes;
  int64_t chunk, chunks;
};
inline BackwardSpace backward_space(int64_t n, int64_t v, int k, int num_sms) {
  auto up = [](int64_t words) { return (static_cast<size_t>(words) * 4 + 255) / 256 * 256; };
  BackwardSpace s;
  s.chunk = chunk_of(n, k / kTile, num_sms);
  s.chunks = (n + s.chunk - 1) / s.chunk;
  const int64_t wave = 24 * static_cast<int64_t>(num_sms) / (k / kTile), most = wave > n / kMostChunk ? wave : n / kMostChunk;
  const int64_t room = (most < n / kLeastChunk ? most : n / kLeastChunk) + 1;
  s.order = 256;
  s.sorted = s.order + up(n);
  s.span = s.sorted + up(n);
  s.used = s.span + up(2 * n);
  s.done = s.used + up((v + 31) / 32);
  s.part = s.done + up(room * (k / kTile));
  s.bytes = s.part + up(room * 2 * k) + (kSpaceAlign - kCallerAlign);
  return s;
}

}  // namespace muse
