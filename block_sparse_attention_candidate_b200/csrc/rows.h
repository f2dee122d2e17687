// Whether the rows of strided operands share memory: what a call writes must not meet
// what it reads, what else it writes, or itself.
//
// No CUDA types here, so the logic is testable on a machine without a GPU.
#pragma once

#include <cstdint>

namespace dynrad {

// Whether two of one operand's rows (D bf16 numbers at t * token_stride + h *
// head_stride, t < tokens, h < heads, strides >= 0) share memory.
inline bool rows_meet_own(int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t heads, int64_t D) {
  using wide = __int128;
  if (tokens == 1) token_stride = 0;
  if (heads == 1) head_stride = 0;
  // the usual order: all of one axis within a step of the other
  const bool token_in = tokens == 1 || (heads > 1 && token_stride < head_stride);
  const wide in = token_in ? token_stride : head_stride, out = token_in ? head_stride : token_stride;
  const int64_t n_in = token_in ? tokens : heads, n_out = token_in ? heads : tokens;
  if ((n_in == 1 || in >= D) && (n_out == 1 || out >= in * (n_in - 1) + D)) return false;
  if ((n_in > 1 && in < D) || (n_out > 1 && out < D)) return true;
  // rows i, j steps apart: for each j > 0 of the wider the two i next to j * out / in
  for (int64_t j = 1; j < n_out; ++j)
    for (wide i = j * out / in, last = i + 1; i <= last; ++i)
      if (i < n_in && j * out - i * in < D && i * in - j * out < D) return true;
  return false;
}

// Whether a row of a shares memory with one of b's, whose own do not meet.  Operands whose
// spans meet count as meeting where their strides differ; with the same strides, as in
// two slices of one tensor, the rows decide.
inline bool rows_meet(const void* a, int64_t a_token, int64_t a_head, const void* b, int64_t b_token,
                      int64_t b_head, int64_t tokens, int64_t heads, int64_t D) {
  using wide = __int128;
  if (tokens == 1) a_token = b_token = 0;
  if (heads == 1) a_head = b_head = 0;
  const wide a_span = static_cast<wide>(a_token) * (tokens - 1) + static_cast<wide>(a_head) * (heads - 1) + D;
  const wide b_span = static_cast<wide>(b_token) * (tokens - 1) + static_cast<wide>(b_head) * (heads - 1) + D;
  const wide d = (static_cast<wide>(reinterpret_cast<uintptr_t>(b)) - static_cast<wide>(reinterpret_cast<uintptr_t>(a))) / 2;
  if (d >= a_span || -d >= b_span) return false;
  if (a_token != b_token || a_head != b_head) return true;
  // rows i tokens and j heads apart lie d + i * token + j * head apart: for each j the
  // two i next to where that is 0
  for (int64_t j = 1 - heads; j < heads; ++j) {
    const wide c = d + static_cast<wide>(j) * a_head;
    wide i = a_token > 0 ? -c / a_token : 0;
    if (i * a_token > -c) --i;
    for (const wide last = i + 1; i <= last; ++i)
      if (i > -tokens && i < tokens && c + i * a_token < D && -c - i * a_token < D) return true;
  }
  return false;
}

}  // namespace dynrad
