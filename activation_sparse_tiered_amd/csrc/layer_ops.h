// Internal declarations of the operators between the projections (not installed).
#pragma once

#include "common.h"
#include "elem.h"

namespace spax {

// A buffer of an operator: [p, p + bytes), of which only the first `row` bytes of every `step`
// are its own (row 0: all of them).
struct Span {
  const void* p;
  size_t bytes;
  bool out;
  const char* name;
  size_t row, step;
};
// True if x and y have a byte in common.  Columns of the same rows (equal steps) are told apart;
// anything else strided counts as all bytes from its first to its last.
bool shares(const Span& x, const Span& y);
constexpr int kMaxSpans = 12;
struct Spans {
  Span s[kMaxSpans];
  int n = 0;
  void add(const void* p, size_t bytes, bool out, const char* name, size_t row = 0,
           size_t step = 0) {
    if (p && bytes) s[n++] = Span{p, bytes, out, name, row, step};
  }
};

// Validation (host only); each also lists the operator's buffers.
int check_kv_append(const spax_kv_append_args* a, Spans* spans);
int check_attention(const spax_attention_args* a, Spans* spans);
int check_residual_norm(const spax_residual_norm_args* a, Spans* spans);
int check_glu(const spax_glu_args* a, Spans* spans);

// How an attention call shares out its keys: every key head's sequences, laid end to end, are cut
// into `shares` equal shares (of the lengths at run time), one workgroup each.
struct AttentionPlan {
  int32_t head_tiles;   // groups of 16 query heads per key head
  int32_t shares;
  int64_t units;        // tiles and fixed costs of n_seqs sequences of max_len
  size_t ws_bytes;
};
AttentionPlan attention_plan(const spax_attention_args* a);

// Launches of validated arguments.
int launch_kv_append(const spax_kv_append_args* a, hipStream_t s);
int launch_attention(const spax_attention_args* a, void* ws, hipStream_t s);
int launch_residual_norm(const spax_residual_norm_args* a, hipStream_t s);
int launch_glu(const spax_glu_args* a, hipStream_t s);

}  // namespace spax
