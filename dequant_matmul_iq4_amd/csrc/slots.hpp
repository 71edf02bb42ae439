// slots.hpp -- tokens' rows into the experts' order and back: the launchers' arguments
// (slots.hip).
#pragma once
#include "common.hpp"

namespace iq4 {

struct SlotArgs {
  const int32_t* slot_row;  // [n_tok][top_k]: each pair's row, or a number outside [0, n_rows)
  const float* w;           // [n_tok][top_k], or null: 1
  int64_t n_tok, n_rows, hidden;
  int top_k;
  const void* tok;          // the tokens' rows: x, dout, or the addend of a combine (or null)
  int64_t ldt;
  const void* rows;         // the experts' rows, read
  int64_t ldr;
  void* out;                // what is written: the experts' rows, or the tokens'
  int64_t ldo;
  float* dw;                // [n_tok][top_k], or null
};

int launch_dispatch(const SlotArgs& a, int x_type, int rows_type, hipStream_t s);
int launch_combine_rows(const SlotArgs& a, int rows_type, int out_type, hipStream_t s);
int launch_combine_grad(const SlotArgs& a, int dout_type, int rows_type, hipStream_t s);

}  // namespace iq4
