// swiglu.hpp -- SwiGLU between two products, and its gradient: the launchers' arguments
// (swiglu.hip).
#pragma once
#include "common.hpp"
#include "rows.hpp"

namespace iq4 {

struct SwigluArgs {
  const void* g;
  const void* u;
  int64_t ldg, ldu;
  int64_t m, k;
  void* y;         // or null
  int y_type;
  int64_t ldy;
  int fmt;         // RowFormat, or -1: no quantised output
  RowsOut o;
};
int launch_swiglu(const SwigluArgs& a, int type, hipStream_t s);

struct SwigluGradArgs {
  const void* dh;
  const void* g;
  const void* u;
  int64_t lddh, ldg, ldu;
  int64_t m, k;
  void* dg;
  void* du;
  int64_t lddg, lddu;
};
int launch_swiglu_grad(const SwigluGradArgs& a, int dh_type, int type, hipStream_t s);

}  // namespace iq4
