// slots.hip -- tokens' rows into the experts' order, back with weights, and the gradient.
// Pair p = t * top_k + j is token t's slot j; slot_row[p] is its row among the experts'
// rows, or a number outside [0, n_rows) for a pair that has none.
//
//   dispatch   R[slot_row[p]] = w[p] * X[t]
//   combine    O[t] = sum_j w[p] * R[slot_row[p]] (+ A[t]), binary32, j ascending
//   gradient   dR[slot_row[p]] = w[p] * dO[t],  dw[p] = sum_h dO[t][h] * R[slot_row[p]][h]
//
// All three go by tokens, so that a token's row is read (or written) once and each expert's
// row once; the order of the rows needs no list of its own.
#include "pieces.hpp"
#include "slots.hpp"

namespace iq4 {

// Elements a lane holds: 16 bytes of the wider of the two types.
template <int T1, int T2>
constexpr int kPiece = (T1 == kF32 || T2 == kF32) ? 4 : 8;

// w * v as a binary32 number: without the barrier a binary16 result would be made of the exact
// product by a mixed-precision instruction, and differ in the last place from the other types' way.
__device__ __forceinline__ float scaled(float w, float v) {
  float p = w * v;
  asm("" : "+v"(p));
  return p;
}

template <int TX, int TR>
__global__ void __launch_bounds__(256) dispatch_kernel(SlotArgs a, uint32_t pieces) {
  constexpr int P = kPiece<TX, TR>;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t t = i / pieces;
  if (t >= a.n_tok) return;
  const int64_t at = (int64_t)(i - t * pieces) * P;
  const int left = (int)min<int64_t>(a.hidden - at, P);
  float v[P];
  load_piece<TX, P>(static_cast<const char*>(a.tok) + t * a.ldt * (TX == kF32 ? 4 : 2), at, left, v);
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t p = (int64_t)t * a.top_k + j;
    const int r = a.slot_row[p];
    if ((uint32_t)r >= a.n_rows) continue;
    float o[P];
    const float w = a.w ? a.w[p] : 1.0f;
#pragma unroll
    for (int e = 0; e < P; ++e) o[e] = a.w ? scaled(w, v[e]) : v[e];
    store_piece<TR, P>(static_cast<char*>(a.out) + r * a.ldo * (TR == kF32 ? 4 : 2), at, left, o);
  }
}

template <int TR, int TO>
__global__ void __launch_bounds__(256) combine_rows_kernel(SlotArgs a, uint32_t pieces) {
  constexpr int P = kPiece<TR, TO>;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t t = i / pieces;
  if (t >= a.n_tok) return;
  const int64_t at = (int64_t)(i - t * pieces) * P;
  const int left = (int)min<int64_t>(a.hidden - at, P);
  float acc[P];
#pragma unroll
  for (int e = 0; e < P; ++e) acc[e] = 0.f;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t p = (int64_t)t * a.top_k + j;
    const int r = a.slot_row[p];
    if ((uint32_t)r >= a.n_rows) continue;
    const float w = a.w ? a.w[p] : 1.0f;
    float v[P];
    load_piece<TR, P>(static_cast<const char*>(a.rows) + r * a.ldr * (TR == kF32 ? 4 : 2), at, left, v);
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = acc[e] + w * v[e];
  }
  if (a.tok) {
    float v[P];
    load_piece<TO, P>(static_cast<const char*>(a.tok) + t * a.ldt * (TO == kF32 ? 4 : 2), at, left, v);
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = acc[e] + v[e];
  }
  store_piece<TO, P>(static_cast<char*>(a.out) + t * a.ldo * (TO == kF32 ? 4 : 2), at, left, acc);
}

// One wave per token.
template <int TD, int TR>
__global__ void __launch_bounds__(64) combine_grad_kernel(SlotArgs a, uint32_t pieces) {
  constexpr int P = kPiece<TD, TR>;
  const int64_t t = blockIdx.x;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t p = t * a.top_k + j;
    const int r = a.slot_row[p];
    float dot = 0.f;
    if ((uint32_t)r < a.n_rows) {
      const float w = a.w ? a.w[p] : 1.0f;
      for (uint32_t q = threadIdx.x; q < pieces; q += 64) {
        const int64_t at = (int64_t)q * P;
        const int left = (int)min<int64_t>(a.hidden - at, P);
        float d[P], v[P], o[P];
        load_piece<TD, P>(static_cast<const char*>(a.tok) + t * a.ldt * (TD == kF32 ? 4 : 2), at, left, d);
        if (a.dw) {
          load_piece<TR, P>(static_cast<const char*>(a.rows) + r * a.ldr * (TR == kF32 ? 4 : 2), at, left, v);
#pragma unroll
          for (int e = 0; e < P; ++e) dot = fmaf(d[e], v[e], dot);
        }
        if (a.out) {
#pragma unroll
          for (int e = 0; e < P; ++e) o[e] = scaled(w, d[e]);
          store_piece<TR, P>(static_cast<char*>(a.out) + r * a.ldo * (TR == kF32 ? 4 : 2), at, left, o);
        }
      }
    }
    if (a.dw) {
      for (int m = 32; m > 0; m >>= 1) dot += __shfl_xor(dot, m);
      if (threadIdx.x == 0) a.dw[p] = dot;
    }
  }
}

// A launch has fewer than 2^32 threads: tokens go in as many launches as that takes.
template <typename F>
static int by_tokens(SlotArgs a, int64_t threads_per_token, int in_type, int out_type, bool out_by_token, F launch) {
  const int64_t most = ((int64_t)1 << 31) / threads_per_token;
  while (a.n_tok > 0) {
    SlotArgs part = a;
    part.n_tok = a.n_tok < most ? a.n_tok : most;
    if (int e = launch(part)) return e;
    const int64_t n = part.n_tok;
    a.n_tok -= n;
    a.slot_row += n * a.top_k;
    if (a.w) a.w += n * a.top_k;
    if (a.dw) a.dw += n * a.top_k;
    if (a.tok) a.tok = static_cast<const char*>(a.tok) + n * a.ldt * type_bytes(in_type);
    if (out_by_token) a.out = static_cast<char*>(a.out) + n * a.ldo * type_bytes(out_type);
  }
  return 0;
}

#define IQ4_TYPES(T1, T2, CALL)                                                               \
  switch (3 * (T1) + (T2)) {                                                                  \
    case 0: CALL(0, 0); break;                                                                \
    case 1: CALL(0, 1); break;                                                                \
    case 2: CALL(0, 2); break;                                                                \
    case 3: CALL(1, 0); break;                                                                \
    case 4: CALL(1, 1); break;                                                                \
    case 5: CALL(1, 2); break;                                                                \
    case 6: CALL(2, 0); break;                                                                \
    case 7: CALL(2, 1); break;                                                                \
    default: CALL(2, 2); break;                                                               \
  }

static uint32_t pieces_of(int64_t hidden, int t1, int t2) {
  const int p = (t1 == kF32 || t2 == kF32) ? 4 : 8;
  return (uint32_t)((hidden + p - 1) / p);
}

int launch_dispatch(const SlotArgs& a, int x_type, int rows_type, hipStream_t s) {
  const uint32_t pieces = pieces_of(a.hidden, x_type, rows_type);
  return by_tokens(a, pieces, x_type, rows_type, false, [&](const SlotArgs& b) {
    const dim3 grid((unsigned)((b.n_tok * pieces + 255) / 256));
#define IQ4_CALL(T1, T2) hipLaunchKernelGGL((dispatch_kernel<T1, T2>), grid, dim3(256), 0, s, b, pieces)
    IQ4_TYPES(x_type, rows_type, IQ4_CALL)
#undef IQ4_CALL
    return check_launch("dispatch_kernel");
  });
}

int launch_combine_rows(const SlotArgs& a, int rows_type, int out_type, hipStream_t s) {
  const uint32_t pieces = pieces_of(a.hidden, rows_type, out_type);
  return by_tokens(a, pieces, out_type, out_type, true, [&](const SlotArgs& b) {
    const dim3 grid((unsigned)((b.n_tok * pieces + 255) / 256));
#define IQ4_CALL(T1, T2) hipLaunchKernelGGL((combine_rows_kernel<T1, T2>), grid, dim3(256), 0, s, b, pieces)
    IQ4_TYPES(rows_type, out_type, IQ4_CALL)
#undef IQ4_CALL
    return check_launch("combine_rows_kernel");
  });
}

int launch_combine_grad(const SlotArgs& a, int dout_type, int rows_type, hipStream_t s) {
  const uint32_t pieces = pieces_of(a.hidden, dout_type, rows_type);
  return by_tokens(a, 64, dout_type, rows_type, false, [&](const SlotArgs& b) {
    const dim3 grid((unsigned)b.n_tok);
#define IQ4_CALL(T1, T2) hipLaunchKernelGGL((combine_grad_kernel<T1, T2>), grid, dim3(64), 0, s, b, pieces)
    IQ4_TYPES(dout_type, rows_type, IQ4_CALL)
#undef IQ4_CALL
    return check_launch("combine_grad_kernel");
  });
}

}  // namespace iq4
