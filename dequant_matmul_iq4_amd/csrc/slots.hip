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

// What a token's slots j0 .. j0 + N - 1 point at: row numbers (-1: none) and weights.
template <int N>
struct Slots {
  int r[N];
  float w[N];
};
template <int N>
__device__ __forceinline__ Slots<N> slots_of(const SlotArgs& a, int64_t t, int j0) {
  Slots<N> s;
  const int64_t p = t * a.top_k + j0;
#pragma unroll
  for (int i = 0; i < N; ++i) s.r[i] = j0 + i < a.top_k ? a.slot_row[p + i] : -1;
#pragma unroll
  for (int i = 0; i < N; ++i) s.w[i] = a.w && j0 + i < a.top_k ? a.w[p + i] : 1.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((uint32_t)s.r[i] >= a.n_rows) s.r[i] = -1;
  return s;
}
// The same where all lanes have one token: lane j loads slot j's, and they are read from there into
// scalar registers, as are the addresses made of them.
struct TokenSlots {
  int r;
  float w;
  __device__ __forceinline__ TokenSlots(const SlotArgs& a, int64_t t) : r(-1), w(1.0f) {
    const int lane = threadIdx.x & 63;
    if (lane < a.top_k) {
      r = a.slot_row[t * a.top_k + lane];
      if (a.w) w = a.w[t * a.top_k + lane];
    }
    if ((uint32_t)r >= a.n_rows) r = -1;
  }
  __device__ __forceinline__ int row(int j) const { return __builtin_amdgcn_readlane(r, j); }
  __device__ __forceinline__ float weight(int j) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j));
  }
};
template <int T>
__device__ __forceinline__ const char* row_of(const void* rows, int64_t r, int64_t ld) {
  return static_cast<const char*>(rows) + r * ld * (T == kF32 ? 4 : 2);
}
template <int T>
__device__ __forceinline__ char* row_of(void* rows, int64_t r, int64_t ld) {
  return static_cast<char*>(rows) + r * ld * (T == kF32 ? 4 : 2);
}

template <int T>
__device__ __forceinline__ void store_one(char* row, int64_t at, float v) {
  if constexpr (T == kF32) reinterpret_cast<float*>(row)[at] = v;
  else reinterpret_cast<uint16_t*>(row)[at] = (uint16_t)pack2<T>(v, 0.f);
}

// A lane per piece, whatever token it belongs to; four slots at a time.  The written rows bound it: 3256
// tokens of 2048 numbers of 16 bits to 8 rows each 22 us (5.4 TB/s), of 2047 28, of float32 42.
template <int TX, int TR, bool STREAM>
__global__ void __launch_bounds__(256) dispatch_kernel(SlotArgs a, Pieces pieces) {
  constexpr int P = kPiece<TX, TR>;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t t = pieces.row(i);
  if (t >= a.n_tok) return;
  const Piece c = piece_of<P>(i - t * pieces.n, a.hidden);
  float v[P];
  load_piece<TX, P>(row_of<TX>(a.tok, t, a.ldt), c.at, c.left, v);
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {
    const Slots<4> s = slots_of<4>(a, t, j0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (s.r[j] < 0) continue;
      float o[P];
#pragma unroll
      for (int e = 0; e < P; ++e) o[e] = a.w ? scaled(s.w[j], v[e]) : v[e];
      // (what two pieces have is written twice, the same)
      store_piece<TR, P, STREAM>(row_of<TR>(a.out, s.r[j], a.ldo), c.at, c.left, o);
    }
  }
}

// The same way; the rows of four slots are under way at once.  The rows read bound it: 3256 tokens of
// 2048, eight rows of 16 bits each, 24 us (5.0 TB/s), of 2047 29, of float32 44; four tokens 3.3.  (While this way took 26.1:
// eight slots at once 31.9; a workgroup per token, its slots in scalar registers, 28.2, and 52 for rows of 700.)
template <int TR, int TO, bool STREAM>
__global__ void __launch_bounds__(256) combine_rows_kernel(SlotArgs a, Pieces pieces) {
  constexpr int P = kPiece<TR, TO>;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t t = pieces.row(i);
  if (t >= a.n_tok) return;
  const Piece c = piece_of<P>(i - t * pieces.n, a.hidden);
  float acc[P];
#pragma unroll
  for (int e = 0; e < P; ++e) acc[e] = 0.f;
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {
    const Slots<4> s = slots_of<4>(a, t, j0);
    float v[4][P];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s.r[j] >= 0) load_piece<TR, P, STREAM>(row_of<TR>(a.rows, s.r[j], a.ldr), c.at, c.left, v[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (s.r[j] >= 0) {
#pragma unroll
        for (int e = 0; e < P; ++e) acc[e] = acc[e] + s.w[j] * v[j][e];
      }
  }
  if (a.tok) {
    float v[P];
    load_piece<TO, P>(row_of<TO>(a.tok, t, a.ldt), c.at, c.left, v);
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = acc[e] + v[e];
  }
  char* out = row_of<TO>(a.out, t, a.ldo);
  if (c.twice == 0) {
    store_piece<TO, P>(out, c.at, c.left, acc);
  } else {
    // out may be the addend: what the piece before has it may have stored already, and the sum here is
    // then wrong; only the others are stored
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if (e >= c.twice) store_one<TO>(out, c.at + e, acc[e]);
    }
  }
}

// The wave's sum in every lane: within 16 lanes by DPP, across them by two exchanges.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(lane_move<CTRL>(__float_as_int(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += moved<0xB1>(v);   // lane ^ 1
  v += moved<0x4E>(v);   // lane ^ 2
  v += moved<0x141>(v);  // half rows mirrored
  v += moved<0x140>(v);  // rows mirrored
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// (Rows both read and written bound it: 3256 tokens of 2048, eight rows of 16 bits each, 47 us, 4.8 TB/s.)
// A workgroup per token: a lane takes every blockDim-th piece of the row, its part of dO and the rows of eight
// slots at once (dO once for every eight slots: twice where top_k is above eight); the slots' dots are summed over the lanes in a fixed order.
template <int TD, int TR, bool STREAM>
__global__ void __launch_bounds__(1024) combine_grad_kernel(SlotArgs a, uint32_t pieces) {
  constexpr int P = kPiece<TD, TR>;
  __shared__ float part[16][16];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const TokenSlots s(a, t);
  const int twice = pieces > 1 ? (int)(pieces * P - a.hidden) : 0;  // what a row's last piece shares with the one before
  const char* dout = row_of<TD>(a.tok, t, a.ldt);
  for (int j0 = 0; j0 < a.top_k; j0 += 8) {
    float dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = 0.f;
    for (uint32_t q = threadIdx.x; q < pieces; q += blockDim.x) {
      const Piece c = piece_of<P>(q, a.hidden);
      float d[P], v[8][P];
      load_piece<TD, P>(dout, c.at, c.left, d);
      if (a.dw) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = s.row(j0 + j);
          if (r >= 0) load_piece<TR, P, STREAM>(row_of<TR>(a.rows, r, a.ldr), c.at, c.left, v[j]);
        }
      }
      if (a.out) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = s.row(j0 + j);
          if (r < 0) continue;
          const float w = s.weight(j0 + j);
          float o[P];
#pragma unroll
          for (int e = 0; e < P; ++e) o[e] = scaled(w, d[e]);
          // (what two pieces have is written twice, the same)
          store_piece<TR, P, STREAM>(row_of<TR>(a.out, r, a.ldo), c.at, c.left, o);
        }
      }
      if (a.dw) {
        if (c.twice) {  // and counted once (both are zero: a zero times an infinity would not be)
#pragma unroll
          for (int e = 0; e < P - 1; ++e) {
            if (e >= twice) break;
            d[e] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j][e] = 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (s.row(j0 + j) >= 0) {
#pragma unroll
            for (int e = 0; e < P; ++e) dot[j] = fmaf(d[e], v[j][e], dot[j]);
          }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sum = wave_sum(dot[j]);
        if (lane == 0) part[wave][j0 + j] = sum;
      }
    }
  }
  if (!a.dw) return;
  __syncthreads();
  if ((int)threadIdx.x < a.top_k) {
    float s = part[0][threadIdx.x];
    for (int v = 1; v < (int)(blockDim.x >> 6); ++v) s = s + part[v][threadIdx.x];
    a.dw[t * a.top_k + threadIdx.x] = s;
  }
}

// Rows of at most 16 pieces: sixteen lanes a token (10000 tokens of 128, two rows each: 6.2 us; a wave a
// token 14).
template <int TD, int TR>
__global__ void __launch_bounds__(256) combine_grad_short_kernel(SlotArgs a, uint32_t pieces) {
  constexpr int P = kPiece<TD, TR>;
  const int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const uint32_t q = threadIdx.x & 15;
  const bool live = t < a.n_tok && q < pieces;  // (the others take part in the sums)
  const Piece c = piece_of<P>(live ? q : 0, a.hidden);
  float d[P];
#pragma unroll
  for (int e = 0; e < P; ++e) d[e] = 0.f;
  if (live) load_piece<TD, P>(row_of<TD>(a.tok, t, a.ldt), c.at, c.left, d);
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {
    Slots<4> s = slots_of<4>(a, t < a.n_tok ? t : 0, j0);
    float v[4][P];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (live && a.dw && s.r[j] >= 0) load_piece<TR, P>(row_of<TR>(a.rows, s.r[j], a.ldr), c.at, c.left, v[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float dot = 0.f;
      if (live && s.r[j] >= 0) {
        if (a.out) {
          float o[P];
#pragma unroll
          for (int e = 0; e < P; ++e) o[e] = scaled(s.w[j], d[e]);
          store_piece<TR, P>(row_of<TR>(a.out, s.r[j], a.ldo), c.at, c.left, o);
        }
        if (a.dw) {  // (what two pieces have is counted once)
#pragma unroll
          for (int e = 0; e < P; ++e) dot = e < c.twice ? dot : fmaf(d[e], v[j][e], dot);
        }
      }
      dot += moved<0xB1>(dot);
      dot += moved<0x4E>(dot);
      dot += moved<0x141>(dot);
      dot += moved<0x140>(dot);
      if (a.dw && q == 0 && t < a.n_tok && j0 + j < a.top_k) a.dw[t * a.top_k + j0 + j] = dot;
    }
  }
}

// Tokens go in as many launches of at most `most` as that takes.
template <typename F>
static int by_tokens(SlotArgs a, int64_t most, int in_type, int out_type, bool out_by_token, F launch) {
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

// The experts' rows pass the caches where they are too many for them (kStreamBytes): each is used once.
// The prompt's dispatch 22.0 us for 23.9, its gradient 47 for 54; 42 for 47 of float32 rows.
static bool streams(const SlotArgs& a, int rows_type) {
  return a.n_tok * a.top_k * a.hidden * type_bytes(rows_type) > kStreamBytes;
}

int launch_dispatch(const SlotArgs& a, int x_type, int rows_type, hipStream_t s) {
  const Pieces pieces(pieces_of(a.hidden, x_type, rows_type));
  // (written rows that do not begin on 16 bytes leave in parts: 2047 numbers of 16 bits 31 us for 27)
  const bool st = streams(a, rows_type) && aligned(a.out, 16) && a.ldo * type_bytes(rows_type) % 16 == 0;
  return by_tokens(a, rows_a_launch(pieces), x_type, rows_type, false, [&](const SlotArgs& b) {
    const dim3 grid((unsigned)((b.n_tok * pieces.n + 255) / 256));
#define IQ4_CALL(T1, T2)                                                                                 \
  if (st) hipLaunchKernelGGL((dispatch_kernel<T1, T2, true>), grid, dim3(256), 0, s, b, pieces);         \
  else hipLaunchKernelGGL((dispatch_kernel<T1, T2, false>), grid, dim3(256), 0, s, b, pieces)
    IQ4_TYPES(x_type, rows_type, IQ4_CALL)
#undef IQ4_CALL
    return check_launch("dispatch_kernel");
  });
}

int launch_combine_rows(const SlotArgs& a, int rows_type, int out_type, hipStream_t s) {
  const Pieces pieces(pieces_of(a.hidden, rows_type, out_type));
  const bool st = streams(a, rows_type);
  return by_tokens(a, rows_a_launch(pieces), out_type, out_type, true, [&](const SlotArgs& b) {
    const dim3 grid((unsigned)((b.n_tok * pieces.n + 255) / 256));
#define IQ4_CALL(T1, T2)                                                                                 \
  if (st) hipLaunchKernelGGL((combine_rows_kernel<T1, T2, true>), grid, dim3(256), 0, s, b, pieces);     \
  else hipLaunchKernelGGL((combine_rows_kernel<T1, T2, false>), grid, dim3(256), 0, s, b, pieces)
    IQ4_TYPES(rows_type, out_type, IQ4_CALL)
#undef IQ4_CALL
    return check_launch("combine_rows_kernel");
  });
}

int launch_combine_grad(const SlotArgs& a, int dout_type, int rows_type, hipStream_t s) {
  const uint32_t pieces = pieces_of(a.hidden, dout_type, rows_type);
  if (pieces <= 16)
    return by_tokens(a, ((int64_t)1 << 31) / 16, dout_type, rows_type, false, [&](const SlotArgs& b) {
      const dim3 grid((unsigned)((b.n_tok + 15) / 16));
#define IQ4_CALL(T1, T2) hipLaunchKernelGGL((combine_grad_short_kernel<T1, T2>), grid, dim3(256), 0, s, b, pieces)
      IQ4_TYPES(dout_type, rows_type, IQ4_CALL)
#undef IQ4_CALL
      return check_launch("combine_grad_kernel");
    });
  // waves a token: a wave per 64 pieces up to four, in rounds of four or of three, whichever fill the last one better
  // (5147 tokens of 2290 numbers of 16 bits, 287 pieces: 35 us with three, 40 with four; 3256 of 2048 59 and 47); up to
  // sixteen where the tokens alone would not fill the device (four tokens of 8192: 6.2 us, 12.9 with four)
  int waves = (int)((pieces + 63) / 64);
  if (pieces > 256 && a.n_tok <= 256) waves = waves < 16 ? waves : 16;
  else if (waves > 2) waves = (pieces + 191) / 192 * 192 < (pieces + 255) / 256 * 256 ? 3 : 4;
  const bool st = streams(a, rows_type);
  return by_tokens(a, ((int64_t)1 << 31) / (64 * waves), dout_type, rows_type, false, [&](const SlotArgs& b) {
    const dim3 grid((unsigned)b.n_tok);
#define IQ4_CALL(T1, T2)                                                                                         \
  if (st) hipLaunchKernelGGL((combine_grad_kernel<T1, T2, true>), grid, dim3(64 * waves), 0, s, b, pieces);      \
  else hipLaunchKernelGGL((combine_grad_kernel<T1, T2, false>), grid, dim3(64 * waves), 0, s, b, pieces)
    IQ4_TYPES(dout_type, rows_type, IQ4_CALL)
#undef IQ4_CALL
    return check_launch("combine_grad_kernel");
  });
}

}  // namespace iq4
