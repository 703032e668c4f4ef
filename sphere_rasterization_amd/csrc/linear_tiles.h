// Products C[i][j] = sum over c of Q[i][c] P[j][c], with j the axis along which C is stored, and
// what is done to C on its way to memory (linear_tiles_kernels.h, a file for each type).
#pragma once
#include "linear_common.h"

// What happens to C: stored, or one layer's bias, activation, dropout and residual first, or stored
// from an operand's two parts of which the second's sums are multiplied by REST (fp16).
enum { OUT_STORE, OUT_LAYER, OUT_PARTS };

struct Operand {
  const void *p;                 // [outer][c] with c contiguous, or [c][outer] (transposed)
  int64_t stride;                // elements between rows of that array
  int64_t rest;                  // bytes from p to what p's rounding lost, an array of its own, or 0
};

struct ProductArgs {
  Operand q, p;
  int64_t I, J, K;               // rows and columns of C, length of the summed axis
  int64_t ti, tj;                // tiles along I and J
  int parts;                     // 2: Q or P comes in two parts, and the summed axis is gone through twice, first with
                                 // what the rounding lost
  int64_t axis, steps, per;      // stages of the summed axis, of all parts, and of one split
  void *c;
  int64_t cs;                    // row stride of C
  float scale;                   // of the sums, where C is stored as it is
  float *part;                   // [splits][I][J] sums where the summed axis is split, else unused
  int splits;
  LayerArgs layer;
};

// How a product is cut: the tile, and pieces of the summed axis that are added by a second
// launch where tiles alone do not fill the chip.
struct Cut {
  int tile;                      // index of the tile's shape
  int splits;
};
struct TileShape {
  int i, j;
};
constexpr TileShape TILES[3] = {{256, 256}, {128, 128}, {64, 128}};
Cut product_cut(int64_t I, int64_t J, int64_t K, int parts, int dtype);

// Products of few rows of Q are cut by columns of C (32, or where P lies transposed as many as
// 16 chunks hold); the axis only where those are too few to fill the chip and every wave keeps
// eight stages: 8 x 8192 by 8192 x 8192 bf16, P transposed, 33 us in 64 x 4 workgroups and 57 in 64.
constexpr int FEW = 16;
static inline int few_splits(int64_t J, int64_t K, bool pt, int dtype) {
  const int64_t e = dtype == SPLAT_F32 ? 4 : 8, side = pt ? 16 * e : 32, groups = (J + side - 1) / side;
  const int64_t most = (K + 4 * e - 1) / (4 * e) / 64, want = groups < 128 ? 256 / groups : 1, n = want < most ? want : most;
  return n < 1 ? 1 : (int)n;
}
static inline size_t product_part_bytes(int64_t I, int64_t J, int64_t K, int parts, int dtype) {
  if (I == 0 || J == 0) return 0;
  int n = product_cut(I, J, K, parts, dtype).splits;
  if (I <= FEW)
    for (int pt = 0; pt < 2; pt++) n = few_splits(J, K, pt, dtype) > n ? few_splits(J, K, pt, dtype) : n;
  return n > 1 ? ws_align(sizeof(float) * (size_t)n * I * J) : 0;
}

// qt, pt: whether Q and P lie transposed; not Q alone.
int launch_product_f32(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t stream);
int launch_product_f16(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t stream);
int launch_product_bf16(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t stream);
template <typename T>
static inline int launch_product(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t stream) {
  if constexpr (sizeof(T) == 4) return launch_product_f32(a, qt, pt, out, stream);
  else if constexpr (__is_same(T, f16_t)) return launch_product_f16(a, qt, pt, out, stream);
  else return launch_product_bf16(a, qt, pt, out, stream);
}
