// 1x1 (pointwise) layers as products of 8-bit floats with one scale per 128
// channels of a pixel and one per 128 x 128 weights: geometry and entry
// points (pointwise8.cu, pointwise8_tc.cu).
#pragma once

#include "act8.cuh"

namespace dwconv {
namespace pw8 {

constexpr int kBlock = 128;  // channels of a scale

// Validated geometry. y[p, yo + o] = act(sum_b sx[p, b] sw[o / 128, b] sum_{c in b} x[p, c] w[o, c] + bias[o])
struct Pw {
  int64_t rows;
  int cin, cout;
  int64_t pitch;    // distance of the weights' rows: cin rounded up to 128
  int64_t ys, yo;   // distance of y's rows, first channel
  int act, dtype;   // of y and bias
  int nkb;          // blocks of channels
};

inline int64_t pitch_of(int64_t cin) { return (cin + kBlock - 1) / kBlock * kBlock; }

enum class Plan { Row, Tile };
Plan plan(const Pw& g);
bool by_pairs(const Pw& g);  // Plan::Tile: by pairs of thread blocks
// rows of codes that are no multiple of 16 bytes are copied to rows that are
size_t workspace_bytes(const Pw& g);

cudaError_t encode_weights(int64_t cout, int64_t cin, bool transpose, int dtype, const void* w, uint8_t* codes,
                           float* scales, cudaStream_t s);
cudaError_t run(const Pw& g, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, const void* bias,
                void* y, void* ws, cudaStream_t s);

// pointwise8_tc.cu: x's rows ldx bytes apart, x, w and ldx on 16 bytes; copied:
// the launch before this one writes x. cudaErrorNotSupported where the tensor
// maps or the device refuse.
cudaError_t run_tc(const Pw& g, int64_t ldx, const uint8_t* x, bool copied, const float* sx, const uint8_t* w,
                   const float* sw, const void* bias, void* y, cudaStream_t s);

}  // namespace pw8
}  // namespace dwconv
