// Arguments of the rotary kernels.
#pragma once
#include <cstdint>
#include "fa2_cache.cuh"

namespace fa2 {

constexpr int kRotThreads = 256;

// Rows of a [B][H][N][d] tensor of 16-bit floats with any strides (elements).
struct RowView {
  uint16_t* p;
  long long sb, sh, sn;
};

// What the kernels do to one of the two tensors (queries, keys).
struct RotarySide {
  RowView x;           // forward: input. Backward: the gradient of the output
  RowView src;         // backward with a norm: the forward's input
  RowView y;           // output, or the gradient of the input
  const void* weight;  // [d], or nullptr: no norm
  void* weight_grad;   // [d]
  int H;               // heads; 0: the tensor is absent
};

// CTAs of the backward with a norm, of queries and of keys. A big one has kRotBig times
// the work of a small one.
constexpr int kRotBig = 6;
struct RotarySplit {
  int big_q, big_k, small_q, small_k;
};

struct RotaryArgs {
  RotarySide q, k;
  const double* freqs;   // [r / 2], radians per position
  const int* positions;  // by pos_mode
  int pos_mode;          // 0: token n of every sequence is at n; 1: at positions[b] + n; 2: at positions[b][n]
  int B, N;
  int r;                 // turned elements of a head
  int interleaved;
  int weight_fp32;       // weights are fp32, else of the tensors' type
  float eps, amplitude;
  float sign;            // -1 turns back
  long long tokens;      // B * N
  FastDiv fT, fN;
  int chunk, chunks;     // heads per work item; items per token
  int chunks_q;          // of them with queries (backward with a norm: no item has both)
  float* part;           // workspace, backward with a norm: [CTAs][d] sums of the weights' gradients
};

}  // namespace fa2
