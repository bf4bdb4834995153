// mss_train.hpp -- shapes and pointers of the operations around the scans of a
// training step: layer norm and its backward, the losses over a vocabulary.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mss_head.hpp"

namespace mss {

struct LayerNormArgs {
  int64_t rows;
  int dim;
  int64_t sx, sr, so, sro;
  float eps;
  const void* x;
  const void* res;
  const float* weight;
  const float* bias;
  void* out;
  float* mean;
  float* rstd;
  void* res_out;
};

struct LayerNormBwdArgs {
  int64_t rows;
  int dim;
  int parts;  // workgroups, each with its own sums over its rows
  int64_t sdy, sr, sdr, sdx, sdres;
  const void* dy;
  const void* r;
  const void* dr;
  const float* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dres;
  float* dweight;
  float* dbias;
  float* sums;  // workspace [2][parts][dim]
};

hipError_t launch_layer_norm(const LayerNormArgs& a, bool io_bf16, bool res_bf16, hipStream_t stream);
int layer_norm_bwd_parts(int64_t rows, int64_t dim);
hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, bool io_bf16, bool r_bf16, hipStream_t stream);

// ---------------------------------------------------------------- losses

struct LossArgs {
  int rows, dim, vocab, entries;
  int64_t sx, sw, sids[2], steach[2], sdx, sdw;
  const void* x;
  const void* weight;
  const int64_t* ids;
  const void* teacher;  // null: cross entropy
  bool teacher_bf16;
  const float* row_weight;
  float inv_tau;   // 1 / temperature
  float scale;     // logit_scale / temperature: x.w to logits
  float back;      // logit_scale * temperature: dz's factor before c
  float tau2;      // temperature^2
  float* loss;
  float* lse;
  float* total;
  void* dx;
  void* dweight;
  // workspace
  int* live;       // [1] rows that count
  int* cuts;       // [pieces] parts of the vocabulary that a piece's dx product is cut into
  int* row_of;     // [rows] row of the i-th of them
  int* place;      // [rows] the i of a row, or -1
  uint8_t* counts; // [rows] whether it counts
  float* share;    // [rows][entries] t_k by row (teacher only)
  float* known;    // [rows] sum_k t_k log t_k (teacher only)
  int* near;       // [rows][entries] ids of the i-th row that counts, -1 for those that do not
  uint32_t* where; // [rows][where_words] the tiles that hold one of them, a bit each
  int where_words;
  float* picked;   // [rows][entries] their logits
  // Rows, weights and dz as bf16 operands of the products: one plane, or three
  // whose sum is the fp32 value.  They lie in panels, [columns / 64][rows][64] (32 in
  // place of 64 for dz, and for all of three planes), so that a tile's part of any
  // of them is one stretch of memory.
  int planes;
  bool direct;     // few rows of fp32: xp and dz are fp32, weights are read where they are
  int64_t dpad;    // columns of x and weight, a multiple of 64
  uint16_t* xp;    // [planes][dpad / 64][xrows][64]
  int64_t xrows;   // a multiple of 64; those behind the last row that counts, to the next 64, are 0
  uint16_t* wp;    // [planes][dpad / 64][vocab][64], or the weight itself
  bool pack_w;
  bool small_logits, small_dx, small_dw;  // small tiles of a product
  int vocab_tile;  // vocabulary entries that share a maximum
  int dw_blocks, dw_splits;  // workgroups of the dweight product, and the parts of the rows they are cut into
  bool dw_vecs;    // dweight's rows are whole aligned 16-byte vectors
  // of a piece of rows
  int piece;       // rows of a piece, a multiple of 64
  int pieces;
  int tiles;       // vocabulary tiles, whose entries share a maximum
  int64_t vpad;    // columns of dz, a multiple of 64
  float2* stats;   // [piece][tiles] the largest logit R and the sum of e^(z - R) without R's own 1
  float2* sums;    // [piece] `from` and c / sum, the row's sum of e^z being sum e^from
  void* probs;     // [piece / 64][vpad / 32][64][32] codes of the logits (bf16), or the logits (fp32; `direct`: then dz)
  uint16_t* dz;    // [planes][piece / 64][vpad / 32][64][32] (bf16: probs itself)
  float* value;    // [piece][entries] dz of the entries
  int2* fix;       // [piece] (bf16) id and what its dz lost by its rounding, as float bits; or id -1
  float* part;     // [splits][piece][dpad]
  int splits;      // at most
  float* dw_sum;   // [dw_splits][vocab][dpad] (more than one part or piece; null otherwise)
};

hipError_t launch_loss(const LossArgs& a, bool io_bf16, hipStream_t stream);
hipError_t launch_scale(const void* in, const float* factor, void* out, int64_t n, bool bf16,
                        hipStream_t stream);

}  // namespace mss
