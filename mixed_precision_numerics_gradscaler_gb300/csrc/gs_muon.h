// gs_muon.h -- the tables of a list of matrices updated by their orthogonalised
// momentum, and the launcher of the update.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gs {

constexpr int kMuonTile = 256;               // rows of a product's tile; its columns are these or half
constexpr int64_t kMuonChunk = 4096;         // elements of an element-wise step's CTA
constexpr int kMuonMaps = 6;                 // tensor maps of a matrix by one box: x, gram, poly, x_lo

// One matrix [rows, cols]; s = min, l = max of the two.  The products' operands
// are fp16 times a power of two each: x by sx, gram and poly by sa and sa / 4.
struct MuonMat {
  float* w;
  uint16_t* wb;              // bf16 copy, or null
  const void* g;
  float* m;
  uint16_t* x[2];            // [rows, ldx], in turns
  uint16_t* x_lo[2];         // what fp16 leaves of x, in fp16
  uint16_t *gram, *poly;     // [s, lds]
  int rows, cols, s, ldx, lds;
  int tall;                  // rows > cols
  float sx, sa;
  int64_t first_chunk;       // of the list's chunks of elements
  int first_sym, first_app;  // of the list's tiles of either kind of product
  int syms, apps;            // this matrix's tiles of either kind
};

struct MuonTable {
  const MuonMat* mats;
  const CUtensorMap* maps;   // per matrix: x[0], x[1], gram, poly, x_lo[0], x_lo[1] by 64 x 64, then by 32 x 64
  double* partials;          // one per chunk
  unsigned int* arrived;     // per matrix, 0 between calls
  unsigned int* done;        // per matrix: warps' parts of tiles (16 each) stored by the call's products
  float* factor;             // per matrix: sx / |u|
  int n;
  int64_t chunks;
  int sym_tiles, app_tiles;
  int tile_n;                // columns of a tile
};

struct MuonArgs {
  float lr, mu, weight_decay, max_norm;
  int nesterov, steps, scale_mode, grad_dtype;
  const float* grad_norm;
  const int32_t* found_inf;
  int32_t* status;
  int stall;
};

// A tensor map of an fp16 matrix [rows, cols] with row distance ld, boxes of
// box_rows x 64 in the 128-byte swizzle.
bool muon_encode(CUtensorMap* map, uint16_t* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);
cudaError_t launch_master_update_muon(const MuonTable& t, const MuonArgs& a, cudaStream_t st);

}  // namespace gs
