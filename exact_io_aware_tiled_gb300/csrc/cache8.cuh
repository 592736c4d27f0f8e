// cache8.cuh -- arguments of the kernels on a paged cache of 8-bit codes.
#pragma once
#include "common.cuh"

namespace fa {

// New rows into the cache, or the cache's rows out of it: sequence b's row n, K/V head h, lies in page
// table[b][n / page], row n % page; codes at stride cs, scales [pages][Hkv].
struct Cache8Rows {
  int B, Hkv, T, d;            // T: new rows (append), rows of the output (read)
  int page, lg, pages, width;  // lg = log2(page)
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
  void* x[2];                  // k, v rows [B,Hkv,T,d]
  Strides xs[2];
  uint8_t* code[2];            // [pages,Hkv,page,d]
  Strides cs[2];               // b: page, h: head, n: row
  float* scale[2];
};

struct Cache8Args {
  int B, H, Hkv, T, G;         // G = H / Hkv
  int r, tile, tiles;          // rows of a K/V head (G T), rows of a tile (8, 16, 32 or 64), tiles
  int page, lg, pages, width, cap;   // cap = width * page
  int window, sinks;
  const void* q;
  void* o;
  Strides qs, os;
  float* lse;
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
  const float* ks;
  const float* vs;             // [pages][Hkv]
  float scale_log2;            // tau * log2(e)
  int* status;
  int* count;                  // [3 kCMax], cleared: pieces left of a group, and groups joined, of rows that were cut
  float2* stat;                // [2 kCMax][tile]: maximum (log2), sum
  float* part;                 // [2 kCMax][tile][D] unnormalised O
  int2* pre;                   // [B + 1] before each sequence: units of the line, sequences with keys, where the
                               // kernel does not sum them itself
};

constexpr int kCMax = 152 * 3;   // CTAs at most: a workspace's size does not depend on the device at hand
// Sequences whose units a CTA sums by itself, as many as its shared memory has room for: 300 sequences of up to 2,047
// keys took 133.5 us so (where 384 fit) and 135 with the kernel that sums them first.
constexpr int kPreMax = 192;

size_t cache8_workspace(const fa_cache8_params* p);
// mk, mv: 4-D byte maps (d, page, Hkv, pages) of the codes, boxes of d x min(page, 64 at d = 64, 32 at d = 128)
cudaError_t launch_cache8_fwd(int dtype, int d, const CUtensorMap& mk, const CUtensorMap& mv, Cache8Args a, uint8_t* ws,
                              cudaStream_t s);
cudaError_t launch_cache8_append(int dtype, const Cache8Rows& a, cudaStream_t s);
cudaError_t launch_cache8_read(int dtype, const Cache8Rows& a, cudaStream_t s);

}  // namespace fa
