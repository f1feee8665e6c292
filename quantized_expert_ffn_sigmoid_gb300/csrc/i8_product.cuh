// Parameters and workspace of the products of 8-bit codes.
#pragma once
#include "mx4_common.cuh"

namespace colimoe {

struct I8Params {
  const int8_t* x;            // activation codes, X rows of pitch ldx
  long long ldx;
  const float* xs;            // [X]
  int X;
  const int32_t* rows;        // [P] activation row of each row of y; null: the row itself
  int P;
  const int8_t* w;            // weight codes: group g at g * wgroup, its rows of pitch ldw
  long long ldw, wgroup;
  const float* ws_;           // their scales: group g at g * wsgroup
  long long wsgroup;
  int G, N, K;
  const int32_t* offsets;     // [G + 1], or null (one group)
  void* y;
  int32_t y_type;
  long long ldy;
  uint8_t* ws;                // status word at 0
};

// The streaming kernel takes up to 4 rows, and up to 8 of several groups, which
// are most often one or two a group: 4096 x 6144 against 4 rows 11 us (13 on the
// tensor cores), against 6 rows of one group 16 (13)
constexpr int I8_FEW = 8;
inline bool i8_few(int P, int G) { return P <= (G > 1 ? I8_FEW : 4); }

// Workspace behind the header, whose words but the status are other operators': a
// word for each CTA that widens activations, a count for each tile of split sums,
// the scales of the rows of y, 128 times the sums of their codes, fp16 copies of
// their activation rows padded to kp codes.
constexpr int I8_WIDEN_CTAS = 1280;
constexpr int I8_SPLIT_TILES = 80;
constexpr size_t I8_OFF_PARTS = WS_HEADER_BYTES + 4 * I8_WIDEN_CTAS;
inline long long i8_kp(int K) { return ((long long)K + 63) / 64 * 64; }
inline size_t i8_off_xs() { return I8_OFF_PARTS + 4 * I8_SPLIT_TILES; }
inline size_t i8_off_xb(int P) { return align_up(i8_off_xs() + 8 * (size_t)P, 256); }
inline size_t i8_off_part(int P, int K) { return align_up(i8_off_xb(P) + 2 * (size_t)P * (size_t)i8_kp(K), 256); }
// then split sums: tiles of 128 weight rows
inline size_t i8_ws_bytes(int P, int K) { return i8_off_part(P, K) + (size_t)I8_SPLIT_TILES * (P <= 32 ? 32 : 64) * 512; }

// First row of group g: offsets clamped to [0, P]; ascending by running maximum
__device__ __forceinline__ int i8_offset(const I8Params& A, int g) { return A.offsets ? min(max(__ldcg(A.offsets + g), 0), A.P) : g * A.P; }

// One element of y: the integer sum, then the scales, in fp32
__device__ __forceinline__ float i8_value(int sum, float sx, float sw) { return __int2float_rn(sum) * sx * sw; }

cudaError_t launch_i8_stream(const I8Params& A, cudaStream_t st);
cudaError_t launch_i8_gemm(const I8Params& A, cudaStream_t st);

}  // namespace colimoe
