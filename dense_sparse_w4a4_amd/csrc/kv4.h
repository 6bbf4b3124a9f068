// The paged 4-bit key/value cache: its layout, shared by the kernel that
// writes it (kv4_append.hip) and the one that reads it (kv4_attn.hip).
//
// One page holds `page` tokens (a power of two, at least 32) of every
// key/value head.  A token's key (or value) of one head is D 4-bit codes u in
// 0..15 and one 32-bit word, the fp16 scale s in its low half and the fp16
// zero point z, a whole number, in its high half; the value held is s*(u + z).
//   kq  [pages][heads][page][D/2]           codes of a token side by side, low
//       nibble first: the 16 tokens x D tile that one score step reads is
//       contiguous, and a lane's D/4 channels of its token are one load.
//   vq  [pages][heads][page/4][D/8][4][4]   channel-major by 8 inside blocks of
//       four tokens: the four tokens x 8 channels that one lane feeds to the
//       matrix core as values are 16 contiguous bytes, and a token's bytes are
//       its own (no two tokens share one, so appending needs no read).
//   ksz, vsz  u32 [pages][heads][page]
#pragma once

#include "mq_internal.h"

namespace mq {

constexpr int kKv4Tile = 32;  // tokens of one wave step; divides every page

// Index of a token's word in ksz / vsz; its code row starts at D/2 times it.
__host__ __device__ inline int64_t kv4_row(int64_t page_index, int64_t head, int64_t offset, int64_t heads,
                                           int64_t page) {
  return (page_index * heads + head) * page + offset;
}

// Byte of channel 8*d8 of token `offset` of a page and head in vq, relative
// to that page and head's first byte.
__host__ __device__ inline int64_t kv4_v_byte(int64_t offset, int d8, int dim) {
  return ((offset >> 2) * (dim / 8) + d8) * 16 + (offset & 3) * 4;
}

struct Kv4Cache {
  uint8_t* kq;
  uint32_t* ksz;
  uint8_t* vq;
  uint32_t* vsz;
  int64_t pages;
  int page;   // tokens of a page, 1 << shift
  int shift;
  int heads;  // key/value heads
  int dim;
};

constexpr int kF16 = MQ_FP16, kBf16 = MQ_BF16;

__device__ __forceinline__ float bf2f(uint32_t b) { return __uint_as_float(b << 16); }
template <int DT>
__device__ __forceinline__ float to_f32(uint16_t b) {
  return DT == kF16 ? h2f(b) : bf2f(b);
}
// fp32 -> fp16 or bf16, round to nearest even (one instruction for two).
template <int DT>
__device__ __forceinline__ uint32_t from_f32(float f) {
  if constexpr (DT == kF16) return f2h_bits(f);
  else return __builtin_bit_cast(uint16_t, (__bf16)f);
}
template <int DT>
__device__ __forceinline__ void unpack16(const uint4& v, float f[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = to_f32<DT>((uint16_t)(w[i] & 0xFFFFu));
    f[2 * i + 1] = to_f32<DT>((uint16_t)(w[i] >> 16));
  }
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef _Float16 v2h __attribute__((ext_vector_type(2)));
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  if constexpr (DT == kF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{lo, hi}, v2h));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{lo, hi}, v2b));
}
template <int DT>
__device__ __forceinline__ uint4 pack16(const float f[8]) {
  return make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
}

typedef _Float16 v2half __attribute__((ext_vector_type(2)));
// Two codes (bits 0..3, or 4..7 when `high`, of each half) as fp16 u - 8.
// `magic`: 0x64006400 in a vector register (kv4_magic): the mask takes the one
// scalar operand of the and-or.
__device__ __forceinline__ uint32_t kv4_centred(uint32_t w, int high, uint32_t magic) {
  const v2half m = __builtin_bit_cast(v2half, (w & (high ? 0x00F000F0u : 0x000F000Fu)) | magic);
  const v2half f = high ? __builtin_elementwise_fma(m, v2half{0.0625f16, 0.0625f16}, v2half{-72.0f16, -72.0f16})
                        : m - v2half{1032.0f16, 1032.0f16};
  return __builtin_bit_cast(uint32_t, f);
}
__device__ __forceinline__ uint32_t kv4_magic(uint32_t bits) {
  uint32_t v;
  asm("v_mov_b32 %0, %1" : "=v"(v) : "s"(bits));  // opaque: stays a vector register
  return v;
}

}  // namespace mq

namespace mq {

struct Kv4AppendArgs {
  Kv4Cache c;
  const uint16_t *q, *k, *v;
  int64_t T, ldq, ldk, ldv;
  int q_heads;
  int dtype;
  const int64_t* slots;
  const int32_t* positions;
  const float* table;  // [n_pos][rot]: cosines then sines, or null
  int64_t n_pos;
  int rot;
  int interleaved;
  const uint16_t *wq, *wk;  // or null: no norm
  float eps;
  uint16_t* q_out;
  int64_t ldqo;
  uint16_t *k_out, *v_out;  // [T][heads][dim] or null
};
hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t st);

struct Kv4AttnArgs {
  Kv4Cache c;
  const uint16_t* q;
  int64_t T, ldq;
  int q_heads;
  int dtype;
  const int32_t* table;  // [seqs][ldt] page indexes
  int64_t seqs, ldt;
  int64_t max_pages;
  const int32_t* kv_len;  // [seqs]
  const int32_t* cu_q;    // [seqs + 1], or null: one query per sequence
  int causal;
  int window;  // 0: none
  float scale;
  uint16_t* out;
  int64_t ldo;
  float* lse;  // [T][q_heads] or null
  float* part;
};
// Workgroups of a launch: at most 2^24 - 1, 2^32 threads.
int64_t kv4_attn_groups(int64_t T, int64_t seqs, int q_heads, int kv_heads, int64_t max_q);
size_t kv4_attn_workspace(int64_t T, int64_t seqs, int q_heads, int kv_heads, int dim, int64_t max_q);
hipError_t launch_kv4_attn(const Kv4AttnArgs& a, int64_t max_q, hipStream_t st);

struct W4a16Args {
  const uint16_t* x;
  int dtype;
  int64_t M, N, K, ldx;
  const uint8_t* qw;
  const uint16_t* sw;
  int block, n_select;
  const int32_t *row_ptr, *col_idx;
  const uint8_t* qr;
  const uint16_t* sr;
  uint16_t* y;
  int64_t ldy;
  float* part;  // K splits' sums [splits][M][N]
};
size_t w4a16_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_w4a16(const W4a16Args& a, hipStream_t st);

}  // namespace mq
