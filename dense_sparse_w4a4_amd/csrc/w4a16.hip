// The packed layer (dense 4-bit base + block-sparse 4-bit residual) on
// unquantised activations, for decoding batches:
//   y[m][n] = sum_j sw[n][j] sum_{k in group j} x[m][k] qw[n][k]
//           + sum_{selected blocks i of n's row} sr_i[n] sum_c x[m][kt_i b + c] qr_i[n][c]
// with fp16 or bf16 x and fp32 sums: the layer for projections whose
// activations do not bear 4 bits, from the same packed weights.
//
// Codes to matrix operands.  A two's-complement code q becomes u = q + 8 (one
// XOR of the word's sign bits), and u is AND-ed out of the word in place and
// OR-ed under an exponent that makes it a number:
//   fp16: 1024 + u (or 1024 + 16u one nibble higher), from which one packed
//         operation on two codes takes 1032 (or a sixteenth, then 72): q
//         exactly, 10 instructions per 8 codes
//   bf16, which has no packed arithmetic: (128 + u) 2^-15; the surplus of 136
//         2^-15 times the token's sum of x over the group enters as the
//         accumulator's start, one chain of products of x with the constant
//         -136 2^-15 per group, shared by all channels of the workgroup.  The
//         terms are up to 18 times the codes' own, and so is the rounding of
//         their fp32 sums (some 2^-17 of sum |x| times the largest code in a
//         group, against the output's 2^-9).  2^-15 keeps the sums of any finite
//         x finite: 128 inputs times 143 2^-15 at most.  Small x loses nothing by
//         it: the matrix core keeps subnormal products
// The group's scale (for bf16, times 2^15) is applied to the fp32 group sum, never
// rounded into a weight.
//
// Mapping: as the streaming kernel of the 4-bit route (slab layout: a group
// of 16 channels is 1 KB contiguous and lane (r, c) holds channel r's 32
// inputs 32c .. 32c+31): NS slabs x 16 MT tokens per workgroup, the K groups
// split into contiguous runs over KS waves, which join through LDS in wave
// order.  A lane's eight inputs of an operand are taken in the order 0, 4, 1,
// 5, 2, 6, 3, 7 that the codes leave their word in; x is permuted to match
// once per group, shared by the slabs.
//
// Bound by the weights' bytes for few tokens (N K/2, read once per 16 MT
// tokens).  For many no unit is full: a wave has few groups, so that the start,
// the residual and the join weigh as much as its stream, and four token tiles with
// four slabs spill some registers.  A tenth of the blocks as residual: 1 token
// 4096->4096 5.9 us (9.6 MB, 1.6 TB/s: a launch and one round of loads); 4 tokens
// 4096->14336 12.2 us (33.6 MB, 2.7 TB/s); 16 tokens 5120->25600 (bf16) 21 us (75
// MB, 3.6 TB/s); 50 tokens 25600->5120 45 us (78 MB and 14.4 GFLOP: 1.7 TB/s, 320
// TFLOP/s; vector unit issuing 37% of the time, matrix core busy 21%); these with
// two layers in turn, the weights partly in the last-level cache; with six in
// turn, from memory, in a graph: 6.7, 12.3, 27.5 (fp16) and 49.6 us.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "kv4.h"

namespace mq {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
// (a plain vector: copies of the uint4 class from memory to LDS go through scratch)
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ v4f mfma_x(const uint4& a, const uint4& b, v4f c) {
  if constexpr (DT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

// Eight two's-complement codes of a word, in the order 0, 4, 1, 5, 2, 6, 3, 7:
// fp16 q, or bf16 (136 + q) 2^-15.
template <int DT>
__device__ __forceinline__ uint4 code_operand(uint32_t w, uint32_t magic) {
  constexpr uint32_t m = 0x000F000Fu;
  w ^= 0x88888888u;
  if constexpr (DT == kF16) {
    const uint32_t h = w >> 8;
    return make_uint4(kv4_centred(w, 0, magic), kv4_centred(w, 1, magic), kv4_centred(h, 0, magic),
                      kv4_centred(h, 1, magic));
  } else {
    return make_uint4((w & m) | magic, ((w >> 4) & m) | magic, ((w >> 8) & m) | magic, ((w >> 12) & m) | magic);
  }
}
// Eight inputs in the same order.
__device__ __forceinline__ uint4 order_x(const v4u& x) {
  return make_uint4(__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                    __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u));
}
// bf16: the constant -136 2^-15 that takes the codes' surplus back out.
__device__ __forceinline__ uint4 surplus_operand() {
  constexpr uint32_t c = 0xBB88BB88u;
  return make_uint4(c, c, c, c);
}

// f(0), f(1), ... with constant arguments, while they return true.
template <int... I, typename F>
__device__ __forceinline__ bool in_turn(std::integer_sequence<int, I...>, F f) {
  return (f(std::integral_constant<int, I>{}) && ...);
}

// One residual block's operands of a lane (entry e of the CSR).
template <int BLK, int NS, int MT>
struct Residual {
  uint4 W[NS];
  v4u X[MT][BLK / 32];
  uint16_t S[NS];
};

// Up to 16 MT tokens.  The weight codes of several groups are in flight per
// wave, in buffers that take turns, x one group ahead; loads past a wave's run
// read its last group again (with scale 0), so that every step issues the same
// loads and no wait covers a later one's.  The scales of the workgroup's
// channels are staged in LDS once.
//
// XL: x through LDS.  An operand's lanes take 16 bytes from each of 16 rows, 64
// pieces of as many cache lines; instead each load takes 256 contiguous bytes
// of four rows, and the wave's own LDS turns rows into operands (piece p of row
// r at place p ^ r, free of bank conflicts either way).  With up to four tokens
// the operand's own loads touch no more lines (rows past M read row M - 1), and
// the detour costs more than it saves.
//
// gridDim.z > 1: the K groups are split over that many workgroups, which leave
// fp32 sums in a.part for w4a16_sum_kernel.
template <int DT, int BLK, int KS, int NS, int MT, bool XL>
__global__ __launch_bounds__(64 * KS) void w4a16_kernel(W4a16Args a) {
  static_assert(16 * NS <= BLK, "the slabs of a workgroup lie in one block row");
  constexpr int CW = 16 * NS;
  constexpr int DEPTH = 2;                // groups' weights in flight
  constexpr int XD = MT == 1 ? DEPTH : 1;  // and x's (as many: loads return in order)
  extern __shared__ __align__(16) unsigned char smem[];
  const int G = (int)(a.K / kGroup);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  uint16_t* const sw = reinterpret_cast<uint16_t*>(smem);                              // [CW][G]
  v4u* const xs = reinterpret_cast<v4u*>(smem + CW * G * 2) + wave * (MT * 256);   // XL: [MT][16][16]
  float(*const red)[16][CW + 1] = reinterpret_cast<float(*)[16][CW + 1]>(smem);        // after the streams
  const int r = lane & 15, ch = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * CW;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int runs = KS * (int)gridDim.z, run = (int)blockIdx.z * KS + wave;  // runs <= G: at least one group each
  const int gb = (int)((int64_t)run * G / runs), ge = (int)((int64_t)(run + 1) * G / runs);

  const uint8_t* const wp = a.qw + n0 * (a.K / 2) + lane * 16;  // group j of slab s at j * 1024 + s * 8 * K
  auto row_of = [&](int i) {  // rows past M read row M - 1 (computed, never stored)
    const int64_t m = m0 + i;
    return a.x + (m < a.M ? m : a.M - 1) * a.ldx;
  };
  const uint16_t* xp[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) xp[t] = row_of(16 * t + r);
  const uint32_t magic = kv4_magic(DT == kF16 ? 0x64006400u : 0x3B803B80u);

  v4f y[MT][NS];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s) y[t][s] = v4f{0.f, 0.f, 0.f, 0.f};

  // ND operand words per slab: y += scale * (x . codes); x(t, j): eight inputs
  auto item = [&](auto nd, const uint4* W, auto x, auto scale) {
    constexpr int ND = decltype(nd)::value;
    uint4 xo[MT][ND];
    v4f c0[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      c0[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < ND; ++j) {
        xo[t][j] = order_x(x(t, j));
        if constexpr (DT == kBf16) c0[t] = mfma_x<DT>(xo[t][j], surplus_operand(), c0[t]);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint32_t w[4] = {W[s].x, W[s].y, W[s].z, W[s].w};
      v4f acc[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = c0[t];
#pragma unroll
      for (int j = 0; j < ND; ++j) {
        const uint4 c = code_operand<DT>(w[j], magic);
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = mfma_x<DT>(xo[t][j], c, acc[t]);
      }
      const float sc = DT == kBf16 ? scale(s) * 0x1p15f : scale(s);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[t][s][i] = fmaf(acc[t][i], sc, y[t][s][i]);
    }
  };

  // ---- the scales' loads first, then the first groups', then the residual's
  // first block's (whose address takes two dependent loads) ----
  constexpr int SMAX = MT > 1 ? 4 : 2;  // 16-byte pieces of the scales issued ahead, per thread
  const uint4* const sg = reinterpret_cast<const uint4*>(a.sw + n0 * G);
  const int pieces = CW * G / 8;
  uint4 sv[SMAX];
#pragma unroll
  for (int k = 0; k < SMAX; ++k) sv[k] = sg[min((int)threadIdx.x + k * 64 * KS, pieces - 1)];

  // Row ranges are clipped to [0, n_select] and a block column outside
  // [0, K/BLK) counts with scale 0, so a corrupt CSR is never read out of
  // bounds.  The CSR is read through the scalar cache: its waits never involve
  // the vector loads in flight.
  typedef const __attribute__((address_space(4))) int32_t* cint_p;
  constexpr int ND = BLK / 32;
  const int nt = (int)(n0 / BLK), rrow = (int)(n0 - (int64_t)nt * BLK) + r;
  int p0 = 0, p1 = 0;
  if (a.n_select > 0) {
    p0 = min(max(((cint_p)a.row_ptr)[nt], 0), a.n_select);
    p1 = min(max(((cint_p)a.row_ptr)[nt + 1], p0), a.n_select);
  }
  // entry e (none from p1 on: group 0's words, with scale 0); lane chunk c
  // holds inputs c*BLK/4 .. of the block
  auto residual = [&](Residual<BLK, NS, MT>& R, int e) {
    const bool has = e < p1;
    const int kt = has ? ((cint_p)a.col_idx)[e] : -1;
    const bool ok = kt >= 0 && kt < (int)(a.K / BLK);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const uint8_t* const q =
          ok ? a.qr + ((int64_t)e * BLK + rrow + 16 * s) * (BLK / 2) + ch * (BLK / 8) : a.qw;
      if constexpr (ND == 4) R.W[s] = *reinterpret_cast<const uint4*>(q);
      else if constexpr (ND == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(q);
        R.W[s] = make_uint4(v.x, v.y, 0, 0);
      } else R.W[s] = make_uint4(*reinterpret_cast<const uint32_t*>(q), 0, 0, 0);
      const uint16_t sc = *(ok ? a.sr + (int64_t)e * BLK + rrow + 16 * s : a.sw);
      R.S[s] = ok ? sc : (uint16_t)0;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < ND; ++j)
        R.X[t][j] = *reinterpret_cast<const v4u*>(xp[t] + (int64_t)(ok ? kt : 0) * BLK + ch * (BLK / 4) + 8 * j);
  };
  auto residual_item = [&](const Residual<BLK, NS, MT>& R) {
    item(std::integral_constant<int, ND>{}, R.W, [&](int t, int j) { return R.X[t][j]; },
         [&](int s) { return h2f(R.S[s]); });
  };

  struct Codes {
    uint4 W[NS];
  };
  struct Acts {
    v4u X[MT][4];
  };
  auto fetch_w = [&](Codes& g, int j) {
    const int jj = min(j, ge - 1);
#pragma unroll
    for (int s = 0; s < NS; ++s)
      g.W[s] = *reinterpret_cast<const uint4*>(wp + (int64_t)jj * 1024 + (int64_t)s * 8 * a.K);
  };
  auto fetch_x = [&](Acts& g, int j) {
    const int jj = min(j, ge - 1);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        g.X[t][i] = *reinterpret_cast<const v4u*>((XL ? row_of(16 * t + 4 * i + ch) + 8 * r : xp[t] + 32 * ch + 8 * i) +
                                                    (int64_t)jj * kGroup);
  };
  Codes W[DEPTH];
  Acts X[XD];
  if constexpr (XD == 1) fetch_x(X[0], gb);
  in_turn(std::make_integer_sequence<int, DEPTH - 1>{}, [&](auto turn) {
    constexpr int d = decltype(turn)::value;
    if constexpr (XD > 1) fetch_x(X[d], gb + d);
    fetch_w(W[d], gb + d);
    return true;
  });
  Residual<BLK, NS, MT> R;
  int e = p0 + run;  // the entry in R
  if constexpr (MT == 1) residual(R, e);

#pragma unroll
  for (int k = 0; k < SMAX; ++k)
    if ((int)threadIdx.x + k * 64 * KS < pieces) reinterpret_cast<uint4*>(sw)[threadIdx.x + k * 64 * KS] = sv[k];
  for (int i = (int)threadIdx.x + SMAX * 64 * KS; i < pieces; i += 64 * KS)  // long K only
    reinterpret_cast<uint4*>(sw)[i] = sg[i];
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // group j; with one buffer for x, group j + 1's is loaded as soon as LDS has
  // group j's
  auto group = [&](const Codes& w, Acts& x, int j) {
    const auto scale = [&](int s) {
      const float sc = h2f(sw[(16 * s + r) * G + min(j, ge - 1)]);
      return j < ge ? sc : 0.0f;
    };
    if constexpr (XL) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 4 * i + ch;
          xs[t * 256 + rr * 16 + (r ^ rr)] = x.X[t][i];
        }
      if constexpr (XD == 1) fetch_x(x, j + 1);
      item(std::integral_constant<int, 4>{}, w.W,
           [&](int t, int jj) { return xs[t * 256 + r * 16 + ((4 * ch + jj) ^ r)]; }, scale);
    } else {
      item(std::integral_constant<int, 4>{}, w.W, [&](int t, int jj) { return x.X[t][jj]; }, scale);
    }
  };
  for (int j = gb;; j += DEPTH) {
    const bool more = in_turn(std::make_integer_sequence<int, DEPTH>{}, [&](auto turn) {
      constexpr int d = decltype(turn)::value, ahead = (d + DEPTH - 1) % DEPTH;
      if constexpr (XD > 1) fetch_x(X[ahead], j + d + DEPTH - 1);
      fetch_w(W[ahead], j + d + DEPTH - 1);
      group(W[d], X[XD > 1 ? d : 0], j + d);
      return j + d + 1 < ge;
    });
    if (!more) break;
    if constexpr (MT == 1) {  // a residual block every DEPTH groups, the next in flight
      if (e < p1) residual_item(R);
      e += runs;
      residual(R, e);
    }
  }
  if constexpr (MT > 1) residual(R, e);
  for (; e < p1; e += runs) {
    residual_item(R);
    residual(R, e + runs);
  }

  // ---- join the waves, in wave order: one pass through LDS ----
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave * MT + t][4 * ch + i][16 * s + r] = y[t][s][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * MT * CW; i += 64 * KS) {
    const int row = i / CW, n = i - row * CW;
    const int64_t m = m0 + row;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < KS; ++w) sum += red[w * MT + row / 16][row % 16][n];
    if (m < a.M) {
      if (gridDim.z > 1) a.part[((int64_t)blockIdx.z * a.M + m) * a.N + n0 + n] = sum;
      else a.y[m * a.ldy + n0 + n] = (uint16_t)from_f32<DT>(sum);
    }
  }
}

// Sums the K splits in their order, four outputs per thread.
template <int DT>
__global__ __launch_bounds__(256) void w4a16_sum_kernel(W4a16Args a, int splits) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= a.M * a.N) return;  // N is a multiple of 32: the four are of one row
  float4 v = *reinterpret_cast<const float4*>(a.part + i);
  for (int z = 1; z < splits; ++z) {
    const float4 u = *reinterpret_cast<const float4*>(a.part + z * a.M * a.N + i);
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  const int64_t m = i / a.N;
  *reinterpret_cast<uint2*>(a.y + m * a.ldy + (i - m * a.N)) = make_uint2(pack2<DT>(v.x, v.y), pack2<DT>(v.z, v.w));
}

// Launch shape: token tiles and slabs per workgroup, waves, K splits.  Figures
// are times of one call in a graph, weights from memory, fp16, a tenth of the
// blocks as residual.
struct Plan {
  int mt, ns, ks, splits;
  bool xl;
};
size_t lds_bytes(int64_t K, const Plan& p) {
  const size_t stage = (size_t)(16 * p.ns) * (size_t)(K / kGroup) * 2 + (p.xl ? (size_t)p.ks * p.mt * 4096 : 0);
  return std::max(stage, (size_t)p.ks * p.mt * 16 * (16 * p.ns + 1) * 4);
}
Plan plan_of(int64_t M, int64_t N, int64_t K, int block) {
  const int64_t groups = K / kGroup;
  const bool four = block >= 64 && N % 64 == 0;
  Plan p;
  // x through LDS from 5 tokens on: 16 tokens 4096->14336 12.5 us against 16.5,
  // 25600->5120 48 against 66; 4 tokens the same, 2 tokens 12.1 against 11.5.
  p.xl = M > 4;
  p.splits = 1;
  // As many tokens as a workgroup can hold: the weights are read and unpacked
  // once for them (64 tokens 5120->25600: 57 us, 61 with two tiles or one;
  // 4096->14336: 24.6, 27.5, 29).
  p.mt = M > 32 ? 4 : M > 16 ? 2 : 1;
  auto tiles = [&](int ns) { return N / (16 * ns) * ((M + 16 * p.mt - 1) / (16 * p.mt)); };
  // K groups over several workgroups of eight waves, every wave keeping four.
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(256 / tiles(4 * four + 2 * !four), groups / 32));
  if (four && groups >= 16 && (p.mt > 1 || (M > 4 && tiles(4) < 256)) && tiles(4) * splits >= 128) {
    // Four slabs (64 channels; x once for all) and eight waves, where that, with
    // K split, still has work for half the compute units: 16 tokens 25600->5120,
    // three splits: 28.5 us, 48 with one slab and no split; 64 tokens
    // 5120->10240, 160 workgroups: 27 us, 37 without.  With fewer than two groups
    // per wave the other way: 50 tokens 1024->8192 11.3 us with, 8.8 without;
    // 64 tokens 2048->14336 17.3 and 18.9.
    p.ns = 4;
    p.ks = 8;
    if (tiles(4) < 256) p.splits = (int)splits;
  } else {
    // A small or shallow layer: one token tile per workgroup (33 tokens
    // 4096->4096: 11.3 us, 14.5 with four; the second tile finds the weights in
    // cache).
    if (tiles(2) < 256 || groups < 16) p.mt = 1;
    // Four slabs, two or one, as the grid still spans every compute unit: 4
    // tokens 4096->14336 12.0 us with two, 14.5 with one; 5120->25600 25.3 with
    // four or two, 30.6 with one.
    p.ns = four && tiles(4) >= 256 ? 4 : tiles(2) >= 256 ? 2 : 1;
    // Eight waves while every one has four groups and the grid stays within one
    // resident round, else four: 2 tokens 4096->14336 11.5 us against 12.5, 16
    // tokens 4096->4096 7.4 against 9.1; with four slabs (fewer waves fit) 8
    // tokens 5120->25600 27.4 with eight, 25.3 with four.
    p.ks = groups >= 32 && p.ns < 4 && tiles(p.ns) * 8 <= 4096 ? 8 : 4;
  }
  if (groups < p.ks) p.ks = groups < 4 ? 1 : 4;
  // long K: the scales and x have to fit 160 KB
  while (p.ns > 1 && lds_bytes(K, p) > 160 * 1024) p.ns /= 2;
  if (lds_bytes(K, p) > 160 * 1024) p.ks = 4;
  return p;
}

template <int DT, int BLK, int KS, int NS, int MT, bool XL>
hipError_t launch_cfg(const W4a16Args& a, const Plan& p, hipStream_t st) {
  const size_t lds = lds_bytes(a.K, p);
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(w4a16_kernel<DT, BLK, KS, NS, MT, XL>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)(a.N / (16 * NS)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)), (unsigned)p.splits);
  hipLaunchKernelGGL((w4a16_kernel<DT, BLK, KS, NS, MT, XL>), grid, dim3(64 * KS), lds, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL((w4a16_sum_kernel<DT>), dim3((unsigned)((a.M * a.N / 4 + 255) / 256)), dim3(256), 0, st, a,
                     p.splits);
  return hipGetLastError();
}
template <int DT, int BLK, int NS, int MT, bool XL>
hipError_t launch_ks(const W4a16Args& a, const Plan& p, hipStream_t st) {
  if constexpr (XL || NS < 4) {  // up to four tokens four slabs go with four waves
    if (p.ks == 8) return launch_cfg<DT, BLK, 8, NS, MT, XL>(a, p, st);
  }
  if constexpr (MT == 1) {  // short K takes one token tile
    if (p.ks == 1) return launch_cfg<DT, BLK, 1, NS, MT, XL>(a, p, st);
  }
  return launch_cfg<DT, BLK, 4, NS, MT, XL>(a, p, st);
}
template <int DT, int BLK, int MT, bool XL>
hipError_t launch_ns(const W4a16Args& a, const Plan& p, hipStream_t st) {
  if constexpr (BLK >= 64) {
    if (p.ns == 4) return launch_ks<DT, BLK, 4, MT, XL>(a, p, st);
  }
  if (p.ns == 2) return launch_ks<DT, BLK, 2, MT, XL>(a, p, st);
  return launch_ks<DT, BLK, 1, MT, XL>(a, p, st);
}
template <int DT, int BLK>
hipError_t launch_blk(const W4a16Args& a, hipStream_t st) {
  const Plan p = plan_of(a.M, a.N, a.K, BLK);
  if (p.mt == 4) return launch_ns<DT, BLK, 4, true>(a, p, st);
  if (p.mt == 2) return launch_ns<DT, BLK, 2, true>(a, p, st);
  if (p.xl) return launch_ns<DT, BLK, 1, true>(a, p, st);
  return launch_ns<DT, BLK, 1, false>(a, p, st);
}
template <int DT>
hipError_t launch_dt(const W4a16Args& a, hipStream_t st) {
  switch (a.block) {
    case 32: return launch_blk<DT, 32>(a, st);
    case 64: return launch_blk<DT, 64>(a, st);
    default: return launch_blk<DT, 128>(a, st);
  }
}

}  // namespace

size_t w4a16_workspace(int64_t M, int64_t N, int64_t K) {
  // whatever the residual block edge
  const int s = std::max(plan_of(M, N, K, 32).splits, plan_of(M, N, K, 64).splits);
  return s == 1 ? 0 : (size_t)s * (size_t)M * (size_t)N * sizeof(float);
}

hipError_t launch_w4a16(const W4a16Args& a, hipStream_t st) {
  return a.dtype == kF16 ? launch_dt<kF16>(a, st) : launch_dt<kBf16>(a, st);
}

}  // namespace mq
