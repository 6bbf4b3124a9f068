// Attention over the paged 4-bit key/value cache (layout: kv4.h):
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q.k_t) over the visible t.
// With k = s_k (u + z_k) and v = s_v (u + z_v), u the 4-bit codes,
//   q.k_t = s_k (q.u + z_k * sum(q)),   sum_t p_t v_t = sum_t (p_t s_v)(u + z_v),
// so both products run on the codes themselves and every scale is one factor
// per token: no cached value is ever dequantised.
//
// Codes to matrix operands.  Keys: a code shifted to bits 4..7 of an fp16 is
// the subnormal u * 2^-20, which V_MFMA_F32_16X16X32_F16 takes: 7 instructions
// per 8 codes, no conversion.  The power of two is undone in the fp32 scores.
// (The matrix core does not normalise such operands, so their leading zeros are
// lost below the products: two bits here.  With the even codes left in bits
// 0..3, 5 instructions, six bits were, and the scores' error was 1.8e-6 of
// their maximum.)  Queries are scaled per row by a power of two to |q| < 2^11
// first, so that bf16 queries fit fp16 too.
// Values: the same would leave a long context's small mean as the difference
// of two large sums (measured 3x the error of fp32 softmax at 131075 tokens),
// so they are centred: OR-ed under the exponent of 1024 the code is 1024 + u
// (or 1024 + 16u), and one packed operation on two codes makes it u - 8,
// exactly; the zero points' sum takes z + 8, as two fp16 whole numbers (its nearest
// and the rest, 0 for |z| <= 2040) in different rows of one product.
//
// Operand layout.  Scores are computed transposed, S^T = K Q^T (A: 16 tokens,
// B: 16 query columns), so that lane (r = lane % 16, c = lane / 16) receives
// column r's scores of tokens 4c .. 4c+3 of each 16: exactly the lane and
// order in which the second product O^T = V^T P^T takes them as its B operand
// when a 32-token step's k index is (token 4c+i, token 16+4c+i).  The weights
// go from one product to the next in registers, no LDS, no lane exchange.
//
// Softmax.  Running maximum m and sum l per lane in fp32, for the lane's own
// tokens of its column; m is shared by the column's four lanes and raised only
// when a score passes it by 2^6 (a rare branch), so the common step has no lane
// exchange.  The weights w = p * s_v are rounded to fp16 for the matrix core
// (to nearest); the zero points' sum (of w (z_v + 8)) is one more product with
// the same rounded w, so that rounding scales v and not its offset.  w is kept
// in fp16's normal range by a power of two of the column's own, which follows the
// largest w that the column has seen: not the largest s_v, since a token that the
// column does not see, or whose weight is next to nothing, would push the weights
// that count into fp16's subnormals.  l sums the unrounded p.
#include <algorithm>

#include "kv4.h"

namespace mq {

// a * b with 0 * anything = 0, NaN and infinities included (V_MUL_LEGACY_F32).
__device__ float mul_zero(float a, float b) __asm("llvm.amdgcn.fmul.legacy");

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// The page table is read through the scalar cache (uniform addresses, never
// written here), so that waiting for a page index never waits for the cache
// words in flight.
typedef const __attribute__((address_space(4))) int32_t* cint_p;

constexpr int kWaves = 4;            // waves of a workgroup
constexpr int kStep = kWaves * kKv4Tile;  // tokens of one step of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMostCs = 0x1p100f;  // of a column that has seen no value but 0
constexpr float kLow = -1e10f;  // below every finite score s_k (q.u + z sum q) of scaled queries, all under 1e8

__device__ __forceinline__ float xor16(float v, bool take_max) {
  const uint32_t b = __float_as_uint(v);
  const v2u s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const float x = __uint_as_float(s[0]), y = __uint_as_float(s[1]);
  return take_max ? fmaxf(x, y) : x + y;
}
__device__ __forceinline__ float xor32(float v, bool take_max) {
  const uint32_t b = __float_as_uint(v);
  const v2u s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const float x = __uint_as_float(s[0]), y = __uint_as_float(s[1]);
  return take_max ? fmaxf(x, y) : x + y;
}
// Over the four lanes r, r + 16, r + 32, r + 48.
__device__ __forceinline__ float column_max(float v) { return xor32(xor16(v, true), true); }
__device__ __forceinline__ float column_sum(float v) { return xor32(xor16(v, false), false); }

// Not shared with the same expression elsewhere: what a rare branch computes
// again stays inside it.
template <typename T>
__device__ __forceinline__ T opaque(T v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Between one lane's LDS stores and other lanes' loads of them in the same wave,
// and before the next stores there: the LDS takes a wave's accesses in order, this
// keeps the compiler from changing it (the words are stored one by one and loaded
// four at a time, types that it may take for distinct memory).  No instruction.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }

__device__ __forceinline__ v4f mfma16(const uint4& a, const uint4& b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Eight codes of one word as an operand: codes 0, 4, 1, 5, 2, 6, 3, 7, times
// 2^-20.
__device__ __forceinline__ uint4 codes8(uint32_t w) {
  return make_uint4((w << 4) & 0x00F000F0u, w & 0x00F000F0u, (w >> 4) & 0x00F000F0u, (w >> 8) & 0x00F000F0u);
}

// One 32-token step's cache words of one lane, and whether its page is one of
// the cache's (uniform).
template <int D>
struct Tile {
  uint32_t k[2][D / 32];  // keys of token 16h + r: channels c*D/4 .. of it
  uint4 v[2];             // values of tokens 16h + 4c + i: eight channels
  uint32_t sz;            // lane t < 32: token t's key (scale, zero point); t >= 32: token t - 32's values'
  bool ok;
};

// A token's (scale, zero point) word as it is computed with: a zero point that is
// not finite becomes a scale of NaN and a zero point of 0.  The scale reaches only
// the rows that see the token (an unseen token's score is replaced, and its weight
// of 0 takes the value scale by mul_zero), but zero points are a matrix operand,
// where 0 * NaN would reach every row of the step.
__device__ __forceinline__ uint32_t finite_zero(uint32_t w) { return (w & 0x7C000000u) == 0x7C000000u ? 0x7E00u : w; }

// z + 8 as its nearest fp16 and the rest, exactly, for whole z: where |z| < 8 the
// sum is exact, above it the larger addend gives the sum's error back.
struct ZeroPair {
  _Float16 near, rest;
};
__device__ __forceinline__ ZeroPair zero_pair(uint32_t word) {
  const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(word >> 16));
  const _Float16 near = z + 8.0f16;
  return {near, 8.0f16 - (near - z)};
}
__device__ __forceinline__ uint32_t with_zero(uint32_t word, _Float16 z) {
  return (word & 0xFFFFu) | ((uint32_t)__builtin_bit_cast(uint16_t, z) << 16);
}

// ONCE: the words pass the caches by.  One wave reads them, with up to 16 query
// columns per key/value head in a sequence; above, every tile of 16 columns reads
// them again (64 sequences of 2048 tokens: 16 columns 35 us, 32 62, 64 109).
template <bool ONCE, typename T>
__device__ __forceinline__ T load_words(const uint8_t* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  else return *reinterpret_cast<const T*>(p);
}

// Where a wave reads one head of the cache for one sequence.
template <int D, bool ONCE>
struct Reader {
  cint_p pages;
  const uint8_t *kq, *vq;  // of the lane within a step
  const uint32_t* sz;
  int64_t n_pages, page_rows, head_rows;
  int shift, mask;

  __device__ __forceinline__ Reader(const Kv4AttnArgs& a, int sq, int head, int lane) {
    const int r = lane & 15, ch = lane >> 4;
    pages = (cint_p)(a.table + (int64_t)sq * a.ldt);
    kq = a.c.kq + r * (D / 2) + ch * (D / 8);
    vq = a.c.vq + (ch * (D / 8) + (D == 128 ? r : r >> 1)) * 16;
    sz = lane < 32 ? a.c.ksz + lane : a.c.vsz + (lane - 32);
    n_pages = a.c.pages;
    page_rows = (int64_t)a.c.heads << a.c.shift;
    head_rows = (int64_t)head << a.c.shift;
    shift = a.c.shift;
    mask = a.c.page - 1;
  }
  __device__ __forceinline__ int page_of(int t0) const { return pages[t0 >> shift]; }
  // (the words of a page index that is none are read from page 0 and not used)
  __device__ __forceinline__ void fetch(Tile<D>& t, int t0, int page) const {
    t.ok = page >= 0 && page < n_pages;
    const int64_t row0 = (t.ok ? page : 0) * page_rows + head_rows + (t0 & mask);
    const uint8_t* const k = kq + row0 * (D / 2);
    const uint8_t* const v = vq + row0 * (D / 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (D == 128) {
        const v4u x = load_words<ONCE, v4u>(k + 16 * h * (D / 2));
        t.k[h][0] = x[0]; t.k[h][1] = x[1]; t.k[h][2] = x[2]; t.k[h][3] = x[3];
      } else {
        const v2u x = load_words<ONCE, v2u>(k + 16 * h * (D / 2));
        t.k[h][0] = x[0]; t.k[h][1] = x[1];
      }
    }
    t.sz = sz[row0];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4u x = load_words<ONCE, v4u>(v + 16 * h * (D / 2));
      t.v[h] = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  // n steps of 32 tokens from token t0, every `stride` tokens: three steps'
  // words in flight, in buffers that take turns; the page indexes one step
  // ahead of them.  Past the end the last step is read again, so that every
  // step issues the same loads and the wait for one step's words never waits
  // for a later one's.  No token past the step at `cap` is read.
  template <typename F>
  __device__ __forceinline__ void walk(int t0, int stride, int n, int cap, F run) const {
    if (n <= 0) return;
    const int last = t0 + (n - 1) * stride, end = min(last, cap);
    int at = min(t0, end), next = page_of(at);
    auto more = [&](Tile<D>& t) {
      const int here = at, page = next;
      at = min(at + stride, end);
      next = page_of(at);
      fetch(t, here, page);
    };
    Tile<D> A, B, C;
    more(A);
    more(B);
    for (;; t0 += 3 * stride) {
      more(C);
      run(A, t0);
      if (t0 + stride > last) break;
      more(A);
      run(B, t0 + stride);
      if (t0 + 2 * stride > last) break;
      more(B);
      run(C, t0 + 2 * stride);
      if (t0 + 3 * stride > last) break;
    }
  }
};

// NC tiles of 16 query columns and their running softmax.  m is in the units
// of the scaled queries' scores; times mul it is the exponent of two.
template <int D, int NC>
struct Columns {
  uint4 q[NC][D / 32];
  float qsum[NC], mul[NC];      // sum of the scaled queries; scores' factor to exponents of two
  int hi[NC], lo[NC];           // the column sees tokens lo <= t < hi
  v4f o[NC][D / 16], z[NC];     // z: rows 0, 4, 8, 12 of the product sum the near parts, the others the rests
  float m[NC], top[NC], l[NC];  // top: the score that raises m
  float cs[NC], big[NC];        // power of two on w = p * s_v; the largest w that was looked for

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      m[n] = kLow;
      top[n] = kLow + 6.0f / mul[n];  // infinite for the smallest factor: p = 1
      l[n] = 0.0f;
      z[n] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i] = v4f{0.f, 0.f, 0.f, 0.f};
      cs[n] = kMostCs;
      big[n] = 0.0f;
    }
  }
  __device__ __forceinline__ float zeros(int n) const { return z[n][0] + z[n][1]; }
  __device__ __forceinline__ void rescale(int n, float f) {
    z[n] *= f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[n][i] *= f;
  }
};

// A column's queries, scaled by a power of two to below 2^11 and ordered as
// codes8 orders the codes.
template <int DT, int D, int NC>
__device__ __forceinline__ void load_queries(Columns<D, NC>& s, int n, const uint16_t* row, bool has, int ch,
                                             float scale) {
  float f[D / 4];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    if (has) unpack16<DT>(*reinterpret_cast<const uint4*>(row + ch * (D / 4) + 8 * j), f + 8 * j);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) f[8 * j + i] = 0.0f;
  }
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 4; ++i) am = fmaxf(am, fabsf(f[i]));
  am = column_max(am);
  const int e = (int)(__float_as_uint(am) >> 23);  // |q| < 2^(e - 126)
  const float f2 = __uint_as_float((uint32_t)min(264 - e, 253) << 23);  // 2^(137 - e): |q * f2| < 2^11
  const float back = __uint_as_float((uint32_t)max(e - 10, 1) << 23);   // 1 / f2
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = f2h_bits(f[8 * j + i] * (scale < 0.0f ? -f2 : f2));
      sum += h2f((uint16_t)h[i]);
    }
    s.q[n][j] = make_uint4(h[0] | (h[4] << 16), h[1] | (h[5] << 16), h[2] | (h[6] << 16), h[3] | (h[7] << 16));
  }
  s.qsum[n] = column_sum(sum) * 0x1p-20f;
  // (neither 0, which would make NaN of an unseen token's -infinity, nor so
  // large that kLow times it is infinite: the softmax is flat, or one-hot, there)
  s.mul[n] = fminf(fmaxf(fabsf(scale) * kLog2e * 0x1p20f * back, 0x1p-126f), 0x1p92f);
}

// Value operand x of a lane's eight tokens: channel (D/16) r + x of each, from
// their words of eight channels (two words' halves side by side, then two codes
// at a time).
template <int D>
__device__ __forceinline__ void value_operands(const Tile<D>& t, int r, uint32_t magic, uint4 v[D / 16]) {
  const uint32_t w[8] = {t.v[0].x, t.v[0].y, t.v[0].z, t.v[0].w, t.v[1].x, t.v[1].y, t.v[1].z, t.v[1].w};
#pragma unroll
  for (int g = 0; g < D / 64; ++g) {  // 16-bit halves of a word that the lane's channels fill
    const uint32_t sel = D == 128 ? (g ? 0x07060302u : 0x05040100u) : (r & 1 ? 0x07060302u : 0x05040100u);
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], sel);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int sh = x & 2 ? 8 : 0;
      v[4 * g + x] = make_uint4(kv4_centred(p[0] >> sh, x & 1, magic), kv4_centred(p[1] >> sh, x & 1, magic),
                                kv4_centred(p[2] >> sh, x & 1, magic), kv4_centred(p[3] >> sh, x & 1, magic));
    }
  }
}

// What a step takes of its 32 tokens: operands, and for the lane's own tokens
// (16h + 4c + i) the words with the keys' zero points, the scales, the zero
// points' operand and the largest value scale.  Here from the wave's own
// registers, the words through 512 bytes of LDS of its own: the keys' words, the
// values' with the near part of z + 8 and once more with the rest, for the rows
// (lanes) that take the one or the other.
template <int D>
struct FromRegisters {
  const Tile<D>& t;
  int r, ch;
  uint32_t magic;
  uint32_t kw[8], vw[8];
  uint4 v[D / 16];

  __device__ __forceinline__ FromRegisters(const Tile<D>& tile, uint32_t* words, int lane, uint32_t m)
      : t(tile), r(lane & 15), ch(lane >> 4), magic(m) {
    const uint32_t word = finite_zero(t.sz);
    const ZeroPair z = zero_pair(word);
    wave_exchange();  // the step before has been read
    words[lane] = lane < 32 ? word : with_zero(word, z.near);
    words[lane ^ 96] = with_zero(word, z.rest);  // 64 .. 95; the keys' lanes' are not used
    const uint32_t* const values = words + (r & 3 ? 64 : 32);
    wave_exchange();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 x = *reinterpret_cast<const uint4*>(words + 16 * h + 4 * ch);
      const uint4 y = *reinterpret_cast<const uint4*>(values + 16 * h + 4 * ch);
      kw[4 * h] = x.x; kw[4 * h + 1] = x.y; kw[4 * h + 2] = x.z; kw[4 * h + 3] = x.w;
      vw[4 * h] = y.x; vw[4 * h + 1] = y.y; vw[4 * h + 2] = y.z; vw[4 * h + 3] = y.w;
    }
  }
  __device__ __forceinline__ uint4 key(int h, int j) const { return codes8(t.k[h][j]); }
  __device__ __forceinline__ float key_zero(int i) const { return half_hi(kw[i]); }
  __device__ __forceinline__ float key_scale(int i) const { return half_lo(kw[i]); }
  __device__ __forceinline__ float value_scale(int i) const { return half_lo(vw[i]); }
  __device__ __forceinline__ float value_scale_again(int i) const { return half_lo(opaque(vw[i])); }
  __device__ __forceinline__ float largest() const {
    v2half m = __builtin_bit_cast(v2half, vw[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2half, vw[i]));  // not NaN
    return (float)m[0];
  }
  __device__ __forceinline__ uint4 zeros() const {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_perm(vw[2 * i + 1], vw[2 * i], 0x07060302u);
    return make_uint4(p[0], p[1], p[2], p[3]);
  }
  __device__ __forceinline__ void prepare_values() { value_operands<D>(t, r, magic, v); }
  __device__ __forceinline__ uint4 value(int x) const { return v[x]; }
};

// One 32-token step from token t0.  edge (uniform): some column may not see
// some token of it.
template <int D, int NC, typename F>
__device__ __forceinline__ void step(Columns<D, NC>& s, F& t, bool edge, int t0, int ch) {
  // scores
  v4f a[NC][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const uint4 k = t.key(h, j);
#pragma unroll
      for (int n = 0; n < NC; ++n)
        a[n][h] = mfma16(k, s.q[n][j], j ? a[n][h] : v4f{0.f, 0.f, 0.f, 0.f});
    }
  float x[NC][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float sk = t.key_scale(i);
#pragma unroll
    for (int n = 0; n < NC; ++n) x[n][i] = fmaf(t.key_zero(i), s.qsum[n], a[n][i >> 2][i & 3]) * sk;
  }
  if (__builtin_expect(edge, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int tok = t0 + 16 * (i >> 2) + 4 * ch + (i & 3);
#pragma unroll
      for (int n = 0; n < NC; ++n) x[n][i] = tok >= s.lo[n] && tok < s.hi[n] ? x[n][i] : -__builtin_inff();
    }
  }

  // rare: a score far above its column's maximum, or a value scale so large that
  // a weight might leave fp16's range (w <= 2^6 * 2^9)
  const float vtop = t.largest();
  bool raise = false;
  float tm[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    tm[n] = fmaxf(fmaxf(fmaxf(x[n][0], x[n][1]), fmaxf(x[n][2], x[n][3])),
                  fmaxf(fmaxf(x[n][4], x[n][5]), fmaxf(x[n][6], x[n][7])));
    raise |= (tm[n] > s.top[n]) | (vtop * s.cs[n] > 512.0f);
  }
  if (__builtin_expect(__any(raise), 0)) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float m = column_max(fmaxf(tm[n], s.m[n]));
      const float g = __builtin_amdgcn_exp2f((s.m[n] - m) * s.mul[n]);
      s.m[n] = m;
      s.top[n] = m + 6.0f / s.mul[n];
      s.l[n] *= g;
      float big = s.big[n] * g;
#pragma unroll
      for (int i = 0; i < 8; ++i)  // (NaN does not count)
        big = fmaxf(big, mul_zero(__builtin_amdgcn_exp2f(fmaf(x[n][i], s.mul[n], -m * s.mul[n])),
                                  t.value_scale_again(i) * s.cs[n]));
      big = column_max(fminf(big, 65504.0f * s.cs[n]));
      // big < 2^(e - 126), and comes to [2^3, 2^4): weights down to 2^-17 of it keep
      // fp16's full precision, and a value scale may be 32 times it before this
      // branch is taken
      const int e = (int)(__float_as_uint(big) >> 23), c = (int)(__float_as_uint(s.cs[n]) >> 23);
      const int to = min(c + 130 - e, (int)(__float_as_uint(kMostCs) >> 23));
      const float f = __uint_as_float((uint32_t)(127 + to - c) << 23);
      s.cs[n] = __uint_as_float((uint32_t)to << 23);
      s.big[n] = big * f;
      s.rescale(n, g * f);
    }
  }

  uint4 w[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const float mm = s.m[n] * s.mul[n];
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __builtin_amdgcn_exp2f(fmaf(x[n][i], s.mul[n], -mm));
      s.l[n] += p;
      y[i] = mul_zero(p, t.value_scale(i) * s.cs[n]);  // an unseen token has no effect
    }
    w[n] = make_uint4(pack2<kF16>(y[0], y[1]), pack2<kF16>(y[2], y[3]), pack2<kF16>(y[4], y[5]), pack2<kF16>(y[6], y[7]));
  }

  // the zero points' sums and the values
  const uint4 z = t.zeros();
#pragma unroll
  for (int n = 0; n < NC; ++n) s.z[n] = mfma16(z, w[n], s.z[n]);
  t.prepare_values();
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint4 v = t.value(i);
#pragma unroll
    for (int n = 0; n < NC; ++n) s.o[n][i] = mfma16(v, w[n], s.o[n][i]);
  }
}

// A lane's accumulators: element i of accumulator x is its output channel
// (D/4) c + (D/16) i + x.

// The first token that a query at position pos sees.  (No difference that may
// pass 31 bits: positions before the context's start are negative, windows go up to
// 2^31 - 1.)
__device__ __forceinline__ int first_seen(const Kv4AttnArgs& a, int pos) {
  return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// A sequence's share of the work: its queries' columns in tiles of `width`
// and the steps over the tokens that any of them sees.
struct Seq {
  int len, q0, n;   // cached tokens, first query row, queries
  int lo, steps, tiles;
};
__device__ __forceinline__ Seq seq_of(const Kv4AttnArgs& a, int s, int group, int width) {
  Seq q;
  q.len = (int)min((int64_t)max(a.kv_len[s], 0), a.max_pages * a.c.page);
  q.q0 = a.cu_q ? min(max(a.cu_q[s], 0), (int)a.T) : s;
  q.n = a.cu_q ? min(max(a.cu_q[s + 1], q.q0), (int)a.T) - q.q0 : 1;
  const int first = q.len - q.n;  // position of the first query
  q.lo = first_seen(a, first) & ~(kKv4Tile - 1);
  q.steps = max((q.len - q.lo + kStep - 1) / kStep, 1);  // at least one: every row is written
  q.tiles = (q.n * group + width - 1) / width;
  return q;
}
__device__ __forceinline__ int64_t seq_work(const Seq& q, int heads) { return (int64_t)q.tiles * heads * q.steps; }

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
// a / b rounded down, exact for 0 <= a < 2^52 (the quotient's distance to the
// next whole number, at least 1/b, is above the rounding of the division).
__device__ __forceinline__ int64_t floor_div(int64_t a, int64_t b) { return (int64_t)((double)a / (double)b); }

// Exclusive prefix and sum over the wave's lanes.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane, int64_t* total) {
  if (__all(v < (1 << 25))) {  // the sum fits 31 bits: row shifts, then the rows' last lanes
    int x = (int)v;
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast 15 to rows 1, 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // row_bcast 31 to rows 2, 3
    *total = __builtin_amdgcn_readlane(x, 63);
    return x - (int)v;
  }
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  *total = uniform(__shfl(x, 63));
  return x - v;
}
__device__ __forceinline__ int64_t lane_value(int64_t v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, l);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), l);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Sum over the batch of work(sequence), and the sequence for which
// mine(sequence index, first, work) holds (-1: none) with the sum before it.
template <typename W, typename M>
__device__ __forceinline__ int64_t batch_scan(int64_t seqs, int lane, W work, M mine, int* sq, int64_t* base) {
  int64_t sum = 0;
  *sq = -1;
  *base = 0;
  for (int64_t s0 = 0; s0 < seqs; s0 += 64) {
    const int64_t s = s0 + lane;
    int64_t t;
    const int64_t w = s < seqs ? work((int)s) : 0;
    const int64_t before = sum + wave_scan(w, lane, &t);
    const uint64_t hit = __ballot(s < seqs && mine((int)s, before, w));
    if (hit && *sq < 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      *sq = (int)s0 + l;
      *base = lane_value(before, l);
    }
    sum += t;
  }
  return sum;
}

// The decoding kernel's work: the whole batch's steps in a row, sequence by
// sequence, head by head, column tile by column tile; workgroup i takes
// steps [i*chunk, (i+1)*chunk) of them, chunk = total / workgroups, rounded up.
__device__ __forceinline__ int64_t chunk_of(int64_t total, int64_t groups) {
  return max(floor_div(total + groups - 1, groups), (int64_t)1);
}

// Partial results of workgroup i: slot 2i for the unit it finishes or goes
// through from a step after its first, slot 2i + 1 for the unit it begins and
// does not finish.  A slot: [16 columns][D] sums, then [16][2] (the maximum as
// an exponent of two, the sum).  After the slots, for every workgroup the unit
// it begins and does not finish: the first query row, its columns' place
// (head, first column, columns) and how many workgroups share it (0: none).
__host__ __device__ constexpr int64_t slot_floats(int D) { return 16 * (int64_t)(D + 2); }
struct Shared {
  int q0, head, col0, cols, parts, pad[3];
};

// Few query columns (a decoding step): the four waves of a workgroup take
// every fourth 32-token step of the same 16 columns and join through LDS.
// Bound by the cache's bytes once contexts are long, by the launches and the
// latency of one pass of dependent loads when short (64 query heads on 8, 128
// channels, with the join): 131075 and 92684 tokens, 244 MB: 54 us, 4.5 TB/s;
// 64 ragged sequences of 512 to 8192 tokens, 199 MB: 58-60 us, 3.4 TB/s; one
// sequence of 1000 tokens (32 heads): 10.8 us.  The work is cut into equal runs
// of steps rather than by sequence or head, so that ragged batches and few long
// contexts fill the card alike.  Eight waves per workgroup, or 384, 768 or 1024
// workgroups instead of 512, gained nothing.
template <int DT, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void kv4_decode_kernel(Kv4AttnArgs a) {
  __shared__ __align__(16) float red[kWaves][16][D + 4];
  __shared__ float red_m[kWaves][16], red_l[kWaves][16];
  __shared__ __align__(16) uint32_t words[kWaves][128];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, ch = lane >> 4;
  const int group = a.q_heads / a.c.heads;
  const uint32_t magic = kv4_magic(0x64006400u);

  auto work = [&](int i) { return seq_work(seq_of(a, i, group, 16), a.c.heads); };
  int sq;
  int64_t base;
  int64_t total, w0 = 0, before0 = 0;
  if (a.seqs <= 64) {  // one scan serves both the sum and the search
    if (lane < a.seqs) w0 = work(lane);
    before0 = wave_scan(w0, lane, &total);
  } else {
    total = batch_scan(a.seqs, lane, work, [](int, int64_t, int64_t) { return false; }, &sq, &base);
  }
  const int64_t chunk = uniform(chunk_of(total, gridDim.x));
  int64_t at = (int64_t)blockIdx.x * chunk;
  Shared* const shared = reinterpret_cast<Shared*>(a.part + 2 * (int64_t)gridDim.x * slot_floats(D)) + blockIdx.x;
  if (threadIdx.x == 0) shared->parts = 0;
  if (at >= total) return;
  const int64_t end = min(at + chunk, total);
  if (a.seqs <= 64) {
    sq = __ffsll((unsigned long long)__ballot(at >= before0 && at < before0 + w0)) - 1;
    base = lane_value(before0, sq);
  } else {
    batch_scan(a.seqs, lane, work, [&](int, int64_t first, int64_t w) { return at >= first && at < first + w; }, &sq,
               &base);
  }
  Seq q = seq_of(a, sq, group, 16);

  while (at < end) {
    while (at >= base + seq_work(q, a.c.heads)) {  // next sequence with work (one exists: at < total)
      base += seq_work(q, a.c.heads);
      q = seq_of(a, ++sq, group, 16);
    }
    const int64_t local = at - base;
    const int unit = (int)uniform(floor_div(local, q.steps));
    const int step0 = (int)(local - (int64_t)unit * q.steps);
    const int nsteps = (int)min((int64_t)(q.steps - step0), end - at);
    const int head = unit / q.tiles, tile = unit - head * q.tiles;
    const int col = tile * 16 + r;
    const bool has = col < q.n * group;
    const int qi = has ? col / group : 0, qh = has ? col - qi * group : 0;
    const int64_t row = q.q0 + qi;
    const int hq = head * group + qh;

    Columns<D, 1> s;
    load_queries<DT>(s, 0, a.q + row * a.ldq + (int64_t)hq * D, has, ch, a.scale);
    s.clear();
    const int pos = q.len - q.n + qi;
    s.hi[0] = has ? (a.causal ? min(pos + 1, q.len) : q.len) : 0;
    s.lo[0] = first_seen(a, pos);
    // tokens that every column of the tile sees
    const int i0 = tile * 16 / group, i1 = min((tile * 16 + 15) / group, q.n - 1);
    const int all_hi = a.causal ? min(q.len - q.n + i0 + 1, q.len) : q.len;
    const int all_lo = first_seen(a, q.len - q.n + i1);

    // this wave's steps: tokens q.lo + 32 * (4 * (step0 + i) + wave)
    const int first = q.lo + kKv4Tile * (kWaves * step0 + wave);
    int left = (q.len - first + kStep - 1) / kStep;
    left = first < q.len ? min(left, nsteps) : 0;
    Reader<D, true>(a, sq, head, lane).walk(first, kStep, left, first + (left - 1) * kStep, [&](const Tile<D>& t, int t0) {
      if (!t.ok) return;
      FromRegisters<D> f(t, words[wave], lane, magic);
      step<D, 1>(s, f, t0 + kKv4Tile > all_hi || t0 < all_lo, t0, ch);
    });

    // join the waves: everything at the largest maximum, in true units
    const float l = column_sum(s.l[0]), z = s.zeros(0), me = s.m[0] * s.mul[0];
    if (ch == 0) red_m[wave][r] = me;
    __syncthreads();
    const float m = fmaxf(fmaxf(red_m[0][r], red_m[1][r]), fmaxf(red_m[2][r], red_m[3][r]));
    const float f = __builtin_amdgcn_exp2f(me - m);
    const float fo = f / s.cs[0];
    if (ch == 0) red_l[wave][r] = l * f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < D / 16; x += 4) {
        float4 v;
        v.x = (s.o[0][x][i] + z) * fo;
        v.y = (s.o[0][x + 1][i] + z) * fo;
        v.z = (s.o[0][x + 2][i] + z) * fo;
        v.w = (s.o[0][x + 3][i] + z) * fo;
        *reinterpret_cast<float4*>(&red[wave][r][ch * (D / 4) + i * (D / 16) + x]) = v;
      }
    __syncthreads();
    const bool whole = step0 == 0 && nsteps == q.steps;
    float* const slot = a.part + (2 * (int64_t)blockIdx.x + (step0 == 0)) * slot_floats(D);
    const int cols = min(q.n * group - tile * 16, 16);
    if (!whole && step0 == 0 && threadIdx.x == 0)
      *shared = Shared{q.q0, head, tile * 16, cols, (int)floor_div(at + q.steps - 1, chunk) - (int)blockIdx.x + 1, {}};
    for (int e = threadIdx.x * 4; e < cols * D; e += 64 * kWaves * 4) {
      const int cc = e / D, d = e - cc * D;
      float4 v = *reinterpret_cast<const float4*>(&red[0][cc][d]);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(&red[w][cc][d]);
        v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
      }
      const float ls = (red_l[0][cc] + red_l[1][cc]) + (red_l[2][cc] + red_l[3][cc]);
      const float ms = fmaxf(fmaxf(red_m[0][cc], red_m[1][cc]), fmaxf(red_m[2][cc], red_m[3][cc]));
      if (whole) {
        const int oi = (tile * 16 + cc) / group, oh = head * group + (tile * 16 + cc) - oi * group;
        const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;  // no visible token: 0
        const uint2 b = make_uint2(pack2<DT>(v.x * inv, v.y * inv), pack2<DT>(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(a.out + (int64_t)(q.q0 + oi) * a.ldo + (int64_t)oh * D + d) = b;
        if (a.lse && d == 0)
          a.lse[(int64_t)(q.q0 + oi) * a.q_heads + oh] =
              ls == 0.0f ? -__builtin_inff() : (ms + __builtin_amdgcn_logf(ls)) * (1.0f / kLog2e);
      } else {
        *reinterpret_cast<float4*>(slot + cc * D + d) = v;
        if (d == 0) {
          slot[16 * D + 2 * cc] = ms;
          slot[16 * D + 2 * cc + 1] = ls;
        }
      }
    }
    __syncthreads();
    at += nsteps;
  }
}

// Joins parts [0, n) of one row and head in their order, W waves taking every
// W-th: slot(p) gives a part's D sums and its (maximum as an exponent of two,
// sum).
template <int DT, int D, int W, typename S>
__device__ __forceinline__ void join_parts(const Kv4AttnArgs& a, int n, S slot, int64_t row, int hq) {
  __shared__ float red[W][D], red_l[W];
  constexpr int PER = D / 64;
  const int wave = W > 1 ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : 0, lane = threadIdx.x & 63;
  const float *o, *ml;
  float m = -3e38f;
  for (int p = lane; p < n; p += 64) {
    slot(p, &o, &ml);
    m = fmaxf(m, ml[0]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  float l = 0.0f, v[PER] = {};
#pragma unroll 8
  for (int p = wave; p < n; p += W) {
    slot(p, &o, &ml);
    const float f = __builtin_amdgcn_exp2f(ml[0] - m);
    l += ml[1] * f;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] += o[lane * PER + i] * f;
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) red[wave][lane * PER + i] = v[i];
    if (lane == 0) red_l[wave] = l;
    __syncthreads();
    if (wave) return;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      l += red_l[w];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] += red[w][lane * PER + i];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no visible token: 0
  uint16_t* const to = a.out + row * a.ldo + (int64_t)hq * D + lane * PER;
  if constexpr (PER == 2) *reinterpret_cast<uint32_t*>(to) = pack2<DT>(v[0] * inv, v[1] * inv);
  else *to = (uint16_t)from_f32<DT>(v[0] * inv);
  if (a.lse && lane == 0)
    a.lse[row * a.q_heads + hq] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * (1.0f / kLog2e);
}

// Joins the units that several workgroups of the decoding kernel shared: a
// workgroup of W waves per (workgroup that began one, column).
template <int DT, int D, int W>
__global__ __launch_bounds__(64 * W) void kv4_join_kernel(Kv4AttnArgs a) {
  const Shared u = *(reinterpret_cast<const Shared*>(a.part + 2 * (int64_t)gridDim.x * slot_floats(D)) + blockIdx.x);
  const int cc = blockIdx.y;
  if (cc >= u.cols || u.parts == 0) return;
  const int group = a.q_heads / a.c.heads;
  const int qi = (u.col0 + cc) / group, hq = u.head * group + u.col0 + cc - qi * group;
  join_parts<DT, D, W>(a, u.parts, [&](int p, const float** o, const float** ml) {
    const float* const s = a.part + (2 * ((int64_t)blockIdx.x + p) + (p == 0)) * slot_floats(D);
    *o = s + cc * D;
    *ml = s + 16 * D + 2 * cc;
  }, u.q0 + qi, hq);
}

// The same of a step that one wave of the workgroup has made operands of.
template <int D>
struct StepLds {
  uint4 k[D / 16][64], v[D / 16][64];  // [operand][lane]
  float kz[32], ks[32], vs[32];  // (widened once here: the fused operation on a half costs two of the fp32 one's)
  _Float16 near[32], rest[32];  // of zero point + 8
  float top;
  int ok;

  __device__ __forceinline__ void fill(const Tile<D>& t, int lane, uint32_t magic) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) k[h * (D / 32) + j][lane] = codes8(t.k[h][j]);
    uint4 o[D / 16];
    value_operands<D>(t, lane & 15, magic, o);
#pragma unroll
    for (int x = 0; x < D / 16; ++x) v[x][lane] = o[x];
    const int i = lane & 31;
    const uint32_t w = finite_zero(t.sz);
    const float sc = half_lo(w);
    if (lane < 32) {
      kz[i] = half_hi(w);
      ks[i] = sc;
    } else {
      vs[i] = sc;
      const ZeroPair z = zero_pair(w);
      near[i] = z.near;
      rest[i] = z.rest;
    }
    float m = sc < 65504.0f ? sc : (sc == sc ? 65504.0f : 0.0f);  // NaN does not count
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    m = fmaxf(m, __shfl_xor(m, 4));
    m = fmaxf(m, __shfl_xor(m, 8));
    m = fmaxf(m, __shfl_xor(m, 16));
    if (lane == 32) top = m;
    if (lane == 0) ok = t.ok;
  }
};
template <int D>
struct FromLds {
  const StepLds<D>& t;
  int lane, ch;
  float kz[8], ks[8], vs[8];

  __device__ __forceinline__ FromLds(const StepLds<D>& s, int l) : t(s), lane(l), ch(l >> 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 a = *reinterpret_cast<const float4*>(t.kz + 16 * h + 4 * ch);
      const float4 b = *reinterpret_cast<const float4*>(t.ks + 16 * h + 4 * ch);
      const float4 c = *reinterpret_cast<const float4*>(t.vs + 16 * h + 4 * ch);
      kz[4 * h] = a.x; kz[4 * h + 1] = a.y; kz[4 * h + 2] = a.z; kz[4 * h + 3] = a.w;
      ks[4 * h] = b.x; ks[4 * h + 1] = b.y; ks[4 * h + 2] = b.z; ks[4 * h + 3] = b.w;
      vs[4 * h] = c.x; vs[4 * h + 1] = c.y; vs[4 * h + 2] = c.z; vs[4 * h + 3] = c.w;
    }
  }
  __device__ __forceinline__ uint4 key(int h, int j) const { return t.k[h * (D / 32) + j][lane]; }
  __device__ __forceinline__ float key_zero(int i) const { return kz[i]; }
  __device__ __forceinline__ float key_scale(int i) const { return ks[i]; }
  __device__ __forceinline__ float value_scale(int i) const { return vs[i]; }
  __device__ __forceinline__ float value_scale_again(int i) const { return opaque(vs[i]); }
  __device__ __forceinline__ float largest() const { return t.top; }
  __device__ __forceinline__ uint4 zeros() const {
    const _Float16* const z = (lane & 3 ? t.rest : t.near) + 4 * ch;
    const uint2 a = *reinterpret_cast<const uint2*>(z), b = *reinterpret_cast<const uint2*>(z + 16);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void prepare_values() {}
  __device__ __forceinline__ uint4 value(int x) const { return t.v[x][lane]; }
};

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Many query columns (prompts and chunks): every wave has NC tiles of 16
// columns of its own; the workgroup walks all tokens that any of them sees,
// 128 at a time: each wave turns one of the four 32-token steps into operands
// in LDS, then every wave takes all four from there, so that unpacking costs a
// column a quarter.  Heads run fastest over the workgroups, so that workgroups
// of one head share an XCD's L2 (with 8 heads), later columns, which see more
// tokens, first.  With few columns the tokens are split over gridDim.y and
// joined by kv4_join_splits_kernel.
// Bound by the vector instructions of the softmax beside the matrix products:
// per 32 x 32 scores of a wave 34 matrix instructions of 16 cycles, and for a
// lane's 16 scores scale, zero point, maximum, exponential (16 cycles), sum,
// weight and conversion, some 800 cycles; and, third, by the operands' way from
// LDS.  1024 queries over 8192 tokens (64 heads on 8, 128 channels, 258 GFLOP): 342
// us in a row of calls, 750 TFLOP/s (384 us as the profiler times it); with every
// wave unpacking for itself 1061 us.  Counters of that run: vector unit issuing 63%
// of the time, matrix core busy 33%, LDS reads some 60%, so no unit is full and
// they overlap in part: between the barriers unpacking comes before use.  Moving
// the next step's scores ahead of this one's exponentials lost 7%, reading
// operands ahead gained nothing.
template <int DT, int D, int NC>
__global__ __launch_bounds__(64 * kWaves, 2) void kv4_tile_kernel(Kv4AttnArgs a) {
  constexpr int WIDTH = kWaves * 16 * NC;
  __shared__ __align__(16) StepLds<D> ops[kWaves];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, ch = lane >> 4;
  const int group = a.q_heads / a.c.heads;
  const uint32_t magic = kv4_magic(0x64006400u);
  const int64_t block = blockIdx.x / (unsigned)a.c.heads;
  const int head = (int)(blockIdx.x - block * a.c.heads);
  int sq;
  int64_t base;
  batch_scan(
      a.seqs, lane, [&](int i) { return (int64_t)seq_of(a, i, group, WIDTH).tiles; },
      [&](int, int64_t first, int64_t w) { return block >= first && block < first + w; }, &sq, &base);
  if (sq < 0) return;
  const Seq q = seq_of(a, sq, group, WIDTH);
  const int c0 = (q.tiles - 1 - (int)(block - base)) * WIDTH + wave * (16 * NC);

  Columns<D, NC> s;
  int64_t row[NC];
  int hq[NC];
  const int first = q.len - q.n;  // position of the sequence's first query
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int col = c0 + 16 * n + r;
    const bool has = col < q.n * group;
    const int qi = has ? col / group : 0;
    row[n] = has ? q.q0 + qi : -1;
    hq[n] = head * group + (has ? col - qi * group : 0);
    load_queries<DT>(s, n, a.q + (q.q0 + qi) * a.ldq + (int64_t)hq[n] * D, has, ch, a.scale);
    const int pos = first + qi;
    s.hi[n] = has ? (a.causal ? min(pos + 1, q.len) : q.len) : 0;
    s.lo[n] = first_seen(a, pos);
  }
  s.clear();
  // tokens that some column of queries i0 .. i1 sees
  auto seen_to = [&](int i1) { return a.causal ? min(first + i1 + 1, q.len) : q.len; };
  auto seen_from = [&](int i0) { return first_seen(a, first + i0); };
  // of the wave: what some, and what every, column sees (no column: nothing)
  const bool any = c0 < q.n * group;
  const int i0 = c0 / group, i1 = min((c0 + 16 * NC - 1) / group, q.n - 1);
  const int all_hi = seen_to(i0), all_lo = seen_from(i1);
  const int hi = any ? seen_to(i1) : 0, lo = seen_from(i0);
  // of the workgroup
  const int w0 = c0 - wave * (16 * NC);
  const int hi_w = seen_to(min((w0 + WIDTH - 1) / group, q.n - 1));
  const int lo_w = seen_from(w0 / group) & ~(kKv4Tile - 1);
  const int steps = hi_w > lo_w ? (hi_w - lo_w + kStep - 1) / kStep : 0;
  const int part = blockIdx.y, parts = gridDim.y;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);

  // (the waves' own steps run to the same count; one past the workgroup's last
  // token reads that token's step again and is not used)
  const int last = max((q.len - 1) & ~(kKv4Tile - 1), 0);
  Reader<D, false>(a, sq, head, lane).walk(lo_w + kStep * s0 + kKv4Tile * wave, kStep, s1 - s0, last, [&](const Tile<D>& t, int t0) {
    lds_barrier();  // the steps before are done with
    ops[wave].fill(t, lane, magic);
    lds_barrier();
    const int base = t0 - kKv4Tile * wave;
#pragma unroll 1
    for (int u = 0; u < kWaves; ++u) {
      const int tu = base + kKv4Tile * u;
      if (tu >= hi || tu + kKv4Tile <= lo || !__builtin_amdgcn_readfirstlane(ops[u].ok)) continue;
      FromLds<D> f(ops[u], lane);
      step<D, NC>(s, f, tu + kKv4Tile > all_hi || tu < all_lo, tu, ch);
    }
  });

#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const float l = column_sum(s.l[n]), me = s.m[n] * s.mul[n];
    if (row[n] < 0) continue;
    const float z = s.zeros(n), unit = 1.0f / s.cs[n];
    const float f = parts == 1 ? (l == 0.0f ? 0.0f : unit / l) : unit;  // no visible token: 0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[D / 16];
#pragma unroll
      for (int x = 0; x < D / 16; ++x) v[x] = (s.o[n][x][i] + z) * f;
      const int d = ch * (D / 4) + i * (D / 16);
      if (parts == 1) {
        uint16_t* const to = a.out + row[n] * a.ldo + (int64_t)hq[n] * D + d;
        if constexpr (D == 128) *reinterpret_cast<uint4*>(to) = pack16<DT>(v);
        else *reinterpret_cast<uint2*>(to) = make_uint2(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]));
      } else {
        float* const to = a.part + (((int64_t)part * a.T + row[n]) * a.q_heads + hq[n]) * D + d;
#pragma unroll
        for (int x = 0; x < D / 16; x += 4)
          *reinterpret_cast<float4*>(to + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
      }
    }
    if (ch == 0) {
      const int64_t at = row[n] * a.q_heads + hq[n];
      if (parts > 1) {
        float* const to = a.part + (int64_t)parts * a.T * a.q_heads * D + ((int64_t)part * a.T * a.q_heads + at) * 2;
        to[0] = me;
        to[1] = l;
      } else if (a.lse) {
        a.lse[at] = l == 0.0f ? -__builtin_inff() : (me + __builtin_amdgcn_logf(l)) * (1.0f / kLog2e);
      }
    }
  }
}

// Joins the token splits of the kernel above: one workgroup per row and head
// (rows outside every sequence are left alone).
template <int DT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv4_join_splits_kernel(Kv4AttnArgs a, int parts) {
  const int64_t row = blockIdx.x / (unsigned)a.q_heads;
  const int hq = (int)(blockIdx.x - row * a.q_heads);
  int sq;
  int64_t base;
  batch_scan(
      a.seqs, threadIdx.x & 63, [](int) { return (int64_t)0; },
      [&](int i, int64_t, int64_t) {
        const Seq q = seq_of(a, i, 1, 1);
        return row >= q.q0 && row < q.q0 + q.n;
      },
      &sq, &base);
  if (sq < 0) return;
  const int64_t rows = a.T * a.q_heads;
  join_parts<DT, D, kWaves>(a, parts, [&](int p, const float** o, const float** ml) {
    *o = a.part + ((int64_t)p * rows + blockIdx.x) * D;
    *ml = a.part + (int64_t)parts * rows * D + ((int64_t)p * rows + blockIdx.x) * 2;
  }, row, hq);
}

// Workgroups of the decoding kernel: two per compute unit.
constexpr int64_t kDecodeGroups = 512;
constexpr int kTileNC = 2;

// Which kernel, by the query columns of a key/value head in one sequence: up to
// 64 the decoding kernel, which unpacks for 16 columns but cuts the work evenly,
// above them the tile kernel.  Times in us, decoding / tile kernel, 64 heads on
// 8:  64 sequences of 2048 tokens, 16 columns 35 / 139, 32: 62 / 126, 64: 109 /
// 136, 128: 179 / 162;  8 of 512, 64 columns 16 / 36, 128: 23 / 40;  one of
// 8192, 32 columns 29 / 27, 64: 31 / 29, 128: 33 / 33.  So on short contexts the
// decoding kernel would win above 64 columns, too; the rule looks at the columns
// alone.
bool takes_tiles(int64_t max_q, int group) { return max_q * group > 64; }
int64_t tile_blocks(int64_t T, int64_t seqs, int group) {
  const int64_t width = kWaves * 16 * kTileNC;
  // every sequence that has queries may end in a part of a block
  return (T * group + width - 1) / width + std::min(T, seqs);
}
// Token splits: enough workgroups for two per compute unit (its registers hold
// no more), at most 16 (each costs the join a read of all outputs).
int tile_splits(int64_t T, int group, int kv_heads) {
  const int64_t width = kWaves * 16 * kTileNC;
  const int64_t blocks = (T * group + width - 1) / width * kv_heads;
  return (int)std::max<int64_t>(1, std::min<int64_t>(16, (512 + blocks / 2) / blocks));
}

}  // namespace

int64_t kv4_attn_groups(int64_t T, int64_t seqs, int q_heads, int kv_heads, int64_t max_q) {
  const int group = q_heads / kv_heads;
  return takes_tiles(max_q, group) ? tile_blocks(T, seqs, group) * kv_heads : kDecodeGroups;
}

size_t kv4_attn_workspace(int64_t T, int64_t, int q_heads, int kv_heads, int dim, int64_t max_q) {
  const int group = q_heads / kv_heads;
  if (!takes_tiles(max_q, group)) return (size_t)kDecodeGroups * (2 * (size_t)slot_floats(dim) * sizeof(float) + sizeof(Shared));
  const int splits = tile_splits(T, group, kv_heads);
  return splits == 1 ? 0 : (size_t)splits * (size_t)T * (size_t)q_heads * (size_t)(dim + 2) * sizeof(float);
}

template <int DT, int D>
static hipError_t launch(const Kv4AttnArgs& a, int64_t max_q, hipStream_t st) {
  const int group = a.q_heads / a.c.heads;
  const dim3 rows((unsigned)(a.T * a.q_heads)), threads(64 * kWaves);
  if (takes_tiles(max_q, group)) {
    const int splits = tile_splits(a.T, group, a.c.heads);
    const dim3 grid((unsigned)(tile_blocks(a.T, a.seqs, group) * a.c.heads), (unsigned)splits);
    hipLaunchKernelGGL((kv4_tile_kernel<DT, D, kTileNC>), grid, threads, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1) return e;
    hipLaunchKernelGGL((kv4_join_splits_kernel<DT, D>), rows, threads, 0, st, a, splits);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((kv4_decode_kernel<DT, D>), dim3((unsigned)kDecodeGroups), threads, 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // four waves per column where there are fewer units than a quarter of the
  // workgroups and so many parts in each, else one (join alone: 2 x 131075 tokens
  // 6.8 us with four, 8.9 with one; 64 ragged sequences 5.5 and 4.7)
  const dim3 cols((unsigned)kDecodeGroups, (unsigned)std::min<int64_t>(16, a.cu_q ? 16 : group));
  if (a.T * a.q_heads < kDecodeGroups / 4 * 16)
    hipLaunchKernelGGL((kv4_join_kernel<DT, D, kWaves>), cols, dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((kv4_join_kernel<DT, D, 1>), cols, dim3(64), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_kv4_attn(const Kv4AttnArgs& a, int64_t max_q, hipStream_t st) {
  const bool h = a.dtype == kF16;
  if (a.c.dim == 128) return h ? launch<kF16, 128>(a, max_q, st) : launch<kBf16, 128>(a, max_q, st);
  return h ? launch<kF16, 64>(a, max_q, st) : launch<kBf16, 64>(a, max_q, st);
}

}  // namespace mq
