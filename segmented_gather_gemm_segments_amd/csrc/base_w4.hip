// Base projection y = x W^T from 4-bit weights with group scales (lora_w4.h).
//
// Per group of k the kernel forms t = sum (128 + u) x and xs = sum x on the
// matrix cores and adds s (t - (128 + z) xs) to the output's fp32 sum.  128 + u
// is exact in bf16 (8 significant bits, unit spacing from 128 to 256), and its
// bit pattern is 0x4300 | u: one AND-OR turns two nibbles of a code word into
// two operand elements, so a word of 8 codes costs 7 vector instructions.  xs
// comes from the same x fragments against a constant operand of ones.
//
// Bound by HBM while the tokens of a decode batch are few, since at 4 bits a weight the codes are nearly all
// the bytes (16 tokens, 28672 x 8192: 28.9 us, 4.2 TB/s).  From 33 tokens on by the latency of a step: one step is in
// flight, behind a wait for all its loads and a barrier, and waves wait for 42 % of their time (8192 x 8192, groups of 64 with
// zero points: 24.6 us, 349 TFLOP/s, with the codes in the last cache, 30.2 from HBM).  The matrix cores are busy for 31 %
// of it, half of that for the sums of x, which each wave forms anew; the LDS for 17 %.  Small calls are a launch and one
// chain of loads (one token, 4096 x 4096: 4.6 us in the kernel).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "lora_internal.h"
#include "lora_w4.h"
#include "lds_load.h"

using namespace lora;

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

constexpr int kTileBytes = 1024;   // codes of 16 rows x 128 k
constexpr int kTileK = 128;
__device__ const uint4 g_zeros = {0, 0, 0, 0};  // x behind the last k
constexpr int kComputeUnits = 256;
// The kernels count rows, columns and bytes of one row in 32 bits.
constexpr int kMaxN = 1 << 26, kMaxK = 1 << 24;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));  // nearest even
}

// Four consecutive scales (or zero points) of one group as they are stored, and widened.
template <typename S>
using Four = std::conditional_t<sizeof(S) == 2, uint2, f32x4_t>;
__device__ __forceinline__ f32x4_t values(f32x4_t u) { return u; }
__device__ __forceinline__ f32x4_t values(uint2 u) {
  return f32x4_t{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xffff0000u)};
}

// The operand of one word of codes: 128 + u, 8 elements.
__device__ __forceinline__ bf16x8_t widen(uint32_t w) {
  uint4 o;
  o.x = (w & 0x000f000fu) | 0x43004300u;
  o.y = ((w >> 4) & 0x000f000fu) | 0x43004300u;
  o.z = ((w >> 8) & 0x000f000fu) | 0x43004300u;
  o.w = ((w >> 12) & 0x000f000fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8_t, o);
}

// One workgroup: R NT row tiles of W (16 rows each) and 16 MT tokens.  Its waves, in groups of R that share
// x and have NT row tiles each, take the steps of KC k in turn, each with the next step's codes,
// scales and x on their way while it works on this one; their fp32 sums are added in order through LDS.
// x goes through two LDS stages of each group: read as operands straight from memory, every lane would
// name a line of its own, and the address units, which take those one by one, would set the time
// (when the stages came, 16 tokens through 28672 x 8192 went from 33.4 to 29.9 us, 64 through 8192 x 8192 from 38.2 to 28.6).
template <int MT>
struct Shape {  // 64 tokens: 8 waves and steps of 128 k take 26.5 us there from the last cache, 29.7 from HBM, these 24.6 and 30.2
  static constexpr int kWaves = MT == 4 ? 16 : 8;
  static constexpr int kStep = MT == 4 ? 64 : 128;  // KC
};

template <int MT, int R, int NT, int G, typename S, bool Z>
__global__ __launch_bounds__(64 * Shape<MT>::kWaves) void base_w4_kernel(int m, int n, int k, int row_tiles, int col_tiles,
                                                              const uint8_t *__restrict__ codes,
                                                              const S *__restrict__ scales,
                                                              const S *__restrict__ zeros,
                                                              const uint16_t *__restrict__ x, int64_t x_stride,
                                                              uint16_t *__restrict__ y, int64_t y_stride) {
  constexpr int WAVES = Shape<MT>::kWaves, KC = Shape<MT>::kStep, W = WAVES / R;
  constexpr int WORDS = KC / 32;                 // words of codes per lane and step
  constexpr int GT = KC > G ? KC / G : 1;        // groups per step (a larger group is met in several)
  constexpr int GW = WORDS / GT;                 // words per group and step
  constexpr int kStage = 16 * MT * KC;           // elements of x
  constexpr int CPR = KC / 8, TPL = 64 / CPR;    // chunks per token, tokens per load
  __shared__ __attribute__((aligned(16))) uint16_t sx[2 * W * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int kw = wave / R, r0 = (blockIdx.x * R + wave % R) * NT, t0 = blockIdx.y * (16 * MT);
  const int groups = k / G, steps = (k + KC - 1) / KC;
  // Addresses are a part that all lanes share, which the scalar unit steps, and a fixed 32-bit offset per lane.
  const uint8_t *cp[NT];
  uint32_t nrow[NT];  // first of the 4 rows that this lane holds results of (clamped: results past n are not stored)
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    cp[a] = codes + (int64_t)min(r0 + a, row_tiles - 1) * col_tiles * kTileBytes;
    nrow[a] = min((r0 + a) * 16 + 4 * fg, n - 4);
  }
  // x: a load takes TPL tokens, lane l 16 bytes of one; chunk c of a token is stored in slot(token, c), so that the 16
  // lanes that read one chunk of 16 tokens hit every bank once
  auto slot = [](int t, int c) { return KC == 128 ? c ^ (t & 15) : c ^ ((t >> 1) & 7); };
  constexpr int LOADS = 16 * MT / TPL / R;
  uint32_t xo[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int t = TPL * (LOADS * (wave % R) + i) + lane / CPR;
    xo[i] = ((uint32_t)min(t, m - 1 - t0) * (uint32_t)x_stride + slot(t, lane % CPR) * 8) * 2;
  }
  const uint16_t *xt = x + (int64_t)t0 * x_stride;
  const uint16_t *stage = sx + kw * 2 * kStage;
  auto load_x = [&](int st, int buf) {
    const uint32_t to = lds_offset(sx) + (uint32_t)((kw * 2 + buf) * kStage + LOADS * (wave % R) * 512) * 2;
    if ((st + 1) * KC <= k) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) load_lds16(xt + st * KC, xo[i], to + i * 1024);
    } else {  // zeros behind the last k
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int t = TPL * (LOADS * (wave % R) + i) + lane / CPR, kk = st * KC + slot(t, lane % CPR) * 8;
        load_lds16(kk < k ? (const char *)(xt + st * KC) + xo[i] : (const char *)&g_zeros, to + i * 1024);
      }
    }
  };
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u));
  f32x4_t sum[NT][MT];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int i = 0; i < MT; ++i) sum[a][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  typedef __attribute__((ext_vector_type(WORDS))) uint32_t words_t;
  struct Step {
    words_t c[NT];
    Four<S> s[NT][GT], z[NT][Z ? GT : 1];
  };
  auto fetch = [&](int st, Step &p) {
    st = min(st, steps - 1);
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int64_t at = (int64_t)(st * KC / kTileK) * kTileBytes + st * KC % kTileK / 8;
      const words_t *c = reinterpret_cast<const words_t *>(cp[a] + at + (uint32_t)lane * 16);
      // Up to 32 tokens the codes are read once, past the caches (16 tokens, 28672 x 8192: 28.9 us, else 31.3); above
      // that, other token tiles may read them again (64 tokens, 8192 x 8192, codes that the last cache still holds: 24.6
      // us, past the caches 28.2; codes from HBM 30.2 and 29.0).
      p.c[a] = MT < 4 ? __builtin_nontemporal_load(c) : *c;
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        const int64_t row = (int64_t)min(st * KC / G + g, groups - 1) * n;
        p.s[a][g] = *reinterpret_cast<const Four<S> *>(scales + row + nrow[a]);
        if constexpr (Z) p.z[a][g] = *reinterpret_cast<const Four<S> *>(zeros + row + nrow[a]);
      }
    }
  };

  Step next;
  fetch(kw, next);
  if (kw < steps) load_x(kw, 0);
  int buf = 0;
  // waves that share stages go through the loop together, the last time some without a step
  for (int st = kw; R > 1 ? st - kw < steps : st < steps; st += W, buf ^= 1) {
    wait_vm<0>();  // this step's loads have landed
    wait_lds();    // and the other stage has been read
    if constexpr (R > 1) {
      __syncthreads();
      if (st >= steps) continue;
    }
    const Step now = next;
    fetch(st + W, next);
    if (st + W < steps) load_x(st + W, buf ^ 1);
    bf16x8_t xf[MT][WORDS];
#pragma unroll
    for (int s = 0; s < WORDS; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        xf[i][s] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const uint4 *>(
            stage + buf * kStage + (16 * i + fr) * KC + slot(fr, 4 * s + fg) * 8));
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      if (st * KC + g * G >= k) break;  // the last step of a k that is no multiple of KC
      f32x4_t xs[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xs[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = g * GW; s < (g + 1) * GW; ++s)
          xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xf[i][s], xs[i], 0, 0, 0);
      }
#pragma unroll
      for (int a = 0; a < NT; ++a) {
        f32x4_t t[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) t[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = g * GW; s < (g + 1) * GW; ++s) {
          const bf16x8_t wf = widen(now.c[a][s]);
#pragma unroll
          for (int i = 0; i < MT; ++i) t[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[i][s], t[i], 0, 0, 0);
        }
        const f32x4_t sc = values(now.s[a][g]);
        f32x4_t off = f32x4_t{136.f, 136.f, 136.f, 136.f};
        if constexpr (Z) off = values(now.z[a][g]) + 128.f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[a][i][j] += sc[j] * (t[i][j] - off[j] * xs[i][0]);
      }
    }
  }
  f32x4_t *red = reinterpret_cast<f32x4_t *>(sx);  // [WAVES][64]
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      __syncthreads();
      red[wave * 64 + lane] = sum[a][i];
      __syncthreads();
      if (kw == (a * MT + i) % W) {
        f32x4_t v = red[wave % R * 64 + lane];
        for (int w = 1; w < W; ++w) v += red[(w * R + wave % R) * 64 + lane];
        const int t = t0 + 16 * i + fr, c = (r0 + a) * 16 + 4 * fg;
        if (t < m && c < n)
          *reinterpret_cast<uint2 *>(y + (int64_t)t * y_stride + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      }
    }
}

// Thread: one 32-bit word of the tiled codes.
__global__ __launch_bounds__(256) void w4_pack_kernel(int n, int k, int col_tiles, int64_t words, uint32_t flip,
                                                      const uint32_t *__restrict__ rows,
                                                      uint32_t *__restrict__ codes) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= words) return;
  const int w = (int)(i & 3), lane = (int)((i >> 2) & 63);
  const int64_t tile = i >> 8;
  const int row = (int)(tile / col_tiles) * 16 + (lane & 15);
  const int k0 = (int)(tile % col_tiles) * kTileK + w * 32 + (lane >> 4) * 8;
  uint32_t out = 0x88888888u;
  if (row < n && k0 < k) {
    const uint32_t src = rows[((int64_t)row * k + k0) >> 3] ^ flip;  // element e in nibble e
    out = 0;
    for (int e = 0; e < 8; ++e) out |= ((src >> (4 * e)) & 15u) << (4 * ((e >> 1) + 4 * (e & 1)));
  }
  codes[i] = out;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

struct W4Call {
  int m, n, k, col_tiles;
  const lora_w4_weights *w;
  const uint16_t *x;
  int64_t xs;
  uint16_t *y;
  int64_t ys;
  hipStream_t stream;
};

template <int MT, int R, int NT, int G, typename S, bool Z>
void launch(const W4Call &c) {
  constexpr int kRows = R * NT;
  const int row_tiles = (c.n + 15) / 16;
  hipLaunchKernelGGL((base_w4_kernel<MT, R, NT, G, S, Z>), dim3((row_tiles + kRows - 1) / kRows, (c.m + 16 * MT - 1) / (16 * MT)),
                     dim3(64 * Shape<MT>::kWaves), 0, c.stream, c.m, c.n, c.k, row_tiles, c.col_tiles, (const uint8_t *)c.w->codes,
                     (const S *)c.w->scales, (const S *)c.w->zeros, c.x, c.xs, c.y, c.ys);
}
// Row tiles per workgroup: as many as still leave every compute unit a workgroup, since they share the
// reads of x, which for 16 tokens are four times those of one row tile's codes.  Up to 32 tokens a wave takes
// them, at most kMost, so that the scales and zero points on their way (kWords registers a tile) and the
// sums fit the registers (16 tokens, 28672 x 8192: 28.9 us, with one row tile 42.0).  For
// more tokens the waves of a group take one each, two of them, so that two stages of each group fit the LDS, or
// four (64 tokens, codes from HBM: through 28672 x 8192 77 us, with two 102; through 8192 x 8192, 128 workgroups of
// four, 42 and 30).
template <int MT, int G, typename S, bool Z>
void pick_tiles(const W4Call &c) {
  const int64_t row_tiles = (c.n + 15) / 16;
  if constexpr (MT == 4) {
    if ((row_tiles + 3) / 4 * ((c.m + 63) / 64) >= kComputeUnits) launch<MT, 4, 1, G, S, Z>(c);
    else launch<MT, 2, 1, G, S, Z>(c);
  } else {
    constexpr int kWords = kTileK / G * (int)sizeof(S) * (Z ? 2 : 1);
    constexpr int kMost = 64 / MT / kWords;
    if (kMost >= 4 && row_tiles >= 4 * kComputeUnits) launch<MT, 1, kMost >= 4 ? 4 : 1, G, S, Z>(c);
    else if (kMost >= 2 && row_tiles >= 2 * kComputeUnits) launch<MT, 1, kMost >= 2 ? 2 : 1, G, S, Z>(c);
    else launch<MT, 1, 1, G, S, Z>(c);
  }
}
template <int MT, int G>
void pick_scale(const W4Call &c) {
  if (c.w->scale_dtype == LORA_BF16)
    c.w->zeros ? pick_tiles<MT, G, uint16_t, true>(c) : pick_tiles<MT, G, uint16_t, false>(c);
  else
    c.w->zeros ? pick_tiles<MT, G, float, true>(c) : pick_tiles<MT, G, float, false>(c);
}
template <int MT>
void pick_group(const W4Call &c) {
  if (c.w->group == 32) pick_scale<MT, 32>(c);
  else if (c.w->group == 64) pick_scale<MT, 64>(c);
  else pick_scale<MT, 128>(c);
}

}  // namespace

extern "C" lora_status lora_w4_bytes(int32_t n, int32_t k, int64_t *bytes) {
  if (!bytes) return fail(LORA_EINVAL, "null bytes");
  *bytes = 0;
  if (n <= 0 || k <= 0) return fail(LORA_EINVAL, "4-bit weights n=%d k=%d", n, k);
  *bytes = (int64_t)kTileBytes * (((int64_t)n + 15) / 16) * (((int64_t)k + kTileK - 1) / kTileK);
  return ok();
}

extern "C" lora_status lora_w4_pack(int32_t n, int32_t k, int32_t twos_complement, const void *rows, void *codes,
                                    hipStream_t stream) {
  int64_t bytes = 0;
  lora_status st = lora_w4_bytes(n, k, &bytes);
  if (st != LORA_OK) return st;
  if (n % 8 || k % 32) return fail(LORA_EUNSUPPORTED, "4-bit weights need n a multiple of 8 and k of 32");
  if (n > kMaxN || k > kMaxK) return fail(LORA_EUNSUPPORTED, "4-bit weights of n=%d k=%d", n, k);
  if (twos_complement != 0 && twos_complement != 1) return fail(LORA_EINVAL, "twos_complement is 0 or 1");
  if (!rows || !codes) return fail(LORA_EINVAL, "null pointer");
  if (!aligned16(rows) || !aligned16(codes)) return fail(LORA_EINVAL, "device arrays must be 16-byte aligned");
  const int64_t words = bytes / 4, blocks = (words + 255) / 256;
  if (blocks > UINT32_MAX / 256) return fail(LORA_EUNSUPPORTED, "4-bit weights too large");
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, n, k, (k + kTileK - 1) / kTileK,
                     words, twos_complement ? 0x88888888u : 0u, (const uint32_t *)rows, (uint32_t *)codes);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "4-bit pack launch");
  return ok();
}

extern "C" lora_status lora_base_w4(int32_t dtype, int32_t m, const lora_w4_weights *w, const void *x,
                                    int64_t x_stride, void *y, int64_t y_stride, hipStream_t stream) {
  if (!w) return fail(LORA_EINVAL, "null weights");
  if (dtype != LORA_BF16) return fail(LORA_EUNSUPPORTED, "4-bit base projection supports bf16 activations only");
  if (m < 0 || w->n <= 0 || w->k <= 0) return fail(LORA_EINVAL, "4-bit base projection m=%d n=%d k=%d", m, w->n, w->k);
  if (w->group != 32 && w->group != 64 && w->group != 128)
    return fail(LORA_EUNSUPPORTED, "group must be 32, 64 or 128 (got %d)", w->group);
  if (w->n % 8 || w->k % w->group)
    return fail(LORA_EUNSUPPORTED, "4-bit base projection needs n a multiple of 8 and k of the group");
  if (w->scale_dtype != LORA_F32 && w->scale_dtype != LORA_BF16)
    return fail(LORA_EUNSUPPORTED, "scale dtype %d", w->scale_dtype);
  if (w->n > kMaxN || w->k > kMaxK) return fail(LORA_EUNSUPPORTED, "4-bit weights of n=%d k=%d", w->n, w->k);
  if (x_stride < w->k || y_stride < w->n || x_stride % 8 || y_stride % 8)
    return fail(LORA_EINVAL, "row strides must be multiples of 8 of at least k and n (got %lld and %lld)",
                (long long)x_stride, (long long)y_stride);
  if (x_stride > kMaxK) return fail(LORA_EUNSUPPORTED, "an x row stride above 2^24");
  if (m == 0) return ok();
  if (!w->codes || !w->scales || !x || !y) return fail(LORA_EINVAL, "null pointer");
  if (!aligned16(w->codes) || !aligned16(w->scales) || !aligned16(w->zeros) || !aligned16(x) || !aligned16(y))
    return fail(LORA_EINVAL, "device arrays must be 16-byte aligned");
  const int mt = m <= 16 ? 1 : m <= 32 ? 2 : 4;
  if ((m + 16 * mt - 1) / (16 * mt) > 65535) return fail(LORA_EUNSUPPORTED, "too many tokens");
  const W4Call c{m, w->n, w->k, (w->k + kTileK - 1) / kTileK, w, (const uint16_t *)x, x_stride, (uint16_t *)y,
                 y_stride, stream};
  if (mt == 1) pick_group<1>(c);
  else if (mt == 2) pick_group<2>(c);
  else pick_group<4>(c);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "4-bit base projection launch");
  return ok();
}
