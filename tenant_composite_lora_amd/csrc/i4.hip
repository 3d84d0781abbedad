// Base projections by 4-bit weights with group scales (include/tcl.h has the
// formulas): bf16 activations, integers 0..15 with a scale and a zero point
// for each group of a channel's weights.
//
// An integer n becomes the bf16 number 16 + n by at most two operations on a
// pair of them (a shift, and its four bits under the exponent of 16), exactly.
// The matrix cores sum x (16 + n) over a group, and with the sums of x over the
// groups
//   y = sum_g s_g sum_g x (n - z) = sum_g s_g (sum_g x (16 + n) - (16 + z_g) sum_g x)
// takes one or two fused operations an output and group, in fp32.  The correction
// is the second of them (i4_rows, i4_direct), what a group's products start from,
// a short product of fp32 numbers in bf16 parts (i4_blocks), or such a product
// every four groups (i4_tile): running sums never hold more than four groups'
// uncorrected.  No weight is rounded.
//
// Four kernels (choose):
//   i4_rows    up to 16 tokens: the weight streams from memory into matrix-core
//              operands, the waves of a workgroup split d_in and add their sums
//              in LDS;
//   i4_direct  more, in tiles of 32: likewise, x turned in LDS;
//   i4_blocks  wide outputs in short groups: likewise, after a launch that lays x
//              out in operands and sums it over the groups (i4_stage_kernel);
//   i4_tile    many tokens, from laid-out activations: tiles of both operands go
//              through LDS.
//
// The packed weight holds blocks of 32 channels by 64 columns, 1 KiB, 16 bytes a
// lane: lane l has channel l % 32 and, in its dwords 0..3, the eights of columns
// o, 4 + o, 2 + o and 6 + o of the block, o = l / 32.  A lane of a 32 x 32 x 16
// product takes all four, one of a 16 x 16 x 32 product one half.  Columns 2 j
// and 2 j + 1 of an eight lie at bits 3 + 4 j and 19 + 4 j, those beyond bit 31
// at its start.  Behind the blocks come the scales, 32 channels of a group side
// by side, and the zero points likewise.
#include <algorithm>
#include <type_traits>

#include "kern_common.hpp"

namespace tcl {
namespace {

constexpr int kWaves = 8;  // a workgroup's, but in i4_tile

struct I4Args {
  const uint8_t *w;       // packed blocks
  const float *scale;     // [32 channels][group][32]
  const uint8_t *zero;    // the same, or NULL: 8
  const uint16_t *x;
  void *y;
  int64_t ldx, ldy;
  int32_t T, K, N, kb, groups;  // kb: 128 columns
  uint64_t per_block;     // 2^32 / blocks of 128 columns of a group, rounded up (group_of)
  const nt_u4 *xb;        // staged activations
  const float *xe;        // and their groups' sums
  int32_t steps;          // corrections of four groups
  int32_t nt, nc;         // tiles of tokens, of channels
  int32_t ks;             // workgroups that share a tile's columns (i4_direct)
  float *part;            // [ks][T][N], where ks > 1
  bool y_f32;
};

// ---------------------------------------------------------------------------
// packing
// ---------------------------------------------------------------------------
struct PackArgs {
  const uint8_t *W, *zero;
  const float *scale;
  uint8_t *w, *pz;
  float *ps;
  int32_t K, N, kb, groups;
  int64_t n_w, n_s;  // 16-byte pieces of the blocks; scales
};

__global__ __launch_bounds__(256) void i4_pack_kernel(PackArgs a) {
  const int64_t step = int64_t(gridDim.x) * 256, at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t p = at; p < a.n_w; p += step) {
    const int lane = int(p & 63);
    const int64_t blk = p >> 6;
    const int c = int(blk / (2 * a.kb)) * 32 + (lane & 31);
    const int k0 = int(blk % (2 * a.kb)) * 64 + 8 * (lane >> 5);
    nt_u4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 16 * ((i & 1) << 1 | i >> 1);
      uint32_t u = 0;
      if (c < a.N && k < a.K) {  // (d_in is a multiple of 32)
        const uint32_t b = *reinterpret_cast<const uint32_t *>(a.W + (int64_t(c) * a.K + k) / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u |= (b >> 8 * j & 15) << 4 * j | (b >> (8 * j + 4) & 15) << (16 + 4 * j);
      }
      out[i] = u << 3 | u >> 29;
    }
    reinterpret_cast<nt_u4 *>(a.w)[p] = out;
  }
  for (int64_t p = at; p < a.n_s; p += step) {
    const int64_t tg = p >> 5;
    const int c = int(tg / a.groups) * 32 + int(p & 31), g = int(tg % a.groups);
    a.ps[p] = c < a.N ? a.scale[int64_t(c) * a.groups + g] : 0.f;
    if (a.zero) a.pz[p] = c < a.N ? a.zero[int64_t(c) * a.groups + g] : 8;
  }
}

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
// For more than a few tokens the activations are laid out once, in the order
// in which the products take them, with zeros behind the last token and
// column: 4 KiB of 32 tokens by 64 columns, piece i of lane l the 16 bytes of
// token l % 32, columns 16 i + 8 (l / 32).  Behind them come the sums of x over
// the groups, fp32: [32 tokens][four groups][4][32].
struct StageArgs {
  const uint16_t *x;
  nt_u4 *xb;
  float *xe;
  int64_t ldx;
  int32_t T, K, kb, steps;  // steps: groups / 4, rounded up
};

// 32 tokens by 128 columns a wave.
template <int GS>
__global__ __launch_bounds__(256) void i4_stage_kernel(StageArgs a) {
  constexpr int PER = 4 / GS;  // blocks of a correction step
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int b = blockIdx.y * 4 + (threadIdx.x >> 6);
  const int t = blockIdx.x * 32 + c;
  if (b >= a.steps * PER) return;
  float sum[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = 128 * b + 16 * i + 8 * h;
    nt_u4 u = {0, 0, 0, 0};
    if (t < a.T && k < a.K) u = *reinterpret_cast<const nt_u4 *>(a.x + t * a.ldx + k);
    if (b < a.kb) a.xb[(int64_t(blockIdx.x) * a.kb + b) * 512 + 64 * i + lane] = u;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[i / 2] += bf16_lo(u[e]) + bf16_hi(u[e]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] += __shfl_xor(sum[i], 32, 64);
  float *xe = a.xe + (int64_t(blockIdx.x) * a.steps + b / PER) * 128 + c;
  if constexpr (GS == 4) {
    xe[32 * h] = h ? sum[1] : sum[0];
    xe[64 + 32 * h] = h ? sum[3] : sum[2];
  } else if constexpr (GS == 2) {
    xe[64 * (b & 1) + 32 * h] = h ? sum[2] + sum[3] : sum[0] + sum[1];
  } else {
    if (h == 0) xe[32 * (b & 3)] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// Eight columns as bf16 numbers 16 + n.  (The mask in a scalar and the exponent
// in a vector register, which the compiler has to be told: it then needs one
// operation for both, with literals two.)
struct Widen {
  uint32_t mask, base;
  __device__ inline Widen() {
    asm("s_mov_b32 %0, 0x780078" : "=s"(mask));
    asm("v_mov_b32 %0, 0x41804180" : "=v"(base));
  }
  __device__ inline bf16x8_t operator()(uint32_t w) const {
    const uint32_t top = __builtin_amdgcn_alignbit(w, w, 12);
    return __builtin_bit_cast(bf16x8_t, nt_u4{(w & mask) | base, (w >> 4 & mask) | base,
                                              (w >> 8 & mask) | base, (top & mask) | base});
  }
};

__device__ inline bf16x8_t ones() {
  return __builtin_bit_cast(bf16x8_t, nt_u4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
}

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
__device__ inline f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16_t nothing() {
  return f32x16_t{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
}
__device__ inline bf16x8_t as_bf16(nt_u4 u) { return __builtin_bit_cast(bf16x8_t, u); }

// The group of block b where groups have blocks of 128 columns, n of them: b /
// n, exact for b and n up to 2^13.
__device__ inline int group_of(const I4Args &a, int b) { return int(uint64_t(unsigned(b)) * a.per_block >> 32); }
// the group of the block's part e (the last block may hold fewer than others)
template <int GS>
__device__ inline int group_at(const I4Args &a, int b, int e) {
  return GS == 1 ? group_of(a, b) : min(b * GS + e, a.groups - 1);
}

// v = p[0] + p[1] + p[2] in bf16 numbers, the rest below 2^-24 of v
__device__ inline void split3(float v, uint32_t *p) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = __builtin_bit_cast(uint16_t, __bf16(v));
    v -= __uint_as_float(p[i] << 16);
  }
}

// The correction of a group, -(s (16 + z)) sum x, as products of bf16 parts on
// the matrix cores (i4_tile): columns 0 .. 5 of a lane's eight hold parts 0 0 1 0 2 1 of
// its group's sum against parts 0 1 0 2 0 1 of its factor, which leaves out less
// than 2^-23 of the product.
__device__ inline bf16x8_t parts_x(float v) {
  uint32_t p[3];
  split3(v, p);
  return as_bf16(nt_u4{p[0] | p[0] << 16, p[1] | p[0] << 16, p[2] | p[1] << 16, 0});
}
__device__ inline bf16x8_t parts_w(float v) {
  uint32_t p[3];
  split3(v, p);
  return as_bf16(nt_u4{p[0] | p[1] << 16, p[0] | p[2] << 16, p[0] | p[1] << 16, 0});
}

// Four channels of a token to y.
__device__ inline void store4(const I4Args &a, int t, int ch, nt_f4 v) {
  const int64_t at = int64_t(t) * a.ldy + ch;
  if (a.y_f32) {
    *reinterpret_cast<nt_f4 *>(static_cast<float *>(a.y) + at) = v;
  } else {
    *reinterpret_cast<nt_u2 *>(static_cast<uint16_t *>(a.y) + at) = nt_u2{uint32_t(f32_to_bf16(v[0])) | uint32_t(f32_to_bf16(v[1])) << 16,
                                          uint32_t(f32_to_bf16(v[2])) | uint32_t(f32_to_bf16(v[3])) << 16};
  }
}

// The waves' sums of a tile of R tokens by 16 CH channels, added in order:
// put(token, channel, four channels) of each; part[wave][token][LD].
template <int R, int CH, int LD, int WV, typename F>
__device__ inline void add_up(const I4Args &a, const float *part, int t0, int c0, F put) {
  for (int o = threadIdx.x; o < R * CH * 4; o += 64 * WV) {
    const int r = o / (4 * CH), t = t0 + r, ch = c0 + o % (4 * CH) * 4;
    if (t >= a.T || ch >= a.N) continue;
    const float *in = part + r * LD + o % (4 * CH) * 4;
    nt_f4 v = *reinterpret_cast<const nt_f4 *>(in);
#pragma unroll
    for (int i = 1; i < WV; ++i) v += *reinterpret_cast<const nt_f4 *>(in + i * R * LD);
    put(t, ch, v);
  }
}

// A wave's blocks first, first + step, ... below n, from slots 0 .. AHEAD - 1 in
// turn: block(slot, number, whether the slot is to be filled again).  No branch
// lies around a load: where two paths meet, the compiler waits for the longer
// one.  (Slots that nothing uses again are filled with the last block, fewer
// than AHEAD of them.)
template <int AHEAD, typename F>
__device__ inline void stream(int first, int step, int n, F block) {
  int b = first;
  for (; b + AHEAD * step < n; b += AHEAD * step)
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) block(d, b + d * step, std::true_type{});
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (b + d * step < n) block(d, b + d * step, std::false_type{});
}

// Few tokens, straight from x.  16 NB channels a workgroup; wave w of WV takes
// the blocks w, w + WV, ... of 128 columns.  Tokens are the rows of a
// result, so that a lane holds one channel, its scale and zero point; the sums
// of x come from an operand of ones.  Operands are on their way up to four
// blocks ahead, since a wave has few: at 1 token, 4096 -> 1024, 64 workgroups of
// 8 waves have 4 blocks each, 4.5 us, a launch and two trips to memory; 4096 ->
// 14336, 31 MB, 8.7 us, 3.6 TB/s.  GS: groups of a block (4, 2, 1; 1 also
// for groups of several blocks).
template <int NB, int GS, bool ZP>
__global__ __launch_bounds__(64 * kWaves) void i4_rows(I4Args a) {
  const Widen widen;
  constexpr int AHEAD = NB > 2 ? 2 : 4;  // blocks on their way
  constexpr int WV = kWaves, LD = 16 * NB + 4;
  __shared__ __align__(16) float part[WV * 16 * LD];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int c0 = blockIdx.x * 16 * NB;
  const int tiles = (a.N + 15) / 16;
  const uint16_t *xp = a.x + int64_t(min(c, a.T - 1)) * a.ldx + 8 * g;
  const uint8_t *wp[NB];
  const float *sp[NB];
  const uint8_t *zp[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    // (channel tiles past the last: the last one again, not stored)
    const int ct = int(min(blockIdx.x * NB + n, unsigned(tiles - 1)));
    const int64_t t32 = ct >> 1;
    wp[n] = a.w + t32 * a.kb * 2048 + (g & 1) * 512 + (ct & 1) * 256 + c * 16 + (g >> 1) * 8;
    sp[n] = a.scale + t32 * a.groups * 32 + (ct & 1) * 16 + c;
    zp[n] = ZP ? a.zero + t32 * a.groups * 32 + (ct & 1) * 16 + c : nullptr;
  }
  f32x4_t acc[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) acc[n] = f32x4_t{0, 0, 0, 0};
  // (operands are replaced as in i4_blocks)
  nt_u2 wq[AHEAD][NB][2];
  nt_u4 xr[AHEAD][4];
  float s[AHEAD][NB][GS], z[AHEAD][NB][GS];
  auto load_w = [&](int d, int n, int k, int b) {
    wq[d][n][k] = *reinterpret_cast<const nt_u2 *>(wp[n] + int64_t(min(b, a.kb - 1)) * 2048 + 1024 * k);
  };
  auto load_s = [&](int d, int n, int b) {
#pragma unroll
    for (int e = 0; e < GS; ++e) {
      const int gr = group_at<GS>(a, min(b, a.kb - 1), e);
      s[d][n][e] = sp[n][gr * 32];
      z[d][n][e] = ZP ? 16.f + float(zp[n][gr * 32]) : 24.f;
    }
  };
  auto load_x = [&](int d, int i, int b) {
    // (columns past the row's end: any of it)
    const int k = b * 128 + 32 * i;
    xr[d][i] = *reinterpret_cast<const nt_u4 *>(xp + (k < a.K ? k : 0));
  };
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) {
    const int b = w + d * WV;
#pragma unroll
    for (int n = 0; n < NB; ++n) load_w(d, n, 0, b), load_w(d, n, 1, b), load_s(d, n, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_x(d, i, b);
    __builtin_amdgcn_sched_barrier(0);
  }
  // block b from slot d, which block b + AHEAD * WV then takes
  auto block = [&](int d, int b, auto more) {
#pragma unroll
    for (int e = 0; e < GS; ++e) {
      f32x4_t sum = {0, 0, 0, 0}, p[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) p[n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 4 / GS * e; i < 4 / GS * (e + 1); ++i) {
        // columns past the row's end: zeros (here, not where they are read,
        // which would wait for them)
        const bf16x8_t x = as_bf16(b * 128 + 32 * i < a.K ? xr[d][i] : nt_u4{0, 0, 0, 0});
        sum = mfma(x, ones(), sum);
#pragma unroll
        for (int n = 0; n < NB; ++n) p[n] = mfma(x, widen(wq[d][n][i >> 1][i & 1]), p[n]);
        if constexpr (more) {
          load_x(d, i, b + AHEAD * WV);
          if (i % 2 == 1)
#pragma unroll
            for (int n = 0; n < NB; ++n) load_w(d, n, i / 2, b + AHEAD * WV);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[n][r] = fmaf(s[d][n][e], fmaf(-z[d][n][e], sum[r], p[n][r]), acc[n][r]);
    }
    if constexpr (more)
#pragma unroll
      for (int n = 0; n < NB; ++n) load_s(d, n, b + AHEAD * WV);
  };
  stream<AHEAD>(w, WV, a.kb, block);
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[(w * 16 + 4 * g + r) * LD + 16 * n + c] = acc[n][r];
  __syncthreads();
  add_up<16, NB, LD, WV>(a, part, 0, c0, [&](int t, int ch, nt_f4 v) { store4(a, t, ch, v); });
}

// The row of a 32 x 32 result that element e of a lane of half h holds.
__device__ inline int row_of(int e, int h) { return 8 * (e / 4) + 4 * h + e % 4; }

// The position in a packed lane of columns 16 i ..
__device__ inline constexpr int place(int i) { return (i & 1) << 1 | i >> 1; }

// A group's correction, -(16 + z) sum x, as a product of bf16 parts: columns 0 ..
// 5 of a lane's eight hold parts 0 0 1 1 2 2 of the sum against the even part of
// 16 + z (at most 270, so exactly a bf16 number) and the odd one (0 or 1) in turn.
__device__ inline nt_u4 parts_sum(float v) {
  uint32_t p[3];
  split3(v, p);
  return nt_u4{p[0] | p[0] << 16, p[1] | p[1] << 16, p[2] | p[2] << 16, 0};
}
__device__ inline bf16x8_t parts_zero(uint32_t z) {  // z: zero point
  const uint32_t n = 16 + z, even = __float_as_uint(-float(n & ~1u)), odd = __float_as_uint(-float(n & 1));
  const uint32_t w = __builtin_amdgcn_perm(odd, even, 0x07060302);
  return as_bf16(nt_u4{w, w, w, 0});
}

constexpr int kBlockTiles = 4;  // tiles of 32 channels of a workgroup of i4_blocks

// More tokens, from staged activations: 128 channels by 32 tokens, the blocks
// dealt out to the waves as in i4_rows.  For groups of 32 and 64: 64 tokens, 4096 ->
// 14336, groups of 32, 24.0 us with the 4.8 of laying the activations out (zero
// points 24.8), 128 tokens 39.2.  A group's products start from its correction, a
// matrix product in which one half of the lanes (the group's, two groups in turn)
// holds the sum of x: what is scaled and added up is then no larger than the
// result's own terms.  (Corrections taken off at the end, all groups' together:
// 65536 columns of activations of one sign, 16 times the error that a group's own
// roundings allow.)  What scales the sums, two operations an element and group in
// i4_direct, one here, shares the issue slots with widening and the matrix
// instructions.
template <int GS, bool ZP>
__global__ __launch_bounds__(64 * kWaves) void i4_blocks(I4Args a) {
  static_assert(GS > 1, "two groups share a correction's operands");
  const Widen widen;
  constexpr int NB = kBlockTiles, WV = kWaves, LD = 32 * NB + 8;
  __shared__ __align__(16) float part[WV * 32 * LD];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int nx = (a.N + 32 * NB - 1) / (32 * NB);
  const int c0 = blockIdx.x % nx * 32 * NB, t0 = blockIdx.x / nx * 32;
  const int tiles = (a.N + 31) / 32;
  const int64_t tile = t0 / 32;
  const nt_u4 *xp = a.xb + tile * a.kb * 512;
  const float *ep = a.xe + tile * a.steps * 128;
  const nt_u4 *wp[NB];
  const float *sp[NB];
  const uint8_t *zp[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    // (channel tiles past the last: the last one again, not stored)
    const int64_t ct = min(c0 / 32 + n, tiles - 1);
    wp[n] = reinterpret_cast<const nt_u4 *>(a.w) + ct * a.kb * 128;
    sp[n] = a.scale + ct * a.groups * 32;
    zp[n] = ZP ? a.zero + ct * a.groups * 32 : nullptr;
  }
  f32x16_t acc[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) acc[n] = nothing();
  // A block's operands, each replaced by that of the next as soon as its
  // products have been issued: loads are always on their way, and no register
  // waits for them twice.  Activations as far ahead as weights, although they
  // come from L2: loads are waited for in the order of their issue.  (The
  // scheduling barriers hold the loads there; left to itself the compiler puts
  // them right before their use.)
  nt_u4 wq[NB][2], xr[8];
  float s[NB][GS], v;
  uint32_t z[NB];
  auto load_w = [&](int n, int k, int b) {
    const nt_u4 *at = wp[n] + int64_t(min(b, a.kb - 1)) * 128 + 64 * k;
    asm("" : "+s"(at));  // (a scalar: else the lane's addresses take eight registers all along)
    wq[n][k] = at[lane];
  };
  auto load_s = [&](int n, int b) {
#pragma unroll
    for (int e = 0; e < GS; ++e) s[n][e] = (sp[n] + group_at<GS>(a, min(b, a.kb - 1), e) * 32)[c];
  };
  auto load_x = [&](int i, int b) { xr[i] = (xp + int64_t(min(b, a.kb - 1)) * 512 + 64 * i)[lane]; };
  // the sum of x of group 2 k + h of the block and its zero points (behind the last
  // group sums of zero), half a block ahead: a whole one takes registers that spill
  auto load_c = [&](int k, int b) {
    const int pair = min(b, a.kb - 1) * (GS / 2) + k;
    v = (ep + int64_t(pair) * 64)[lane];
#pragma unroll
    for (int n = 0; n < NB; ++n) z[n] = ZP ? zp[n][unsigned(min(2 * pair + h, a.groups - 1) * 32 + c)] : 8;
  };
  load_c(0, w);
#pragma unroll
  for (int n = 0; n < NB; ++n) load_w(n, 0, w), load_w(n, 1, w), load_s(n, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) load_x(i, w);
  __builtin_amdgcn_sched_barrier(0);
  auto block = [&](int, int b, auto more) {
#pragma unroll
    for (int e = 0; e < GS; ++e) {
      f32x16_t p[NB];
      const nt_u4 sum = parts_sum(h == (e & 1) ? v : 0.f);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        p[n] = mfma(as_bf16(sum), parts_zero(z[n]), nothing());
        __builtin_amdgcn_sched_barrier(0);
      }
      if (e == 1 && GS == 4) load_c(1, b);
      if constexpr (more)
        if (e == GS - 1) load_c(0, b + WV);
#pragma unroll
      for (int i = 8 / GS * e; i < 8 / GS * (e + 1); ++i) {
#pragma unroll
        for (int n = 0; n < NB; ++n) p[n] = mfma(as_bf16(xr[i]), widen(wq[n][i / 4][place(i % 4)]), p[n]);
        if constexpr (more) {
          load_x(i, b + WV);
          if (i % 4 == 3)
#pragma unroll
            for (int n = 0; n < NB; ++n) load_w(n, i / 4, b + WV);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[n][r] = fmaf(s[n][e], p[n][r], acc[n][r]);
    }
    if constexpr (more)
#pragma unroll
      for (int n = 0; n < NB; ++n) load_s(n, b + WV);
  };
  stream<1>(w, WV, a.kb, block);
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) part[(w * 32 + row_of(r, h)) * LD + 32 * n + c] = acc[n][r];
  __syncthreads();
  add_up<32, 2 * NB, LD, WV>(a, part, t0, c0, [&](int t, int ch, nt_f4 v) { store4(a, t, ch, v); });
}

// Loads straight into LDS: 64 lanes write 16 (or 4) bytes each, in a row from
// `to`; the compiler does not count them (arrived).  An immediate offset moves
// source and destination alike.
__device__ inline uint32_t lds_at(const void *p) {
  return uint32_t(uintptr_t((__attribute__((address_space(3))) const char *)(p)));
}
template <int N>
__device__ inline void move16(uint32_t to, const void *from, uint32_t off) {
  static_assert(N == 1 || N == 2 || N == 4, "pieces of 1 KiB");
  if constexpr (N == 4)
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
        "global_load_lds_dwordx4 %1, %2 offset:1024\n\tglobal_load_lds_dwordx4 %1, %2 offset:2048\n\t"
        "global_load_lds_dwordx4 %1, %2 offset:3072" ::"s"(to), "v"(off), "s"(from) : "memory", "m0");
  else if constexpr (N == 2)
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
        "global_load_lds_dwordx4 %1, %2 offset:1024" ::"s"(to), "v"(off), "s"(from) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off),
                 "s"(from)
                 : "memory", "m0");
}
__device__ inline void move4(uint32_t to, const void *from, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(off), "s"(from)
               : "memory", "m0");
}
__device__ inline void move16(uint32_t to, const void *from) {  // an address a lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}

// The same without a launch that lays out the activations: a wave moves its
// block of them, rows of 256 bytes, into LDS, a block ahead, and turns it in
// reading; the sums of x come from an operand of ones.  32 NB channels by 32
// tokens; with ks > 1 as many workgroups, blockIdx.y, share their columns.  32 x
// 4096 -> 4096 8.1 us, 64 8.7; 64 x 4096 -> 14336 15.6; 23 tokens, 14336 -> 4096 in
// four, groups of 32, 13.5 us of 37 MB and 4.0 joining.  With a block of rows and
// one of weights on their way a wave, a CU takes in 26 to 41 GB/s, rows and weights
// together (23 tokens, 14336 -> 4096: 364 KB a workgroup; 64, 4096 -> 14336: 528; 32,
// 4096 -> 4096: 324): no rate of its own, rather too little on its way.  A last tile of fewer than 32 tokens
// takes in its last row again for those that it lacks.  (Rows through registers take 32 more of them:
// 64 x 4096 -> 14336, 30 spilled, 20.7.  Weights two blocks ahead: 32 x 4096 ->
// 14336 12.6 where one takes 11.4.)
template <int NB, int GS, bool ZP>
__global__ __launch_bounds__(64 * kWaves) void i4_direct(I4Args a) {
  const Widen widen;
  constexpr int WV = kWaves, LD = 32 * NB + 8;
  __shared__ __align__(16) union {
    float part[WV * 32 * LD];
    nt_u4 x[WV][2][32 * 16];  // chunk c of row r at 16 r + (c ^ r % 16)
  } l;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int nx = (a.N + 32 * NB - 1) / (32 * NB);
  const int c0 = blockIdx.x % nx * 32 * NB, t0 = blockIdx.x / nx * 32;
  const int first = blockIdx.y * WV + w, stride = a.ks * WV;
  const int tiles = (a.N + 31) / 32;
  const nt_u4 *wp[NB];
  const float *sp[NB];
  const uint8_t *zp[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    // (channel tiles past the last: the last one again, not stored)
    const int64_t ct = min(c0 / 32 + n, tiles - 1);
    wp[n] = reinterpret_cast<const nt_u4 *>(a.w) + ct * a.kb * 128;
    sp[n] = a.scale + ct * a.groups * 32;
    zp[n] = ZP ? a.zero + ct * a.groups * 32 : nullptr;
  }
  f32x16_t acc[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) acc[n] = nothing();
  nt_u4 wq[NB][2];
  float s[NB][GS], z[NB][GS];
  auto load_w = [&](int n, int k, int b) { wq[n][k] = (wp[n] + int64_t(min(b, a.kb - 1)) * 128 + 64 * k)[lane]; };
  auto load_s = [&](int n, int b) {
#pragma unroll
    for (int e = 0; e < GS; ++e) {
      const int gr = group_at<GS>(a, min(b, a.kb - 1), e);
      s[n][e] = (sp[n] + gr * 32)[c];
      z[n][e] = ZP ? 16.f + float((zp[n] + gr * 32)[c]) : 24.f;
    }
  };
  // rows of a block into LDS, four an instruction (columns past the row's end:
  // any of it; rows past the last: the last)
  auto load_x = [&](int b, int slot) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = 4 * j + (lane >> 4), k = b * 128 + 8 * ((lane ^ row) & 15);
      move16(lds_at(&l.x[w][slot][64 * j]), a.x + int64_t(min(t0 + row, a.T - 1)) * a.ldx + (k < a.K ? k : 0));
    }
  };
  load_x(first, 0);
#pragma unroll
  for (int n = 0; n < NB; ++n) load_w(n, 0, first), load_w(n, 1, first), load_s(n, first);
  int slot = 0;
  auto block = [&](int, int b, auto more) {
    // The block's rows have come: at least the 2 NB loads of its weights were
    // issued behind them.  What the next rows replace has been read.
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * NB) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (more) load_x(b + stride, slot ^ 1);
    __builtin_amdgcn_sched_barrier(0);
    const nt_u4 *xl = &l.x[w][slot][16 * c];
    slot ^= 1;
#pragma unroll
    for (int e = 0; e < GS; ++e) {
      f32x16_t sum = nothing();
      f32x16_t p[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) p[n] = nothing();
      nt_u4 xo[2];
      auto read = [&](int i) { xo[i & 1] = xl[(2 * i + h) ^ (c & 15)]; };
      read(8 / GS * e);
#pragma unroll
      for (int i = 8 / GS * e; i < 8 / GS * (e + 1); ++i) {
        if (i + 1 < 8 / GS * (e + 1)) read(i + 1);
        // (a row's last block may end before 128 columns)
        const bf16x8_t x = as_bf16(more || b * 128 + 8 * (2 * i + h) < a.K ? xo[i & 1] : nt_u4{0, 0, 0, 0});
        sum = mfma(x, ones(), sum);
#pragma unroll
        for (int n = 0; n < NB; ++n) p[n] = mfma(x, widen(wq[n][i / 4][place(i % 4)]), p[n]);
        if constexpr (more)
          if (i % 4 == 3)
#pragma unroll
            for (int n = 0; n < NB; ++n) load_w(n, i / 4, b + stride);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          acc[n][r] = fmaf(s[n][e], fmaf(-z[n][e], sum[r], p[n][r]), acc[n][r]);
    }
    if constexpr (more)
#pragma unroll
      for (int n = 0; n < NB; ++n) load_s(n, b + stride);
    __builtin_amdgcn_sched_barrier(0);
  };
  stream<1>(first, stride, a.kb, block);
  // the waves' activations lie where their sums go; rows of a wave without a
  // block may still be on their way
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) l.part[(w * 32 + row_of(r, h)) * LD + 32 * n + c] = acc[n][r];
  __syncthreads();
  add_up<32, 2 * NB, LD, WV>(a, l.part, t0, c0, [&](int t, int ch, nt_f4 v) {
    if (a.ks == 1)
      store4(a, t, ch, v);
    else
      *reinterpret_cast<nt_f4 *>(a.part + ((int64_t(blockIdx.y) * a.T + t) * a.N + ch)) = v;
  });
}

// Adds the parts of the workgroups that shared columns, in order.
__global__ __launch_bounds__(256) void i4_join_kernel(I4Args a) {
  const int64_t n4 = a.N / 4, all = a.T * n4;
  for (int64_t o = int64_t(blockIdx.x) * 256 + threadIdx.x; o < all; o += int64_t(gridDim.x) * 256) {
    const nt_f4 *in = reinterpret_cast<const nt_f4 *>(a.part) + o;
    nt_f4 v = in[0];
#pragma unroll 4
    for (int z = 1; z < a.ks; ++z) v += in[z * all];
    store4(a, int(o / n4), int(o % n4) * 4, v);
  }
}

// Many tokens: tiles of 256 channels by BT tokens, four by two waves.  Blocks
// of 128 columns go through LDS in three stages, activations and weights alike,
// each filled while the block two before it is multiplied (a wave's own
// registers hold no load: one block's time does not cover a trip to memory);
// scales, zero points and sums of x come with every four groups.  2048 tokens,
// 4096 -> 14336: 258 to 272 us with the 10 of laying x out, 0.9 P operations a second
// (launch by launch: 267 in the median and at first, 310 to 330 from the fourth or
// seventh launch behind a pause on for a while); the same matrix instructions alone take 176 (the clock under full load), what
// comes on top is LDS filled (31), sums scaled (31), corrections (16), operands
// read (16); widening, dealt out among the products, 3.
template <int BT, int GS, bool ZP>
__global__ __launch_bounds__(512, 2) void i4_tile(I4Args a) {
  const Widen widen;
  constexpr int BC = 256, WV = 8, WC = 4, WT = WV / WC, NB = BC / WC / 32, MT = BT / WT / 32, PER = 4 / GS;
  constexpr int NX = BT / 32;  // KiB of activations a wave moves a block
  __shared__ struct {
    nt_u4 x[3][BT / 32 * 512];
    nt_u4 w[3][BC / 32 * 128];
    float sum[2][BT / 32 * 128];  // of four groups
    float s[2][BC / 32 * 128];
    uint8_t z[2][BC / 32 * 128];
  } l;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups go to the eight XCDs in turn: each gets a run of tiles, token
  // tiles next to each other, so that its L2 holds their weights
  const int n_all = a.nt * a.nc, per = (n_all + 7) / 8;
  const int id = int(blockIdx.x & 7) * per + int(blockIdx.x >> 3);
  if (int(blockIdx.x >> 3) >= per || id >= n_all) return;
  const int c0 = id / a.nt * BC, t0 = id % a.nt * BT;
  const int wc = (w % WC) * NB, wt = (w / WC) * MT;  // the wave's first tiles
  const int tiles = (a.N + 31) / 32, tt = (a.T + 31) / 32;
  // (tiles past the last: the last again, not stored)
  auto c_tile = [&](int i) { return int64_t(min(c0 / 32 + i, tiles - 1)); };
  auto t_tile = [&](int i) { return int64_t(min(t0 / 32 + i, tt - 1)); };
  auto stage = [&](int b, int slot) {
    move16<NX>(lds_at(&l.x[slot][w * NX * 64]),
               a.xb + (t_tile(w * NX / 8) * a.kb + b) * 512 + w * NX % 8 * 64, 16 * lane);
    move16<2>(lds_at(&l.w[slot][w * 128]), a.w + (c_tile(w) * a.kb + b) * 2048, 16 * lane);
  };
  // A step's groups; lanes of groups behind the last take the last one's
  // factors, their sums are zero.
  auto group = [&](int st, int i) { return min(GS == 1 ? group_of(a, 4 * st + i) : 4 * st + i, a.groups - 1); };
  auto stage_step = [&](int st) {
    const int sl = st & 1, p = w % (BT / 16);  // 64 sums a wave
    move4(lds_at(&l.sum[sl][p * 64]), a.xe + (t_tile(p / 2) * a.steps + st) * 128 + p % 2 * 64, 4 * lane);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      move4(lds_at(&l.s[sl][w * 128 + 64 * i]), a.scale + c_tile(w) * a.groups * 32,
            4 * (group(st, 2 * i + h) * 32 + c));
    if constexpr (ZP) {
      // two channel tiles an instruction, four channels a lane
      const int i = w % 4 * 2;
      move4(lds_at(&l.z[sl][i * 128]), a.zero + c_tile(i) * a.groups * 32,
            uint32_t((c_tile(i + h) - c_tile(i)) * a.groups * 32 + group(st, lane >> 3 & 3) * 32 +
                     4 * (lane & 7)));
    }
  };
  f32x16_t acc[MT][NB];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = nothing();
  stage_step(0);
  stage(0, 0);
  stage(min(1, a.kb - 1), 1);
  int slot = 0;
  for (int b = 0; b < a.kb; ++b) {
    // all but the newest block's loads have come; every wave is done with
    // what the next loads write
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NX + 2) : "memory");
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    if ((b + 1) % PER == 0) stage_step(min((b + 1) / PER, a.steps - 1));
    stage(min(b + 2, a.kb - 1), slot == 0 ? 2 : slot - 1);
    const int sl = b / PER & 1;
    // Sixteen columns at a time; the next ones are read and widened between
    // the matrix instructions of these.
    nt_u4 q[NB][2], xf[2][MT];
    bf16x8_t wf[2][NB];
    float sc[NB][GS];
    f32x16_t p[MT][NB];
    auto read = [&](int i) {
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[i & 1][m] = l.x[slot][(wt + m) * 512 + 64 * i + lane];
    };
    auto widen_all = [&](int i) {
#pragma unroll
      for (int n = 0; n < NB; ++n) wf[i & 1][n] = widen(q[n][i / 4][place(i % 4)]);
    };
    auto multiply = [&](int i) {
      constexpr int LEN = 8 / GS;  // steps of sixteen of a group
      if (i % LEN == 0)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NB; ++n) p[m][n] = nothing();
      if (i < 7) {
        read(i + 1);
        widen_all(i + 1);
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) p[m][n] = mfma(as_bf16(xf[i & 1][m]), wf[i & 1][n], p[m][n]);
      __builtin_amdgcn_sched_group_barrier(0x100, MT, 0);  // LDS reads
#pragma unroll
      for (int k = 0; k < MT * NB; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);       // a matrix instruction
        __builtin_amdgcn_sched_group_barrier(0x2, 8 / MT, 0);  // widening
      }
      __builtin_amdgcn_sched_barrier(0);
      if (i % LEN == LEN - 1)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[m][n][r] = fmaf(sc[n][i / LEN], p[m][n][r], acc[m][n][r]);
    };
    read(0);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int k = 0; k < 2; ++k) q[n][k] = l.w[slot][(wc + n) * 128 + 64 * k + lane];
#pragma unroll
      for (int e = 0; e < GS; ++e) sc[n][e] = l.s[sl][(wc + n) * 128 + (b % PER * GS + e) * 32 + c];
    }
    widen_all(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) multiply(i);
    // corrections every four groups, so that sums stay small
    if (b % PER == PER - 1 || b == a.kb - 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        bf16x8_t f[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int at = (wc + n) * 128 + 64 * k + lane;
          f[n] = parts_w(-l.s[sl][at] * (ZP ? 16.f + float(l.z[sl][at]) : 24.f));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const bf16x8_t x = parts_x(l.sum[sl][(wt + m) * 128 + 64 * k + lane]);
#pragma unroll
          for (int n = 0; n < NB; ++n) acc[m][n] = mfma(x, f[n], acc[m][n]);
        }
      }
    }
    slot = slot == 2 ? 0 : slot + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  // Results through LDS, a wave's 32 tokens at a time, so that a store covers
  // whole lines of y.
  constexpr int LD = 32 * NB + 8;
  static_assert(WV * 32 * LD * 4 <= int(sizeof(l)), "LDS of the results");
  float *out = reinterpret_cast<float *>(&l) + w * 32 * LD;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) out[row_of(r, h) * LD + 32 * n + c] = acc[m][n][r];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#pragma unroll
    for (int k = 0; k < 4 * NB; ++k) {
      const int o = k * 64 + lane, x = o / (8 * NB), t = t0 + 32 * (wt + m) + x;
      const int ch = o % (8 * NB) * 4, at = c0 + 32 * wc + ch;
      if (t < a.T && at < a.N) store4(a, t, at, *reinterpret_cast<const nt_f4 *>(out + x * LD + ch));
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
  }
}

// ---------------------------------------------------------------------------
// checks and launches
// ---------------------------------------------------------------------------
bool misaligned(const void *p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) & (m - 1); }

constexpr int kMaxChannels = 1 << 26, kMaxTokens = 1 << 24;

// up to as many tokens are taken from x as it is, in one launch
constexpr int kRows = 16;

// Which kernel.  Measured on captured calls with weights from memory, groups of
// 128, us, staging and joins included; d_in 4096 unless said.
//   i4_rows, as many channels a workgroup as leave 192 of them: 1 token, 1024
//     channels: 16 channels 4.5, 32 5.7; 4096 channels 4.9, 6.1; 14336: 16
//     channels 10.6, 64 8.7 (16 tokens: 19.1, 9.9).
//   The others by whole rounds over the CUs (half_us: one workgroup a CU).
//     i4_direct with 32 channels a workgroup, 64, 128: 64 tokens, 4096 channels
//     8.7, 9.7, 13.2; 32 x 14336 16.1, 11.4, 14.4; 64 x 14336 29.7, 20.1, 15.6
//     (i4_blocks, that is the launch that lays out the activations, 18.2); 192 x
//     4096 21.4, 18.1, 14.2 (16.8).  In groups of 32 128 channels with their
//     factors do not fit the registers: 64 x 14336 35.8, 25.6, 30.6 (24.0), 128 x
//     14336 57.1, 46.4, 54.8 (39.2); there i4_blocks takes them.
//     128 channels, i4_tile of 64 tokens, of 128: 512 tokens, 4096 channels 28.7,
//     44.3, 60.4; 1024: 55.3, 49.3, 62.5; 2048: 111, 101, 78; 256 x 14336: 56.3,
//     49.8, 62.7; 512 x 14336: 101, 87, 68.
//   What bounds all of these is how long a CU takes to take its operands in, so that
//     few workgroups with long rows are split over d_in (ks) and joined by a
//     launch more, of 64 channels where that leaves them 256 parts, since rows
//     are most of what they take in.  From 8192 columns on; between 4096 and
//     that neither side has been measured.  d_in 14336: 23 tokens, 4096 channels 19.3, 32
//     channels in two 15.4, 64 in four 14.2; 32, 2048 channels 18.4, 32 in four
//     11.6, 64 in eight 11.4; 64, 4096 channels 22.3, 64 in two 19.1; d_in 8192, 17
//     tokens, 1024 channels 11.6, 32 in eight 7.7, 64 in eight 8.5.  d_in 4096: 17
//     tokens, 1024 channels 7.2, in two 7.4.
struct Choice {
  enum { kFew, kDirect, kBlocks, kTile64, kTile128 } kernel;
  int nb;  // 16 (few) or 32 (direct, blocks) channels a workgroup times this
  int ks;
};

int64_t rounds(int64_t workgroups) { return (workgroups + 255) / 256; }

Choice choose(int32_t n_tokens, int32_t d_out, int32_t kb, bool shorter) {  // groups of less than 128
  const int64_t T = n_tokens, N = d_out;
  auto over = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  if (T <= kRows) return {Choice::kFew, over(N, 64) >= 192 ? 4 : over(N, 32) >= 192 ? 2 : 1, 1};
  const int64_t tb = over(T, 32), w1 = tb * over(N, 32), w2 = tb * over(N, 64);
  if (kb >= 64 && w2 <= 128)
    return w1 < 64 ? Choice{Choice::kDirect, 1, int(std::min<int64_t>(256 / w1, kb / 8))}
                   : Choice{Choice::kDirect, 2, int(256 / w2)};
  const int64_t half_us[5] = {3 + 14 * rounds(w1), 3 + 19 * rounds(w2),
                              (shorter ? 10 : 5) + (shorter ? 24 : 26) * rounds(tb * over(N, 128)),
                              16 + 80 * rounds(over(T, 64) * over(N, 256)),
                              10 + 132 * rounds(over(T, 128) * over(N, 256))};
  switch (std::min_element(half_us, half_us + 5) - half_us) {
    case 0: return {Choice::kDirect, 1, 1};
    case 1: return {Choice::kDirect, 2, 1};
    case 2: return {shorter ? Choice::kBlocks : Choice::kDirect, 4, 1};
    case 3: return {Choice::kTile64, 0, 1};
    default: return {Choice::kTile128, 0, 1};
  }
}

struct Layout {
  int64_t tiles;
  int32_t kb, groups;
  size_t w, scale, total;  // bytes of the blocks; where the zero points are; all
};

int check_weight(const tcl_i4_weight *w, Layout *l) {
  if (!w) return fail(TCL_EINVAL, "i4: weight is NULL");
  if (w->d_in < 32 || w->d_out < 0)
    return fail(TCL_EINVAL, "i4: d_in %d < 32 or d_out %d < 0", w->d_in, w->d_out);
  if (w->group != 32 && w->group != 64 && (w->group < 128 || w->group % 128))
    return fail(TCL_EUNSUPPORTED, "i4: group %d is not 32, 64 or a multiple of 128", w->group);
  if (w->d_in % w->group) return fail(TCL_EINVAL, "i4: d_in %d is not whole groups of %d", w->d_in, w->group);
  if (w->d_in > TCL_I4_MAX_D_IN)
    return fail(TCL_EUNSUPPORTED, "i4: d_in %d beyond %d", w->d_in, TCL_I4_MAX_D_IN);
  if (w->d_out >= kMaxChannels) return fail(TCL_EUNSUPPORTED, "i4: d_out %d, 2^26 or more", w->d_out);
  if (w->d_out % 8) return fail(TCL_EALIGN, "i4: d_out %d is not a multiple of 8", w->d_out);
  if (w->zeros != 0 && w->zeros != 1) return fail(TCL_EINVAL, "i4: zeros %d is not 0 or 1", w->zeros);
  if (misaligned(w->W, 16) || misaligned(w->scale, 4) || misaligned(w->W_p, 256))
    return fail(TCL_EALIGN, "i4: W must be 16-byte, scale 4-byte, W_p 256-byte aligned");
  l->tiles = (int64_t(w->d_out) + 31) / 32;
  l->kb = (w->d_in + 127) / 128;
  l->groups = w->d_in / w->group;
  l->w = size_t(l->tiles) * l->kb * 2048;
  l->scale = l->w + size_t(l->tiles) * l->groups * 128;
  l->total = (l->scale + (w->zeros ? size_t(l->tiles) * l->groups * 32 : 0) + 255) / 256 * 256;
  if (l->total >= size_t(1) << 36) return fail(TCL_EUNSUPPORTED, "i4: a packed copy of 2^36 bytes or more");
  return TCL_OK;
}

template <int NB, int GS, bool ZP>
void go_rows(const I4Args &a, hipStream_t s) {
  hipLaunchKernelGGL((i4_rows<NB, GS, ZP>), dim3((a.N + 16 * NB - 1) / (16 * NB)), dim3(64 * kWaves), 0, s, a);
}

template <int NB, int GS, bool ZP>
void go_direct(const I4Args &a, hipStream_t s) {
  hipLaunchKernelGGL((i4_direct<NB, GS, ZP>),
                     dim3(unsigned((a.N + 32 * NB - 1) / (32 * NB)) * ((a.T + 31) / 32), a.ks), dim3(64 * kWaves),
                     0, s, a);
  if (a.ks > 1) {
    const int64_t n = (int64_t(a.T) * a.N / 4 + 255) / 256;
    hipLaunchKernelGGL(i4_join_kernel, dim3(unsigned(n < 2048 ? n : 2048)), dim3(256), 0, s, a);
  }
}

template <int GS>
void go_stage(const I4Args &a, hipStream_t s) {
  const StageArgs g{a.x, const_cast<nt_u4 *>(a.xb), const_cast<float *>(a.xe), a.ldx, a.T, a.K, a.kb, a.steps};
  hipLaunchKernelGGL(i4_stage_kernel<GS>, dim3((a.T + 31) / 32, (a.steps * (4 / GS) + 3) / 4), dim3(256), 0, s,
                     g);
}

template <int GS, bool ZP>
void go_blocks(const I4Args &a, hipStream_t s) {
  go_stage<GS>(a, s);
  constexpr int channels = 32 * kBlockTiles;
  hipLaunchKernelGGL((i4_blocks<GS, ZP>), dim3(unsigned((a.N + channels - 1) / channels) * ((a.T + 31) / 32)),
                     dim3(64 * kWaves), 0, s, a);
}

template <int BT, int GS, bool ZP>
void go_tile(I4Args a, hipStream_t s) {
  go_stage<GS>(a, s);
  a.nt = (a.T + BT - 1) / BT;
  a.nc = (a.N + 255) / 256;
  hipLaunchKernelGGL((i4_tile<BT, GS, ZP>), dim3((a.nt * a.nc + 7) / 8 * 8), dim3(512), 0, s, a);
}

template <int GS, bool ZP>
void product(const I4Args &a, hipStream_t s) {
  const Choice c = choose(a.T, a.N, a.kb, GS > 1);
  switch (c.kernel) {
    case Choice::kFew:
      return c.nb == 4 ? go_rows<4, GS, ZP>(a, s) : c.nb == 2 ? go_rows<2, GS, ZP>(a, s) : go_rows<1, GS, ZP>(a, s);
    case Choice::kDirect:
      if constexpr (GS == 1)
        if (c.nb == 4) return go_direct<4, GS, ZP>(a, s);
      return c.nb == 2 ? go_direct<2, GS, ZP>(a, s) : go_direct<1, GS, ZP>(a, s);
    case Choice::kBlocks:
      if constexpr (GS > 1) go_blocks<GS, ZP>(a, s);
      return;
    case Choice::kTile64:
      return go_tile<64, GS, ZP>(a, s);
    case Choice::kTile128:
      return go_tile<128, GS, ZP>(a, s);
  }
}

template <int GS>
void product(const I4Args &a, hipStream_t s) {
  if (a.zero)
    product<GS, true>(a, s);
  else
    product<GS, false>(a, s);
}

}  // namespace
}  // namespace tcl

using namespace tcl;

extern "C" int tcl_i4_pack_bytes(const tcl_i4_weight *w, size_t *bytes) {
  Layout l;
  if (!bytes) return fail(TCL_EINVAL, "i4: bytes is NULL");
  const int rc = check_weight(w, &l);
  if (rc) return rc;
  *bytes = l.total;
  return TCL_OK;
}

extern "C" int tcl_i4_pack(tcl_i4_weight *w, void *W_p, size_t bytes, void *stream) {
  Layout l;
  int rc = check_weight(w, &l);
  if (rc) return rc;
  if (!W_p) return fail(TCL_EINVAL, "i4: W_p is NULL");
  if (misaligned(W_p, 256)) return fail(TCL_EALIGN, "i4: W_p must be 256-byte aligned");
  if (bytes < l.total) return fail(TCL_ENOSPC, "i4: W_p holds %zu bytes, needs %zu", bytes, l.total);
  if (w->d_out > 0) {
    if (!w->W || !w->scale || (w->zeros && !w->zero)) return fail(TCL_EINVAL, "i4: weight arrays are NULL");
    uint8_t *p = static_cast<uint8_t *>(W_p);
    PackArgs a{w->W, w->zeros ? w->zero : nullptr, w->scale, p, p + l.scale,
               reinterpret_cast<float *>(p + l.w), w->d_in, w->d_out, l.kb, l.groups,
               int64_t(l.w / 16), int64_t(l.scale - l.w) / 4};
    const int64_t blocks = (a.n_w + 255) / 256;
    hipLaunchKernelGGL(i4_pack_kernel, dim3(unsigned(blocks < 1 << 16 ? blocks : 1 << 16)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    TCL_HIP(hipGetLastError());
  }
  w->W_p = W_p;
  return TCL_OK;
}

namespace tcl {
namespace {

// Bytes of the staged activations, with their sums, and of the parts of
// workgroups that share columns.
struct Space {
  size_t x, total;
  int32_t steps, ks;
};
Space space(const tcl_i4_weight *w, const Layout &l, int32_t n_tokens) {
  const int32_t groups = w->group < 128 ? l.groups : l.kb;  // longer ones count by their blocks
  const int32_t steps = (groups + 3) / 4;
  if (n_tokens == 0 || w->d_out == 0) return {0, 0, steps, 1};
  const Choice c = choose(n_tokens, w->d_out, l.kb, w->group < 128);
  if (c.kernel == Choice::kFew || c.kernel == Choice::kDirect)
    return {0, c.ks > 1 ? size_t(c.ks) * n_tokens * w->d_out * 4 : 0, steps, c.ks};
  const size_t tiles = (size_t(n_tokens) + 31) / 32, x = tiles * l.kb * 8192;
  return {x, x + tiles * steps * 512, steps, 1};
}

int check_tokens(const tcl_i4_weight *w, int32_t n_tokens) {
  if (n_tokens < 0) return fail(TCL_EINVAL, "i4: n_tokens %d < 0", n_tokens);
  if (n_tokens >= kMaxTokens) return fail(TCL_EUNSUPPORTED, "i4: n_tokens %d, 2^24 or more", n_tokens);
  if (int64_t(n_tokens) * w->d_out >= int64_t(1) << 36)
    return fail(TCL_EUNSUPPORTED, "i4: n_tokens * d_out of 2^36 or more");
  if (int64_t(n_tokens) * w->d_in >= int64_t(1) << 40)
    return fail(TCL_EUNSUPPORTED, "i4: n_tokens * d_in of 2^40 or more");
  return TCL_OK;
}

}  // namespace
}  // namespace tcl

extern "C" int tcl_i4_workspace_bytes(const tcl_i4_weight *w, int32_t n_tokens, size_t *bytes) {
  Layout l;
  if (!bytes) return fail(TCL_EINVAL, "i4: bytes is NULL");
  int rc = check_weight(w, &l);
  if (rc || (rc = check_tokens(w, n_tokens))) return rc;
  *bytes = space(w, l, n_tokens).total;
  return TCL_OK;
}

extern "C" int tcl_i4_linear(const tcl_i4_weight *w, const void *x, int64_t ldx, int32_t n_tokens, void *y,
                             int64_t ldy, tcl_dtype yd, void *ws, size_t ws_bytes, void *stream) {
  Layout l;
  int rc = check_weight(w, &l);
  if (rc || (rc = check_tokens(w, n_tokens))) return rc;
  if (yd != TCL_BF16 && yd != TCL_F32) return fail(TCL_EUNSUPPORTED, "i4: y dtype %d", int(yd));
  if (w->d_out == 0) return TCL_OK;  // nothing is written
  if (ldx < w->d_in || ldy < w->d_out) return fail(TCL_EINVAL, "i4: ldx < d_in or ldy < d_out");
  if (misaligned(x, 16) || misaligned(y, 16) || ldx % 8 || ldy % 8)
    return fail(TCL_EALIGN, "i4: x and y must be 16-byte aligned, ldx and ldy multiples of 8");
  if (n_tokens == 0) return TCL_OK;
  if (!x || !y || !w->W_p) return fail(TCL_EINVAL, "i4: x, y and the packed weight are required");
  const Space sp = space(w, l, n_tokens);
  if (sp.total) {
    if (!ws) return fail(TCL_EINVAL, "i4: ws is NULL");
    if (misaligned(ws, 256)) return fail(TCL_EALIGN, "i4: ws must be 256-byte aligned");
    if (ws_bytes < sp.total)
      return fail(TCL_ENOSPC, "i4: workspace holds %zu bytes, needs %zu", ws_bytes, sp.total);
  }
  const uint8_t *p = static_cast<const uint8_t *>(w->W_p);
  char *q = static_cast<char *>(ws);
  I4Args a{p, reinterpret_cast<const float *>(p + l.w), w->zeros ? p + l.scale : nullptr,
           static_cast<const uint16_t *>(x), y, ldx, ldy, n_tokens, w->d_in, w->d_out, l.kb, l.groups,
           w->group < 128 ? 0 : ((uint64_t(1) << 32) + w->group / 128 - 1) / (w->group / 128), reinterpret_cast<nt_u4 *>(q),
           reinterpret_cast<float *>(q + sp.x), sp.steps, 0, 0, sp.ks,
           reinterpret_cast<float *>(q), yd == TCL_F32};
  hipStream_t s = static_cast<hipStream_t>(stream);
  logf("i4: tokens=%d d_in=%d d_out=%d group=%d zeros=%d", a.T, a.K, a.N, w->group, w->zeros);
  if (w->group == 32)
    product<4>(a, s);
  else if (w->group == 64)
    product<2>(a, s);
  else
    product<1>(a, s);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}
