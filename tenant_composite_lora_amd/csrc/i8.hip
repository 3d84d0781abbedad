// Int8 base projections: token-scaled activations in 8 bits, their product
// with channel-scaled weights on the int8 matrix cores (include/tcl.h has the
// formulas).  Two product kernels:
//   i8_skinny  few tokens: the weight streams once from memory straight into
//              matrix-core operands, the waves of a workgroup split d_in and
//              add their integer sums in LDS;
//   i8_tile    many tokens: tiles of both operands go through LDS, three
//              stages deep, and the time is the matrix cores'.
// Integer sums are exact in any order, so neither split changes a result.
//
// Both read their operands in blocks of 16 rows by 64 bytes, the 16-byte
// chunk g of row r at 256 g + 16 r: the order in which the lanes of a wave
// take them, so that a load instruction reads 1 KiB in a row.  The packed
// weight (tcl_i8_pack) and the activations tcl_i8_linear rounds itself are
// stored so.  From rows in memory the same instruction touches 16 lines a row
// stride apart: 16 tokens, d_in 4096 to 4096 channels, 8.3 us for the product
// against 5.9 packed; 177 tokens, d_in 14336, 62 against 35.
#include <cmath>

#include "i8_index.hpp"
#include "kern_common.hpp"

namespace tcl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// activations to 8 bits
// ---------------------------------------------------------------------------
// chunks of 16 elements a thread keeps in registers between the two passes;
// longer rows are read again from L2
constexpr int kQKeep = 4;

struct QuantArgs {
  const void *x;
  int64_t ldx, ldq;
  int32_t T, d, kb, packed;
  int8_t *q;
  float *scale;
};

template <typename T>
struct Raw16;  // 16 elements as loaded

template <>
struct Raw16<bf16_t> {
  nt_u4 u[2];
  __device__ inline void load(const void *row, int c) {
    const nt_u4 *p = reinterpret_cast<const nt_u4 *>(row) + 2 * c;
    u[0] = p[0];
    u[1] = p[1];
  }
  __device__ inline float at(int i) const {
    const uint32_t w = u[i >> 3][(i >> 1) & 3];
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
  }
};

template <>
struct Raw16<float> {
  nt_f4 f[4];
  __device__ inline void load(const void *row, int c) {
    const nt_f4 *p = reinterpret_cast<const nt_f4 *>(row) + 4 * c;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = p[i];
  }
  __device__ inline float at(int i) const { return f[i >> 2][i & 3]; }
};

// The largest magnitude as raw bits without the sign: their order is the
// numbers' order, and a NaN (above infinity's bits) wins over everything.
template <typename R>
__device__ inline uint32_t absmax16(const R &c, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(c.at(i)) & 0x7fffffffu);
  return m;
}

// rint(v / s) of the real quotient.  The fp32 quotient is correctly rounded,
// so it leaves a tie's wrong side only by landing on the tie itself; there
// the remainder v - t * s, exact by fma, tells the side.  For scales below
// 2^-125 that remainder may be half the smallest number and round to zero, so
// small v and s are both raised by a power of two first, which is exact.
__device__ inline float round_quotient(float v, float s) {
  if (s < 0x1p-100f) v *= 0x1p64f, s *= 0x1p64f;
  const float t = v / s;
  float n = rintf(t);
  const float d = t - n;
  if (fabsf(d) == 0.5f) {
    const float rem = fmaf(-t, s, v);
    if (rem != 0.f) n = rem > 0.f ? ceilf(t) : floorf(t);
  }
  return fminf(fmaxf(n, -127.f), 127.f);
}

// 16 quotients to bytes.  v * inv, inv = 1 / s rounded, is off by less than
// 2^-22 of at most 127.5, so unless it lies within 2^-14 of a tie its nearest
// integer is the quotient's; four values of a wave rarely do (the full
// division on all of them costs as much time as the row's memory traffic).
// Below 2^-100 a scale's reciprocal is not relied on.
template <typename R>
__device__ inline i32x4 quant16(const R &x, float s, float inv) {
  i32x4 w = {0, 0, 0, 0};
  if (!(s > 0.f)) return w;  // a row of zeros, or a NaN scale
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float n[4], d = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = x.at(4 * i + j) * inv;
      n[j] = rintf(t);
      d = fmaxf(d, fabsf(t - n[j]));
    }
    if (d > 0.5f - 0x1p-14f || s < 0x1p-100f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) n[j] = round_quotient(x.at(4 * i + j), s);
    }
    // (bytes of n + 128, then the sign bit turned)
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) b = __builtin_amdgcn_cvt_pk_u8_f32(n[j] + 128.f, j, b);
    w[i] = int(b ^ 0x80808080u);
  }
  return w;
}

// WPR waves a row, ROWS rows a workgroup: a row is read once into registers,
// its largest magnitude reduced, the integers written.  A wave takes 1024
// elements at a time; with a wave a row, every wave is resident at once and
// all load, round and store in turn, with too many the short rows' idle ones
// cost.  bf16, us, 1 x 4, 2 x 4, 4 x 2, 8 x 1 waves and rows: 4224 x 1024: 7,
// 8, 11, 16; 4224 x 2048: 12, 11, 14, 19; 4224 x 4096: 20, 19, 18, 22 (52 MB);
// 4224 x 14336: 86, 70, 63, 75; 256 x 4096: 9.8, 6.7, 5.0, 5.3; 256 x 14336:
// 33, 19, 12, 9; 1024 x 5120: 14.5, 10.9, 10.3, 10.7.  (Two rows a wave, the
// second's loads ahead of the first's rounding: 21 for 17 at 4224 x 4096.)
template <typename T, int WPR, int ROWS>
__global__ __launch_bounds__(64 * WPR * ROWS) void i8_quant_kernel(QuantArgs a) {
  __shared__ uint32_t wmax[ROWS][WPR];
  constexpr int TH = 64 * WPR;
  const int tid = threadIdx.x % TH, r = threadIdx.x / TH;
  const int t = blockIdx.x * ROWS + r;
  const bool live = t < a.T;
  const char *row = static_cast<const char *>(a.x) + int64_t(live ? t : 0) * a.ldx * int64_t(sizeof(T));
  const int nc = live ? a.d / 16 : 0;
  Raw16<T> keep[kQKeep];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kQKeep; ++i)
    if (tid + i * TH < nc) keep[i].load(row, tid + i * TH);
#pragma unroll
  for (int i = 0; i < kQKeep; ++i)
    if (tid + i * TH < nc) m = absmax16(keep[i], m);
  for (int c = tid + kQKeep * TH; c < nc; c += TH) {
    Raw16<T> x;
    x.load(row, c);
    m = absmax16(x, m);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o, 64)));
  if constexpr (WPR > 1) {
    if ((tid & 63) == 0) wmax[r][tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) m = max(m, wmax[r][w]);
  }
  if (!live) return;
  const float s = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.f;
  const float inv = 1.f / s;
  if (tid == 0) a.scale[t] = s;
  auto put = [&](int c, i32x4 w) {
    int8_t *p = a.packed ? a.q + (int64_t(t >> 4) * a.kb + (c >> 2)) * 1024 + (c & 3) * 256 + (t & 15) * 16
                         : a.q + int64_t(t) * a.ldq + 16 * c;
    *reinterpret_cast<i32x4 *>(p) = w;
  };
#pragma unroll
  for (int i = 0; i < kQKeep; ++i)
    if (tid + i * TH < nc) put(tid + i * TH, quant16(keep[i], s, inv));
  for (int c = tid + kQKeep * TH; c < nc; c += TH) {
    Raw16<T> x;
    x.load(row, c);
    put(c, quant16(x, s, inv));
  }
  // the last block's chunks behind the row
  if (a.packed && tid < 4 * a.kb - nc) put(nc + tid, i32x4{0, 0, 0, 0});
}

// Rows to blocks, zeros behind them; a thread a chunk.
__global__ __launch_bounds__(256) void i8_pack_kernel(const int8_t *W, int32_t K, int32_t N,
                                                      int32_t kb, int8_t *out) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t blk = i >> 6;
  const int64_t rb = blk / kb;
  if (rb >= (N + 15) / 16) return;
  const int r = int(rb) * 16 + int(i & 15), k = int(blk % kb) * 64 + 16 * int((i >> 4) & 3);
  i32x4 v = {0, 0, 0, 0};
  if (r < N && k < K) v = *reinterpret_cast<const i32x4 *>(W + int64_t(r) * K + k);
  reinterpret_cast<i32x4 *>(out)[i] = v;
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
struct ProdArgs {
  Mat8 w, x;
  const float *ws, *xs;
  void *y;
  int64_t ldy;
  int32_t T, K, N;
  int32_t t0;      // first token
  int32_t nt, nc;  // i8_tile: token tiles, channel tiles
};

// four neighbouring channels of one token
template <typename TY>
__device__ inline void store_y4(const ProdArgs &a, int t, int c, i32x4 s, float xs) {
  const nt_f4 w = *reinterpret_cast<const nt_f4 *>(a.ws + c);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = float(s[i]) * xs * w[i];
  TY *p = static_cast<TY *>(a.y) + int64_t(t) * a.ldy + c;
  if constexpr (sizeof(TY) == 4) {
    *reinterpret_cast<nt_f4 *>(p) = nt_f4{v[0], v[1], v[2], v[3]};
  } else {
    *reinterpret_cast<nt_u2 *>(p) =
        nt_u2{uint32_t(f32_to_bf16(v[0])) | uint32_t(f32_to_bf16(v[1])) << 16,
              uint32_t(f32_to_bf16(v[2])) | uint32_t(f32_to_bf16(v[3])) << 16};
  }
}
template <typename TY>
__device__ inline void store_y4(const ProdArgs &a, int t, int c, i32x4 s) {
  store_y4<TY>(a, t, c, s, a.xs[t]);
}

// 16 * MB channels by 16 * NB tokens; wave w of WV takes the pairs of 64-byte
// blocks w, w + WV, ... of d_in.  v_mfma_i32_16x16x64_i8 with the weight's
// rows as the first operand: a lane of the result holds four channels of one
// token.  The operands of P pairs are in flight or in use at a time.  Bound by
// the weight's bytes at few tokens (16 x 4096 of 4096: 5.9 us, 2.9 TB/s; 64 x
// 14336: 16.8 us, 3.7 TB/s), by the activations' way from L2 at more: a
// workgroup reads (MB + NB) * 16 rows for MB * NB blocks of products (177 x
// 4096 of 14336: 33 us, 530 MB from L2).
template <int MB, int NB, int WV, int P, typename TY>
__global__ __launch_bounds__(64 * WV) void i8_skinny(ProdArgs a) {
  __shared__ i32x4 part[WV / 2][MB * NB][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c0 = blockIdx.x * 16 * MB, t0 = a.t0 + blockIdx.y * 16 * NB;
  const int r = lane & 15, g = lane >> 4;
  const int8_t *wp[MB], *xp[NB];
#pragma unroll
  for (int m = 0; m < MB; ++m) wp[m] = a.w.p + mat_at(a.w, c0 + 16 * m + r, g);
#pragma unroll
  for (int n = 0; n < NB; ++n) xp[n] = a.x.p + mat_at(a.x, t0 + 16 * n + r, g);
  const int sw = mat_step(a.w), sx = mat_step(a.x);
  const int kb = (a.K + 63) / 64;
  i32x4 acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = i32x4{0, 0, 0, 0};
  i32x4 wf[P][2][MB], xf[P][2][NB];
  auto load = [&](int p, int pair) {
    int b[2];
    bool in[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // past the row's end: any bytes of the weight times zeros
      in[h] = chunk_in(a.K, 2 * pair + h, g);
      b[h] = block_or_first(a.K, 2 * pair + h, g);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wf[p][h][m] = *reinterpret_cast<const i32x4 *>(wp[m] + int64_t(b[h]) * sw);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xf[p][h][n] = *reinterpret_cast<const i32x4 *>(xp[n] + int64_t(b[h]) * sx);
        if (!in[h]) xf[p][h][n] = i32x4{0, 0, 0, 0};
      }
  };
  const int pairs = (kb + 1) / 2;
#pragma unroll
  for (int p = 0; p < P; ++p) load(p, w + p * WV);
  for (int i = w; i < pairs; i += P * WV) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int n = 0; n < NB; ++n)
            acc[m][n] =
                __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[p][h][m], xf[p][h][n], acc[m][n], 0, 0, 0);
      load(p, i + (P + p) * WV);  // (zeros past the end)
    }
  }
  // the waves' sums, halves added to halves
#pragma unroll
  for (int s = WV / 2; s > 0; s >>= 1) {
    if (w >= s && w < 2 * s) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) part[w - s][m * NB + n][lane] = acc[m][n];
    }
    __syncthreads();
    if (w < s) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] += part[w][m * NB + n][lane];
    }
    if (s > 1) __syncthreads();
  }
  if (w == 0) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int c = c0 + 16 * m + 4 * g, t = t0 + 16 * n + r;
        if (c < a.N && t < a.T) store_y4<TY>(a, t, c, acc[m][n]);
      }
  }
}

// Up to kFewTok tokens in one launch: each workgroup rounds the tokens itself
// (16 channels, 8 waves; the weight's first operands are on their way
// meanwhile).  The integers lie in LDS, chunk c of token t at 16 (kFewTok c +
// t).  (One token, d_in 4096 to 1024 channels: 4.8 us, in two launches 7.4;
// two tokens 5.8; with four, the repeated rounding made it 9.3.)
constexpr int kFewTok = 2;
constexpr int kFewBytes = 32768;  // LDS for the integers

template <typename TX, typename TY>
__global__ __launch_bounds__(512) void i8_token(ProdArgs a, const void *x, int64_t ldx) {
  __shared__ i32x4 lq[kFewBytes / 16];
  __shared__ i32x4 part[4][64];
  __shared__ uint32_t wmax[kFewTok][8];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int c0 = blockIdx.x * 16, r = lane & 15, g = lane >> 4;
  const int8_t *wp = a.w.p + mat_at(a.w, c0 + r, g);
  const int sw = mat_step(a.w), kb = (a.K + 63) / 64, nc = a.K / 16;
  i32x4 wf[4];
  auto load = [&](int p, int b) {
    wf[p] = *reinterpret_cast<const i32x4 *>(wp + int64_t(block_or_first(a.K, b, g)) * sw);
  };
#pragma unroll
  for (int p = 0; p < 4; ++p) load(p, w + 8 * p);

  // (a chunk of 16 elements a thread; the second pass finds rows in L2)
  for (int t = 0; t < a.T; ++t) {
    const char *row = static_cast<const char *>(x) + t * ldx * int64_t(sizeof(TX));
    uint32_t v = 0;
    for (int c = tid; c < nc; c += 512) {
      Raw16<TX> e;
      e.load(row, c);
      v = absmax16(e, v);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, uint32_t(__shfl_xor(int(v), o, 64)));
    if (lane == 0) wmax[t][w] = v;
  }
  __syncthreads();
  float mine = 0.f;  // the scale of token r
  for (int t = 0; t < a.T; ++t) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v = max(v, wmax[t][i]);
    const float s = v >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(v) / 127.f;
    const float inv = 1.f / s;
    if (t == r) mine = s;
    const char *row = static_cast<const char *>(x) + t * ldx * int64_t(sizeof(TX));
    for (int c = tid; c < nc; c += 512) {
      Raw16<TX> e;
      e.load(row, c);
      lq[kFewTok * c + t] = quant16(e, s, inv);
    }
  }
  __syncthreads();
  i32x4 acc = {0, 0, 0, 0};
  for (int b = w; b < kb; b += 32) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int c = 4 * (b + 8 * p) + g;
      const i32x4 xf = r < a.T && c < nc ? lq[kFewTok * c + r] : i32x4{0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[p], xf, acc, 0, 0, 0);
      load(p, b + 8 * (p + 4));
    }
  }
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) {
    if (w >= s && w < 2 * s) part[w - s][lane] = acc;
    __syncthreads();
    if (w < s) acc += part[w][lane];
    if (s > 1) __syncthreads();
  }
  const int c = c0 + 4 * g;
  if (w == 0 && r < a.T && c < a.N) store_y4<TY>(a, r, c, acc, mine);
}

// BC channels by BT tokens, WC x WT waves, one 64-byte block of d_in a step.
// LDS holds three steps in the blocks' own order, which every operand load
// reads in a row.  At the end of a step its successor lies in LDS whole, so a
// wave reads its next operands before the barrier and goes on multiplying
// behind it; the step after that is written from registers, and the loads of
// the one after go out.  Reads and writes are dealt out among the matrix
// instructions (sched_group_barrier): issued in one go they held the first
// one back by some hundred cycles a step (256 x 256 tiles of 4096 tokens x
// 4096 channels, one a CU: 115 us, dealt out 97).
// 4224 x 14336 of d_in 4096: 264 us, 1.9 P operations a second.  Operand reads
// and matrix instructions alone take 250 us at that size on random bytes, with
// 64 workgroups instead of 952 they run at twice that rate: the clock bounds
// it.
template <int BC, int BT, int WC, int WT, typename TY>
__global__ __launch_bounds__(64 * WC * WT, 2) void i8_tile(ProdArgs a) {
  constexpr int TH = 64 * WC * WT;
  constexpr int NW = BC * 4 / TH, NX = BT * 4 / TH;      // chunks a thread moves a step
  constexpr int FC = BC / WC / 32, FT = BT / WT / 32;    // 32-row operands of a wave
  __shared__ struct {
    i32x4 w[3][BC * 4], x[3][BT * 4];
  } l;
  auto &lw = l.w;
  auto &lx = l.x;
  float *lo = reinterpret_cast<float *>(&l);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  // workgroups go to the eight XCDs in turn: each gets a run of tiles, token
  // tiles next to each other, so that its L2 holds their weight rows
  const int n = a.nt * a.nc, per = (n + 7) / 8;
  const int id = int(blockIdx.x & 7) * per + int(blockIdx.x >> 3);
  if (int(blockIdx.x >> 3) >= per || id >= n) return;
  const int c0 = id / a.nt * BC, t0 = a.t0 + id % a.nt * BT;

  const int kb = (a.K + 63) / 64, sw = mat_step(a.w), sx = mat_step(a.x);
  const int8_t *pw[NW], *px[NX];
  const int g = (tid >> 4) & 3;  // the thread's chunk of a block's row
#pragma unroll
  for (int i = 0; i < NW; ++i)
    pw[i] = a.w.p + mat_at(a.w, c0 + ((tid + i * TH) >> 6) * 16 + (tid & 15), g);
#pragma unroll
  for (int i = 0; i < NX; ++i)
    px[i] = a.x.p + mat_at(a.x, t0 + ((tid + i * TH) >> 6) * 16 + (tid & 15), g);
  i32x4 rw[NW], rx[NX];
  auto load = [&](int st) {
    const int b = block_or_first(a.K, st, g);
#pragma unroll
    for (int i = 0; i < NW; ++i)
      rw[i] = *reinterpret_cast<const i32x4 *>(pw[i] + int64_t(b) * sw);
#pragma unroll
    for (int i = 0; i < NX; ++i)
      rx[i] = *reinterpret_cast<const i32x4 *>(px[i] + int64_t(b) * sx);
  };
  auto put = [&](int b, int st) {
    const bool in = chunk_in(a.K, st, g);  // zeros past the row's end
#pragma unroll
    for (int i = 0; i < NW; ++i) lw[b][tid + i * TH] = rw[i];
#pragma unroll
    for (int i = 0; i < NX; ++i) lx[b][tid + i * TH] = in ? rx[i] : i32x4{0, 0, 0, 0};
  };
  i32x16 acc[FC][FT];
#pragma unroll
  for (int i = 0; i < FC; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  const int r = lane & 31, h = lane >> 5;
  // operand rows r, r + 32, ... of the wave, chunk 2 s + h
  const int aw = (w % WC) * (BC / WC) * 4 + (r >> 4) * 64 + h * 16 + (r & 15);
  const int ax = (w / WC) * (BT / WT) * 4 + (r >> 4) * 64 + h * 16 + (r & 15);
  i32x4 fw[2][FC], fx[2][FT];
  auto read = [&](int b, int s) {
#pragma unroll
    for (int i = 0; i < FC; ++i) fw[s][i] = lw[b][aw + i * 128 + s * 32];
#pragma unroll
    for (int i = 0; i < FT; ++i) fx[s][i] = lx[b][ax + i * 128 + s * 32];
  };
  auto multiply = [&](int s) {
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[s][i], fx[s][j], acc[i][j], 0, 0, 0);
  };
  // (LDS only: global loads stay in flight across it)
  auto barrier = [&] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };
  constexpr int M = FC * FT, RD = FC + FT, WR = NW + NX, WRI = (WR + M / 2 - 1) / (M / 2);
  load(0);
  put(0, 0);
  load(1);
  put(1, 1);
  load(2);
  barrier();
  read(0, 0);
  int b0 = 0, b1 = 1, b2 = 2;
  for (int st = 0; st < kb; ++st) {
    read(b0, 1);
    put(b2, st + 2);
    load(st + 3);
    multiply(0);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);                  // a matrix instruction
      if (i < RD) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // an LDS read
      if (i >= M / 2) {
        __builtin_amdgcn_sched_group_barrier(0x200, WRI, 0);            // LDS writes
        __builtin_amdgcn_sched_group_barrier(0x20, WRI, 0);             // loads
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    read(b1, 0);
    multiply(1);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      if (i < RD) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    const int t = b0;
    b0 = b1, b1 = b2, b2 = t;
  }
  // The results go through LDS, a wave's 32 tokens at a time, so that a store
  // covers whole lines of y: straight from the registers (16 bytes a token
  // and lane half) fp32 rows were written to memory twice over, 133 MB for 67.
  constexpr int CW = BC / WC, LD = CW + 4;  // channels of a wave; row of LDS, floats
  static_assert(WC * WT * 32 * LD * 4 <= int(sizeof(l)), "LDS of the results");
  const int wc = c0 + (w % WC) * CW, wt = t0 + (w / WC) * (BT / WT);
  float *out = lo + w * 32 * LD;
  nt_f4 ws[FC][4];
#pragma unroll
  for (int i = 0; i < FC; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      ws[i][e] = *reinterpret_cast<const nt_f4 *>(a.ws + min(wc + 32 * i + 8 * e + 4 * h, a.N - 4));
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const float xs = a.xs[min(wt + 32 * j + r, a.T - 1)];
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        nt_f4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = float(acc[i][j][4 * e + x]) * xs * ws[i][e][x];
        *reinterpret_cast<nt_f4 *>(out + r * LD + 32 * i + 8 * e + 4 * h) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    constexpr int PER = sizeof(TY) == 4 ? 4 : 8;          // channels a lane stores: 16 bytes
    constexpr int LPT = CW / PER;                          // lanes a token
#pragma unroll
    for (int k = 0; k < LPT / 2; ++k) {
      const int x = k * (64 / LPT) + lane / LPT, t = wt + 32 * j + x, c = wc + lane % LPT * PER;
      const float *in = out + x * LD + lane % LPT * PER;
      if (t >= a.T || c >= a.N) continue;
      TY *p = static_cast<TY *>(a.y) + int64_t(t) * a.ldy + c;
      const nt_f4 u = *reinterpret_cast<const nt_f4 *>(in);
      if constexpr (sizeof(TY) == 4) {
        *reinterpret_cast<nt_f4 *>(p) = u;
      } else {
        const nt_f4 v = *reinterpret_cast<const nt_f4 *>(in + 4);
        auto two = [](float x0, float x1) {
          return uint32_t(f32_to_bf16(x0)) | uint32_t(f32_to_bf16(x1)) << 16;
        };
        *reinterpret_cast<nt_u4 *>(p) =
            nt_u4{two(u[0], u[1]), two(u[2], u[3]), two(v[0], v[1]), two(v[2], v[3])};
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
  }
}

// ---------------------------------------------------------------------------
// checks and launches
// ---------------------------------------------------------------------------
bool misaligned(const void *p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) & (m - 1); }

// A launch's threads stay below 2^32: 512 for 16 channels (few tokens), up to
// 256 a token (quantiser), 512 for 128 x 128 results (tiles), one for 16 bytes
// of a packed copy.
constexpr int kMaxChannels = 1 << 27, kMaxTokens = 1 << 24;
constexpr int64_t kMaxResults = int64_t(1) << 36;
constexpr size_t kMaxPacked = size_t(1) << 36;

int check_weight(const tcl_i8_weight *w) {
  if (!w) return fail(TCL_EINVAL, "i8: weight is NULL");
  if (w->d_in < 16 || w->d_out < 0)
    return fail(TCL_EINVAL, "i8: d_in %d < 16 or d_out %d < 0", w->d_in, w->d_out);
  if (w->d_in > TCL_I8_MAX_D_IN)
    return fail(TCL_EUNSUPPORTED, "i8: d_in %d beyond %d", w->d_in, TCL_I8_MAX_D_IN);
  if (w->d_out >= kMaxChannels)
    return fail(TCL_EUNSUPPORTED, "i8: d_out %d, 2^27 or more", w->d_out);
  if (w->d_in % 16 || w->d_out % 8)
    return fail(TCL_EALIGN, "i8: d_in %d is not a multiple of 16 or d_out %d not of 8", w->d_in,
                w->d_out);
  if (w->d_out > 0 && ((!w->W && !w->W_p) || !w->scale)) return fail(TCL_EINVAL, "i8: weight arrays are NULL");
  if (misaligned(w->W, 16) || misaligned(w->W_p, 256))
    return fail(TCL_EALIGN, "i8: W must be 16-byte, W_p 256-byte aligned");
  if (misaligned(w->scale, 4)) return fail(TCL_EALIGN, "i8: scale must be 4-byte aligned");
  return TCL_OK;
}

int check_quant(const void *x, int64_t ldx, int xd, int32_t n_tokens, int32_t d) {
  if (n_tokens < 0 || d < 16)
    return fail(TCL_EINVAL, "i8: n_tokens %d < 0 or d %d < 16", n_tokens, d);
  if (xd != TCL_BF16 && xd != TCL_F32) return fail(TCL_EUNSUPPORTED, "i8: x dtype %d", xd);
  if (n_tokens >= kMaxTokens) return fail(TCL_EUNSUPPORTED, "i8: n_tokens %d, 2^24 or more", n_tokens);
  if (ldx < d) return fail(TCL_EINVAL, "i8: ldx < d");
  if (d % 16 || ldx % 8) return fail(TCL_EALIGN, "i8: d must be a multiple of 16, ldx of 8");
  if (n_tokens > 0 && !x) return fail(TCL_EINVAL, "i8: x is NULL");
  if (misaligned(x, 16)) return fail(TCL_EALIGN, "i8: x must be 16-byte aligned");
  return TCL_OK;
}

int check_y(const tcl_i8_weight *w, int32_t n_tokens, const void *y, int64_t ldy, int yd) {
  if (n_tokens < 0) return fail(TCL_EINVAL, "i8: n_tokens %d < 0", n_tokens);
  if (yd != TCL_BF16 && yd != TCL_F32) return fail(TCL_EUNSUPPORTED, "i8: y dtype %d", yd);
  if (n_tokens >= kMaxTokens) return fail(TCL_EUNSUPPORTED, "i8: n_tokens %d, 2^24 or more", n_tokens);
  if (int64_t(n_tokens) * w->d_out >= kMaxResults)
    return fail(TCL_EUNSUPPORTED, "i8: n_tokens * d_out of 2^36 or more");
  if (w->d_out == 0) return TCL_OK;  // nothing is written
  if (ldy < w->d_out) return fail(TCL_EINVAL, "i8: ldy < d_out");
  if (n_tokens > 0 && !y) return fail(TCL_EINVAL, "i8: y is NULL");
  if (misaligned(y, 16) || ldy % 8)
    return fail(TCL_EALIGN, "i8: y must be 16-byte aligned, ldy a multiple of 8");
  return TCL_OK;
}

int32_t blocks_of(int32_t d) { return (d + 63) / 64; }

int launch_quant(const void *x, int64_t ldx, int xd, int32_t n, int32_t d, int8_t *q, int64_t ldq,
                 bool packed, float *scale, hipStream_t s) {
  if (n == 0) return TCL_OK;
  QuantArgs a{x, ldx, ldq, n, d, blocks_of(d), packed, q, scale};
#define QUANT(T, W, R) \
  hipLaunchKernelGGL((i8_quant_kernel<T, W, R>), dim3((n + R - 1) / R), dim3(64 * W * R), 0, s, a)
#define QUANT_D(T)                       \
  if (d <= 1024) QUANT(T, 1, 4);         \
  else if (d <= 2048 || n > 1 << 23) QUANT(T, 2, 4); /* (128 threads a token) */ \
  else if (d <= 4096 || n > 512) QUANT(T, 4, 2); \
  else QUANT(T, 8, 1)
  if (xd == TCL_BF16) {
    QUANT_D(bf16_t);
  } else {
    QUANT_D(float);
  }
#undef QUANT_D
#undef QUANT
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

template <int MB, int NB, int WV, int P, typename TY>
void go_skinny(const ProdArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((i8_skinny<MB, NB, WV, P, TY>),
                     dim3((a.N + 16 * MB - 1) / (16 * MB), (a.T - a.t0 + 16 * NB - 1) / (16 * NB)),
                     dim3(64 * WV), 0, s, a);
}

template <int BC, int BT, int WC, int WT, typename TY>
void go_tile(ProdArgs a, hipStream_t s) {
  a.nt = (a.T - a.t0 + BT - 1) / BT;
  a.nc = (a.N + BC - 1) / BC;
  hipLaunchKernelGGL((i8_tile<BC, BT, WC, WT, TY>), dim3((a.nt * a.nc + 7) / 8 * 8),
                     dim3(64 * WC * WT), 0, s, a);
}

// Which kernel: by how many workgroups each would have, for 256 CUs (us on
// packed operands of uniform random bytes, d_in 4096 unless said).
//   up to 16 tokens: 16 channels a workgroup, 8 waves over d_in (1 token,
//     1024 channels: 4.1; 32 channels: 5.5);
//   up to 32: the same with two token blocks (4096 channels: 7.4; 32: 8.3);
//   more, as long as 128 x 128 tiles are fewer than 192 (and further for up
//     to 64 tokens, few_wide): by what runs in one
//     round, two workgroups a CU (with the quantiser): 32 channels x 64
//     tokens, 4 waves, up to 512 of them (256 x 4096: 22.2; 64 x 48 24.2; 64 x
//     64 27.2), else 64 x 48 (333 x 4096: 24.8, 32 x 64 28.8, 64 x 64 28.5; 72
//     x 14336: 27.7, 34.8, 31.0), else 64 x 64 (100 x 14336: 31.4, 32 x 64
//     36.5, 64 x 48 35.6), else 64 x 48 again (560 x 4096: 34.6, 40.7, 38.3);
//     and 32 x 32 with 8 waves where 32 x 64 are at most 256 (128 x 4096:
//     17.2, 32 x 64 19.0).
// Tiles: by whole rounds over the CUs, two workgroups of 128 x 128 or 256 x
// 128 each or one of 256 x 256 (tile_cost).
template <typename TY>
void product_skinny(const ProdArgs &a, hipStream_t s) {
  const int64_t t = a.T - a.t0, tb = (t + 63) / 64, n64 = (a.N + 63) / 64, n32 = (a.N + 31) / 32;
  if (t <= 16)
    go_skinny<1, 1, 8, 2, TY>(a, s);
  else if (t <= 32)
    go_skinny<1, 2, 8, 2, TY>(a, s);
  else if (tb * n32 <= 256)
    go_skinny<2, 2, 8, 2, TY>(a, s);
  else if (tb * n32 <= 512)
    go_skinny<2, 4, 4, 2, TY>(a, s);
  else if ((t + 47) / 48 * n64 > 512 && tb * n64 <= 512)
    go_skinny<4, 4, 4, 2, TY>(a, s);
  else
    go_skinny<4, 3, 4, 2, TY>(a, s);
}

enum Kernel { kSkinny, kTile11, kTile21, kTile22 };

int64_t tiles(int64_t n, int64_t d) { return (n + d - 1) / d; }

// What a kernel costs, in tenths of 8 us at d_in 4096 (every one's time grows
// with d_in alike).  Measured with the quantiser, us: 1024 x 4096: tiles of
// 128 x 128 39, 256 x 128 48, 256 x 256 63; 2048: 61, 59, 68; 2304: 75, 78,
// 69; 4096: 108, 96, 89; 5120: 132, 128, 140; 6144: 154, 138, 148; 8192: 202,
// 178, 172; 2048 x 14336: 159, 155, 142; 4224 x 14336: 338, 301, 288.
int64_t tile_cost(Kernel k, int64_t T, int64_t N) {
  switch (k) {
    case kSkinny: return 10 + 22 * T * N / (1 << 20);
    case kTile11: return 20 + 25 * tiles(tiles(T, 128) * tiles(N, 128), 256);
    case kTile21: return 50 * tiles(tiles(T, 128) * tiles(N, 256), 256);
    default: return 90 * tiles(tiles(T, 256) * tiles(N, 256), 256);
  }
}

Kernel cheapest(int64_t T, int64_t N, int64_t *cost) {
  Kernel best = kSkinny;
  if (T > 32 && tiles(T, 128) * tiles(N, 128) >= 192) {
    best = kTile11;
    for (Kernel k : {kTile21, kTile22})
      if (tile_cost(k, T, N) < tile_cost(best, T, N)) best = k;
  }
  *cost = tile_cost(best, T, N);
  return best;
}

// Up to 64 tokens leave half of every 128 x 128 tile to padding, while one
// round of 64-channel blocks reads the weight once as well.  Blocks and tiles,
// us, 48 and 64 tokens: d_in 14336, 24576 channels 87, 98 and 142, 143; 32768
// 98, 107 and 148, 149; 8192 x 32768 54, 57 and 77, 77; 4096 x 24576 29, 31
// and 32, 33; 4096 x 32768 33, 36 and 34, 34.  Past one round: 14336 x 33024
// 132, 203 and 161, 162.  Shorter rows: 2560 x 28672 25, 28 and 25, 26; 1536
// 21, 23 and 19, 19.
bool few_wide(int64_t T, int64_t K, int64_t N) { return T <= 64 && K >= 4096 && tiles(N, 64) <= 512; }

template <typename TY>
void go(Kernel k, const ProdArgs &a, hipStream_t s) {
  switch (k) {
    case kSkinny: product_skinny<TY>(a, s); break;
    case kTile11: go_tile<128, 128, 4, 2, TY>(a, s); break;
    case kTile21: go_tile<256, 128, 4, 2, TY>(a, s); break;
    default: go_tile<256, 256, 4, 2, TY>(a, s); break;
  }
}

template <typename TY>
void product(ProdArgs &a, hipStream_t s) {
  int64_t cost, rest_cost;
  if (few_wide(a.T, a.K, a.N)) return product_skinny<TY>(a, s);
  const Kernel k = cheapest(a.T, a.N, &cost);
  // or the tokens of whole rounds of the largest tiles, and the rest in a
  // launch of their own (4224 x 4096: 107 in one launch, 101)
  const int64_t nc = tiles(a.N, 256), rounds = tiles(a.T, 256) * nc / 256;
  const int T = a.T, first = int(rounds * 256 / nc * 256);
  if (first > 0 && first < T) {
    const Kernel rest = cheapest(T - first, a.N, &rest_cost);
    if (90 * rounds + rest_cost < cost) {
      a.T = first;
      go<TY>(kTile22, a, s);
      a.t0 = first;
      a.T = T;
      return go<TY>(rest, a, s);
    }
  }
  go<TY>(k, a, s);
}

Mat8 weight_of(const tcl_i8_weight *w) {
  const int32_t kb = blocks_of(w->d_in);
  return w->W_p ? Mat8{static_cast<const int8_t *>(w->W_p), 0, w->d_out, w->d_in / 16, kb, 1}
                : Mat8{w->W, w->d_in, w->d_out, w->d_in / 16, kb, 0};
}

int launch_product(const tcl_i8_weight *w, const Mat8 &x, const float *scale, void *y, int64_t ldy,
                   int yd, hipStream_t s) {
  if (x.n == 0 || w->d_out == 0) return TCL_OK;
  ProdArgs a{weight_of(w), x, w->scale, scale, y, ldy, x.n, w->d_in, w->d_out, 0, 0, 0};
  logf("i8 product: tokens=%d d_in=%d d_out=%d packed=%d", x.n, w->d_in, w->d_out, a.w.packed);
  if (yd == TCL_BF16)
    product<uint16_t>(a, s);
  else
    product<float>(a, s);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

int launch_token(const tcl_i8_weight *w, const void *x, int64_t ldx, int xd, int32_t n, void *y,
                 int64_t ldy, int yd, hipStream_t s) {
  ProdArgs a{weight_of(w), {}, w->scale, nullptr, y, ldy, n, w->d_in, w->d_out, 0, 0, 0};
  const dim3 grid((w->d_out + 15) / 16), block(512);
#define TOKEN(TX, TY) hipLaunchKernelGGL((i8_token<TX, TY>), grid, block, 0, s, a, x, ldx)
  if (xd == TCL_BF16) {
    if (yd == TCL_BF16) TOKEN(bf16_t, uint16_t);
    else TOKEN(bf16_t, float);
  } else {
    if (yd == TCL_BF16) TOKEN(float, uint16_t);
    else TOKEN(float, float);
  }
#undef TOKEN
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

// workspace of tcl_i8_linear: the integers in blocks, then the scales
size_t ws_q_bytes(const tcl_i8_weight *w, int32_t n) {
  return (size_t(n) + 15) / 16 * size_t(blocks_of(w->d_in)) * 1024;
}

size_t ws_bytes_of(const tcl_i8_weight *w, int32_t n) {
  return ws_q_bytes(w, n) + (size_t(n) * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace tcl

using namespace tcl;

extern "C" int tcl_i8_quant(const void *x, int64_t ldx, tcl_dtype xd, int32_t n_tokens, int32_t d,
                            int8_t *q, int64_t ldq, float *scale, void *stream) {
  int rc = check_quant(x, ldx, xd, n_tokens, d);
  if (rc) return rc;
  if (ldq < d) return fail(TCL_EINVAL, "i8: ldq < d");
  if (n_tokens > 0 && (!q || !scale)) return fail(TCL_EINVAL, "i8: q and scale are required");
  if (misaligned(q, 16) || ldq % 16)
    return fail(TCL_EALIGN, "i8: q must be 16-byte aligned, ldq a multiple of 16");
  if (misaligned(scale, 4)) return fail(TCL_EALIGN, "i8: scale must be 4-byte aligned");
  return launch_quant(x, ldx, xd, n_tokens, d, q, ldq, false, scale,
                      static_cast<hipStream_t>(stream));
}

extern "C" int tcl_i8_product(const tcl_i8_weight *w, const int8_t *q, int64_t ldq,
                              const float *scale, int32_t n_tokens, void *y, int64_t ldy,
                              tcl_dtype yd, void *stream) {
  int rc = check_weight(w);
  if (rc) return rc;
  if ((rc = check_y(w, n_tokens, y, ldy, yd))) return rc;
  if (ldq < w->d_in) return fail(TCL_EINVAL, "i8: ldq < d_in");
  if (n_tokens > 0 && (!q || !scale)) return fail(TCL_EINVAL, "i8: q and scale are required");
  if (misaligned(q, 16) || ldq % 16)
    return fail(TCL_EALIGN, "i8: q must be 16-byte aligned, ldq a multiple of 16");
  if (misaligned(scale, 4)) return fail(TCL_EALIGN, "i8: scale must be 4-byte aligned");
  return launch_product(w, Mat8{q, ldq, n_tokens, w->d_in / 16, blocks_of(w->d_in), 0}, scale, y,
                        ldy, yd, static_cast<hipStream_t>(stream));
}

extern "C" int tcl_i8_pack_bytes(const tcl_i8_weight *w, size_t *bytes) {
  if (!bytes) return fail(TCL_EINVAL, "i8: bytes is NULL");
  int rc = check_weight(w);
  if (rc) return rc;
  *bytes = (size_t(w->d_out) + 15) / 16 * size_t(blocks_of(w->d_in)) * 1024;
  return TCL_OK;
}

extern "C" int tcl_i8_pack(tcl_i8_weight *w, void *W_p, size_t bytes, void *stream) {
  size_t need = 0;
  int rc = tcl_i8_pack_bytes(w, &need);
  if (rc) return rc;
  if (w->d_out == 0) return TCL_OK;
  if (need >= kMaxPacked) return fail(TCL_EUNSUPPORTED, "i8: a packed copy of 2^36 bytes or more");
  if (!w->W || !W_p) return fail(TCL_EINVAL, "i8: pack needs W and W_p");
  if (misaligned(W_p, 256)) return fail(TCL_EALIGN, "i8: W_p must be 256-byte aligned");
  if (bytes < need) return fail(TCL_ENOSPC, "i8: W_p holds %zu bytes, needs %zu", bytes, need);
  hipLaunchKernelGGL(i8_pack_kernel, dim3(unsigned((need / 16 + 255) / 256)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), w->W, w->d_in, w->d_out,
                     blocks_of(w->d_in), static_cast<int8_t *>(W_p));
  TCL_HIP(hipGetLastError());
  w->W_p = W_p;
  return TCL_OK;
}

extern "C" int tcl_i8_workspace_bytes(const tcl_i8_weight *w, int32_t n_tokens, size_t *bytes) {
  if (!bytes) return fail(TCL_EINVAL, "i8: bytes is NULL");
  int rc = check_weight(w);
  if (rc) return rc;
  if (n_tokens < 0) return fail(TCL_EINVAL, "i8: n_tokens %d < 0", n_tokens);
  *bytes = ws_bytes_of(w, n_tokens);
  return TCL_OK;
}

extern "C" int tcl_i8_linear(const tcl_i8_weight *w, const void *x, int64_t ldx, tcl_dtype xd,
                             int32_t n_tokens, void *y, int64_t ldy, tcl_dtype yd, void *ws,
                             size_t ws_bytes, void *stream) {
  int rc = check_weight(w);
  if (rc) return rc;
  if ((rc = check_quant(x, ldx, xd, n_tokens, w->d_in))) return rc;
  if ((rc = check_y(w, n_tokens, y, ldy, yd))) return rc;
  if (n_tokens == 0) return TCL_OK;
  if (!ws) return fail(TCL_EINVAL, "i8: workspace is NULL");
  if (misaligned(ws, 256)) return fail(TCL_EALIGN, "i8: workspace must be 256-byte aligned");
  const size_t need = ws_bytes_of(w, n_tokens);
  if (ws_bytes < need)
    return fail(TCL_ENOSPC, "i8: workspace holds %zu bytes, needs %zu", ws_bytes, need);
  if (n_tokens <= kFewTok && w->d_in <= kFewBytes / kFewTok && w->d_out > 0)
    return launch_token(w, x, ldx, xd, n_tokens, y, ldy, yd, static_cast<hipStream_t>(stream));
  int8_t *q = static_cast<int8_t *>(ws);
  float *scale = reinterpret_cast<float *>(q + ws_q_bytes(w, n_tokens));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((rc = launch_quant(x, ldx, xd, n_tokens, w->d_in, q, 0, true, scale, s))) return rc;
  return launch_product(w, Mat8{q, 0, n_tokens, w->d_in / 16, blocks_of(w->d_in), 1}, scale, y, ldy,
                        yd, s);
}
