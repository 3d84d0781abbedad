// Int8 base projections: token-scaled activations in 8 bits, their product
// with channel-scaled weights on the int8 matrix cores (include/tcl.h has the
// formulas).  Two product kernels:
//   i8_skinny  few tokens: the weight streams once from memory straight into
//              matrix-core operands, the waves of a workgroup split d_in and
//              add their integer sums in LDS;
//   i8_tile    many tokens: tiles of both operands go through LDS, double
//              buffered, and the time is the matrix cores'.
// Integer sums are exact in any order, so neither split changes a result.
#include <cmath>

#include "kern_common.hpp"

namespace tcl {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// activations to 8 bits
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;
// chunks of 16 elements a thread keeps in registers between the two passes;
// longer rows are read again from L2
constexpr int kQKeep = 4;

struct QuantArgs {
  const void *x;
  int64_t ldx, ldq;
  int32_t d;
  int8_t *q;
  float *scale;
};

struct Chunk16 {
  float v[16];
};

template <typename T>
__device__ inline void load16(const void *row, int c, Chunk16 &o);

template <>
__device__ inline void load16<bf16_t>(const void *row, int c, Chunk16 &o) {
  const uint4 *p = reinterpret_cast<const uint4 *>(row) + 2 * c;
  uint4 u[2] = {p[0], p[1]};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[8 * h + 2 * i] = bf16_lo(w[i]);
      o.v[8 * h + 2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

template <>
__device__ inline void load16<float>(const void *row, int c, Chunk16 &o) {
  const float4 *p = reinterpret_cast<const float4 *>(row) + 4 * c;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 f = p[h];
    o.v[4 * h] = f.x;
    o.v[4 * h + 1] = f.y;
    o.v[4 * h + 2] = f.z;
    o.v[4 * h + 3] = f.w;
  }
}

// The largest magnitude as raw bits without the sign: their order is the
// numbers' order, and a NaN (above infinity's bits) wins over everything.
__device__ inline uint32_t absmax16(const Chunk16 &c, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(c.v[i]) & 0x7fffffffu);
  return m;
}

// rint(v / s) of the real quotient.  The fp32 quotient is correctly rounded,
// so it leaves a tie's wrong side only by landing on the tie itself; there
// the remainder v - t * s, exact by fma, tells the side.
__device__ inline int round_quotient(float v, float s) {
  const float t = v / s;
  float n = rintf(t);
  const float d = t - n;
  if (fabsf(d) == 0.5f) {
    const float rem = fmaf(-t, s, v);
    if (rem != 0.f) n = rem > 0.f ? ceilf(t) : floorf(t);
  }
  return int(fminf(fmaxf(n, -127.f), 127.f));
}

__device__ inline void store_q(int8_t *row, int c, const Chunk16 &x, float s) {
  const bool zero = !(s > 0.f);  // a row of zeros, or a NaN scale
  int w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b |= uint32_t(uint8_t(zero ? 0 : round_quotient(x.v[4 * i + j], s))) << (8 * j);
    w[i] = int(b);
  }
  reinterpret_cast<i32x4 *>(row)[c] = i32x4{w[0], w[1], w[2], w[3]};
}

// One workgroup a token: the row is read once into registers, its largest
// magnitude reduced, the integers written.
template <typename T>
__global__ __launch_bounds__(kQThreads) void i8_quant_kernel(QuantArgs a) {
  __shared__ uint32_t wmax[kQThreads / 64];
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const char *row = static_cast<const char *>(a.x) + t * a.ldx * int64_t(sizeof(T));
  int8_t *qrow = a.q + t * a.ldq;
  const int nc = a.d / 16;
  Chunk16 keep[kQKeep];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kQKeep; ++i) {
    const int c = tid + i * kQThreads;
    if (c < nc) {
      load16<T>(row, c, keep[i]);
      m = absmax16(keep[i], m);
    }
  }
  for (int c = tid + kQKeep * kQThreads; c < nc; c += kQThreads) {
    Chunk16 x;
    load16<T>(row, c, x);
    m = absmax16(x, m);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o, 64)));
  if ((tid & 63) == 0) wmax[tid >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 64; ++w) m = max(m, wmax[w]);
  const float s = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.f;
  if (tid == 0) a.scale[t] = s;
#pragma unroll
  for (int i = 0; i < kQKeep; ++i) {
    const int c = tid + i * kQThreads;
    if (c < nc) store_q(qrow, c, keep[i], s);
  }
  for (int c = tid + kQKeep * kQThreads; c < nc; c += kQThreads) {
    Chunk16 x;
    load16<T>(row, c, x);
    store_q(qrow, c, x, s);
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
struct ProdArgs {
  const int8_t *W, *q;
  const float *ws, *xs;
  void *y;
  int64_t ldq, ldy;
  int32_t T, K, N;
  int32_t nt, nc;  // i8_tile: token tiles, channel tiles
};

// four neighbouring channels of one token
template <typename TY>
__device__ inline void store_y4(const ProdArgs &a, int t, int c, i32x4 s) {
  const float xs = a.xs[t];
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

// 16 * MB channels by 16 * NB tokens; wave w of WV takes the 128-byte groups
// of d_in w, w + WV, ...  v_mfma_i32_16x16x64_i8 with the weight's rows as
// the first operand: a lane of the result holds four channels of one token.
// U groups are loaded before their products.
template <int MB, int NB, int WV, int U, typename TY>
__global__ __launch_bounds__(64 * WV) void i8_skinny(ProdArgs a) {
  __shared__ i32x4 part[WV][MB * NB][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c0 = blockIdx.x * 16 * MB, t0 = blockIdx.y * 16 * NB;
  const int r = lane & 15, kg = 16 * (lane >> 4);
  const int8_t *wp[MB], *xp[NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
    wp[m] = a.W + int64_t(min(c0 + 16 * m + r, a.N - 1)) * a.K;
#pragma unroll
  for (int n = 0; n < NB; ++n)
    xp[n] = a.q + int64_t(min(t0 + 16 * n + r, a.T - 1)) * a.ldq;
  i32x4 acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = i32x4{0, 0, 0, 0};
  const int groups = (a.K + 127) / 128;
  for (int g = w; g < groups; g += WV * U) {
    i32x4 wf[U][2][MB], xf[U][2][NB];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // past the row's end: any bytes of the weight's row times zeros
        const int k = (g + u * WV) * 128 + 64 * h + kg;
        const bool in = k < a.K;
        const int kc = in ? k : 0;
#pragma unroll
        for (int m = 0; m < MB; ++m) wf[u][h][m] = *reinterpret_cast<const i32x4 *>(wp[m] + kc);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          xf[u][h][n] = *reinterpret_cast<const i32x4 *>(xp[n] + kc);
          if (!in) xf[u][h][n] = i32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int n = 0; n < NB; ++n)
            acc[m][n] =
                __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[u][h][m], xf[u][h][n], acc[m][n], 0, 0, 0);
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) part[w][m * NB + n][lane] = acc[m][n];
  __syncthreads();
  for (int j = threadIdx.x; j < MB * NB * 64; j += 64 * WV) {
    const int b = j >> 6, l = j & 63;
    i32x4 s = part[0][b][l];
#pragma unroll
    for (int v = 1; v < WV; ++v) s += part[v][b][l];
    const int c = c0 + 16 * (b / NB) + 4 * (l >> 4), t = t0 + 16 * (b % NB) + (l & 15);
    if (c < a.N && t < a.T) store_y4<TY>(a, t, c, s);
  }
}

// 128 channels by 128 tokens, 4 waves of 64 x 64, 128 bytes of d_in a step.
// LDS holds rows of eight 16-byte chunks; chunk c of row r lies at c ^ ((r >>
// 1) & 7), so that the 32 rows an operand load touches fall on all banks.
constexpr int kTB = 128;

template <typename TY>
__global__ __launch_bounds__(256, 2) void i8_tile(ProdArgs a) {
  __shared__ i32x4 lw[2][kTB * 8], lx[2][kTB * 8];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  // workgroups go to the eight XCDs in turn: each gets a run of tiles, token
  // tiles next to each other, so that its L2 holds their weight rows
  const int n = a.nt * a.nc, per = (n + 7) / 8;
  const int id = int(blockIdx.x & 7) * per + int(blockIdx.x >> 3);
  if (int(blockIdx.x >> 3) >= per || id >= n) return;
  const int c0 = id / a.nt * kTB, t0 = id % a.nt * kTB;
  const int wc = (w & 1) * 64, wt = (w >> 1) * 64;

  const int8_t *gw[4], *gx[4];
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = tid + 256 * i, row = p >> 3, c = p & 7;
    gw[i] = a.W + int64_t(min(c0 + row, a.N - 1)) * a.K;
    gx[i] = a.q + int64_t(min(t0 + row, a.T - 1)) * a.ldq;
    pos[i] = row * 8 + (c ^ ((row >> 1) & 7));
  }
  const int kc = 16 * (tid & 7);
  i32x4 rw[4], rx[4];
  auto load = [&](int k0) {
    const int k = k0 + kc;
    const bool in = k < a.K;
    const int kk = in ? k : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rw[i] = *reinterpret_cast<const i32x4 *>(gw[i] + kk);
      rx[i] = *reinterpret_cast<const i32x4 *>(gx[i] + kk);
      if (!in) rx[i] = i32x4{0, 0, 0, 0};
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lw[b][pos[i]] = rw[i];
      lx[b][pos[i]] = rx[i];
    }
  };
  i32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  load(0);
  put(0);
  __syncthreads();
  const int r = lane & 31, h = lane >> 5;
  int b = 0;
  for (int k0 = 0; k0 < a.K; k0 += 128, b ^= 1) {
    const bool more = k0 + 128 < a.K;
    if (more) load(k0 + 128);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      i32x4 fw[2], fx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rw_ = wc + 32 * i + r, rx_ = wt + 32 * i + r;
        fw[i] = lw[b][rw_ * 8 + ((2 * s + h) ^ ((rw_ >> 1) & 7))];
        fx[i] = lx[b][rx_ * 8 + ((2 * s + h) ^ ((rx_ >> 1) & 7))];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fx[j], acc[i][j], 0, 0, 0);
    }
    if (more) put(b ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = t0 + wt + 32 * j + r;
    if (t >= a.T) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = c0 + wc + 32 * i + 8 * g + 4 * h;
        if (c < a.N)
          store_y4<TY>(a, t, c, i32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                      acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
      }
  }
}

// ---------------------------------------------------------------------------
// checks and launches
// ---------------------------------------------------------------------------
bool misaligned(const void *p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) & (m - 1); }

int check_weight(const tcl_i8_weight *w) {
  if (!w) return fail(TCL_EINVAL, "i8: weight is NULL");
  if (w->d_in < 16 || w->d_out < 0)
    return fail(TCL_EINVAL, "i8: d_in %d < 16 or d_out %d < 0", w->d_in, w->d_out);
  if (w->d_in > TCL_I8_MAX_D_IN)
    return fail(TCL_EUNSUPPORTED, "i8: d_in %d beyond %d", w->d_in, TCL_I8_MAX_D_IN);
  if (w->d_in % 16 || w->d_out % 8)
    return fail(TCL_EALIGN, "i8: d_in %d is not a multiple of 16 or d_out %d not of 8", w->d_in,
                w->d_out);
  if (w->d_out > 0 && (!w->W || !w->scale)) return fail(TCL_EINVAL, "i8: weight arrays are NULL");
  if (misaligned(w->W, 16)) return fail(TCL_EALIGN, "i8: W must be 16-byte aligned");
  if (misaligned(w->scale, 4)) return fail(TCL_EALIGN, "i8: scale must be 4-byte aligned");
  return TCL_OK;
}

int check_quant(const void *x, int64_t ldx, int xd, int32_t n_tokens, int32_t d) {
  if (n_tokens < 0 || d < 16)
    return fail(TCL_EINVAL, "i8: n_tokens %d < 0 or d %d < 16", n_tokens, d);
  if (xd != TCL_BF16 && xd != TCL_F32) return fail(TCL_EUNSUPPORTED, "i8: x dtype %d", xd);
  if (ldx < d) return fail(TCL_EINVAL, "i8: ldx < d");
  if (d % 16 || ldx % 8) return fail(TCL_EALIGN, "i8: d must be a multiple of 16, ldx of 8");
  if (n_tokens > 0 && !x) return fail(TCL_EINVAL, "i8: x is NULL");
  if (misaligned(x, 16)) return fail(TCL_EALIGN, "i8: x must be 16-byte aligned");
  return TCL_OK;
}

int check_y(const tcl_i8_weight *w, int32_t n_tokens, const void *y, int64_t ldy, int yd) {
  if (n_tokens < 0) return fail(TCL_EINVAL, "i8: n_tokens %d < 0", n_tokens);
  if (yd != TCL_BF16 && yd != TCL_F32) return fail(TCL_EUNSUPPORTED, "i8: y dtype %d", yd);
  if (w->d_out == 0) return TCL_OK;  // nothing is written
  if (ldy < w->d_out) return fail(TCL_EINVAL, "i8: ldy < d_out");
  if (n_tokens > 0 && !y) return fail(TCL_EINVAL, "i8: y is NULL");
  if (misaligned(y, 16) || ldy % 8)
    return fail(TCL_EALIGN, "i8: y must be 16-byte aligned, ldy a multiple of 8");
  return TCL_OK;
}

int launch_quant(const void *x, int64_t ldx, int xd, int32_t n, int32_t d, int8_t *q, int64_t ldq,
                 float *scale, hipStream_t s) {
  if (n == 0) return TCL_OK;
  QuantArgs a{x, ldx, ldq, d, q, scale};
  if (xd == TCL_BF16)
    hipLaunchKernelGGL(i8_quant_kernel<bf16_t>, dim3(n), dim3(kQThreads), 0, s, a);
  else
    hipLaunchKernelGGL(i8_quant_kernel<float>, dim3(n), dim3(kQThreads), 0, s, a);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

template <int MB, int NB, int WV, int U, typename TY>
void go_skinny(const ProdArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((i8_skinny<MB, NB, WV, U, TY>),
                     dim3((a.N + 16 * MB - 1) / (16 * MB), (a.T + 16 * NB - 1) / (16 * NB)),
                     dim3(64 * WV), 0, s, a);
}

template <int NB, typename TY>
void skinny(const ProdArgs &a, hipStream_t s) {
  const int64_t tb = (a.T + 16 * NB - 1) / (16 * NB);
  if (tb * (a.N / 64) >= 192)
    go_skinny<4, NB, 4, 1, TY>(a, s);
  else if (tb * (a.N / 32) >= 192)
    go_skinny<2, NB, 8, 1, TY>(a, s);
  else
    go_skinny<1, NB, 16, 1, TY>(a, s);
}

template <typename TY>
void product(ProdArgs &a, hipStream_t s) {
  if (a.T <= 256) {
    if (a.T <= 16)
      skinny<1, TY>(a, s);
    else if (a.T <= 32)
      skinny<2, TY>(a, s);
    else
      skinny<4, TY>(a, s);
    return;
  }
  a.nt = (a.T + kTB - 1) / kTB;
  a.nc = (a.N + kTB - 1) / kTB;
  const int per = (a.nt * a.nc + 7) / 8;
  hipLaunchKernelGGL(i8_tile<TY>, dim3(8 * per), dim3(256), 0, s, a);
}

int launch_product(const tcl_i8_weight *w, const int8_t *q, int64_t ldq, const float *scale,
                   int32_t n, void *y, int64_t ldy, int yd, hipStream_t s) {
  if (n == 0 || w->d_out == 0) return TCL_OK;
  ProdArgs a{w->W, q, w->scale, scale, y, ldq, ldy, n, w->d_in, w->d_out, 0, 0};
  if (yd == TCL_BF16)
    product<uint16_t>(a, s);
  else
    product<float>(a, s);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

// workspace of tcl_i8_linear: the integers, then the scales
size_t ws_q_bytes(const tcl_i8_weight *w, int32_t n) {
  return (size_t(n) * size_t(w->d_in) + 255) / 256 * 256;
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
  return launch_quant(x, ldx, xd, n_tokens, d, q, ldq, scale, static_cast<hipStream_t>(stream));
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
  return launch_product(w, q, ldq, scale, n_tokens, y, ldy, yd, static_cast<hipStream_t>(stream));
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
  int8_t *q = static_cast<int8_t *>(ws);
  float *scale = reinterpret_cast<float *>(q + ws_q_bytes(w, n_tokens));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((rc = launch_quant(x, ldx, xd, n_tokens, w->d_in, q, w->d_in, scale, s))) return rc;
  return launch_product(w, q, w->d_in, scale, n_tokens, y, ldy, yd, s);
}
