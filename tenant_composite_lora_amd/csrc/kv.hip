// Appending to a paged key/value cache, with the position rotation on the way
// (include/tcl.h has the formulas).
//
// One launch.  The work of a token is cut into units of 16 elements: a
// rotated pair of 8-element chunks (or 16 neighbouring elements of
// interleaved pairs), or 16 elements that are only copied.  A thread owns a
// unit, so every element of q, k and v is read and written once, 16 bytes a
// lane.  The angles of a token are computed once a workgroup, in 64 bits
// (positions reach far beyond what an fp32 product resolves), reduced to one
// turn there and handed to the fp32 sine and cosine.
// Bound by memory for many tokens (4224 tokens, 32 + 8 + 8 heads of 128, fp32
// in: 156 MB in 24.2 us, 6.4 TB/s, part of it from the last-level cache); 64
// tokens take 3.6 us (3.3 in a captured graph), a launch and two round trips
// to memory.
#include <cmath>
#include <type_traits>

#include "kern_common.hpp"
#include "kv.hpp"

namespace tcl {
namespace {

constexpr int kAppThreads = 256;

struct AppendArgs {
  KvArgs c;
  const void *k, *v, *q;
  uint16_t *q_out;
  int64_t ldk, ldv, ldq, ldqo;
  const float *inv_freq;
  const int32_t *pos;
  const int64_t *slot;
  int32_t T, Hq, rot, inter;
  int32_t units;  // units of a token
};

template <typename T>
__device__ inline void load8(const T *p, float *v);

template <>
__device__ inline void load8<bf16_t>(const bf16_t *p, float *v) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <>
__device__ inline void load8<float>(const float *p, float *v) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ inline void store8(uint16_t *p, const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = uint32_t(f32_to_bf16(v[2 * i])) | uint32_t(f32_to_bf16(v[2 * i + 1])) << 16;
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of pos * f.  The 64-bit product of a 32-bit integer and an fp32
// number is off by half a step of the angle at most (1e-10 at a million
// radians); whole turns are taken off with 2 pi in two parts, which adds less.
__device__ inline float2 turn(int32_t pos, float f) {
  const double a = double(pos) * double(f);
  const double n = rint(a * 0.15915494309189535);
  const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, a));
  float s, c;
  sincosf(float(r), &s, &c);
  return make_float2(c, s);
}

// grid: (token, part); a workgroup takes its part's units of the token
template <typename T>
__global__ __launch_bounds__(kAppThreads) void kv_append_kernel(AppendArgs a) {
  __shared__ float2 cs[128];  // rot_dim / 2 <= 128 pairs
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int D = a.c.D, half = a.rot / 2;
  if (tid < half) cs[tid] = turn(a.pos[t], a.inv_freq[tid]);
  const int64_t slot = a.slot[t];
  const bool live = slot >= 0 && slot < int64_t(a.c.n_pages) << a.c.page_shift;
  const int64_t at = live ? kv_slot(a.c, slot) : 0;
  __syncthreads();
  const int per = D / 16, rper = a.rot / 16;  // units of a head, of its rotated part
  for (int u = blockIdx.y * kAppThreads + tid; u < a.units; u += gridDim.y * kAppThreads) {
    const int head = u / per, e = u % per;
    const T *src;
    uint16_t *dst;
    bool rotate = e < rper, keep = true;
    if (head < a.Hq) {
      src = static_cast<const T *>(a.q) + t * a.ldq + int64_t(head) * D;
      dst = a.q_out + t * a.ldqo + int64_t(head) * D;
    } else if (head < a.Hq + a.c.H) {
      const int h = head - a.Hq;
      src = static_cast<const T *>(a.k) + t * a.ldk + int64_t(h) * D;
      dst = a.c.K + at + h * a.c.s_head;
      keep = live;
    } else {
      const int h = head - a.Hq - a.c.H;
      src = static_cast<const T *>(a.v) + t * a.ldv + int64_t(h) * D;
      dst = a.c.V + at + h * a.c.s_head;
      rotate = false;
      keep = live;
    }
    if (!keep) continue;
    const bool split = rotate && !a.inter;
    const int i0 = split ? 8 * e : 16 * e, i1 = split ? i0 + half : i0 + 8;
    float x[8], y[8];
    load8<T>(src + i0, x);
    load8<T>(src + i1, y);
    if (split) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 r = cs[i0 + i];
        const float p = x[i] * r.x - y[i] * r.y, q = y[i] * r.x + x[i] * r.y;
        x[i] = p;
        y[i] = q;
      }
    } else if (rotate) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 r = cs[8 * e + i / 2], s = cs[8 * e + 4 + i / 2];
        const float p = x[i] * r.x - x[i + 1] * r.y, q = x[i + 1] * r.x + x[i] * r.y;
        const float v = y[i] * s.x - y[i + 1] * s.y, w = y[i + 1] * s.x + y[i] * s.y;
        x[i] = p, x[i + 1] = q, y[i] = v, y[i + 1] = w;
      }
    }
    store8(dst + i0, x);
    store8(dst + i1, y);
  }
}

// ---------------------------------------------------------------------------
// with norms of queries and keys
// ---------------------------------------------------------------------------
struct NormArgs {
  AppendArgs a;
  const float *wq, *wk;
  int64_t sq, sk;  // elements between the weights of neighbouring heads
  float eps;
  int32_t lanes_log2;  // lanes of a head: D / 16 rounded up to a power of two
};

// The sum over a head's 2^n neighbouring lanes, n <= 4, the same in all of
// them: lane moves inside rows of 16, no trip through LDS.
__device__ inline float head_sum(float v, int n) {
  auto add = [&v](auto ctrl) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf,
                                                    true));
  };
  if (n > 0) add(std::integral_constant<int, 0xb1>{});   // lane ^ 1
  if (n > 1) add(std::integral_constant<int, 0x4e>{});   // lane ^ 2
  if (n > 2) add(std::integral_constant<int, 0x141>{});  // 7 - lane, of 8
  if (n > 3) add(std::integral_constant<int, 0x140>{});  // 15 - lane, of 16
  return v;
}

// The append, where the heads of q and k are divided by their root mean square
// and multiplied by a weight on the way.  A head belongs to neighbouring lanes
// that hold 16 elements each, as in kv_append_kernel, so that its sum of
// squares takes up to four lane moves and its elements are still read once.
// Squares are summed in fp32; a head whose sum is not between 1e-20 and 1e37
// (zeros, numbers whose squares leave fp32's range, infinities) is summed again
// in 64 bits, so that no finite head overflows or vanishes.  Bound by the rows'
// bytes as the plain append is: 4224 tokens of 32 + 8 + 8 heads of 128 in fp32,
// 156 MB, 28.4 us, 5.5 TB/s (without the norms 24.2); 64 tokens 4.0 us, a launch.
template <typename T>
__global__ __launch_bounds__(kAppThreads) void kv_append_norm_kernel(NormArgs n) {
  __shared__ float2 cs[128];
  const AppendArgs &a = n.a;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int D = a.c.D, half = a.rot / 2;
  if (tid < half) cs[tid] = turn(a.pos[t], a.inv_freq[tid]);
  const int64_t slot = a.slot[t];
  const bool live = slot >= 0 && slot < int64_t(a.c.n_pages) << a.c.page_shift;
  const int64_t at = live ? kv_slot(a.c, slot) : 0;
  __syncthreads();
  const int per = D / 16, rper = a.rot / 16, lg = n.lanes_log2;
  const int heads = a.Hq + 2 * a.c.H, e = tid & ((1 << lg) - 1);
  for (int head = (blockIdx.y * kAppThreads + tid) >> lg; head < heads; head += gridDim.y * kAppThreads >> lg) {
    const T *src;
    uint16_t *dst;
    const float *w = nullptr;
    bool rotate = e < rper;
    if (head < a.Hq) {
      src = static_cast<const T *>(a.q) + t * a.ldq + int64_t(head) * D;
      dst = a.q_out + t * a.ldqo + int64_t(head) * D;
      if (n.wq) w = n.wq + head * n.sq;
    } else {
      const bool key = head < a.Hq + a.c.H;
      const int h = key ? head - a.Hq : head - a.Hq - a.c.H;
      if (!live) continue;
      src = key ? static_cast<const T *>(a.k) + t * a.ldk + int64_t(h) * D
                : static_cast<const T *>(a.v) + t * a.ldv + int64_t(h) * D;
      dst = (key ? a.c.K : a.c.V) + at + h * a.c.s_head;
      if (key && n.wk) w = n.wk + h * n.sk;
      rotate &= key;
    }
    const bool mine = e < per, split = rotate && !a.inter;
    const int i0 = split ? 8 * e : 16 * e, i1 = split ? i0 + half : i0 + 8;
    float x[8], y[8], wx[8], wy[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    if (mine) {
      load8<T>(src + i0, x);
      load8<T>(src + i1, y);
    }
    if (w) {
      if (mine) {
        load8<float>(w + i0, wx);
        load8<float>(w + i1, wy);
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
      ss = head_sum(ss, lg);
      if (ss >= 1e-20f && ss <= 1e37f) {
        const float r = rsqrtf(ss / float(D) + n.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r, y[i] *= r;
      } else {
        double s2 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          s2 = fma(double(x[i]), double(x[i]), fma(double(y[i]), double(y[i]), s2));
        for (int o = 1; o < 1 << lg; o <<= 1) s2 += __shfl_xor(s2, o, 64);
        const double r = 1 / sqrt(s2 / D + double(n.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = float(x[i] * r), y[i] = float(y[i] * r);
      }
      if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= wx[i], y[i] *= wy[i];
      }
    }
    if (!mine) continue;
    if (split) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 r = cs[i0 + i];
        const float p = x[i] * r.x - y[i] * r.y, q = y[i] * r.x + x[i] * r.y;
        x[i] = p;
        y[i] = q;
      }
    } else if (rotate) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 r = cs[8 * e + i / 2], s = cs[8 * e + 4 + i / 2];
        const float p = x[i] * r.x - x[i + 1] * r.y, q = x[i + 1] * r.x + x[i] * r.y;
        const float v = y[i] * s.x - y[i + 1] * s.y, u = y[i + 1] * s.x + y[i] * s.y;
        x[i] = p, x[i + 1] = q, y[i] = v, y[i + 1] = u;
      }
    }
    store8(dst + i0, x);
    store8(dst + i1, y);
  }
}

bool misaligned(const void *p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) & (m - 1); }

// The checks of both appends; *launch says whether there is anything to do.
int append_args(const tcl_kv_cache *c, const tcl_rope *rope, const void *k, int64_t ldk, const void *v,
                int64_t ldv, const void *q, int64_t ldq, int32_t n_q_heads, tcl_dtype xd, void *q_out,
                int64_t ldqo, int32_t n_tokens, const int32_t *pos, const int64_t *slot, AppendArgs *out,
                bool *launch);

}  // namespace

int kv_check(const tcl_kv_cache *c, KvArgs *out) {
  if (!c) return fail(TCL_EINVAL, "kv: cache is NULL");
  if (c->n_pages < 1 || c->n_kv_heads < 1)
    return fail(TCL_EINVAL, "kv: n_pages %d and n_kv_heads %d must be >= 1", c->n_pages,
                c->n_kv_heads);
  if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(TCL_EUNSUPPORTED, "kv: page_size %d is not a power of two in 1..1024",
                c->page_size);
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
    return fail(TCL_EUNSUPPORTED, "kv: head_dim %d is not a multiple of 16 in 16..256",
                c->head_dim);
  if (!c->K || !c->V) return fail(TCL_EINVAL, "kv: K and V are required");
  if (c->stride_page < 0 || c->stride_slot < 0 || c->stride_head < 0)
    return fail(TCL_EINVAL, "kv: strides must not be negative");
  if (misaligned(c->K, 16) || misaligned(c->V, 16) || c->stride_page % 8 || c->stride_slot % 8 ||
      c->stride_head % 8)
    return fail(TCL_EALIGN, "kv: K and V must be 16-byte aligned, strides multiples of 8");
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  *out = KvArgs{static_cast<uint16_t *>(c->K), static_cast<uint16_t *>(c->V), c->stride_page,
                c->stride_slot, c->stride_head, c->n_pages, shift, c->n_kv_heads, c->head_dim};
  return TCL_OK;
}

}  // namespace tcl

using namespace tcl;

namespace tcl {
namespace {

int append_args(const tcl_kv_cache *c, const tcl_rope *rope, const void *k, int64_t ldk, const void *v,
                int64_t ldv, const void *q, int64_t ldq, int32_t n_q_heads, tcl_dtype xd, void *q_out,
                int64_t ldqo, int32_t n_tokens, const int32_t *pos, const int64_t *slot, AppendArgs *out,
                bool *launch) {
  AppendArgs &a = *out;
  *launch = false;
  int rc = kv_check(c, &a.c);
  if (rc) return rc;
  if (!rope) return fail(TCL_EINVAL, "kv: rope is NULL");
  if (rope->rot_dim < 0 || rope->rot_dim > c->head_dim || rope->rot_dim % 16)
    return fail(TCL_EUNSUPPORTED, "kv: rot_dim %d is not a multiple of 16 in 0..head_dim",
                rope->rot_dim);
  if (rope->rot_dim > 0 && !rope->inv_freq) return fail(TCL_EINVAL, "kv: inv_freq is NULL");
  if (xd != TCL_BF16 && xd != TCL_F32) return fail(TCL_EUNSUPPORTED, "kv: dtype %d", int(xd));
  if (n_tokens < 0) return fail(TCL_EINVAL, "kv: n_tokens %d < 0", n_tokens);
  const int64_t row = int64_t(c->n_kv_heads) * c->head_dim;
  if (ldk < row || ldv < row) return fail(TCL_EINVAL, "kv: ldk or ldv below the heads of a row");
  if (ldk % 8 || ldv % 8) return fail(TCL_EALIGN, "kv: ldk and ldv must be multiples of 8");
  if (q) {
    if (n_q_heads < 1) return fail(TCL_EINVAL, "kv: n_q_heads %d < 1", n_q_heads);
    const int64_t qrow = int64_t(n_q_heads) * c->head_dim;
    if (!q_out || ldq < qrow || ldqo < qrow)
      return fail(TCL_EINVAL, "kv: q_out is NULL, or ldq or ldqo below the heads of a row");
    if (q == q_out && (xd != TCL_BF16 || ldq != ldqo))
      return fail(TCL_EINVAL, "kv: q_out may be q only in bf16 with one leading dimension");
    if (misaligned(q, 16) || misaligned(q_out, 16) || ldq % 8 || ldqo % 8)
      return fail(TCL_EALIGN, "kv: q and q_out must be 16-byte aligned, ldq and ldqo multiples of 8");
  }
  if (int64_t(q ? n_q_heads : 0) + 2 * int64_t(c->n_kv_heads) > (int64_t(1) << 26))
    return fail(TCL_EUNSUPPORTED, "kv: too many heads");
  if (n_tokens >= 1 << 24)  // (a launch's threads, 256 a token, below 2^32)
    return fail(TCL_EUNSUPPORTED, "kv: n_tokens %d, 2^24 or more", n_tokens);
  if (n_tokens == 0) return TCL_OK;
  if (!k || !v || !pos || !slot) return fail(TCL_EINVAL, "kv: k, v, pos and slot are required");
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slot, 8) || misaligned(pos, 4) ||
      misaligned(rope->inv_freq, 4))
    return fail(TCL_EALIGN, "kv: k and v must be 16-byte, slot 8-byte, pos and inv_freq 4-byte "
                            "aligned");
  a.k = k, a.v = v, a.q = q, a.q_out = static_cast<uint16_t *>(q_out);
  a.ldk = ldk, a.ldv = ldv, a.ldq = ldq, a.ldqo = ldqo;
  a.inv_freq = rope->inv_freq, a.pos = pos, a.slot = slot;
  a.T = n_tokens, a.Hq = q ? n_q_heads : 0, a.rot = rope->rot_dim, a.inter = rope->interleaved;
  a.units = (a.Hq + 2 * c->n_kv_heads) * (c->head_dim / 16);
  *launch = true;
  return TCL_OK;
}

}  // namespace
}  // namespace tcl

extern "C" int tcl_kv_append(const tcl_kv_cache *c, const tcl_rope *rope, const void *k,
                             int64_t ldk, const void *v, int64_t ldv, const void *q, int64_t ldq,
                             int32_t n_q_heads, tcl_dtype xd, void *q_out, int64_t ldqo,
                             int32_t n_tokens, const int32_t *pos, const int64_t *slot,
                             void *stream) {
  AppendArgs a{};
  bool go;
  const int rc = append_args(c, rope, k, ldk, v, ldv, q, ldq, n_q_heads, xd, q_out, ldqo, n_tokens, pos,
                             slot, &a, &go);
  if (rc || !go) return rc;
  const int parts = (a.units + kAppThreads - 1) / kAppThreads;
  const dim3 grid(n_tokens, parts < 64 ? parts : 64);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (xd == TCL_BF16)
    hipLaunchKernelGGL(kv_append_kernel<bf16_t>, grid, dim3(kAppThreads), 0, s, a);
  else
    hipLaunchKernelGGL(kv_append_kernel<float>, grid, dim3(kAppThreads), 0, s, a);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

extern "C" int tcl_kv_append_norm(const tcl_kv_cache *c, const tcl_rope *rope, const tcl_head_norm *norm,
                                  const void *k, int64_t ldk, const void *v, int64_t ldv, const void *q,
                                  int64_t ldq, int32_t n_q_heads, tcl_dtype xd, void *q_out, int64_t ldqo,
                                  int32_t n_tokens, const int32_t *pos, const int64_t *slot,
                                  void *stream) {
  NormArgs n{};
  if (!norm) return fail(TCL_EINVAL, "kv: norm is NULL");
  if (!(norm->eps >= 0.f && std::isfinite(norm->eps)))
    return fail(TCL_EINVAL, "kv: eps is negative or not finite");
  if (norm->stride_q < 0 || norm->stride_k < 0)
    return fail(TCL_EINVAL, "kv: strides of the norm weights must not be negative");
  if (misaligned(norm->w_q, 16) || misaligned(norm->w_k, 16) || norm->stride_q % 4 || norm->stride_k % 4)
    return fail(TCL_EALIGN, "kv: norm weights must be 16-byte aligned, their strides multiples of 4");
  bool go;
  const int rc = append_args(c, rope, k, ldk, v, ldv, q, ldq, n_q_heads, xd, q_out, ldqo, n_tokens, pos,
                             slot, &n.a, &go);
  if (rc || !go) return rc;
  n.wq = norm->w_q, n.wk = norm->w_k, n.sq = norm->stride_q, n.sk = norm->stride_k, n.eps = norm->eps;
  while ((16 << n.lanes_log2) < c->head_dim) ++n.lanes_log2;
  const int64_t lanes = (int64_t(n.a.Hq) + 2 * c->n_kv_heads) << n.lanes_log2;
  const int64_t parts = (lanes + kAppThreads - 1) / kAppThreads;
  const dim3 grid(n_tokens, parts < 64 ? unsigned(parts) : 64);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (xd == TCL_BF16)
    hipLaunchKernelGGL(kv_append_norm_kernel<bf16_t>, grid, dim3(kAppThreads), 0, s, n);
  else
    hipLaunchKernelGGL(kv_append_norm_kernel<float>, grid, dim3(kAppThreads), 0, s, n);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}
