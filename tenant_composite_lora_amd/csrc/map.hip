// Pages, positions and slots of a batch's new tokens, from the requests'
// lengths (include/tcl.h has the formulas).
//
// Whether a batch is good is known only once all of it has been looked over
// (lengths, page ids, pages left), and nothing of a bad one may be written, so
// one workgroup checks and then writes what belongs to requests: pointers,
// lengths, page tables.  What belongs to tokens (positions and slots) it writes
// as well in small batches, where a launch more is what would cost; in larger
// ones a second launch does, from what the first has left.
// Bound by the launch and some ten round trips to memory and barriers, one
// behind the other: 64 requests of one token 5.8 us, 1152 requests with 43 000
// tokens 10.4 and, by the second launch, 3.9.
#include "kern_common.hpp"
#include "kv.hpp"
#include "scan.hpp"

namespace tcl {
namespace {

// Tokens that the first launch writes itself (captured, by the first and by the
// second: 300 tokens 5.6 us, 7.2; 4000 7.8, 8.7; 8000 10.4, 8.7; 43 000 48, 13.5).
constexpr int kMapOne = 4096;
// Requests whose pointers the second launch searches in LDS.
constexpr int kMapPtr = 8191;

struct MapArgs {
  int32_t S, G, T, n_free, ld;
  int32_t n_pages, shift;
  const int32_t *n_new, *group_seq, *prefix_len, *own_len, *free_pages, *used;
  int32_t *own_pages, *seq_tok, *pos, *own_out, *used_out, *status;
  int64_t *slot;
};

// The workgroup's sums of u and v, and whether any thread has found it bad.
__device__ inline void block_sums(int64_t &u, int64_t &v, bool &bad, int64_t (*lds)[kMapThreads / 64], int *flag) {
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) {
    u += __shfl_xor(u, x, 64);
    v += __shfl_xor(v, x, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    lds[0][threadIdx.x >> 6] = u;
    lds[1][threadIdx.x >> 6] = v;
  }
  if (bad) *flag = 1;
  __syncthreads();
  u = v = 0;
#pragma unroll
  for (int i = 0; i < kMapThreads / 64; ++i) {
    u += lds[0][i];
    v += lds[1][i];
  }
  bad = *flag;
}

__device__ inline int pages_of(const MapArgs &a, int n) {
  return (n >> a.shift) + ((n & ((1 << a.shift) - 1)) != 0);
}

// The groups' tables, in LDS where they fit (a search in memory is a round trip
// a step).
struct Groups {
  int32_t seq[kMapThreads + 1], prefix[kMapThreads];
  __device__ inline void load(const MapArgs &a) {
    if (a.G > kMapThreads) return;
    for (int g = threadIdx.x; g < a.G; g += blockDim.x) {
      seq[g] = a.group_seq[g];
      prefix[g] = a.prefix_len[g];
    }
    if (threadIdx.x == 0 && a.G > 0) seq[a.G] = a.group_seq[a.G];
  }
  // prefix of the group of request s
  __device__ inline int prefix_of(const MapArgs &a, int s) const {
    return a.G > kMapThreads ? a.prefix_len[upper(a.group_seq, a.G, s)] : prefix[upper(seq, a.G, s)];
  }
};

// A chunk of kMapThreads requests in LDS: tokens and pages before each, its
// keys before, its prefix.
struct Chunk {
  int32_t tok[kMapThreads], page[kMapThreads], have[kMapThreads], prefix[kMapThreads];
};

// The tokens [t0, t1) of the chunk's requests s0 .. s0 + n - 1.
__device__ inline void put_tokens(const MapArgs &a, const Chunk &c, int s0, int n, int t0, int t1, int used) {
  const int mask = (1 << a.shift) - 1;
  for (int t = t0 + threadIdx.x; t < t1; t += kMapThreads) {
    const int i = upper(c.tok, n, t), have = c.have[i];
    const int key = have + (t - c.tok[i]), p = key >> a.shift, hp = pages_of(a, have);
    const int id = p < hp ? a.own_pages[int64_t(s0 + i) * a.ld + p] : a.free_pages[used + c.page[i] + p - hp];
    a.pos[t] = c.prefix[i] + key;
    a.slot[t] = (int64_t(id) << a.shift) + (key & mask);
  }
}

// The pages [g0, g1) that the chunk's requests take (counted over all requests).
__device__ inline void put_pages(const MapArgs &a, const Chunk &c, int s0, int n, int g0, int g1, int used) {
  for (int g = g0 + threadIdx.x; g < g1; g += kMapThreads) {
    const int i = upper(c.page, n, g), p = pages_of(a, c.have[i]) + g - c.page[i];
    a.own_pages[int64_t(s0 + i) * a.ld + p] = a.free_pages[used + g];
  }
}

__device__ inline void pad(const MapArgs &a, int t0, int t1) {
  for (int t = t0 + threadIdx.x; t < t1; t += kMapThreads) {
    a.pos[t] = 0;
    a.slot[t] = -1;
  }
}

__global__ __launch_bounds__(kMapThreads) void kv_map_kernel(MapArgs a) {
  __shared__ int lds[2][kMapThreads / 64];
  __shared__ int64_t sums[2][kMapThreads / 64];
  __shared__ int s_bad;
  __shared__ Groups groups;
  __shared__ Chunk chunk;
  const int tid = threadIdx.x;
  const int used = a.used[0];
  // (the first chunk's requests stay in registers)
  const int q0 = tid < a.S ? a.n_new[tid] : 0, n0 = tid < a.S ? a.own_len[tid] : 0;
  groups.load(a);
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // the batch
  bool bad = used < 0 || used > a.n_free;
  if (a.S > 0 && tid == 0) bad |= a.group_seq[0] != 0 || a.group_seq[a.G] != a.S;
  if (a.G <= kMapThreads) {
    if (tid < a.G) bad |= groups.seq[tid + 1] < groups.seq[tid] || groups.prefix[tid] < 0;
  } else {
    for (int g = tid; g < a.G; g += kMapThreads)
      bad |= a.group_seq[g + 1] < a.group_seq[g] || a.prefix_len[g] < 0;
  }
  int64_t tokens = 0, pages = 0;
  for (int s = tid; s < a.S; s += kMapThreads) {
    const int64_t q = s == tid ? q0 : a.n_new[s], n = s == tid ? n0 : a.own_len[s];
    const int64_t cap = int64_t(a.ld) << a.shift;
    const int32_t prefix = groups.prefix_of(a, s);
    // (the last new key's position; without one nothing has a position)
    if (q < 0 || n < 0 || n + q > cap || (q > 0 && prefix + n + q - 1 > int64_t(0x7fffffff))) {
      bad = true;
      continue;
    }
    // the page that the first new key may share with keys before it
    if (q > 0 && (n & ((1 << a.shift) - 1))) {
      const int id = a.own_pages[int64_t(s) * a.ld + (n >> a.shift)];
      bad |= id < 0 || id >= a.n_pages;
    }
    tokens += q;
    pages += pages_of(a, int(n + q)) - pages_of(a, int(n));
  }
  block_sums(tokens, pages, bad, sums, &s_bad);
  bad |= tokens > a.T;
  const bool enough = pages <= int64_t(a.n_free) - used;
  // the page ids that are taken
  if (!bad && enough) {
#pragma unroll 4
    for (int i = tid; i < int(pages); i += kMapThreads) {
      const int id = a.free_pages[used + i];
      bad |= id < 0 || id >= a.n_pages;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const int code = s_bad ? TCL_EINVAL : (enough ? TCL_OK : TCL_ENOSPC);
  if (tid == 0) {
    a.status[0] = code;
    a.status[1] = code == TCL_OK ? int(tokens) : 0;
    a.status[2] = code == TCL_OK ? int(pages) : 0;
    a.status[3] = a.n_free - used - (code == TCL_OK ? int(pages) : 0);
    a.used_out[0] = used + (code == TCL_OK ? int(pages) : 0);
  }
  const bool all = a.T <= kMapOne;
  if (code != TCL_OK) {
    for (int s = tid; s <= a.S; s += kMapThreads) {
      a.seq_tok[s] = 0;
      if (s < a.S) a.own_out[s] = a.own_len[s];
    }
    if (all) pad(a, 0, a.T);
    return;
  }
  int tok = 0, page = 0;
  for (int s0 = 0; s0 < a.S; s0 += kMapThreads) {
    const int s = s0 + tid, n = min(kMapThreads, a.S - s0);
    int q = 0, have = 0, v[2] = {0, 0}, total[2], prefix = 0;
    if (s < a.S) {
      q = s0 ? a.n_new[s] : q0;
      have = s0 ? a.own_len[s] : n0;
      prefix = groups.prefix_of(a, s);
      v[0] = q;
      v[1] = pages_of(a, have + q) - pages_of(a, have);
    }
    block_scan(v, total, lds);  // (its barriers also end the chunk before)
    chunk.tok[tid] = tok + v[0];
    chunk.page[tid] = page + v[1];
    chunk.have[tid] = have;
    chunk.prefix[tid] = prefix;
    if (s < a.S) {
      a.seq_tok[s] = tok + v[0];
      a.own_out[s] = have + q;
    }
    __syncthreads();
    put_pages(a, chunk, s0, n, page, page + total[1], used);
    if (all) put_tokens(a, chunk, s0, n, tok, tok + total[0], used);
    tok += total[0];
    page += total[1];
  }
  if (tid == 0) a.seq_tok[a.S] = tok;
  if (all) pad(a, tok, a.T);
}

// The tokens of a batch that kv_map_kernel has looked over, kMapThreads a
// workgroup: token t of request s is key own_out[s] - (seq_tok[s + 1] - t).
template <bool LDS>
__global__ __launch_bounds__(kMapThreads) void kv_map_fill_kernel(MapArgs a) {
  __shared__ Groups groups;
  __shared__ int32_t l_ptr[LDS ? kMapPtr + 1 : 1];
  const int t = blockIdx.x * kMapThreads + threadIdx.x, tokens = a.status[1];
  if (int(blockIdx.x) * kMapThreads < tokens) {
    groups.load(a);
    if (LDS)
      for (int s = threadIdx.x; s <= a.S; s += kMapThreads) l_ptr[s] = a.seq_tok[s];
    __syncthreads();
  }
  if (t >= a.T) return;
  if (t >= tokens) {
    a.pos[t] = 0;
    a.slot[t] = -1;
    return;
  }
  const int32_t *ptr = LDS ? l_ptr : a.seq_tok;
  const int s = upper(ptr, a.S, t), key = a.own_out[s] - (ptr[s + 1] - t);
  const int id = a.own_pages[int64_t(s) * a.ld + (key >> a.shift)];
  a.pos[t] = groups.prefix_of(a, s) + key;
  a.slot[t] = (int64_t(id) << a.shift) + (key & ((1 << a.shift) - 1));
}

bool misaligned(const void *p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) & (m - 1); }

}  // namespace
}  // namespace tcl

using namespace tcl;

extern "C" int tcl_kv_map(const tcl_kv_cache *c, const tcl_kv_batch *b, void *stream) {
  KvArgs kv;
  const int rc = kv_check(c, &kv);
  if (rc) return rc;
  if (!b) return fail(TCL_EINVAL, "map: batch is NULL");
  if (b->n_seqs < 0 || b->n_groups < 0 || b->n_tokens < 0 || b->n_free < 0 || b->ld_own < 0)
    return fail(TCL_EINVAL, "map: negative size");
  if (b->n_seqs > 0 && b->n_groups < 1) return fail(TCL_EINVAL, "map: requests without a group");
  if (b->n_seqs >= 1 << 24 || b->n_groups >= 1 << 24 || b->n_tokens >= 1 << 24)
    return fail(TCL_EUNSUPPORTED, "map: n_seqs, n_groups or n_tokens of 2^24 or more");
  if (int64_t(b->ld_own) * c->page_size >= int64_t(1) << 29)
    return fail(TCL_EUNSUPPORTED, "map: page tables of 2^29 keys or more");
  if (!b->seq_tok_ptr || !b->used || !b->used_out || !b->status)
    return fail(TCL_EINVAL, "map: seq_tok_ptr, used, used_out and status are required");
  if (b->n_seqs > 0 && (!b->n_new || !b->group_seq_ptr || !b->prefix_len || !b->own_len ||
                        !b->own_len_out || (b->ld_own > 0 && !b->own_pages)))
    return fail(TCL_EINVAL, "map: an array of the requests is NULL");
  if (b->n_free > 0 && !b->free_pages) return fail(TCL_EINVAL, "map: free_pages is NULL");
  if (b->n_tokens > 0 && (!b->pos || !b->slot)) return fail(TCL_EINVAL, "map: pos and slot are required");
  const void *p[] = {b->n_new, b->group_seq_ptr, b->prefix_len, b->own_len, b->own_pages, b->free_pages,
                     b->used, b->seq_tok_ptr, b->pos, b->own_len_out, b->used_out, b->status};
  for (const void *x : p)
    if (misaligned(x, 4)) return fail(TCL_EALIGN, "map: arrays must be 4-byte aligned");
  if (misaligned(b->slot, 8)) return fail(TCL_EALIGN, "map: slot must be 8-byte aligned");
  MapArgs a{b->n_seqs, b->n_seqs ? b->n_groups : 0, b->n_tokens, b->n_free, b->ld_own, kv.n_pages,
            kv.page_shift, b->n_new, b->group_seq_ptr, b->prefix_len, b->own_len, b->free_pages, b->used,
            b->own_pages, b->seq_tok_ptr, b->pos, b->own_len_out, b->used_out, b->status, b->slot};
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(kv_map_kernel, dim3(1), dim3(kMapThreads), 0, s, a);
  TCL_HIP(hipGetLastError());
  if (a.T > kMapOne) {
    const dim3 grid((a.T + kMapThreads - 1) / kMapThreads);
    if (a.S <= kMapPtr)
      hipLaunchKernelGGL(kv_map_fill_kernel<true>, grid, dim3(kMapThreads), 0, s, a);
    else
      hipLaunchKernelGGL(kv_map_fill_kernel<false>, grid, dim3(kMapThreads), 0, s, a);
    TCL_HIP(hipGetLastError());
  }
  return TCL_OK;
}
