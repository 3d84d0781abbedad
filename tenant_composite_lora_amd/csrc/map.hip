// Pages, positions and slots of a batch's new tokens, from the requests'
// lengths (include/tcl.h has the formulas).
//
// Whether a batch is good is known only once all of it has been looked over
// (lengths, page ids, pages left), and nothing of a bad one may be written, so
// one workgroup checks and then writes what belongs to requests.  What belongs
// to tokens (positions, slots, the page ids of new pages) it writes as well in
// small batches, where a launch more is what would cost; in larger ones a
// second launch does, whose workgroups take kMapThreads tokens each and repeat
// the scan over the requests, which is cheaper than a round trip of its
// results through memory.
#include "kern_common.hpp"
#include "kv.hpp"
#include "scan.hpp"

namespace tcl {
namespace {

// Tokens that the first launch writes itself.
constexpr int kMapOne = 8192;

struct MapArgs {
  int32_t S, G, T, n_free, ld;
  int32_t n_pages, shift;
  const int32_t *n_new, *group_seq, *prefix_len, *own_len, *free_pages, *used;
  int32_t *own_pages, *seq_tok, *pos, *own_out, *used_out, *status;
  int64_t *slot;
};

__device__ inline int64_t block_sum(int64_t v, int64_t *lds) {
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) v += __shfl_xor(v, x, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  int64_t s = 0;
#pragma unroll
  for (int i = 0; i < kMapThreads / 64; ++i) s += lds[i];
  return s;
}

__device__ inline int pages_of(const MapArgs &a, int n) {
  return (n >> a.shift) + ((n & ((1 << a.shift) - 1)) != 0);
}

// A chunk of kMapThreads requests in LDS: tokens and pages before each, its
// keys before, its prefix.
struct Chunk {
  int32_t tok[kMapThreads], page[kMapThreads], have[kMapThreads], prefix[kMapThreads];
};

// Tokens [t0, t1) of the chunk's requests s0 .. s0 + n - 1.
__device__ inline void fill(const MapArgs &a, const Chunk &c, int s0, int n, int t0, int t1, int used) {
  const int mask = (1 << a.shift) - 1;
  for (int t = t0 + threadIdx.x; t < t1; t += kMapThreads) {
    const int i = upper(c.tok, n, t), have = c.have[i];
    const int key = have + (t - c.tok[i]), p = key >> a.shift, hp = pages_of(a, have);
    int32_t *row = a.own_pages + int64_t(s0 + i) * a.ld;
    const int id = p < hp ? row[p] : a.free_pages[used + c.page[i] + p - hp];
    // (a page's first key brings it into the table)
    if ((key & mask) == 0) row[p] = id;
    a.pos[t] = c.prefix[i] + key;
    a.slot[t] = (int64_t(id) << a.shift) + (key & mask);
  }
}

__device__ inline void pad(const MapArgs &a, int t0, int t1) {
  for (int t = t0 + threadIdx.x; t < t1; t += kMapThreads) {
    a.pos[t] = 0;
    a.slot[t] = -1;
  }
}

// The scan over the requests; the chunk's tokens are written where `tokens`.
// OLD: own_len as before the call (else as after it).  WRITE: pointers,
// lengths and the count of pages in use.
template <bool OLD, bool WRITE>
__device__ inline void walk(const MapArgs &a, Chunk &c, int (*lds)[kMapThreads / 64], int used, int t0,
                            int t1) {
  const int tid = threadIdx.x;
  int tok = 0, page = 0;
  for (int s0 = 0; s0 < a.S; s0 += kMapThreads) {
    const int s = s0 + tid, n = min(kMapThreads, a.S - s0);
    int q = 0, have = 0, v[2] = {0, 0}, total[2], prefix = 0;
    if (s < a.S) {
      q = a.n_new[s];
      have = OLD ? a.own_len[s] : a.own_out[s] - q;
      prefix = a.prefix_len[upper(a.group_seq, a.G, s)];
      v[0] = q;
      v[1] = pages_of(a, have + q) - pages_of(a, have);
    }
    block_scan(v, total, lds);  // (its barriers also end the chunk before)
    c.tok[tid] = tok + v[0];
    c.page[tid] = page + v[1];
    c.have[tid] = have;
    c.prefix[tid] = prefix;
    if (WRITE && s < a.S) {
      a.seq_tok[s] = tok + v[0];
      a.own_out[s] = have + q;
    }
    __syncthreads();
    const int end = tok + total[0];
    fill(a, c, s0, n, max(t0, tok), min(t1, end), used);
    tok = end;
    page += total[1];
    if (!WRITE && tok >= t1) break;
  }
  if (WRITE && tid == 0) {
    a.seq_tok[a.S] = tok;
    a.used_out[0] = used + page;
  }
}

__global__ __launch_bounds__(kMapThreads) void kv_map_kernel(MapArgs a) {
  __shared__ int lds[2][kMapThreads / 64];
  __shared__ int64_t sums[kMapThreads / 64];
  __shared__ int s_bad;
  __shared__ Chunk chunk;
  const int tid = threadIdx.x;
  const int used = a.used[0];
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // the batch
  bool bad = used < 0 || used > a.n_free;
  if (a.S > 0 && tid == 0) bad |= a.group_seq[0] != 0 || a.group_seq[a.G] != a.S;
  for (int g = tid; g < a.G; g += kMapThreads)
    bad |= a.group_seq[g + 1] < a.group_seq[g] || a.prefix_len[g] < 0;
  int64_t tokens = 0, pages = 0;
  for (int s = tid; s < a.S; s += kMapThreads) {
    const int64_t q = a.n_new[s], n = a.own_len[s];
    const int64_t cap = int64_t(a.ld) << a.shift;
    const int32_t prefix = a.prefix_len[upper(a.group_seq, a.G, s)];
    if (q < 0 || n < 0 || n + q > cap || prefix + n + q > int64_t(0x7fffffff)) {
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
  tokens = block_sum(tokens, sums);
  pages = block_sum(pages, sums);
  bad |= tokens > a.T;
  const bool enough = pages <= int64_t(a.n_free) - used;
  // the page ids that are taken
  if (!bad && enough)
    for (int i = tid; i < int(pages); i += kMapThreads) {
      const int id = a.free_pages[used + i];
      bad |= id < 0 || id >= a.n_pages;
    }
  if (bad) s_bad = 1;
  __syncthreads();
  const int code = s_bad ? TCL_EINVAL : (enough ? TCL_OK : TCL_ENOSPC);
  if (tid == 0) {
    a.status[0] = code;
    a.status[1] = code == TCL_OK ? int(tokens) : 0;
    a.status[2] = code == TCL_OK ? int(pages) : 0;
    a.status[3] = a.n_free - used - (code == TCL_OK ? int(pages) : 0);
  }
  const bool all = a.T <= kMapOne;
  if (code != TCL_OK) {
    for (int s = tid; s <= a.S; s += kMapThreads) {
      a.seq_tok[s] = 0;
      if (s < a.S) a.own_out[s] = a.own_len[s];
    }
    if (tid == 0) a.used_out[0] = used;
    if (all) pad(a, 0, a.T);
    return;
  }
  walk<true, true>(a, chunk, lds, used, 0, all ? a.T : 0);
  if (all) pad(a, int(tokens), a.T);
}

// the tokens of a batch that kv_map_kernel has looked over
__global__ __launch_bounds__(kMapThreads) void kv_map_fill_kernel(MapArgs a) {
  __shared__ int lds[2][kMapThreads / 64];
  __shared__ Chunk chunk;
  const int t0 = blockIdx.x * kMapThreads, t1 = min(a.T, t0 + kMapThreads);
  const int tokens = a.status[1];
  if (t0 < tokens) walk<false, false>(a, chunk, lds, a.used_out[0] - a.status[2], t0, min(t1, tokens));
  pad(a, max(t0, tokens), t1);
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
    hipLaunchKernelGGL(kv_map_fill_kernel, dim3((a.T + kMapThreads - 1) / kMapThreads), dim3(kMapThreads),
                       0, s, a);
    TCL_HIP(hipGetLastError());
  }
  return TCL_OK;
}
