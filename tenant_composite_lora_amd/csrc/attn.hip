// Attention of a batch over a paged key/value cache whose requests share
// their group's prefix (include/tcl.h has the formulas).
//
// A query row is one head of one token.  Rows that read the same keys through
// the same key/value head form a tile: the tokens of one request, or, over a
// prefix, the tokens of all the short requests of its group, so that the
// prefix is read once for all of them.  The mapping launch (attn_plan_kernel)
// cuts the tiles' keys into items of even length; attn_kernel computes an
// item a workgroup; attn_join_kernel joins the items of rows that have
// several.
//
// attn_kernel computes the transposed products S' = K Q' and O' = V' P' on
// the matrix cores: a lane then holds scores of one query row only, so that
// the running maximum and sum are per-lane numbers with one exchange between
// lane halves (or quarters) a step, and the probabilities leave the first
// product in the very registers the second wants them in.
#include <algorithm>
#include <cmath>
#include <limits>
#include <type_traits>

#include "kern_common.hpp"
#include "kv.hpp"

namespace tcl {
namespace {

constexpr int kRows = 128;      // query rows of a tile of many rows
constexpr int kFew = 16;        // rows of a tile of few rows (keys split over the waves)
constexpr int kKeys = 64;       // keys of a step
constexpr int kMinChunk = 128;  // smallest key range an item is cut to
// Workgroups that a batch is cut into where it has fewer tiles.  Few rows:
// four a CU (with two, four and eight: 64 requests of 8 tenants 174, 160 and
// 155 us, 16 requests of 4 tenants 30, 29 and 32).  Many: two, as many as run
// at a time; their partial outputs weigh more (64 requests over a prefix of
// 8192: 35 + 8 us, with 1024 41 + 10; chunks of 256..512 tokens over 4096: 41
// us of joining, with 1024 107).
constexpr int kTargetFew = 1024, kTargetMany = 512;
// a request whose rows fill half a tile reads its prefix by itself
constexpr int kShortRows = 64;
constexpr int kMagic = 0x41747432;
// workgroups of a launch (of 256 threads, below 2^32 of them)
constexpr int kMaxGrid = 1 << 24;

// A request's keys are numbered with its own ones starting on a step of their
// own: key j < prefix is the prefix's, key j >= whole(prefix) is own key j -
// whole(prefix), and the numbers between name none.  A step then never holds
// keys of both, and every 16 keys of a step lie in one page of 16 or more.
__host__ __device__ inline int whole(int prefix) { return (prefix + kKeys - 1) / kKeys * kKeys; }
// the number behind the first n keys
__device__ inline int key_end(int prefix, int n) {
  return n <= prefix ? n : n + whole(prefix) - prefix;
}

enum { H_CODE, H_MAGIC, H_SEQS, H_GROUPS, H_TOKENS, H_HEADS, H_KVHEADS, H_DIM, H_PAGES, H_SHIFT,
       H_LDO, H_LDP, H_ITEMS, H_TILES, H_SHARED, H_FLAGS = 16, H_WORDS = 64 };
constexpr int kPageGroups = 16;  // workgroups that look page ids over, a flag each

struct alignas(16) Work {
  int32_t tok0;     // first token, or first entry of the token list (list 1)
  int32_t list;
  int32_t n_tok;    // tokens
  int32_t seq, group;
  int32_t prefix;   // keys of the prefix
  int32_t lo, hi;   // keys [lo, hi), lo a whole step
  int32_t part;     // first partial row, -1: write the output itself
  int32_t fine;     // weights in two parts (attend_many)
  int32_t pad[2];
};

struct alignas(16) Tile {
  int32_t n_tok;    // tokens
  int32_t n_split;  // items
  int32_t part0;    // first partial row, -1: its one item writes the output
  int32_t pad;
};

// A token: where the partial rows of its first head lie.  Item i of its own
// range has row own + i * own_step, i < own_n; of its group's prefix likewise.
struct alignas(16) TokRec {
  int32_t vis;  // keys the token sees, -1: no request owns it
  int32_t own, own_n, own_step;
  int32_t pre, pre_n, pre_step;
  int32_t join;  // 0: an item wrote the output
};

struct PlanArgs {
  // table
  const int32_t *seq_tok, *group_seq, *prefix_len, *prefix_pages, *own_len, *own_pages;
  int32_t S, G, T, ldp, ldo;
  int32_t Hq, Hkv, D, n_pages, page_shift;
  int32_t tpt_many, tpt_few;  // whole tokens in a tile
  int32_t cap_tiles, cap_items, cap_rows, target_few, target_many;
  // plan
  int32_t *hdr;
  TokRec *tok;
  Tile *tiles;
  Work *items;
  int32_t *list;       // [T]
  int32_t *short_tok;  // [S + 1] tokens of short requests before this one
  int32_t *short_seq;  // [S + 1] short requests before this one
  int32_t *utile;      // [G + S] first tile of a unit (groups first)
};

// The mapping's view of the small arrays: in LDS for up to kMapThreads
// requests and groups (every phase reads them, and a round trip to memory
// each made up most of the launch), else in memory.
struct MapView {
  const int32_t *seq_tok, *group_seq, *prefix_len, *own_len;
  int32_t *short_tok, *short_seq, *utile;
};

struct Layout {
  size_t o_tok, o_tiles, o_items, o_list, o_stok, o_sseq, o_utile, total;
};

// ---------------------------------------------------------------------------
// mapping
// ---------------------------------------------------------------------------
constexpr int kMapThreads = 1024;

// Inclusive scan over a wave by lane moves: 1, 2, 4 and 8 lanes inside each
// row of 16, then the last lane of rows 0 and 2 into the row behind, then the
// last lane of row 1 into rows 2 and 3.  ROWS false: inside rows only.
template <bool ROWS>
__device__ inline int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  if constexpr (ROWS) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  }
  return v;
}

// Exclusive scans of N numbers a thread over the workgroup: v becomes the sum
// before the thread, total the workgroup's.
template <int N>
__device__ inline void block_scan(int (&v)[N], int (&total)[N], int (*lds)[kMapThreads / 64]) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int W = kMapThreads / 64;
  static_assert(W == 16, "the waves' sums fill a row of lanes");
  int inc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) inc[i] = lane_scan<true>(v[i]);
  __syncthreads();
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds[i][w] = inc[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // the waves' sums, scanned by every wave
    const int x = lds[i][lane & (W - 1)], y = lane_scan<false>(x);
    total[i] = __builtin_amdgcn_readlane(y, W - 1);
    v[i] = inc[i] - v[i] + __builtin_amdgcn_readlane(y - x, w);
  }
}

__device__ inline int upper(const int32_t *ptr, int n, int x) {
  // the last i in [0, n) with ptr[i] <= x
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (ptr[m] <= x)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

struct Unit {
  int rows, n_tok, tpt;  // rows, tokens, tokens a tile
  int tok0, list, seq, group, prefix, lo, hi, n_q;
};

__device__ inline bool is_short(const PlanArgs &a, int q) {
  return q > 0 && int64_t(q) * (a.Hq / a.Hkv) < kShortRows;
}

__device__ inline bool shares(const PlanArgs &a, const MapView &m, int g) {
  const int b = m.group_seq[g], e = m.group_seq[g + 1];
  return m.prefix_len[g] > 0 && m.short_seq[e] - m.short_seq[b] >= 2;
}

// unit u: group u's prefix for u < G, request u - G's own keys (and its
// prefix, if it does not share it) above
__device__ inline Unit unit_of(const PlanArgs &a, const MapView &m, int u) {
  Unit x{};
  const int gq = a.Hq / a.Hkv;
  if (u < a.G) {
    if (!shares(a, m, u)) return x;
    const int b = m.group_seq[u], e = m.group_seq[u + 1];
    x.tok0 = m.short_tok[b];
    x.n_tok = m.short_tok[e] - x.tok0;
    x.list = 1;
    x.group = u;
    x.prefix = x.hi = m.prefix_len[u];
  } else {
    const int s = u - a.G;
    x.tok0 = m.seq_tok[s];
    x.n_tok = x.n_q = m.seq_tok[s + 1] - x.tok0;
    x.seq = s;
    x.group = upper(m.group_seq, a.G, s);
    // (empty groups: the one whose range holds s)
    x.prefix = m.prefix_len[x.group];
    x.lo = is_short(a, x.n_q) && shares(a, m, x.group) ? whole(x.prefix) : 0;
    x.hi = x.prefix + m.own_len[s];  // (a count here)
  }
  x.rows = x.n_tok * gq;
  x.tpt = x.rows <= kFew ? a.tpt_few : a.tpt_many;
  return x;
}

__device__ inline int unit_tiles(const Unit &x) {
  return x.n_tok == 0 ? 0 : (x.n_tok + x.tpt - 1) / x.tpt;
}

// last key + 1 of tile i of a unit: the keys its last token sees
__device__ inline int tile_hi(const Unit &x, int i) {
  if (x.list) return x.hi;
  const int last = min(x.n_tok, (i + 1) * x.tpt) - 1;
  return max(x.lo, key_end(x.prefix, max(0, x.hi - x.n_q + last + 1)));
}

// 64 requests 10.4 us, 8 prompts of 512 tokens 11.2, 3 requests 7.8: a launch
// and the round trips of some fifteen phases.
// Workgroups 1 .. kPageGroups look page ids over, a row of a page table a wave,
// and leave a flag each; workgroup 0 does the rest.  One launch: the flags
// are read with the header.
template <bool LDS>
__global__ __launch_bounds__(kMapThreads) void attn_plan_kernel(PlanArgs a) {
  __shared__ int lds[3][kMapThreads / 64];
  __shared__ int s_err, s_chunk[2];
  __shared__ unsigned long long s_work;
  constexpr int NS = LDS ? kMapThreads + 1 : 1;
  __shared__ int32_t l_seq_tok[NS], l_group_seq[NS], l_prefix_len[NS], l_own_len[NS],
      l_short_tok[NS], l_short_seq[NS], l_utile[2 * NS];
  __shared__ int32_t l_unit[kMapThreads], l_place[kMapThreads], l_item[kMapThreads], l_row[kMapThreads];
  const int tid = threadIdx.x, gq = a.Hq / a.Hkv;
  const int page = 1 << a.page_shift;
  if (tid == 0) {
    s_err = 0;
    s_work = 0;
  }
  if (blockIdx.x > 0) {
    __syncthreads();
    const int w = (int(blockIdx.x) - 1) * (kMapThreads / 64) + (tid >> 6), lane = tid & 63;
    bool bad = false;
    for (int r = w; r < a.S + a.G; r += kPageGroups * (kMapThreads / 64)) {
      const bool own = r < a.S;
      const int g = r - a.S, ld = own ? a.ldo : a.ldp;
      // (a length that does not fit is workgroup 0's finding)
      const int len = min(max(own ? a.own_len[r] : a.prefix_len[g], 0), ld * page);
      const int n = (len + page - 1) >> a.page_shift;
      const int32_t *p = own ? a.own_pages + int64_t(r) * a.ldo : a.prefix_pages + int64_t(g) * a.ldp;
#pragma unroll 4
      for (int i = lane; i < n; i += 64) bad |= p[i] < 0 || p[i] >= a.n_pages;
    }
    if (bad) s_err = 1;
    __syncthreads();
    if (tid == 0) a.hdr[H_FLAGS + blockIdx.x - 1] = s_err;
    return;
  }
  MapView m{a.seq_tok, a.group_seq, a.prefix_len, a.own_len, a.short_tok, a.short_seq, a.utile};
  if constexpr (LDS) {
    if (a.S > 0) {
      for (int i = tid; i <= a.S; i += kMapThreads) l_seq_tok[i] = a.seq_tok[i];
      for (int i = tid; i <= a.G; i += kMapThreads) l_group_seq[i] = a.group_seq[i];
      if (tid < a.S) l_own_len[tid] = a.own_len[tid];
      if (tid < a.G) l_prefix_len[tid] = a.prefix_len[tid];
    }
    m = MapView{l_seq_tok, l_group_seq, l_prefix_len, l_own_len, l_short_tok, l_short_seq, l_utile};
  }
  if (tid == 0) {
    a.hdr[H_MAGIC] = kMagic, a.hdr[H_SEQS] = a.S, a.hdr[H_GROUPS] = a.G, a.hdr[H_TOKENS] = a.T;
    a.hdr[H_HEADS] = a.Hq, a.hdr[H_KVHEADS] = a.Hkv, a.hdr[H_DIM] = a.D;
    a.hdr[H_PAGES] = a.n_pages, a.hdr[H_SHIFT] = a.page_shift;
    a.hdr[H_LDO] = a.ldo, a.hdr[H_LDP] = a.ldp;
    a.hdr[H_CODE] = TCL_OK, a.hdr[H_ITEMS] = 0, a.hdr[H_TILES] = 0, a.hdr[H_SHARED] = 0;
  }
  __syncthreads();
  // the table
  bool bad = false;
  if (tid == 0 && a.S > 0)
    bad = m.seq_tok[0] != 0 || m.seq_tok[a.S] > a.T || m.group_seq[0] != 0 ||
          m.group_seq[a.G] != a.S;
  for (int s = tid; s < a.S; s += kMapThreads) {
    bad |= m.seq_tok[s + 1] < m.seq_tok[s];
    bad |= m.own_len[s] < 0 || m.own_len[s] > a.ldo * page;
  }
  for (int g = tid; g < a.G; g += kMapThreads) {
    bad |= m.group_seq[g + 1] < m.group_seq[g];
    bad |= m.prefix_len[g] < 0 || m.prefix_len[g] > a.ldp * page;
  }
  if (bad) s_err = 1;
  __syncthreads();
  if (s_err) {
    if (tid == 0) a.hdr[H_CODE] = TCL_EINVAL;
    return;
  }
  // requests and tokens that may share a prefix, counted in order
  int tok_base = 0, seq_base = 0;
  for (int s0 = 0; s0 < a.S; s0 += kMapThreads) {
    const int s = s0 + tid;
    const int q = s < a.S ? m.seq_tok[s + 1] - m.seq_tok[s] : 0;
    const bool sh = is_short(a, q);
    int v[2] = {sh ? q : 0, sh ? 1 : 0}, total[2];
    block_scan(v, total, lds);
    if (s < a.S) {
      m.short_tok[s] = tok_base + v[0];
      m.short_seq[s] = seq_base + v[1];
    }
    tok_base += total[0];
    seq_base += total[1];
  }
  if (tid == 0) {
    m.short_tok[a.S] = tok_base;
    m.short_seq[a.S] = seq_base;
  }
  __syncthreads();
  // keys over all tiles: the length of an item
  const int U = a.G + a.S;
  unsigned long long work = 0;
  for (int u = tid; u < U; u += kMapThreads) {
    const Unit x = unit_of(a, m, u);
    const int n = unit_tiles(x);
    for (int i = 0; i < n; ++i) work += unsigned(tile_hi(x, i) - x.lo);
  }
  if (work) atomicAdd(&s_work, work);  // (an integer sum: any order)
  __syncthreads();
  if (tid < 2) {
    const unsigned t = tid ? a.target_many : a.target_few;
    const unsigned long long r = ((s_work + t - 1) / t + kKeys - 1) / kKeys * kKeys;
    s_chunk[tid] = r < kMinChunk ? kMinChunk : (r > 0x40000000ull ? 0x40000000 : int(r));
  }
  __syncthreads();
  // the units' first tiles
  int n_tiles = 0;
  for (int u0 = 0; u0 < U; u0 += kMapThreads) {
    const int u = u0 + tid;
    int v[1] = {u < U ? unit_tiles(unit_of(a, m, u)) : 0}, total[1];
    block_scan(v, total, lds);
    if (u < U) m.utile[u] = n_tiles + v[0];
    n_tiles += total[0];
  }
  __syncthreads();
  // tiles, a thread each, then their items, a thread each
  // (the capacities hold every table of these sizes; what lies beyond them
  // could only come from a table that changed under the launch)
  n_tiles = min(n_tiles, a.cap_tiles);
  int item_base = 0, row_base = 0;
  struct Cut {
    Unit x;
    int i, hi, nt, ns, per;
  };
  auto cut = [&](int u, int i) {
    Cut c{unit_of(a, m, u), i, 0, 0, 0, 0};
    c.hi = tile_hi(c.x, i);
    const int len = c.hi - c.x.lo, chunk = s_chunk[c.x.rows > kFew];
    c.nt = min(c.x.n_tok, (i + 1) * c.x.tpt) - i * c.x.tpt;
    c.ns = max(1, (len + chunk - 1) / chunk);
    // even lengths, whole steps
    c.per = max(kKeys, ((len + c.ns - 1) / c.ns + kKeys - 1) / kKeys * kKeys);
    return c;
  };
  auto direct = [](const Cut &c) { return c.ns == 1 && !c.x.list && c.x.lo == 0; };
  for (int t0 = 0; t0 < n_tiles; t0 += kMapThreads) {
    const int t = t0 + tid, here = min(kMapThreads, n_tiles - t0);
    int v[2] = {0, 0}, total[2];
    Cut c{};
    if (tid < here) {
      const int u = upper(m.utile, U, t);
      c = cut(u, t - m.utile[u]);
      v[0] = c.ns;
      v[1] = c.ns * c.nt * gq;
      l_unit[tid] = u;
      l_place[tid] = c.i;
    }
    block_scan(v, total, lds);
    if (tid < here) {
      l_item[tid] = v[0];
      l_row[tid] = row_base + v[1];
      a.tiles[t] = Tile{c.nt, c.ns, direct(c) ? -1 : row_base + v[1], 0};
    }
    __syncthreads();
    for (int k = tid; k < total[0]; k += kMapThreads) {
      const int j = upper(l_item, here, k), n = k - l_item[j];
      c = cut(l_unit[j], l_place[j]);
      const int lo = min(c.hi, c.x.lo + n * c.per), row = l_row[j] + n * c.nt * gq;
      if (item_base + k >= a.cap_items || row + c.nt * gq > a.cap_rows) continue;
      a.items[item_base + k] = Work{c.x.tok0 + c.i * c.x.tpt, c.x.list, c.nt, c.x.seq, c.x.group,
                                    c.x.prefix, lo, min(c.hi, lo + c.per), direct(c) ? -1 : row,
                                    c.x.list || is_short(a, c.x.n_q), {}};
    }
    item_base += total[0], row_base += total[1];
    __syncthreads();
  }
  // tokens
  for (int t = tid; t < a.T; t += kMapThreads) {
    TokRec r{-1, 0, 0, 0, 0, 0, 0, 0};
    if (a.S > 0 && t < m.seq_tok[a.S]) {
      const int s = upper(m.seq_tok, a.S, t);
      const Unit x = unit_of(a, m, a.G + s);
      const int i = t - x.tok0;
      r.vis = max(0, x.hi - x.n_q + i + 1);  // (a count)
      const Tile o = a.tiles[min(m.utile[a.G + s] + i / x.tpt, a.cap_tiles - 1)];
      r.own = o.part0 + i % x.tpt * gq;
      r.own_n = o.n_split;
      r.own_step = o.n_tok * gq;
      r.join = o.part0 >= 0;
      if (is_short(a, x.n_q) && shares(a, m, x.group)) {
        const Unit p = unit_of(a, m, x.group);
        const int at = m.short_tok[s] + i;
        a.list[min(at, a.T - 1)] = t;
        const Tile q = a.tiles[min(m.utile[x.group] + (at - p.tok0) / p.tpt, a.cap_tiles - 1)];
        r.pre = q.part0 + (at - p.tok0) % p.tpt * gq;
        r.pre_n = q.n_split;
        r.pre_step = q.n_tok * gq;
      }
    }
    a.tok[t] = r;
  }
  if (tid == 0) {
    a.hdr[H_ITEMS] = min(item_base, a.cap_items);
    a.hdr[H_TILES] = n_tiles;
    a.hdr[H_SHARED] = tok_base;
  }
}

__device__ inline bool pages_ok(const int32_t *hdr) {
  int bad = 0;
#pragma unroll
  for (int i = 0; i < kPageGroups; ++i) bad |= hdr[H_FLAGS + i];
  return bad == 0;
}

__global__ void attn_status_kernel(const int32_t *hdr, int32_t *out) {
  if (threadIdx.x > 0) return;
  const bool ok = hdr[H_CODE] == TCL_OK && pages_ok(hdr);
  out[0] = ok ? TCL_OK : TCL_EINVAL;
  out[1] = ok ? hdr[H_ITEMS] : 0;
  out[2] = ok ? hdr[H_TILES] : 0;
  out[3] = ok ? hdr[H_SHARED] : 0;
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
struct AttnArgs {
  KvArgs c;
  const uint16_t *q;
  uint16_t *o;
  float *lse;
  int64_t ldq, ldo;
  float scale2;    // |scale| * log2(e)
  int32_t q_sign;  // the sign bit of a bf16 number where scale is negative
  int32_t S, G, T, ldp, ld_own, Hq;
  const int32_t *prefix_pages, *own_pages;
  const int32_t *hdr;
  const TokRec *tok;
  const Work *items;
  const int32_t *list;
  float *part_o;   // [rows][Hkv][D], not divided by the sum
  float2 *part_ml; // [rows][Hkv]: running maximum (of base-2 scores), sum
};

// the plan belongs to these sizes (a plan of other sizes: nothing is done)
__device__ inline bool plan_fits(const AttnArgs &a) {
  const int32_t *h = a.hdr;
  return h[H_MAGIC] == kMagic && h[H_CODE] == TCL_OK && h[H_SEQS] == a.S && h[H_GROUPS] == a.G &&
         h[H_TOKENS] == a.T && h[H_HEADS] == a.Hq && h[H_KVHEADS] == a.c.H && h[H_DIM] == a.c.D &&
         h[H_PAGES] == a.c.n_pages && h[H_SHIFT] == a.c.page_shift && h[H_LDO] == a.ld_own &&
         h[H_LDP] == a.ldp && pages_ok(h);
}

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef short s16x4 __attribute__((__vector_size__(4 * sizeof(short))));
typedef short s16x8 __attribute__((__vector_size__(8 * sizeof(short))));

// LDS holds a step's keys (or values) as rows of D / 8 16-byte chunks; chunk
// c of row r lies at c ^ swz(r).  A key operand reads one chunk of 16 or 32
// rows, a transposed value operand four chunks of 4 or 8 rows: both then
// fall on all banks.
template <int D>
__device__ inline int swz(int r) {
  if constexpr (D == 64)
    return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
  else
    return (r & 3) << 2 | ((r >> 2) & 3);
}

// Four keys' values of one dimension: lane l of a group of 16 names four
// neighbouring elements of key l / 4 and receives element l of keys 0..3.
__device__ inline s16x4 read_tr(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}

__device__ inline uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 v = {__bf16(a), __bf16(b)};
  return __builtin_bit_cast(uint32_t, v);
}

template <int D>
struct Smem {
  uint16_t k[2][kKeys * D];
  uint16_t v[2][kKeys * D];
};

// Writes four neighbouring dimensions of a row: the output itself, or a
// partial one.
__device__ inline void put4(uint16_t *o, const float *v, float f) {
  *reinterpret_cast<nt_u2 *>(o) = nt_u2{pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f)};
}

// A step's keys: key i0 + r of the part (prefix or own) for row r, the part's
// last key again behind it (masked where it is used).
struct Part {
  const int32_t *table;
  int i0, last;
};
__device__ inline Part part_of(const AttnArgs &a, const Work &t, int j0) {
  const int w = whole(t.prefix);
  if (j0 < w) return {a.prefix_pages + int64_t(t.group) * a.ldp, j0, min(t.prefix, t.hi) - 1};
  return {a.own_pages + int64_t(t.seq) * a.ld_own, j0 - w, t.hi - w - 1};
}

// Infinities and NaNs among the values of keys that a row does not see must
// not reach it, and a zero weight does not keep them out (0 * inf is NaN).
// Where a step hides keys from some row, the values are looked over as they
// pass through registers; where any is not finite, its products are added one
// by one to the rows that see it, zero takes its place in LDS, and the matrix
// product goes on as ever.
__device__ inline bool bad_bf16(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }
__device__ inline nt_u4 cleaned(nt_u4 u) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    u[e] = (bad_bf16(u[e]) ? 0 : u[e] & 0xffffu) | (bad_bf16(u[e] >> 16) ? 0 : u[e] & 0xffff0000u);
  return u;
}

// Moves an item's keys and values, 64 a step, through registers into LDS:
// wave w the rows 16 w .. 16 w + 15 of a step.  Where those lie in one page
// its id is read two steps ahead, and the rows' addresses are a scalar and
// lane offsets that never change; else (small pages, a part's last step) each
// lane looks its rows up.  Page ids are held to the cache's pages, so that a
// table that changed after its mapping reads other keys, never other memory.
template <int D>
struct Stage {
  static constexpr int CH = D / 8;     // chunks of a row
  static constexpr int RPI = 64 / CH;  // rows a wave loads an instruction
  static constexpr int NI = 16 / RPI;  // instructions for a wave's 16 rows
  nt_u4 k[NI], v[NI];
  int page;  // of the wave's rows of the next step to be loaded
  int w, row, col;
  unsigned lane_off;  // bytes, of the wave's first RPI rows
  int64_t head;
  bool paged;

  __device__ inline void init(const AttnArgs &a, int h) {
    const int lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    row = lane / CH;
    col = lane % CH;
    head = int64_t(h) * a.c.s_head;
    paged = a.c.page_shift >= 4 && a.c.s_slot < (int64_t(1) << 26);
    lane_off = 2 * (unsigned(row) * unsigned(a.c.s_slot) + 8 * col);
  }
  __device__ inline int clamp(const AttnArgs &a, int p) const {
    return min(max(p, 0), a.c.n_pages - 1);
  }
  __device__ inline void pages(const AttnArgs &a, const Work &t, int j0) {
    if (!paged || j0 >= t.hi) return;
    const Part p = part_of(a, t, j0);
    page = p.table[min(p.i0 + 16 * w, p.last) >> a.c.page_shift];
  }
  __device__ inline void load(const AttnArgs &a, const Work &t, int j0) {
    const Part p = part_of(a, t, j0);
    const int mask = (1 << a.c.page_shift) - 1;
    if (paged && p.i0 + kKeys - 1 <= p.last) {
      const int64_t at = int64_t(clamp(a, __builtin_amdgcn_readfirstlane(page))) * a.c.s_page +
                         int64_t((p.i0 + 16 * w) & mask) * a.c.s_slot + head;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const char *bk = reinterpret_cast<const char *>(a.c.K + at + i * RPI * a.c.s_slot);
        const char *bv = reinterpret_cast<const char *>(a.c.V + at + i * RPI * a.c.s_slot);
        k[i] = *reinterpret_cast<const nt_u4 *>(bk + lane_off);
        v[i] = *reinterpret_cast<const nt_u4 *>(bv + lane_off);
      }
      return;
    }
    int64_t at[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int j = min(p.i0 + 16 * w + row + i * RPI, p.last);
      at[i] = int64_t(clamp(a, p.table[j >> a.c.page_shift])) * a.c.s_page +
              int64_t(j & mask) * a.c.s_slot + head + 8 * col;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      k[i] = *reinterpret_cast<const nt_u4 *>(a.c.K + at[i]);
      v[i] = *reinterpret_cast<const nt_u4 *>(a.c.V + at[i]);
    }
  }
  // a value that is not finite among those in registers
  __device__ inline bool bad() const {
    // (magnitudes in order of their bits, two at a time)
    typedef uint16_t us2 __attribute__((ext_vector_type(2)));
    us2 x = {0, 0};
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x = __builtin_elementwise_max(x, __builtin_bit_cast(us2, v[i][e] & 0x7fff7fffu));
    return x[0] >= 0x7f80 || x[1] >= 0x7f80;
  }
  // zero for those among the wave's own rows in LDS
  __device__ inline void clean(uint16_t *sv) const {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = 16 * w + row + i * RPI;
      nt_u4 *p = reinterpret_cast<nt_u4 *>(sv + r * D + 8 * (col ^ swz<D>(r)));
      *p = cleaned(*p);
    }
  }
  __device__ inline void put(uint16_t *sk, uint16_t *sv) const {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = 16 * w + row + i * RPI, p = r * D + 8 * (col ^ swz<D>(r));
      *reinterpret_cast<nt_u4 *>(sk + p) = k[i];
      *reinterpret_cast<nt_u4 *>(sv + p) = v[i];
    }
  }
};

// The number behind the keys that a row with `vis` keys sees of the step at
// j0.
__device__ inline int step_end(const Work &t, int vis, int j0) {
  const int w = whole(t.prefix);
  return j0 < w ? min(vis, t.prefix) : vis + w - t.prefix;
}

// value d of row r in LDS
template <int D>
__device__ inline uint32_t value_at(const uint16_t *sv, int r, int d) {
  return sv[r * D + 8 * ((d >> 3) ^ swz<D>(r)) + (d & 7)];
}

// The step's barrier: LDS only, global loads stay in flight across it.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ inline int token_of(const AttnArgs &a, const Work &t, int gq, int r) {
  const int i = t.tok0 + r / gq;
  return t.list ? a.list[i] : i;
}

// What a row's sums are multiplied by at the end.  Without any weight a row
// that sees no key is zero; one that sees keys, all with a score of -infinity,
// has no softmax and is NaN.
__device__ inline float over_sum(float l, int vis) {
  return l > 0.f || l != l ? 1.f / l : (vis > 0 ? NAN : 0.f);
}

__device__ inline float log_sum(float m, float l) {
  return (m + __log2f(l)) * 0.69314718055994531f;
}

// A maximum that only follows the scores when they pass it by kSlack (in
// powers of two): weights then reach 2^kSlack, which neither fp32 sums nor
// bf16's relative rounding mind, and the outputs are rescaled a few times an
// item instead of every step.
constexpr float kSlack = 8.f;

// The larger of two numbers as a median with infinity: fmaxf first passes each
// score of a matrix instruction through a multiplication by one.
__device__ inline float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }

// the larger of a lane's value and that of the lane 32 away
__device__ inline float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Few rows: every wave holds all of them, over its own 16 keys of a step, and
// needs no barrier; the waves' results are joined through LDS.  Bound by the
// keys' and values' bytes: 64 requests of 8 tenants, 760 MB with the prefixes,
// 150 us, 5.1 TB/s.
template <int D>
__device__ inline void attend_few(const AttnArgs &a, const Work &t, int h, int gq, Smem<D> &sm) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int rows = t.n_tok * gq, steps = (t.hi - t.lo + kKeys - 1) / kKeys;
  Stage<D> st;
  st.init(a, h);
  if (steps > 0) st.pages(a, t, t.lo);
  const int c = lane & 15, g = lane >> 4;
  const bool live = c < rows;
  const int tok = token_of(a, t, gq, live ? c : 0);
  const int hq = h * gq + (live ? c : 0) % gq;
  if (steps > 0) {
    st.load(a, t, t.lo);
    st.pages(a, t, t.lo + kKeys);
  }
  const int vis = live ? a.tok[tok].vis : 0;
  s16x8 qf[D / 32];
#pragma unroll
  for (int s = 0; s < D / 32; ++s)
    qf[s] = *reinterpret_cast<const s16x8 *>(a.q + tok * a.ldq + int64_t(hq) * D + 32 * s + 8 * g) ^
            short(a.q_sign);
  f32x4_t o[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i] = f32x4_t{0, 0, 0, 0};
  float m = -INFINITY, l = 0.f;
  for (int n = 0; n < steps; ++n) {
    const int j0 = t.lo + n * kKeys, b = n & 1;
    st.put(sm.k[b], sm.v[b]);
    // (here in every step: a weight's second part may be zero or negative)
    const bool rare = __any(st.bad());
    if (n + 1 < steps) {
      st.load(a, t, j0 + kKeys);
      st.pages(a, t, j0 + 2 * kKeys);
    }
    // (a wave reads only what it wrote)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    f32x4_t s4 = {0, 0, 0, 0};
    const int kr = 16 * w + c;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const bf16x8_t kf =
          *reinterpret_cast<const bf16x8_t *>(&sm.k[b][kr * D + 8 * ((4 * s + g) ^ swz<D>(kr))]);
      s4 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, __builtin_bit_cast(bf16x8_t, qf[s]), s4, 0, 0, 0);
    }
    float p[4], mx = -INFINITY;
    // visible keys of the lane's four
    const int left = min(step_end(t, vis, j0), t.hi) - (j0 + 16 * w + 4 * g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = i < left ? s4[i] : -INFINITY;
      mx = fmaxf(mx, p[i]);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64)) * a.scale2;
    if (__any(mx > m + kSlack)) {
      const float mn = fmaxf(m, mx), al = mn == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= al;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[d] *= al;
    }
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], a.scale2, -mu));
      l += p[i];
    }
    // probabilities in two bf16 parts: the matrix cores idle here, and the
    // rounding of one part would show beside the output's own
    uint32_t hi2[2], lo2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hi2[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
      lo2[i] = pack_bf16(p[2 * i] - bf16_lo(hi2[i]), p[2 * i + 1] - bf16_hi(hi2[i]));
    }
    const s16x4 ph = __builtin_bit_cast(s16x4, nt_u2{hi2[0], hi2[1]});
    const s16x4 pl = __builtin_bit_cast(s16x4, nt_u2{lo2[0], lo2[1]});
    if (rare) {
#pragma unroll 1
      for (int k = 0; k < 16; ++k) {
        const float q = k & 2 ? (k & 1 ? p[3] : p[2]) : (k & 1 ? p[1] : p[0]);
        const float pk = __shfl(q, c + 16 * (k >> 2), 64);
        if (k >= left + 4 * g) continue;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t u = value_at<D>(sm.v[b], 16 * w + k, 16 * d + 4 * g + e);
            if (bad_bf16(u)) o[d][e] += pk * __uint_as_float(u << 16);
          }
      }
      st.clean(sm.v[b]);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    }
    const int vr = 16 * w + 4 * g + (c >> 2);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const s16x4 vf = read_tr(&sm.v[b][vr * D + 8 * ((2 * d + ((c & 3) >> 1)) ^ swz<D>(vr)) + 4 * (c & 1)]);
      o[d] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(vf, ph, o[d], 0, 0, 0);
      o[d] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(vf, pl, o[d], 0, 0, 0);
    }
  }
  // join the waves: maxima and sums, then outputs, through LDS
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  __syncthreads();
  float *jo = reinterpret_cast<float *>(&sm);  // [4][16][D]
  static_assert(sizeof(sm) >= 4 * 16 * D * 4 + 4 * 16 * 8, "LDS of the join");
  float2 *jm = reinterpret_cast<float2 *>(jo + 4 * 16 * D);  // [4][16]
  if (g == 0) jm[w * 16 + c] = make_float2(m, l);
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
    *reinterpret_cast<f32x4_t *>(&jo[(w * 16 + c) * D + 16 * d + 4 * g]) = o[d];
  __syncthreads();
  for (int x = tid; x < rows * (D / 4); x += 256) {
    const int r = x / (D / 4), d = x % (D / 4) * 4;
    float M = -INFINITY, L = 0.f, f[4], v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) M = fmaxf(M, jm[i * 16 + r].x);
    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __builtin_amdgcn_exp2f(jm[i * 16 + r].x - mu);
      L += jm[i * 16 + r].y * f[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t u = *reinterpret_cast<const f32x4_t *>(&jo[(i * 16 + r) * D + d]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e] * f[i];
    }
    const int tk = token_of(a, t, gq, r), hh = h * gq + r % gq;
    if (t.part < 0) {
      put4(a.o + tk * a.ldo + int64_t(hh) * D + d, v, over_sum(L, L == 0.f ? a.tok[tk].vis : 0));
      if (a.lse && d == 0) a.lse[int64_t(tk) * a.Hq + hh] = log_sum(M, L);
    } else {
      const int64_t pr = int64_t(t.part + r) * a.c.H + h;
      *reinterpret_cast<f32x4_t *>(a.part_o + pr * D + d) = f32x4_t{v[0], v[1], v[2], v[3]};
      if (d == 0) a.part_ml[pr] = make_float2(M, L);
    }
  }
}

// Moves a step's keys and values straight into LDS, wave w the rows 16 w .. 16
// w + 15: 64 lanes write 1 KiB in a row, so a lane fetches the chunk that
// belongs where it writes.  Such loads take no registers and are not counted
// by the compiler; arrived() waits for all of them.  Their immediate offset
// moves source and destination alike, so one M0 serves four instructions.
template <int D>
struct Direct {
  static constexpr int CH = D / 8;     // chunks of a row
  static constexpr int RPI = 64 / CH;  // rows an instruction moves
  static constexpr int NI = 16 / RPI;  // instructions for a wave's 16 rows
  static_assert(NI == 2 || NI == 4 || NI == 8, "head dimension");
  int w, row, page;
  unsigned off[NI];  // bytes from the wave's first row, less the immediate offset
  int64_t head;
  bool paged;

  __device__ inline void init(const AttnArgs &a, int h) {
    const int lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    row = lane / CH;
    head = int64_t(h) * a.c.s_head;
    paged = a.c.page_shift >= 4 && a.c.s_slot >= D && a.c.s_slot < (int64_t(1) << 26);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + row;
      off[i] = 2 * (unsigned(r) * unsigned(a.c.s_slot) + 8 * (lane % CH ^ swz<D>(r))) - 1024 * (i & 3);
    }
  }
  __device__ inline int clamp(const AttnArgs &a, int p) const {
    return min(max(p, 0), a.c.n_pages - 1);
  }
  // reads the page of the wave's rows of the next step to be loaded
  __device__ inline void pages(const AttnArgs &a, const Work &t, int j0) {
    if (!paged || j0 >= t.hi) return;
    const Part p = part_of(a, t, j0);
    page = p.table[min(p.i0 + 16 * w, p.last) >> a.c.page_shift];
  }
  __device__ static inline uint32_t lds(const uint16_t *p) {
    return uint32_t(uintptr_t((__attribute__((address_space(3))) const uint16_t *)(p)));
  }
  __device__ inline void load(const AttnArgs &a, const Work &t, int j0, uint16_t *sk,
                              uint16_t *sv) const {
    const Part p = part_of(a, t, j0);
    const int mask = (1 << a.c.page_shift) - 1;
    const uint32_t to[2] = {lds(sk + 16 * w * D), lds(sv + 16 * w * D)};
    if (paged && p.i0 + kKeys - 1 <= p.last) {
      const int64_t at = int64_t(clamp(a, __builtin_amdgcn_readfirstlane(page))) * a.c.s_page +
                         int64_t((p.i0 + 16 * w) & mask) * a.c.s_slot + head;
      const uint16_t *from[2] = {a.c.K + at, a.c.V + at};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if constexpr (NI == 2)
          asm volatile(
              "s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %3\n\t"
              "global_load_lds_dwordx4 %2, %3 offset:1024" ::"s"(to[x]),
              "v"(off[0]), "v"(off[1]), "s"(from[x])
              : "memory", "m0");
        else
#pragma unroll
          for (int i = 0; i < NI; i += 4)
            asm volatile(
                "s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %5\n\t"
                "global_load_lds_dwordx4 %2, %5 offset:1024\n\t"
                "global_load_lds_dwordx4 %3, %5 offset:2048\n\t"
                "global_load_lds_dwordx4 %4, %5 offset:0xc00" ::"s"(to[x] + 1024 * i),
                "v"(off[i]), "v"(off[i + 1]), "v"(off[i + 2]), "v"(off[i + 3]), "s"(from[x])
                : "memory", "m0");
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = 16 * w + i * RPI + row, j = min(p.i0 + r, p.last);
      const int64_t at = int64_t(clamp(a, p.table[j >> a.c.page_shift])) * a.c.s_page +
                         int64_t(j & mask) * a.c.s_slot + head +
                         8 * ((threadIdx.x & 63) % CH ^ swz<D>(r));
      const uint16_t *from[2] = {a.c.K + at, a.c.V + at};
#pragma unroll
      for (int x = 0; x < 2; ++x)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to[x] + 1024 * i),
                     "v"(from[x])
                     : "memory", "m0");
    }
  }
  __device__ inline void arrived() const { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

  // values that are not finite among the wave's rows in LDS; zero for them
  __device__ inline nt_u4 *chunk(uint16_t *sv, int i) const {
    return reinterpret_cast<nt_u4 *>(sv + 16 * w * D) + 64 * i + (threadIdx.x & 63);
  }
  __device__ inline bool bad(uint16_t *sv) const {
    bool x = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const nt_u4 u = *chunk(sv, i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x |= bad_bf16(u[e]) || bad_bf16(u[e] >> 16);
    }
    return x;
  }
  __device__ inline void clean(uint16_t *sv) const {
#pragma unroll
    for (int i = 0; i < NI; ++i) *chunk(sv, i) = cleaned(*chunk(sv, i));
  }
};

// Many rows: wave w holds rows 32 w .. 32 w + 31 over all keys of a step.
// Operands are read from LDS some instructions before the matrix instruction
// that takes them (sched_group_barrier): left to itself the compiler reads
// each right before, and the LDS latencies, 48 a step, are twice the matrix
// cores' time (8 requests of 256..512 new tokens over 2048..4096 keys, 244 G
// operations: 366 us, read ahead 290, 840 T a second).  What is left is the
// exponentials and maxima between the two products: two waves a SIMD overlap
// them in part.
//
// FINE: the weights enter the second product as two bf16 parts, less than
// 2^-14 of them lost, else as one, 2^-8.  Two for every tile of short
// requests, so that a token's accuracy does not depend on how many others
// share its prefix and thus its tile (attend_few has two as well): the error
// of the output is then that of its own rounding, 1.66e-3 in the mean against
// 2.2e-3 to 2.3e-3 with one part, and the keys' bytes bound such batches
// anyway (64 requests over a prefix of 8192: 43 us with one part, 46 with two;
// of 8 tenants 158 and 159).  One for long requests, where the matrix cores
// bound (chunks of 8 requests over 4096: 296 us, with two 391).
template <int D, bool FINE>
__device__ inline void attend_many(const AttnArgs &a, const Work &t, int h, int gq, Smem<D> &sm) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int rows = t.n_tok * gq, steps = (t.hi - t.lo + kKeys - 1) / kKeys;
  Direct<D> st;
  st.init(a, h);
  st.pages(a, t, t.lo);
  const int c = lane & 31, g = lane >> 5;
  const int r = 32 * w + c;
  const bool live = r < rows, busy = 32 * w < rows;
  const int tok = token_of(a, t, gq, live ? r : 0);
  const int hq = h * gq + (live ? r : 0) % gq;
  if (steps > 0) st.load(a, t, t.lo, sm.k[0], sm.v[0]);
  st.pages(a, t, t.lo + kKeys);
  const int vis = a.tok[tok].vis;
  // the fewest keys a row of the wave sees: a step beyond them hides some
  int least = live ? vis : 0x7fffffff;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) least = min(least, __shfl_xor(least, x, 64));
  least = __builtin_amdgcn_readfirstlane(least);
  s16x8 qf[D / 16];
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    qf[s] = *reinterpret_cast<const s16x8 *>(a.q + tok * a.ldq + int64_t(hq) * D + 16 * s + 8 * g) ^
            short(a.q_sign);
  f32x16_t o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
  float m = -INFINITY, l = 0.f;
  // operand positions in LDS: key row c and value row vr[x] of the first
  // chunks; chunk 2 s (or block i of 32 dimensions) on, the position's bits
  // change as by the swizzle, by exclusive or
  const int i16 = lane & 15, sub = (lane >> 4) & 1;
  const int kpos = c * D + 8 * (g ^ swz<D>(c));
  int vpos[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int vr = 8 * x + 4 * g + (i16 >> 2);
    vpos[x] = vr * D + 8 * ((2 * sub + ((i16 & 3) >> 1)) ^ swz<D>(vr)) + 4 * (i16 & 1);
  }
  // the whole tile's fewest keys: steps beyond them look their values over
  __shared__ int s_least[4];
  if (lane == 0) s_least[w] = least;
  __syncthreads();
  const int tile_least = __builtin_amdgcn_readfirstlane(
      min(min(s_least[0], s_least[1]), min(s_least[2], s_least[3])));
  auto hides = [&](int j0, int least_) { return j0 + kKeys > min(step_end(t, least_, j0), t.hi); };
  for (int n = 0; n < steps; ++n) {
    const int j0 = t.lo + n * kKeys, b = n & 1;
    // this step's keys and values have come; every wave is done with the
    // buffers that the next loads write
    st.arrived();
    lds_barrier();
    if (n + 1 < steps) {
      st.load(a, t, j0 + kKeys, sm.k[b ^ 1], sm.v[b ^ 1]);
      st.pages(a, t, j0 + 2 * kKeys);
    }
    bool rare = false;
    if (hides(j0, tile_least)) rare = __syncthreads_or(st.bad(sm.v[b]));
    uint32_t pw[4][4], pl[4][4];
    if (busy) {
      const uint16_t *sk = sm.k[0];
      const int kp = kpos + b * kKeys * D;
      f32x16_t s2[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) s2[x][e] = 0.f;
      constexpr int AHEAD = 6;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bf16x8_t kf = *reinterpret_cast<const bf16x8_t *>(sk + ((kp ^ (16 * s)) + 32 * x * D));
          s2[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, __builtin_bit_cast(bf16x8_t, qf[s]),
                                                          s2[x], 0, 0, 0);
        }
      __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (i + AHEAD < D / 8) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (hides(j0, least)) {
        const int end = min(step_end(t, vis, j0), t.hi);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 16; ++e)  // (a constant against the lane's limit)
            if (32 * x + 8 * (e / 4) + e % 4 >= end - j0 - 4 * g) s2[x][e] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = larger(mx, s2[x][e]);
      mx = half_max(mx) * a.scale2;
      if (__any(mx > m + kSlack)) {
        const float mn = fmaxf(m, mx), al = mn == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= al;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[i][e] *= al;
      }
      const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float p = __builtin_amdgcn_exp2f(fmaf(s2[x][e], a.scale2, -mu));
          const float q = __builtin_amdgcn_exp2f(fmaf(s2[x][e + 1], a.scale2, -mu));
          l += p;
          l += q;
          uint32_t &hi = pw[2 * x + e / 8][e % 8 / 2];
          if constexpr (FINE) {
            // (the high part cut off, not rounded, and 2^-20 added, so that the
            // low part of a weight is never zero or negative: either would
            // make a NaN of a seen infinity)
            hi = __builtin_amdgcn_perm(__float_as_uint(q), __float_as_uint(p), 0x07060302);
            pl[2 * x + e / 8][e % 8 / 2] =
                pack_bf16(fmaf(p, 1 + 0x1p-20f, -bf16_lo(hi)), fmaf(q, 1 + 0x1p-20f, -bf16_hi(hi)));
          } else {
            hi = pack_bf16(p, q);
          }
        }
    }
    if (rare) {
      if (busy) {
        const int end = min(step_end(t, vis, j0), t.hi);
#pragma unroll 1
        for (int k = 0; k < kKeys; ++k) {
          // key k's weights: word k / 16, k / 8 % 2, k / 2 % 2 of the lane
          // half k / 4 % 2
          uint32_t u = 0;
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (s == k >> 4 && x == ((k >> 3 & 1) << 1 | (k >> 1 & 1))) u = pw[s][x];
          u = __shfl(int(u), c + 32 * (k >> 2 & 1), 64);
          const float wk = k & 1 ? bf16_hi(u) : bf16_lo(u);
          if (j0 + k >= end) continue;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t y = value_at<D>(sm.v[b], k, 32 * i + 8 * (e / 4) + 4 * g + e % 4);
              if (bad_bf16(y)) o[i][e] += wk * __uint_as_float(y << 16);
            }
        }
      }
      lds_barrier();
      st.clean(sm.v[b]);
      lds_barrier();
    }
    if (!busy) continue;
    const uint16_t *sv = sm.v[0];
    const int vp0 = vpos[0] + b * kKeys * D, vp1 = vpos[1] + b * kKeys * D;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // keys 16 s + {4 g + 0..3, 8 + 4 g + 0..3}: the lane's eight, in order
      const bf16x8_t pf = __builtin_bit_cast(bf16x8_t, nt_u4{pw[s][0], pw[s][1], pw[s][2], pw[s][3]});
      const bf16x8_t pg = __builtin_bit_cast(bf16x8_t, nt_u4{pl[s][0], pl[s][1], pl[s][2], pl[s][3]});
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const s16x4 x = read_tr(sv + ((vp0 ^ (32 * i)) + 16 * s * D));
        const s16x4 y = read_tr(sv + ((vp1 ^ (32 * i)) + 16 * s * D));
        const s16x8 vv = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, vv);
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf, o[i], 0, 0, 0);
        if constexpr (FINE) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pg, o[i], 0, 0, 0);
      }
    }
    constexpr int AHEAD = 6;
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 0);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, FINE ? 2 : 1, 0);
      if (i + AHEAD < D / 8) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (!live) return;
  l += __shfl_xor(l, 32, 64);
  const float f = t.part >= 0 ? 1.f : over_sum(l, vis);
  const int64_t pr = int64_t(t.part + r) * a.c.H + h;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 32 * i + 8 * e + 4 * g;
      const float v[4] = {o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
      if (t.part < 0)
        put4(a.o + tok * a.ldo + int64_t(hq) * D + d, v, f);
      else
        *reinterpret_cast<f32x4_t *>(a.part_o + pr * D + d) = f32x4_t{v[0], v[1], v[2], v[3]};
    }
  if (g == 0) {
    if (t.part >= 0)
      a.part_ml[pr] = make_float2(m, l);
    else if (a.lse)
      a.lse[int64_t(tok) * a.Hq + hq] = log_sum(m, l);
  }
}

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_kernel(AttnArgs a) {
  __shared__ __align__(16) Smem<D> sm;
  if (!plan_fits(a)) return;
  // (workgroups go to the XCDs in turn: with eight key heads each XCD's L2
  // holds one head)
  const int h = blockIdx.x % a.c.H, id = blockIdx.x / a.c.H;
  if (id >= a.hdr[H_ITEMS]) return;
  const Work t = a.items[id];
  const int gq = a.Hq / a.c.H;
  if (t.n_tok * gq <= kFew)
    attend_few<D>(a, t, h, gq, sm);
  else if (t.fine)
    attend_many<D, true>(a, t, h, gq, sm);
  else
    attend_many<D, false>(a, t, h, gq, sm);
}

// Joins the items of a token's rows, a row a wave at a time: maxima first,
// then the weighted sums in item order (own items, then the prefix's).  64
// tokens of 32 heads, 16 items a row: 7 us for 17 MB, load latencies.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int tk = blockIdx.x;
  const TokRec r = a.tok[tk];
  if (!plan_fits(a) || r.vis < 0 || !r.join) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gq = a.Hq / a.c.H;
  constexpr int E = D / 64;
  typedef float fe __attribute__((ext_vector_type(E)));
  for (int hh = blockIdx.y * 4 + w; hh < a.Hq; hh += gridDim.y * 4) {
    const int h = hh / gq;
    // partial row (times heads) of item k: first + k * step
    const int64_t first[2] = {int64_t(r.own + hh % gq) * a.c.H + h, int64_t(r.pre + hh % gq) * a.c.H + h};
    const int64_t step[2] = {int64_t(r.own_step) * a.c.H, int64_t(r.pre_step) * a.c.H};
    const int n[2] = {r.own_n, r.pre_n};
    float M = -INFINITY;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      for (int k = lane; k < n[s]; k += 64) M = fmaxf(M, a.part_ml[first[s] + k * step[s]].x);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor(M, x, 64));
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    fe v;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      auto add = [&](auto n_, int k0) {
        constexpr int N = decltype(n_)::value;
        float2 ml[N];
        fe u[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int64_t p = first[s] + (k0 + k) * step[s];
          ml[k] = a.part_ml[p];
          u[k] = *reinterpret_cast<const fe *>(a.part_o + p * D + lane * E);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float f = __builtin_amdgcn_exp2f(ml[k].x - mu);
          L += ml[k].y * f;
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += u[k][e] * f;
        }
      };
      int k = 0;
      for (; k + 8 <= n[s]; k += 8) add(std::integral_constant<int, 8>{}, k);
      for (; k + 2 <= n[s]; k += 2) add(std::integral_constant<int, 2>{}, k);
      if (k < n[s]) add(std::integral_constant<int, 1>{}, k);
    }
    const float f = over_sum(L, r.vis);
#pragma unroll
    for (int e = 0; e < E; ++e)
      a.o[tk * a.ldo + int64_t(hh) * D + lane * E + e] = f32_to_bf16(v[e] * f);
    if (a.lse && lane == 0) a.lse[int64_t(tk) * a.Hq + hh] = log_sum(M, L);
  }
}

// ---------------------------------------------------------------------------
// checks and launches
// ---------------------------------------------------------------------------
bool misaligned(const void *p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) & (m - 1); }

int check_batch(const tcl_attn_batch *b, const tcl_kv_cache *c, int32_t Hq, KvArgs *kv) {
  int rc = kv_check(c, kv);
  if (rc) return rc;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(TCL_EUNSUPPORTED, "attn: head_dim %d is not 64, 128 or 256", c->head_dim);
  if (!b) return fail(TCL_EINVAL, "attn: batch is NULL");
  if (b->n_seqs < 0 || b->n_groups < 0 || b->n_tokens < 0 || b->ld_own < 0 || b->ld_prefix < 0)
    return fail(TCL_EINVAL, "attn: negative size");
  if (Hq < 1 || Hq % c->n_kv_heads)
    return fail(TCL_EINVAL, "attn: n_q_heads %d is not a multiple of n_kv_heads %d", Hq,
                c->n_kv_heads);
  if (Hq / c->n_kv_heads > kRows)
    return fail(TCL_EUNSUPPORTED, "attn: more than %d query heads a key head", kRows);
  const int64_t lim = int64_t(1) << 30;
  if (int64_t(b->ld_own) * c->page_size >= lim / 2 ||
      int64_t(b->ld_prefix) * c->page_size >= lim / 2)
    return fail(TCL_EUNSUPPORTED, "attn: page tables of 2^29 keys or more");
  if (int64_t(b->n_tokens) * Hq >= lim / 2 || b->n_tokens >= kMaxGrid || b->n_seqs >= kMaxGrid ||
      b->n_groups >= kMaxGrid)
    return fail(TCL_EUNSUPPORTED, "attn: n_tokens * n_q_heads, n_tokens, n_seqs or n_groups too large");
  const int gq = Hq / c->n_kv_heads;
  const int64_t items = 2 * int64_t(b->n_tokens / (kRows / gq)) + b->n_seqs + b->n_groups +
                        (kTargetFew + c->n_kv_heads - 1) / c->n_kv_heads;
  if (items * c->n_kv_heads >= kMaxGrid)
    return fail(TCL_EUNSUPPORTED, "attn: 2^24 row tiles, requests and groups times key heads");
  if (b->n_seqs > 0 && (!b->seq_tok_ptr || !b->group_seq_ptr || !b->own_len))
    return fail(TCL_EINVAL, "attn: batch arrays are NULL");
  if (b->n_seqs > 0 && b->n_groups < 1) return fail(TCL_EINVAL, "attn: requests without a group");
  if (b->n_seqs > 0 && (!b->prefix_len || (b->ld_own > 0 && !b->own_pages) ||
                        (b->ld_prefix > 0 && !b->prefix_pages)))
    return fail(TCL_EINVAL, "attn: prefix_len or page tables are NULL");
  const void *p[] = {b->seq_tok_ptr, b->group_seq_ptr, b->prefix_len,
                     b->prefix_pages, b->own_len, b->own_pages};
  for (const void *x : p)
    if (misaligned(x, 4)) return fail(TCL_EALIGN, "attn: batch arrays must be 4-byte aligned");
  return TCL_OK;
}

void sizes(const tcl_attn_batch *b, const KvArgs &kv, int32_t Hq, PlanArgs *a, Layout *L) {
  const int gq = Hq / kv.H;
  a->S = b->n_seqs, a->G = b->n_groups, a->T = b->n_tokens;
  a->ldp = b->ld_prefix, a->ldo = b->ld_own;
  a->Hq = Hq, a->Hkv = kv.H, a->D = kv.D, a->n_pages = kv.n_pages, a->page_shift = kv.page_shift;
  a->tpt_many = kRows / gq;
  a->tpt_few = gq <= kFew ? kFew / gq : a->tpt_many;
  a->target_few = (kTargetFew + kv.H - 1) / kv.H;
  a->target_many = (kTargetMany + kv.H - 1) / kv.H;
  // tiles: whole ones of all tokens twice (own ranges, prefixes) and a
  // broken one a unit; items: one a tile and the larger target; partial rows:
  // every row twice and a whole tile for each item beyond its tile's first
  a->cap_tiles = 2 * (b->n_tokens / a->tpt_many) + b->n_seqs + b->n_groups;
  a->cap_items = a->cap_tiles + a->target_few;
  a->cap_rows = 2 * b->n_tokens * gq + a->target_many * kRows + a->target_few * kFew;
  size_t at = H_WORDS * 4;
  auto take = [&](size_t n) {
    const size_t o = at;
    at = (at + n + 255) / 256 * 256;
    return o;
  };
  L->o_tok = take(size_t(a->T) * sizeof(TokRec));
  L->o_tiles = take(size_t(a->cap_tiles) * sizeof(Tile));
  L->o_items = take(size_t(a->cap_items) * sizeof(Work));
  L->o_list = take(size_t(a->T) * 4);
  L->o_stok = take((size_t(a->S) + 1) * 4);
  L->o_sseq = take((size_t(a->S) + 1) * 4);
  L->o_utile = take((size_t(a->S) + a->G) * 4);
  L->total = at;
}

size_t ws_rows_bytes(const PlanArgs &a) { return size_t(a.cap_rows) * a.Hkv * a.D * 4; }
size_t ws_total(const PlanArgs &a) { return ws_rows_bytes(a) + size_t(a.cap_rows) * a.Hkv * 8; }

int check_plan(const void *plan, size_t bytes, size_t need) {
  if (!plan) return fail(TCL_EINVAL, "attn: plan is NULL");
  if (misaligned(plan, 256)) return fail(TCL_EALIGN, "attn: plan must be 256-byte aligned");
  if (bytes < need) return fail(TCL_ENOSPC, "attn: plan holds %zu bytes, needs %zu", bytes, need);
  return TCL_OK;
}

template <int D>
void launch(const AttnArgs &a, int cap_items, hipStream_t s) {
  hipLaunchKernelGGL(attn_kernel<D>, dim3(unsigned(cap_items) * a.c.H), dim3(256), 0, s, a);
  // a row a wave, until that is eight workgroups a CU and more
  const int by_row = (a.Hq + 3) / 4, parts = a.T >= 2048 ? 1 : std::min(by_row, 4096 / a.T + 1);
  hipLaunchKernelGGL(attn_join_kernel<D>, dim3(a.T, parts), dim3(256), 0, s, a);
}

}  // namespace
}  // namespace tcl

using namespace tcl;

extern "C" int tcl_attn_plan_bytes(const tcl_attn_batch *b, const tcl_kv_cache *c,
                                   int32_t n_q_heads, size_t *bytes) {
  if (!bytes) return fail(TCL_EINVAL, "attn: bytes is NULL");
  KvArgs kv;
  int rc = check_batch(b, c, n_q_heads, &kv);
  if (rc) return rc;
  PlanArgs a{};
  Layout L;
  sizes(b, kv, n_q_heads, &a, &L);
  *bytes = L.total;
  return TCL_OK;
}

extern "C" int tcl_attn_workspace_bytes(const tcl_attn_batch *b, const tcl_kv_cache *c,
                                        int32_t n_q_heads, size_t *bytes) {
  if (!bytes) return fail(TCL_EINVAL, "attn: bytes is NULL");
  KvArgs kv;
  int rc = check_batch(b, c, n_q_heads, &kv);
  if (rc) return rc;
  PlanArgs a{};
  Layout L;
  sizes(b, kv, n_q_heads, &a, &L);
  *bytes = ws_total(a);
  return TCL_OK;
}

extern "C" int tcl_attn_plan(const tcl_attn_batch *b, const tcl_kv_cache *c, int32_t n_q_heads,
                             void *plan, size_t plan_bytes, void *stream) {
  KvArgs kv;
  int rc = check_batch(b, c, n_q_heads, &kv);
  if (rc) return rc;
  PlanArgs a{};
  Layout L;
  sizes(b, kv, n_q_heads, &a, &L);
  if ((rc = check_plan(plan, plan_bytes, L.total))) return rc;
  if (b->n_seqs == 0) {
    // no table is read
    a.S = a.G = 0;
  }
  char *p = static_cast<char *>(plan);
  a.seq_tok = b->seq_tok_ptr, a.group_seq = b->group_seq_ptr, a.prefix_len = b->prefix_len;
  a.prefix_pages = b->prefix_pages, a.own_len = b->own_len, a.own_pages = b->own_pages;
  a.hdr = reinterpret_cast<int32_t *>(p);
  a.tok = reinterpret_cast<TokRec *>(p + L.o_tok);
  a.tiles = reinterpret_cast<Tile *>(p + L.o_tiles);
  a.items = reinterpret_cast<Work *>(p + L.o_items);
  a.list = reinterpret_cast<int32_t *>(p + L.o_list);
  a.short_tok = reinterpret_cast<int32_t *>(p + L.o_stok);
  a.short_seq = reinterpret_cast<int32_t *>(p + L.o_sseq);
  a.utile = reinterpret_cast<int32_t *>(p + L.o_utile);
  const dim3 grid(1 + kPageGroups), block(kMapThreads);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.S <= kMapThreads && a.G <= kMapThreads)
    hipLaunchKernelGGL(attn_plan_kernel<true>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(attn_plan_kernel<false>, grid, block, 0, s, a);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

extern "C" int tcl_attn_status_async(const void *plan, int32_t *dev_status, void *stream) {
  if (!plan || !dev_status) return fail(TCL_EINVAL, "attn: plan and dev_status are required");
  if (misaligned(plan, 256) || misaligned(dev_status, 4))
    return fail(TCL_EALIGN, "attn: plan must be 256-byte, dev_status 4-byte aligned");
  hipLaunchKernelGGL(attn_status_kernel, dim3(1), dim3(64), 0, static_cast<hipStream_t>(stream),
                     static_cast<const int32_t *>(plan), dev_status);
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}

extern "C" int tcl_attn_apply(const tcl_attn_batch *b, const tcl_kv_cache *c, int32_t n_q_heads,
                              const void *plan, size_t plan_bytes, const void *q, int64_t ldq,
                              void *o, int64_t ldo, float *lse, float scale, void *ws,
                              size_t ws_bytes, void *stream) {
  AttnArgs a{};
  int rc = check_batch(b, c, n_q_heads, &a.c);
  if (rc) return rc;
  PlanArgs s{};
  Layout L;
  sizes(b, a.c, n_q_heads, &s, &L);
  if ((rc = check_plan(plan, plan_bytes, L.total))) return rc;
  const int64_t row = int64_t(n_q_heads) * c->head_dim;
  if (ldq < row || ldo < row) return fail(TCL_EINVAL, "attn: ldq or ldo below the heads of a row");
  if (ldq % 8 || ldo % 8) return fail(TCL_EALIGN, "attn: ldq and ldo must be multiples of 8");
  if (!std::isfinite(scale * 1.44269504088896341f))  // (scores are in powers of two)
    return fail(TCL_EINVAL, "attn: scale is not finite, or 2^127 and more");
  if (b->n_tokens == 0 || b->n_seqs == 0) return TCL_OK;
  if (!q || !o || !ws) return fail(TCL_EINVAL, "attn: q, o and ws are required");
  if (misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4) || misaligned(ws, 256))
    return fail(TCL_EALIGN, "attn: q and o must be 16-byte, lse 4-byte, ws 256-byte aligned");
  if (ws_bytes < ws_total(s))
    return fail(TCL_ENOSPC, "attn: workspace holds %zu bytes, needs %zu", ws_bytes, ws_total(s));
  const char *p = static_cast<const char *>(plan);
  a.q = static_cast<const uint16_t *>(q), a.o = static_cast<uint16_t *>(o), a.lse = lse;
  a.ldq = ldq, a.ldo = ldo;
  // (never zero: a hidden key's -infinity times zero would be a NaN; the
  // smallest number there is, so that no finite score shows it)
  a.scale2 = std::fmax(std::fabs(scale) * 1.44269504088896341f,
                       std::numeric_limits<float>::denorm_min());
  a.q_sign = scale < 0 ? 0x8000 : 0;
  a.S = b->n_seqs, a.G = b->n_groups, a.T = b->n_tokens, a.ldp = b->ld_prefix;
  a.ld_own = b->ld_own, a.Hq = n_q_heads;
  a.prefix_pages = b->prefix_pages, a.own_pages = b->own_pages;
  a.hdr = reinterpret_cast<const int32_t *>(p);
  a.tok = reinterpret_cast<const TokRec *>(p + L.o_tok);
  a.items = reinterpret_cast<const Work *>(p + L.o_items);
  a.list = reinterpret_cast<const int32_t *>(p + L.o_list);
  a.part_o = static_cast<float *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + ws_rows_bytes(s));
  hipStream_t st = static_cast<hipStream_t>(stream);
  logf("attn: tokens=%d requests=%d groups=%d heads=%d/%d dim=%d items<=%d", a.T, a.S, a.G, a.Hq,
       a.c.H, a.c.D, s.cap_items);
  switch (c->head_dim) {
    case 64: launch<64>(a, s.cap_items, st); break;
    case 128: launch<128>(a, s.cap_items, st); break;
    default: launch<256>(a, s.cap_items, st); break;
  }
  TCL_HIP(hipGetLastError());
  return TCL_OK;
}
