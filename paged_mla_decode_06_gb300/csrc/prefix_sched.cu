// prefix_sched.cu -- the work list and the merge of a batch that shares prefixes.
//
// The keys of a request are those of its group's prefix (whole blocks, the same in
// all its requests' tables) and its own behind them. The rows of all tokens of a
// group make the tiles of its prefix, the rows of a request those of its own
// keys; an item is a tile of 128 rows and a range of 128-key groups. The tiles
// are laid end to end, those of the prefixes first, each as long as its groups
// and, where workers run items one after another, kItemCost more for what an item
// costs besides; the sequence is cut at every multiple of W = cdiv(its length,
// workers), at least kMinShare. Cuts within kLeastEnd groups of a tile's ends are
// dropped, and those of tiles of less than kLeastCut. A worker's items are those with
// their middle in its share. (Kernels of one item a pair get the longest first instead, cut
// no nearer than W / 8 to an end and not in tiles of half a share, and the short ones
// fill what the others leave.) A row's pieces, of either kind, write base-2
// partials; rows of one piece in all write their output.
//
// A request takes part in its group's prefix when all its tokens see all of it
// (seq_len - qlen >= prefix); the others take all their keys as their own. So a call
// gives what mla_decode_fwd gives for any lengths, and only the tables are trusted to
// share their blocks. A prefix is shared where that saves more than it costs: the
// tiles that its participants would have of their own against those of the group's
// tokens, times its key groups; the cost is a partial more for each own tile,
// which takes about as long as kPieceCost key groups (its store 4 us of an SM
// pair, its part in the merge). With 128 heads a request fills its tiles
// alone, and the common keys come from L2 as they are.
//
// Bound by latency: 6 to 7 us a launch (57 to 66 requests), 12000 cycles of which with 512
// threads were 1700 of reading the lengths, 900 and 900 of participants and groups, 1900 of own
// keys, 2400 and 2600 of the tables, 1600 of the cuts; much of it waiting for code that
// runs once. One CTA, a thread to a tile's first piece and one to the piece behind each cut.
// Lengths and group records are kept in shared memory (of the first 1024 requests and
// 256 groups): it runs beside the decode's start, and before all of its work.
#include "common.cuh"
#include "internal.h"
#include "merge_row.cuh"

namespace mla {
namespace {

// Threads: few wait for one another sooner, many take more requests at once (57 requests of 3
// tokens: 64.8 us with 128, 65.9 with 512; 128 requests in 16 groups: 45.0 and 44.1).
constexpr int kMaxThreads = 512, kFewThreads = 128;
constexpr int kFewReqs = 96;
constexpr int kGroupKeys = 128;
constexpr int kTileRows = 128;
constexpr int kBins = 512;
constexpr int kCache = 256;       // groups and
constexpr int kCacheReqs = 1024;  // requests that are kept in shared memory
constexpr int kItemCost = 4;     // of a worker's item: its start and its output, in groups
constexpr int kMinShare = 4;     // groups: pieces of less cost more than they save
constexpr int kLeastCut = 6, kLeastEnd = 2;  // of a worker's tile: groups to be cut at all, and on either side of a cut

struct Shared {
  int red[kMaxThreads / 32];
  int hist[kBins];   // items by size
  int start[kBins];
  int4 groups[kCache];
  int pos[kCache];
  int req_pos[kCacheReqs];
  int req_item[kCacheReqs];
  int edge[kCache + 1];
  int4 reqs[kCacheReqs];
};

// Exclusive prefix of v over the block. (Out of line, as the loops are not unrolled: the
// kernel runs once a call, and mostly waits for its own code.)
template <int THREADS>
__device__ __noinline__ int block_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  __syncthreads();
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  // (every warp scans the warps' sums)
  const int mine = lane < THREADS / 32 ? red[lane] : 0;
  int all = mine;
#pragma unroll
  for (int o = 1; o < THREADS / 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += n;
  }
  *total = __shfl_sync(0xffffffffu, all, THREADS / 32 - 1);
  return __shfl_sync(0xffffffffu, all - mine, warp) + inc - v;
}

template <int THREADS>
__device__ __forceinline__ int2 block_scan2(int2 v, int* red, int2* total) {
  int2 r;
  int2 all;
  r.x = block_scan<THREADS>(v.x, red, &all.x);
  r.y = block_scan<THREADS>(v.y, red, &all.y);
  *total = all;
  return r;
}

// Last i in [0, n) with at(i) <= v (at does not decrease; 0 if none).
template <typename F>
__device__ __forceinline__ int last_at(int n, int v, F at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at(mid) <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int group_edge(const PrefixParams& p, int g) {  // first request of group g
  return p.group_indptr == nullptr ? (g == 0 ? 0 : p.num_reqs) : min(max(p.group_indptr[g], 0), p.num_reqs);
}
__device__ __forceinline__ int token_edge(const PrefixParams& p, int r) {  // first token of request r
  return p.qo_indptr == nullptr ? min(r, p.num_tokens) : min(max(p.qo_indptr[r], 0), p.num_tokens);
}
__device__ __forceinline__ int groups_of(int keys) { return keys > 0 ? keys / kGroupKeys + (keys % kGroupKeys != 0) : 0; }

// Where a tile may be cut: at the multiples of W in its part of the sequence.
struct Cutter {
  int W, cost;   // shares; length of an item besides its groups
  int least, d;  // groups of a tile that may be cut; of its ends that may not
  unsigned inv;  // (2^32 - 1) / W
  // v / W for 0 <= v < 2^31: the product is at most one too small. (A division is some
  // thirty instructions in a row, and code that the kernel runs once.)
  __device__ __forceinline__ int over(int v) const {
    const int q = static_cast<int>(__umulhi(static_cast<unsigned>(v), inv));
    return q + (v - q * W >= W ? 1 : 0);
  }
  // the first cut, as a multiple of W, of the tile of g groups at place a; and their number
  __device__ __forceinline__ int first(int a) const { return over(a + cost + d + W - 1); }
  __device__ __forceinline__ int count(int a, int g) const {
    return g < least ? 0 : max(over(a + cost + g - d) - first(a) + 1, 0);
  }
};
// Piece j of a tile with `cuts` cuts: groups [from, to).
struct Piece {
  int from, to;
};
__device__ __forceinline__ Piece piece_of(const Cutter& c, int a, int g, int cuts, int j) {
  const int z = c.first(a) * c.W - a - c.cost;
  return Piece{j == 0 ? 0 : z + (j - 1) * c.W, j == cuts ? g : z + j * c.W};
}

template <bool SORTED, int THREADS>
__global__ void __launch_bounds__(THREADS) prefix_schedule_kernel(const PrefixParams p) {
  __shared__ Shared s;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int tid = threadIdx.x;
  const int G = p.num_groups, R = p.num_reqs, H = p.num_heads;
  constexpr int cost = SORTED ? 0 : kItemCost;
  Cutter cut;
  cut.cost = cost;
  int4* const out_groups = reinterpret_cast<int4*>(p.groups);
  // {first request, shared keys, tiles of the participants, -}, then as in PrefixParams
  int4* const gr = G <= kCache ? s.groups : out_groups;
  int* const gp = G <= kCache ? s.pos : p.group_pos;  // places of the groups' first tiles
  int* const rp = R <= kCacheReqs ? s.req_pos : p.req_pos;  // and of the requests',
  int* const ri = R <= kCacheReqs ? s.req_item : p.req_pos + R;  // and the requests' first items
  auto edge = [&](int g) { return G <= kCache ? s.edge[g] : group_edge(p, g); };
  auto tiles_of = [&](int64_t tokens) { return static_cast<int>((tokens * H + kTileRows - 1) / kTileRows); };
  // {first token, tokens, length, group of the prefix that the request takes part in or -1}
  auto request = [&](int r) {
    if (r < kCacheReqs) return s.reqs[r];
    const int t0 = token_edge(p, r);
    return make_int4(t0, max(token_edge(p, r + 1) - t0, 0), p.seq_lens[r], p.req_group[r]);
  };
  auto first_token = [&](int r) { return r < min(R, kCacheReqs) ? s.reqs[r].x : token_edge(p, r); };
  auto group_tokens = [&](int g) {  // {first, number}
    const int t0 = first_token(edge(g));
    return make_int2(t0, max(first_token(edge(g + 1)) - t0, 0));
  };
  auto set_group = [&](int r, int g) {
    p.req_group[r] = g;
    if (r < kCacheReqs) s.reqs[r].w = g;
  };
#pragma unroll 1
  for (int r = tid; r < min(R, kCacheReqs); r += THREADS) {
    const int t0 = token_edge(p, r);
    s.reqs[r] = make_int4(t0, max(token_edge(p, r + 1) - t0, 0), p.seq_lens[r], -1);
  }
  if (SORTED)
    for (int b = tid; b < kBins; b += THREADS) s.hist[b] = 0;
  bool falls = false;
#pragma unroll 1
  for (int g = tid; g < G; g += THREADS) {
    const int first = group_edge(p, g), end = group_edge(p, g + 1);
    const int whole = min(max(p.prefix_lens[g], 0) / p.block_size, p.cols);
    falls |= first > end;
    if (G <= kCache) {
      s.edge[g] = first;
      s.edge[g + 1] = end;  // (the next thread's first)
    }
    gr[g] = make_int4(INT32_MAX, whole * p.block_size, 0, 0);
  }
  // (groups that overlap would have more tiles than the workspace has room for)
  const bool apart = __syncthreads_or(falls) == 0;
#pragma unroll 1
  for (int r = tid; r < R; r += THREADS) {
    const int4 q = request(r);
    int g = last_at(G, r, edge);
    const bool in = apart && r >= edge(g) && r < edge(g + 1);
    const int keys = gr[g].y;
    if (in && keys > 0 && q.y > 0 && q.z - q.y >= keys) {
      atomicMin(&gr[g].x, r);
      atomicAdd(&gr[g].z, min(tiles_of(q.y), p.tiles_max));
    } else {
      g = -1;
    }
    set_group(r, g);
  }
  __syncthreads();
  // prefix tiles and their places in the sequence
  int ptiles = 0, prefix_end = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < G; g0 += THREADS) {
    const int g = g0 + tid;
    int tiles = 0, keys = 0, tok0 = 0, first = 0;
    if (g < G) {
      const int2 tokens = group_tokens(g);
      tok0 = tokens.x;
      tiles = tiles_of(tokens.y);
      const int4 v = gr[g];
      first = v.x;
      const bool share = static_cast<int64_t>(v.z - tiles) * groups_of(v.y) >= static_cast<int64_t>(kPieceCost) * v.z;
      if (share && v.z > 0) keys = v.y;
      else tiles = 0;
    }
    const int length = tiles * (groups_of(keys) + cost);
    int2 sum = make_int2(tiles, length), at = make_int2(0, 0);
    if (G > 1) at = block_scan2<THREADS>(sum, s.red, &sum);
    const int t = ptiles + at.x, a = prefix_end + at.y;
    if (G > 1) {
      ptiles += sum.x;
      prefix_end += sum.y;
    }
    if (g < G) {
      const int4 v = make_int4(first, keys, tok0, t);
      gr[g] = v;
      out_groups[g] = v;
      gp[g] = a;
      if (G == 1) s.start[0] = tiles;
    }
  }
  __syncthreads();
  if (G == 1) {
    ptiles = s.start[0];
    prefix_end = ptiles * (groups_of(gr[0].y) + cost);
  }
  // own keys of request r
  struct Own {
    int4 q;
    int first, groups, tiles;
  };
  auto own_keys = [&](int r) {
    Own o;
    o.q = request(r);
    o.first = o.q.w >= 0 ? gr[o.q.w].y : 0;
    o.groups = groups_of(o.q.z - o.first);
    o.tiles = min(tiles_of(o.q.y), p.tiles_max);
    return o;
  };
  int total = prefix_end;
#pragma unroll 1
  for (int r0 = 0; r0 < R; r0 += THREADS) {
    const int r = r0 + tid;
    int length = 0;
    if (r < R) {
      const int g = request(r).w;
      if (g >= 0 && gr[g].y == 0) set_group(r, -1);
      const Own o = own_keys(r);
      length = o.tiles * (o.groups + cost);
    }
    int sum;
    const int a = total + block_scan<THREADS>(length, s.red, &sum);
    total += sum;
    if (r < R) rp[r] = a;
  }
  cut.W = max((total + p.workers - 1) / p.workers, kMinShare);
  cut.inv = 0xffffffffu / static_cast<unsigned>(cut.W);
  cut.least = SORTED ? cut.W / 2 + 1 : kLeastCut;
  cut.d = SORTED ? max(cut.W / 8, 1) : kLeastEnd;
  __syncthreads();
  const int W = cut.W;
  // A tile: its place, its groups, what its items say.
  struct Tile {
    int a, n, unit, tile, first, end;
    int4 second;
    int stride;  // rows of a piece's partial
  };
  auto prefix_tile = [&](int t) {
    const int g = last_at(G, t, [&](int i) { return gr[i].w; });
    const int4 v = gr[g];
    const int n = groups_of(v.y);
    const int tokens = group_tokens(g).y;
    return Tile{gp[g] + (t - v.w) * (n + cost), n, v.x, t - v.w, 0, v.y, make_int4(-1, v.z, tokens | kItemPrefix, 0), kTileRows};
  };
  auto own_tile = [&](const Own& o, int r, int t) {
    return Tile{rp[r] + t * (o.groups + cost), o.groups, r, t, o.first, max(o.q.z, o.first),
                make_int4(-1, o.q.x, o.q.y, o.q.z - o.q.y + 1), min(kTileRows, o.q.y * H - t * kTileRows)};
  };
  // Cut w of the sequence: the tile that place w W lies in, its entry in the tables and,
  // of an own tile, its first item; false where it is no tile's.
  struct At {
    Tile t;
    const int2* tab;
    int item;
  };
  auto at_cut = [&](int w, At& c) {
    const int at = w * W;
    if (at < prefix_end) {
      const int g = last_at(G, at, [&](int i) { return gp[i]; });
      const int i = min(gr[g].w + (at - gp[g]) / (groups_of(gr[g].y) + cost), ptiles - 1);
      c.t = prefix_tile(i);
      c.tab = reinterpret_cast<const int2*>(p.prefix_tab) + i;
      c.item = c.tab->x / kTileRows;
      return true;
    }
    const int r = last_at(R, at, [&](int i) { return rp[i]; });
    const Own o = own_keys(r);
    if (o.tiles == 0) return false;
    const int i = min((at - rp[r]) / (o.groups + cost), o.tiles - 1);
    c.t = own_tile(o, r, i);
    c.tab = reinterpret_cast<const int2*>(p.unit_tab) + static_cast<int64_t>(r) * p.tiles_max + i;
    if (!SORTED) {
      c.item = ri[r];
#pragma unroll 1
      for (int t = 0; t < i; ++t) {
        const Tile v = own_tile(o, r, t);
        c.item += cut.count(v.a, v.n) + 1;
      }
    }
    return true;
  };
  auto emit = [&](Tile t, int cuts, int j, int base, int at) {
    const Piece q = piece_of(cut, t.a, t.n, cuts, j);
    if (SORTED) at = atomicAdd(&s.start[kBins - 1 - min(q.to - q.from, kBins - 1)], 1);
    if (at >= p.max_items) return;
    int4* it = reinterpret_cast<int4*>(p.items) + 2 * static_cast<int64_t>(at);
    it[0] = make_int4(t.unit, t.tile, t.first + q.from * kGroupKeys, j == cuts ? t.end : t.first + q.to * kGroupKeys);
    t.second.x = base < 0 ? -1 : base + j * t.stride;
    it[1] = t.second;
  };
  const int all_cuts = (total - 1) / W;
  if constexpr (SORTED) {
    // the places of the items by their size: how many are larger
    auto count = [&](const Tile& t, int j) {
      const int cuts = cut.count(t.a, t.n);
      const Piece q = piece_of(cut, t.a, t.n, cuts, j);
      atomicAdd(&s.hist[kBins - 1 - min(q.to - q.from, kBins - 1)], 1);
    };
#pragma unroll 1
    for (int t = tid; t < ptiles; t += THREADS) count(prefix_tile(t), 0);
#pragma unroll 1
    for (int r = tid; r < R; r += THREADS) {
      const Own o = own_keys(r);
#pragma unroll 1
      for (int t = 0; t < o.tiles; ++t) count(own_tile(o, r, t), 0);
    }
#pragma unroll 1
    for (int w = tid + 1; w <= all_cuts; w += THREADS) {
      At c;
      if (!at_cut(w, c)) continue;
      const int j = w - cut.first(c.t.a) + 1;
      if (j >= 1 && j <= cut.count(c.t.a, c.t.n)) count(c.t, j);
    }
    __syncthreads();
    constexpr int kPer = kBins / THREADS;  // bins of a thread
    int mine = 0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) mine += s.hist[kPer * tid + b];
    int all;
    int at = block_scan<THREADS>(mine, s.red, &all);
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      s.start[kPer * tid + b] = at;
      at += s.hist[kPer * tid + b];
    }
    if (tid == 0) *p.n_items = min(all, p.max_items);
    __syncthreads();
  }
  // the tables, and each tile's first item
  int rows = 0, items = 0;  // of the partials, of the list
#pragma unroll 1
  for (int t0 = 0; t0 < ptiles; t0 += THREADS) {
    const int t = t0 + tid;
    Tile v{};
    int cuts = -1;
    if (t < ptiles) {
      v = prefix_tile(t);
      cuts = cut.count(v.a, v.n);
    }
    int sum;
    const int at = items + block_scan<THREADS>(cuts + 1, s.red, &sum);
    items += sum;
    rows += sum * kTileRows;
    if (t < ptiles) {
      reinterpret_cast<int2*>(p.prefix_tab)[t] = make_int2(at * kTileRows, cuts + 1);
      emit(v, cuts, 0, at * kTileRows, at);
    }
  }
#pragma unroll 1
  for (int r0 = 0; r0 < R; r0 += THREADS) {
    const int r = r0 + tid;
    Own o{};
    if (r < R) o = own_keys(r);
    const bool part = r < R && o.q.w >= 0;
    int2 mine = make_int2(0, 0);
#pragma unroll 1
    for (int t = 0; t < o.tiles; ++t) {
      const Tile v = own_tile(o, r, t);
      const int k = cut.count(v.a, v.n) + 1;
      mine.x += k;
      if (part || k > 1) mine.y += k * v.stride;
    }
    int2 sum;
    const int2 before = block_scan2<THREADS>(mine, s.red, &sum);
    int at = items + before.x, base = rows + before.y;
    items += sum.x;
    rows += sum.y;
    if (r < R) ri[r] = at;
#pragma unroll 1
    for (int t = 0; t < o.tiles; ++t) {
      const Tile v = own_tile(o, r, t);
      const int cuts = cut.count(v.a, v.n);
      const bool split = part || cuts > 0;
      reinterpret_cast<int2*>(p.unit_tab)[static_cast<int64_t>(r) * p.tiles_max + t] = make_int2(split ? base : -1, cuts + 1);
      emit(v, cuts, 0, split ? base : -1, at);
      at += cuts + 1;
      if (split) base += (cuts + 1) * v.stride;
    }
  }
  __syncthreads();
  // the items behind the cuts; and each worker's first item: of the piece that the start
  // of its share lies in, or the next where that one's middle is before it
  items = min(items, p.max_items);
#pragma unroll 1
  for (int w = tid + 1; w <= (SORTED ? all_cuts : max(all_cuts, p.workers)); w += THREADS) {
    At c;
    if (w > all_cuts || !at_cut(w, c)) {
      if (!SORTED && w <= p.workers) p.worker_first[w] = items;
      continue;
    }
    const int cuts = cut.count(c.t.a, c.t.n), j = w - cut.first(c.t.a) + 1;
    const bool here = j >= 1 && j <= cuts;
    if (here) emit(c.t, cuts, j, c.tab->x, c.item + j);
    if (!SORTED && w <= p.workers) {
      int at = c.item + (here ? j : j < 1 ? 0 : cuts);
      if (!here) {
        const Piece q = piece_of(cut, c.t.a, c.t.n, cuts, j < 1 ? 0 : cuts);
        const int begin = c.t.a + (q.from > 0 ? cost + q.from : 0);
        at += (begin + c.t.a + cost + q.to) / 2 < w * W ? 1 : 0;
      }
      p.worker_first[w] = min(at, items);
    }
  }
  if (!SORTED && tid == 0) {
    p.worker_first[0] = 0;
    *p.n_items = items;
  }
}

// One warp a row, or (SLICED, few rows) four, each of 128 of its columns: the
// row's pieces over the prefix, then those over its own keys, in their order,
// weighted as mla_merge_segments does. The tables are read while the decode may still
// run; the first pieces' outputs are loaded with their weights, not after them, and two
// at a time (eight of a slice), so that 32 warps fit an SM (four at a time and behind the
// weights: 14 us against 8 for 8192 rows of two pieces). Rows without pieces leave at
// once, but in the first block, by leave_merge.
constexpr int kMergeWarps = 4;

template <bool SLICED>
__global__ void __launch_bounds__(kMergeWarps * 32, 8) prefix_merge_kernel(const PrefixParams p) {
  constexpr int kVec = SLICED ? 1 : 4;    // float4 of a lane
  constexpr int kBatch = SLICED ? 8 : 2;  // pieces loaded at once
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = SLICED ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp;
  const int first = SLICED ? 32 * warp + lane : lane;  // float4 of the row
  if (row >= static_cast<int64_t>(p.num_tokens) * p.num_heads) return leave_merge();
  const int H = p.num_heads;
  const int t = static_cast<int>(row / H), h = static_cast<int>(row - static_cast<int64_t>(t) * H);
  // (the tables come from the schedule, which completed before the decode began)
  int r = t, tok0 = t;
  if (p.qo_indptr != nullptr) {
    if (t < p.qo_indptr[0] || t >= p.qo_indptr[p.num_reqs]) return leave_merge();  // padding of the batch
    r = last_at(p.num_reqs, t, [&](int i) { return p.qo_indptr[i]; });
    tok0 = p.qo_indptr[r];
  }
  const int own_row = (t - tok0) * H + h;
  if (own_row / kTileRows >= p.tiles_max) return leave_merge();
  const int g = p.req_group[r];
  const int2 own = reinterpret_cast<const int2*>(p.unit_tab)[static_cast<int64_t>(r) * p.tiles_max + own_row / kTileRows];
  if (own.x < 0) return leave_merge();  // one piece in all: written by the decode
  const int end = token_edge(p, r + 1);
  const int own_stride = min(kTileRows, (end - tok0) * H - own_row / kTileRows * kTileRows);
  int2 pre = make_int2(0, 0);
  int pre_row = 0;
  if (g >= 0) {
    const int4 gi = reinterpret_cast<const int4*>(p.groups)[g];
    pre_row = (t - gi.z) * H + h;
    pre = reinterpret_cast<const int2*>(p.prefix_tab)[gi.w + pre_row / kTileRows];
  }
  const int live = pre.y + own.y;
  auto at = [&](int s) {  // row of piece s among the partials
    return s < pre.y ? static_cast<int64_t>(pre.x) + s * kTileRows + pre_row % kTileRows
                     : static_cast<int64_t>(own.x) + static_cast<int64_t>(s - pre.y) * own_stride + own_row % kTileRows;
  };
  const float sink2 = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float4 x[kBatch][kVec];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + u >= live) continue;
      const float4* src = reinterpret_cast<const float4*>(p.segm_out + at(s0 + u) * kRank);
#pragma unroll
      for (int v = 0; v < kVec; ++v) x[u][v] = __ldcg(src + v * 32 + first);
    }
  };
  float M = sink2;
  float m0 = -INFINITY, l0 = 0.f;  // of piece `lane`
  if (lane < live) {
    l0 = __ldcg(p.segm_expsum + at(lane));
    m0 = __ldcg(p.segm_max + at(lane));
  }
  load(0);
  if (l0 > 0.f) M = fmaxf(M, m0);
  for (int s = lane + 32; s < live; s += 32) {
    const float m = __ldcg(p.segm_max + at(s));
    if (__ldcg(p.segm_expsum + at(s)) > 0.f) M = fmaxf(M, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * kRank);
  // (a sink that is NaN leaves M to the others and makes the sum NaN)
  if (M == -INFINITY && !(sink2 != sink2)) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) out[v * 32 + first] = make_uint2(0u, 0u);
    if (first == 0) p.lse[row] = -INFINITY;
    return;
  }
  float acc[kVec][4] = {};
  float sum = sink2 == -INFINITY ? 0.f : exp2f(sink2 - M);
  for (int s0 = 0; s0 < live; s0 += 32) {
    if (s0 > 0) {
      const int s = s0 + lane;
      l0 = s < live ? __ldcg(p.segm_expsum + at(s)) : 0.f;
      m0 = s < live ? __ldcg(p.segm_max + at(s)) : -INFINITY;
    }
    const float mine = l0 > 0.f ? l0 * exp2f(m0 - M) : 0.f;
#pragma unroll 1
    for (int k = 0; k < 32 && s0 + k < live; k += kBatch) {
      if (s0 + k > 0) load(s0 + k);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float w = __shfl_sync(0xffffffffu, mine, k + u);
        if (s0 + k + u >= live || w == 0.f) continue;  // (a piece without mass may hold anything)
        sum += w;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          acc[v][0] += w * x[u][v].x;
          acc[v][1] += w * x[u][v].y;
          acc[v][2] += w * x[u][v].z;
          acc[v][3] += w * x[u][v].w;
        }
      }
    }
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[v][0] * inv, acc[v][1] * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[v][2] * inv, acc[v][3] * inv);
    out[v * 32 + first] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (first == 0) p.lse[row] = kLn2 * (M + log2f(sum));
}

}  // namespace

cudaError_t launch_prefix_schedule(const PrefixParams& p, cudaStream_t stream) {
  const bool few = p.num_reqs <= kFewReqs;
  if (p.worker_first == nullptr) {
    if (few) prefix_schedule_kernel<true, kFewThreads><<<1, kFewThreads, 0, stream>>>(p);
    else prefix_schedule_kernel<true, kMaxThreads><<<1, kMaxThreads, 0, stream>>>(p);
  } else {
    if (few) prefix_schedule_kernel<false, kFewThreads><<<1, kFewThreads, 0, stream>>>(p);
    else prefix_schedule_kernel<false, kMaxThreads><<<1, kMaxThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_prefix_merge(const PrefixParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.num_heads;
  if (rows == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  const bool sliced = rows <= 2048;
  cfg.gridDim = dim3(static_cast<unsigned>(sliced ? rows : (rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return sliced ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<true>, p)
                : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<false>, p);
}

}  // namespace mla
