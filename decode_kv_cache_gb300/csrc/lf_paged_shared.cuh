// Before a shared prefix: which rows and keys a block takes.
#pragma once

#include "lf_paged.cuh"
#include "lf_ranges.h"

namespace lf {

// A segment's rows and keys: the group's sequences b0 .. b0 + members - 1, KV head g, key tiles first .. last - 1
// of the pages that sequence `leader` lists.
struct Segment {
  int b0, members, g, leader, first, last;
  int prefix;                // the group's
  int p_lo, p_hi;            // least and largest last position that a row sees of it
  int64_t row;               // of part_o
};

// What a group asks for: `pieces` pieces of `tiles` key tiles, of each KV head.  Its prefix ends where its members' do: what
// prefix_lens holds behind their lengths, or in padded rows, costs nothing (32 sequences behind 8192 and 32 empty groups whose
// prefixes of 60000 are left from another step: 35 us, with those tiles planned for 847).
struct Family {
  int start, members, prefix, tiles, pieces;
  bool right;
};

__device__ __forceinline__ Family family_from(const PagedSharedArgs& a, int start, int end, int prefix, int keys) {
  Family f;
  f.start = start;
  f.right = start >= 0 && end >= start && end <= a.pool.batch;
  f.members = f.right ? end - start : 0;
  f.prefix = f.tiles = f.pieces = 0;
  if (f.members > 0) {
    f.prefix = prefix;
    f.tiles = (prefix + keys - 1) / keys;
    const int each = a.rows / a.group;
    f.pieces = (f.members + each - 1) / each;
  }
  return f;
}

// The groups of a call, kept in shared memory where there are up to kN: where they start, the prefix of their first sequence,
// the most that a member sees of its own.  Of more groups a launch ahead has written what they see to a.seen.
template <int kN>
struct FamilyTable {
  int start[kN + 1], lead[kN], most[kN];

  // For the whole block together.
  template <int kThreads>
  __device__ __forceinline__ void fill(const PagedSharedArgs& a) {
    const int tid = threadIdx.x, n = a.groups, batch = a.pool.batch;
    if (n > kN) return;
    const int64_t room = (int64_t)a.pool.max_pages * a.pool.page_size;
    // (on their way together with the starts)
    const int own_prefix = tid < batch ? a.prefix_lens[tid] : 0, own_len = tid < batch ? a.pool.lens[tid] : 0;
    // (no loop of the plan is unrolled: code that runs once costs what it takes to fetch)
#pragma unroll 1
    for (int i = tid; i <= n; i += kThreads) {
      start[i] = a.group_start[i];
      if (i < n) lead[i] = most[i] = 0;
    }
    __syncthreads();
    const int to = min(start[n], batch);
#pragma unroll 1
    for (int b = min(max(start[0], 0), batch) + tid; b < to; b += kThreads) {
      int lo = 0, hi = n;   // the last group that starts at or before b
#pragma unroll 1
      while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= b) lo = mid;
        else hi = mid;
      }
      const int first = start[lo], end = start[lo + 1];
      if (first < 0 || b < first || b >= end || end > batch) continue;   // of no group
      const int prefix = b == tid ? own_prefix : a.prefix_lens[b], len = b == tid ? own_len : a.pool.lens[b];
      if (b == first) lead[lo] = (int)min((int64_t)max(prefix, 0), room);
      const int mine = shared_len(prefix, (int)min((int64_t)max(len, 0), room), a.fresh != 0);
      if (mine > 0) atomicMax(&most[lo], mine);
    }
    __syncthreads();
  }

  __device__ __forceinline__ Family at(const PagedSharedArgs& a, int i, int keys) const {
    if (a.groups > kN) return family_from(a, a.group_start[i], a.group_start[i + 1], a.seen[i], keys);
    return family_from(a, start[i], start[i + 1], min(lead[i], most[i]), keys);
  }
};

// The last position that sequence b of a segment sees of its group's prefix, -1: none.
__device__ __forceinline__ int last_seen(const PagedSharedArgs& a, int prefix, int b) {
  return min(shared_len(a.prefix_lens[b], paged_len(a.pool, b), a.fresh != 0), prefix) - 1;
}

// Tiles of a segment.  A block costs its tiles and, for its start and its rows' way out, about as much as
// kSegmentStart of them; `units` units of `tiles` tiles in all, the longest of `longest`, are cut so that r rounds of `slots` blocks
// take them, with the r, up to `rounds`, that costs least; `least` tiles or more.
constexpr int kSegmentStart = 4;

__device__ __forceinline__ int segment_tiles(int slots, int rounds, int least, int64_t units, int64_t tiles, int longest) {
  int best = longest;
  int64_t cost = INT64_MAX;
  const int64_t r0 = units / slots + 1;
  for (int64_t r = r0; r < r0 + 2 && r <= rounds; ++r) {
    const int64_t room = r * slots - units;
    const int64_t c = min((int64_t)longest, max((int64_t)least, (tiles + room - 1) / room));
    const int64_t used = c == longest ? (units + slots - 1) / slots : r;
    if (used * (c + kSegmentStart) < cost) {
      cost = used * (c + kSegmentStart);
      best = (int)c;
    }
  }
  return best;
}

// Segment number blockIdx.x, where each block takes one; false: there is none.  The segments of all groups are numbered group
// by group, piece by piece, head by head.  Every block goes through the groups itself: a launch that did so for all would be
// one more to wait for.  Block 0 tells the join.  For the whole block together.
template <int kThreads, int kN>
__device__ __forceinline__ bool take_segment(const PagedSharedArgs& a, int keys, FamilyTable<kN>& table, Segment* out) {
  constexpr int kW = kThreads / 32;
  __shared__ int64_t s_all[2][kW], s_sum[2][kW];
  __shared__ int s_max[kW], s_lo[kW], s_hi[kW];
  __shared__ Segment s_seg;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.pool.kv_heads, id = blockIdx.x;
  table.template fill<kThreads>(a);
  const int per = (a.groups + kThreads - 1) / kThreads;
  const int from = min(tid * per, a.groups), to = min(from + per, a.groups);   // this thread's groups

  // Units, tiles and the longest unit's tiles of all groups.
  int64_t units = 0, tiles = 0;
  int longest = 0;
#pragma unroll 1
  for (int i = from; i < to; ++i) {
    const Family f = table.at(a, i, keys);
    if (f.tiles > 0) {
      units += (int64_t)f.pieces * H;
      tiles += (int64_t)f.pieces * H * f.tiles;
      longest = max(longest, f.tiles);
    }
    if (!f.right && blockIdx.x == 0 && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, o);
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) {
    s_all[0][warp] = units;
    s_all[1][warp] = tiles;
    s_max[warp] = longest;
  }
  if (tid == 0) s_seg.members = 0;
  __syncthreads();
  units = tiles = 0;
  longest = 0;
#pragma unroll 1
  for (int w = 0; w < kW; ++w) {
    units += s_all[0][w];
    tiles += s_all[1][w];
    longest = max(longest, s_max[w]);
  }
  const int chunk = units > 0 ? segment_tiles(a.slots, a.rounds, a.least, units, tiles, longest) : 1;

  // Segments and their rows of part_o in front of each thread's groups.
  auto cuts = [&](const Family& f) { return (f.tiles + chunk - 1) / chunk; };
  int64_t own_seg = 0, own_row = 0;
#pragma unroll 1
  for (int i = from; i < to; ++i) {
    const Family f = table.at(a, i, keys);
    own_seg += (int64_t)f.pieces * H * cuts(f);
    own_row += (int64_t)f.members * a.q_heads * cuts(f);
  }
  int64_t seg = own_seg, row = own_row;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, seg, o), y = __shfl_up_sync(0xffffffffu, row, o);
    if (lane >= o) {
      seg += x;
      row += y;
    }
  }
  if (lane == 31) {
    s_sum[0][warp] = seg;
    s_sum[1][warp] = row;
  }
  __syncthreads();
  seg -= own_seg;
  row -= own_row;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) {
    seg += s_sum[0][w];
    row += s_sum[1][w];
  }
  if (id == 0 || (id >= seg && id < seg + own_seg)) {
#pragma unroll 1
    for (int i = from; i < to; ++i) {
      const Family f = table.at(a, i, keys);
      const int n = cuts(f);
      const int64_t mine = (int64_t)f.pieces * H * n;
      if (id >= seg && id < seg + mine) {
        const int64_t unit = (id - seg) / n;
        const int j = (int)(id - seg - unit * n), piece = (int)(unit / H), each = a.rows / a.group;
        Segment s;
        s.g = (int)(unit - (int64_t)piece * H);
        s.b0 = f.start + piece * each;
        s.members = min(each, f.members - piece * each);
        s.leader = f.start;
        s.first = (int)((int64_t)f.tiles * j / n);
        s.last = (int)((int64_t)f.tiles * (j + 1) / n);
        s.prefix = f.prefix;
        s.p_lo = s.p_hi = -1;
        s.row = row + (int64_t)piece * each * a.q_heads * n + ((int64_t)s.g * n + j) * s.members * a.group;
        s_seg = s;
      }
      if (id == 0) {
        a.segments[i] = n;
        a.first_row[i] = row;
      }
      seg += mine;
      row += (int64_t)f.members * a.q_heads * n;
    }
  }
  if (id == 0 && tid == 0) a.ranges[0] = 0;
  __syncthreads();
  Segment s = s_seg;
  // What its sequences see of the prefix.
  int lo = INT_MAX, hi = -1;
#pragma unroll 1
  for (int i = tid; i < s.members; i += kThreads) {
    const int p = last_seen(a, s.prefix, s.b0 + i);
    lo = min(lo, p);
    hi = max(hi, p);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    s_lo[warp] = lo;
    s_hi[warp] = hi;
  }
  __syncthreads();
  // (Starts that decrease may ask for more than there is room for.)
  if (s.members == 0 || s.row + (int64_t)s.members * a.group > a.part_rows) return false;
  s.p_lo = s_lo[0];
  s.p_hi = s_hi[0];
#pragma unroll 1
  for (int w = 1; w < kW; ++w) {
    s.p_lo = min(s.p_lo, s_lo[w]);
    s.p_hi = max(s.p_hi, s_hi[w]);
  }
  s.last = max(s.first, min(s.last, s.p_hi < 0 ? 0 : s.p_hi / keys + 1));
  *out = s;
  return true;
}

// ---- ranges: prefixes and the rest in one launch ------------------------------------------
//
// The units of all groups (group by group, piece by piece, head by head) lie one behind another, each `start` places, for what
// a CTA spends on a unit besides its tiles, and then a place for each of its tiles.  The first `ctas` CTAs take equal ranges of the
// list, the others the rest of the sequences.  Numbers are below 2^31 (the entry point sees to it).

// What a prefix's tile costs, for one query tile and for two, and a unit's start, in tiles of the rest.  Beside
// CTAs that take the rest, with memory as busy as it gets, a tile of theirs took 1.1 to 1.6 us, one of a prefix 1.5 to 1.9 and
// 1.8 to 2.5, and a segment 8 to 10 us besides: heads of 128.  Heads of 64 take the same numbers; of 0.75, 1.3 and 1.6 times these
// none is better throughout (64 sequences, 8 heads a group, behind 8192: 43, 45 and 55 us, with these 42; 256 of 4 heads a group
// behind 16384: 101, 86 and 85, 94; 32 behind 60000: 62, 60 and 58, 59).
constexpr float kOneTile = 1.35f, kTwoTiles = 1.8f;
constexpr int kUnitStart = 6;

template <int kThreads>
struct RangeList {
  unsigned places, start;      // in all, in front of a unit's tiles
  int ctas;                    // that take prefixes

  // For the whole block together, with the table filled.  `rest`: this thread's share of the rest, in key tiles of a head; `keep`: room for what each
  // group's members see, where there are few groups.
  template <int kN>
  __device__ __forceinline__ void plan(const PagedSharedArgs& a, int keys, float rest, FamilyTable<kN>& table, int32_t* keep) {
    constexpr int kW = kThreads / 32;
    __shared__ unsigned s_units[kW], s_tiles[kW], s_members[kW];
    __shared__ float s_rest[kW], s_mine[kW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.groups + kThreads - 1) / kThreads;
    const int from = min(tid * per, a.groups), to = min(from + per, a.groups);   // this thread's groups
    unsigned own_units = 0, own_tiles = 0, members = 0;
    float mine = 0.f;
#pragma unroll 1
    for (int i = from; i < to; ++i) {
      const Family f = table.at(a, i, keys);
      if (a.groups <= kN) keep[i] = f.prefix;
      members += f.members;
      const unsigned u = f.tiles > 0 ? f.pieces * a.pool.kv_heads : 0;
      own_units += u;
      own_tiles += u * f.tiles;
      mine += (float)u * ((f.members * a.group > 128 ? kTwoTiles : kOneTile) * (float)f.tiles + (float)kUnitStart);
      if (!f.right && blockIdx.x == 0 && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
    }
    unsigned u = own_units, t = own_tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, u, o), y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) {
        u += x;
        t += y;
      }
      rest += __shfl_xor_sync(0xffffffffu, rest, o);
    }
    members = __reduce_add_sync(0xffffffffu, members);
    mine = warp_sum(mine);
    if (lane == 31) {
      s_units[warp] = u;
      s_tiles[warp] = t;
      s_members[warp] = members;
      s_rest[warp] = rest;
      s_mine[warp] = mine;
    }
    fence_proxy_async_smem();   // (copies come in where the table was)
    __syncthreads();
    // Lane w of every warp has warp w's sums.
    const bool in = lane < kW;
    const unsigned wu = in ? s_units[lane] : 0, wt = in ? s_tiles[lane] : 0;
    unsigned units = __reduce_add_sync(0xffffffffu, wu);
    const unsigned tiles = __reduce_add_sync(0xffffffffu, wt);
    const unsigned before_units = u - own_units + __reduce_add_sync(0xffffffffu, lane < warp ? wu : 0);
    const unsigned before_tiles = t - own_tiles + __reduce_add_sync(0xffffffffu, lane < warp ? wt : 0);
    members = __reduce_add_sync(0xffffffffu, in ? s_members[lane] : 0);
    rest = warp_sum(in ? s_rest[lane] : 0.f);
    mine = warp_sum(in ? s_mine[lane] : 0.f);
    // Starts that decrease: groups overlap, and their units may be more than there is room for.
    const bool none = members > (unsigned)a.pool.batch;
    if (none) units = 0;
    // As many CTAs for the prefixes as they are of the work; whole numbers of CTAs for each unit, or of a few units for each CTA.
    const int n = gridDim.x;
    ctas = 0;
    if (units > 0) {
      const float others = rest * (float)a.pool.kv_heads;
      ctas = max(1, min(n - 1, __float2int_rn((float)n * mine / (mine + others))));
      // With a whole number of CTAs for each unit none has the end of one and the start of the next.
      const int u = min(units, (unsigned)n), near = (ctas + u / 2) / u * u;
      if (near > 0 && near < n &&
          fmaxf(mine / (float)near, others / (float)(n - near)) <=
              fmaxf(mine / (float)ctas + (float)kUnitStart, others / (float)(n - ctas)))
        ctas = near;
      ctas = min(ctas, (int)min(tiles, (unsigned)n));
    }
    start = ctas > 0 && (unsigned)ctas % max(units, 1u) != 0 ? kUnitStart : 0;
    places = tiles + start * units;
    if (blockIdx.x == 0) {   // for the join
      unsigned at = before_tiles + start * before_units;
#pragma unroll 1
      for (int i = from; i < to; ++i) {
        const Family f = table.at(a, i, keys);
        a.segments[i] = none ? 0 : f.tiles;
        a.first_row[i] = at;
        at += f.pieces * a.pool.kv_heads * (f.tiles > 0 ? f.tiles + start : 0);
      }
      if (tid == 0) {
        a.ranges[0] = ctas;
        a.ranges[1] = (int)places;
        a.ranges[2] = (int)start;
      }
      __syncthreads();   // the table has been read
    }
  }
};

// What the range that starts at place x and ends at `end` has of the unit at x: a segment, and in `next` where the unit ends.
// members = 0: the range ends within the unit's start.  For one warp together; it goes through the groups again (`seen`: what
// each one's members see), 32 at a time, so that no thread holds what it knew of them.
__device__ __forceinline__ void find_segment(const PagedSharedArgs& a, int keys, const int32_t* seen, unsigned start, unsigned x,
                                             unsigned end, int lane, Segment* s, unsigned* next) {
  unsigned before = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < a.groups; i0 += 32) {
    Family f;
    f.tiles = f.pieces = 0;
    if (i0 + lane < a.groups) f = family_from(a, a.group_start[i0 + lane], a.group_start[i0 + lane + 1], seen[i0 + lane], keys);
    const unsigned size = f.tiles + start, all = f.tiles > 0 ? f.pieces * a.pool.kv_heads * size : 0;
    unsigned at = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    at += before;   // behind this lane's group
    const bool mine = x < at && x >= at - all;
    if (mine) {
      at -= all;
      const unsigned unit = (x - at) / size, piece = unit / a.pool.kv_heads;
      const int each = a.rows / a.group;
      const unsigned t0 = at + unit * size + start, t1 = t0 + f.tiles;   // the unit's tiles
      s->g = unit - piece * a.pool.kv_heads;
      s->b0 = f.start + piece * each;
      s->leader = f.start;
      s->prefix = f.prefix;
      s->first = max(x, t0) - t0;
      s->last = min(end, t1) - t0;
      s->members = end > t0 ? min(each, f.members - (int)piece * each) : 0;
      s->row = (int64_t)blockIdx.x * a.slot_rows + (int64_t)s->b0 * a.q_heads + (int64_t)s->g * s->members * a.group;
      *next = t1;
    }
    if (__any_sync(0xffffffffu, mine)) break;
    before = __shfl_sync(0xffffffffu, at, 31);
  }
  __syncwarp();
}

// What a segment's rows see, by one warp.
__device__ __forceinline__ void see_segment(const PagedSharedArgs& a, int keys, Segment& s, int lane) {
  int lo = INT_MAX, hi = -1;
  for (int i = lane; i < s.members; i += 32) {
    const int p = last_seen(a, s.prefix, s.b0 + i);
    lo = min(lo, p);
    hi = max(hi, p);
  }
  s.p_lo = __reduce_min_sync(0xffffffffu, lo);
  s.p_hi = __reduce_max_sync(0xffffffffu, hi);
  s.last = max(s.first, min(s.last, s.p_hi < 0 ? 0 : s.p_hi / keys + 1));
}

// Byte offset in the pools of the prefix's position `pos`, -1: nothing to read.
__device__ __forceinline__ int64_t shared_offset(const PagedSharedArgs& a, const Segment& s, int pos) {
  if (pos > s.p_hi) return -1;
  int pi, slot;
  paged_split(a.pool, pos, &pi, &slot);
  const int page = a.pool.table[(int64_t)s.leader * a.pool.max_pages + pi];
  if (page >= 0 && page < a.pool.num_pages)
    return page * a.pool.page_stride + slot * a.pool.token_stride + s.g * a.pool.head_stride;
  if (a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
  return -1;
}

// Row r of a segment as a row of q.
__device__ __forceinline__ int64_t shared_row(const PagedSharedArgs& a, const Segment& s, int r) {
  return (int64_t)(s.b0 + r / a.group) * a.q_heads + s.g * a.group + r % a.group;
}

// Row r's share by the definition, a warp at a time, where values that are not finite lie where some row
// does not look (0 * NaN is NaN).
template <typename T, int D>
__device__ __forceinline__ void shared_row_by_hand(const PagedSharedArgs& a, const Segment& s, int keys, int r, int limit,
                                                   int lane) {
  constexpr int E = D >= 32 ? D / 32 : 1;
  const bool mine = lane * E < D;   // lanes past a short row take nothing
  const T* q = reinterpret_cast<const T*>(a.q) + shared_row(a, s, r) * D + lane * E;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = mine ? to_f32(q[e]) : 0.f;
    acc[e] = 0.f;
  }
  float m = kNegInf, l = 0.f;
  const int64_t end = min((int64_t)s.last * keys, (int64_t)limit + 1);
  for (int64_t key = (int64_t)s.first * keys; key < end; ++key) {
    const int64_t off = shared_offset(a, s, (int)key);
    if (off < 0) continue;
    const T* k = reinterpret_cast<const T*>(a.pool.k + off) + lane * E;
    const T* v = reinterpret_cast<const T*>(a.pool.v + off) + lane * E;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (mine) x = fmaf(qv[e], to_f32(k[e]), x);
    x = warp_sum(x);
    const float mn = fmaxf(m, x * a.scale_log2), mu = mn == kNegInf ? 0.f : mn;
    const float f = ex2(m - mu), w = ex2(fmaf(x, a.scale_log2, -mu));
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (mine) acc[e] = acc[e] * f + w * to_f32(v[e]);
  }
  float* o = a.part_o + (s.row + r) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (mine) o[e] = acc[e];
  if (lane == 0) {
    a.part_ml[2 * (s.row + r)] = m;
    a.part_ml[2 * (s.row + r) + 1] = l;
  }
}

}  // namespace lf
