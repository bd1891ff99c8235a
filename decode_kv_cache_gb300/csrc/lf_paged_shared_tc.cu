// Attention of one new token per sequence behind shared prefixes, bf16 caches, head_dim 64 and 128: the prefixes on the
// tensor cores (tcgen05), as lf_paged_prompt_tc.cu does a prompt's rows, and the rest by lf_paged_decode.cu's walk, side by
// side in one launch; the formula and the join are lf_paged_shared.cu's.
//
// Work.  One CTA per SM.  Some take segments of the prefixes, the others ranges of the rest, as many of
// each as there are key tiles (each CTA works that out from the lengths): one kind behind the other would wait for the first's last
// tiles and the second's first ones.  A prefix CTA takes up to 256 rows of one KV head, (sequence, head of the group)
// pairs with the head inner, as one or two tiles of 128, and a segment of the key tiles of their prefix: every key and value that it
// loads serves all of its group's sequences.  Its rows' shares (fp32, with their maximum and sum) go to the workspace.
//
// A prefix CTA's roles are the prompt kernel's: a loader that gathers K and V by page with TMA, a warp that issues S = Q K^T and
// O += P V for the query tiles in turn, two groups of softmax warps with a thread per row, and a scrubber for the tiles
// that some row does not see all of (prefixes of other lengths, or the last tile).
//
// The rest's walk has twelve warps of two stages here, where lf_paged_decode.cu's kernel has eight of three: fewer SMs take it, and
// more warps hide more of each other's steps (256 sequences in 16 groups: the walk 94 us, 85).  Groups of eight heads take ten:
// twelve do not fit beside each other in shared memory with heads of 128, and with heads of 64 they are no faster (64 sequences
// behind 8192: 43 us, ten 42; 200 of up to 3000 behind 2000: 156, 147).
//
// Bound by HBM while a KV head has fewer than about 500 rows, by the key tiles' way in and the products above, and for short
// calls by the steps before the first tile: 3 us until every CTA knows its part, 7 to 10 until a prefix's first products, 4 for its rows'
// way out, and the join.  Measured with the join, bf16, 32 / 8 heads of 128, other inputs every time, against the bytes
// at a plain copy's rate: 64 sequences of 100 to 1000 tokens behind 8192, 50 us, 25; 32 of 50 to 500 behind 60000, 67 us, 41; 256 in 16
// groups behind 500 to 4000, 110 us, 76; 256 of 64 to 512 behind 16384, 110 us, 52 (36 by its products).  lf_paged_decode, which reads
// each prefix for every sequence and most of it from L2, takes 261, 855, 296 and 1889 us.  Heads of 64: 38, 49, 94 and 96 us.  Two query tiles take 1.7 us a key tile where four CTAs read it, as the prompt
// kernel does on such rows; 1.45 where sixteen do.  Not taken: the next tiles asked for into L2 ahead of their copies (64 behind 8192
// 60 us instead of 52).
#include <type_traits>

#include "lf_paged_decode.cuh"
#include "lf_paged_shared.cuh"
#include "lf_paged_tc.cuh"
#include "longflow.h"

namespace lf {

namespace {

struct SharedTcArgs {
  CUtensorMap q, k, v;
  PagedSharedArgs a;
  PagedDecodeArgs rest;
  int box_rows;      // tokens of one TMA box: min(page_size, 128)
  int group_shift;
};

// Shared memory of a prefix CTA: the prompt kernel's, with the room of its output rows for a fifth stage of heads of 128.
template <int D>
struct SharedPlanTc {
  static constexpr int kTileBytes = TcPlan<D>::kTileBytes;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kOffQ = 1024;
  static constexpr int kOffRing = kOffQ + 2 * kTileBytes;
  static constexpr int kSmem = kOffRing + kStages * kTileBytes + 1024;   // + alignment slack
};

template <int D, int G>
using Walk = MmaWalk<D, G, G == 8 ? 10 : 12, 2>;

constexpr int kKept = 56;   // groups whose numbers a CTA keeps in shared memory, from byte 544 to 768

__device__ __forceinline__ void mbar_inval(uint64_t* bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// `bytes` bytes of shared memory to global memory, as a group of copies of this thread's; 16-byte aligned.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
// This thread's copies have been read, or are done.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int D, int G>
__global__ void __launch_bounds__(kThreadsTc, 1) paged_shared_tc_kernel(const __grid_constant__ SharedTcArgs ta) {
  using P = SharedPlanTc<D>;
  using C = Walk<D, G>;
  constexpr int S = P::kStages;
  const PagedSharedArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform for the compiler too
  const int gs = ta.group_shift;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  if (warp == kLoadWarp && lane < 3) tma_prefetch_desc(lane == 0 ? &ta.q : lane == 1 ? &ta.k : &ta.v);
  // Everything below reads what earlier launches of the stream wrote.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint64_t* full = reinterpret_cast<uint64_t*>(smem);   // [S] a tile is ready for the MMAs
  uint64_t* raw = full + S;                             // [S] V landed, to be scrubbed
  uint64_t* qfull = raw + S;
  uint64_t* sfull = qfull + 1;                          // [t][j & 3] S_t of key tile j ready, and
                                                        // every MMA before it done
  uint64_t* pfull = sfull + 8;                          // [2][2] half of P_t written (O_t scaled)
  uint64_t* ofull = pfull + 4;                          // [2] O_t final
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + 528);   // [0] a wait expired, [1] by hand
  Segment* s_seg = reinterpret_cast<Segment*>(smem + 768);
  unsigned* s_next = reinterpret_cast<unsigned*>(smem + 960);
  static_assert(2 * S + 1 + 8 + 4 + 2 <= 64 && sizeof(Segment) <= 192, "in front of kOffQ");
  unsigned char* qs = smem + P::kOffQ;
  unsigned char* ring = smem + P::kOffRing;

  // ---- who does what ------------------------------------------------------------------
  using Families = FamilyTable<kTableTensor>;
  static_assert(sizeof(Families) <= P::kSmem - 2048, "the groups' table lies where the tiles will");
  // What each group's members see, for the segments: of few groups in front of kOffQ.  (Where it lies is kept there too: a
  // pointer that lives through the softmax takes registers that it has not to spare: 64 behind 8192 53.0 us, 51.2.)
  int32_t* const keep = a.groups > kTableTensor ? a.seen
                        : a.groups <= kKept ? reinterpret_cast<int32_t*>(smem + 544)
                                            : a.seen + (int64_t)blockIdx.x * a.groups;
  int32_t* volatile* const s_keep = reinterpret_cast<int32_t* volatile*>(smem + 536);
  if (tid == 0) *s_keep = keep;
  Families& families = *reinterpret_cast<Families*>(smem + 1024);
  families.fill<kThreadsTc>(a);
  RangeList<kThreadsTc> list;
  const int ctas = gridDim.x;
  float rest = 0.f;
#pragma unroll 1
  for (int b = tid; b < a.pool.batch; b += kThreadsTc) {   // a unit costs about a tile of the walk's besides its own
    const int own = seen_of<C::kTokens, true>(ta.rest, b).tiles;
    if (own > 0) rest += (float)(own + 1);
  }
  list.plan(a, kTile, rest * ((float)C::kTokens / kTile), families, keep);
  if ((int)blockIdx.x >= list.ctas) {
    if (warp < C::kWarps)
      decode_walk<C, D, G, true>(ta.rest, smem, blockIdx.x - list.ctas, ctas - list.ctas,
                           [] { named_bar_sync(1, C::kWarps * 32); });
    return;
  }
  if (tid == 0) ta.rest.part_unit[ctas - 1 - blockIdx.x] = -1;   // the ranges that are not taken
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  const unsigned start = list.start;
  unsigned x, x_end;
  {
    const Ranges ranges(list.places, list.ctas);
    x = ranges.first(blockIdx.x);
    x_end = ranges.first(blockIdx.x + 1);
  }
  bool again = false;
#pragma unroll 1
  while (x < x_end) {
  if (warp == kLoadWarp && lane == 0) {
    if (again)   // every wait on them is over, and every copy and product that arrives at them
      for (int i = 0; i < 2 * S + 15; ++i) mbar_inval(full + i);
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&raw[i], 1);
    }
    mbar_init(qfull, 1);
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 4; ++i) mbar_init(&sfull[4 * t + i], 1);
      mbar_init(&pfull[2 * t], 4);
      mbar_init(&pfull[2 * t + 1], 4);
      mbar_init(&ofull[t], 1);
    }
    fence_mbar_init();
    misc[0] = misc[1] = 0;
  }
  again = true;
  if (warp == kLoadWarp) {
    find_segment(a, kTile, *s_keep, start, x, x_end, lane, s_seg, s_next);
    Segment s = *s_seg;
    see_segment(a, kTile, s, lane);
    __syncwarp();
    if (lane == 0) *s_seg = s;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (Read where they are needed: the softmax threads have no registers to spare.)
  volatile Segment& seg = *s_seg;
  x = *reinterpret_cast<volatile unsigned*>(s_next);
  if (seg.members == 0) break;   // (it was the range's last)
  const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int rows = seg.members << gs, nt = seg.last - seg.first;
  const int nq = rows > kTile ? 2 : 1;   // query tiles
  // From this key tile of the segment on some row does not see some key.
  const int clear = ((seg.p_lo + 1) >> 7) - seg.first;
  static_assert(kTile == 1 << 7, "");

  // The loader starts on the queries and the first key tile.
  const int boxes = kTile / ta.box_rows, box = lane % boxes, blk = lane / boxes;
  auto page_of = [&](int j, int* slot) {   // of this lane's box of key tile j; num_pages: zeros
    const int p = (seg.first + j) * kTile + box * ta.box_rows;
    *slot = 0;
    if (lane >= boxes * (D / 64) || p > seg.p_hi) return a.pool.num_pages;
    int pi;
    paged_split(a.pool, p, &pi, slot);
    const int page = a.pool.table[(int64_t)seg.leader * a.pool.max_pages + pi];
    if (page >= 0 && page < a.pool.num_pages) return page;
    if (a.pool.err) atomicOr(a.pool.err, LF_DEVERR_STATE);
    return a.pool.num_pages;
  };
  auto load = [&](int i, bool scrub, int page, int slot) {   // K (i even) or V of key tile i / 2
    const int st = i % S;
    uint64_t* bar = (i & 1) && scrub ? &raw[st] : &full[st];
    if (lane == 0) mbar_arrive_expect_tx(bar, P::kTileBytes);
    __syncwarp();
    if (lane < boxes * (D / 64))
      tma_load_4d(ring + st * P::kTileBytes + blk * kBlk + box * ta.box_rows * 128, (i & 1) ? &ta.v : &ta.k,
                  blk * 64, slot, seg.g, page, bar);
  };
  int page = 0, slot = 0;
  if (warp == kLoadWarp) {
    if (nt > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(qfull, nq * P::kTileBytes);
        for (int t = 0; t < nq; ++t)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(qs + t * P::kTileBytes + c * kBlk, &ta.q, c * 64, seg.g << gs, seg.b0 + t * (kTile >> gs), qfull);
      }
      page = page_of(0, &slot);
      load(0, 0 >= clear, page, slot);
      load(1, 0 >= clear, page, slot);
    }
  }
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_longer(bar, parity, misc);
  };

  if (warp == kLoadWarp) {
    // ---- loader ---------------------------------------------------------------------
    bool ok = true;
    uint64_t* done = sfull + 4 * (nq - 1);   // S of the last query tile: the others' are done too
    if (nt > 1) page = page_of(1, &slot);
    for (int j = 1; j < nt && ok; ++j) {
      const int cur_page = page, cur_slot = slot;
      if (j + 1 < nt) page = page_of(j + 1, &slot);   // a tile ahead
      const bool scrub = j >= clear;
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        // The stage held load i - S, K or V of key tile u: K_u has been read once the last S
        // of tile u is there, V_u once that of tile u + 1 is.  (u >= j - 4, and S of
        // tile j waits for this load: of four barriers in turn none is a lap ahead.)
        const int u = (i - S + 1) >> 1;
        static_assert(S <= 8, "sfull barriers");
        if (i >= S) ok = wait(&done[u & 3], (uint32_t)((u >> 2) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        load(i, scrub, cur_page, cur_slot);
      }
    }
    // The MMAs wait for every copy, so none is in flight when the CTA exits, unless a
    // wait ran out: then give the copies a second.
    if (!ok) {
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < kWaitLimitNs) {}
    }
    __syncwarp();
  } else if (warp == kScrubWarp) {
    // ---- scrubber -------------------------------------------------------------------
    uint32_t phase = 0;   // a bit per stage: its raw barrier's next parity
    for (int j = max(clear, 0); j < nt; ++j) {
      const int k0 = (seg.first + j) * kTile;
      const int st = (2 * j + 1) % S;
      const bool ok = wait(&raw[st], (phase >> st) & 1u);
      if (!__all_sync(0xffffffffu, ok)) break;
      phase ^= 1u << st;
      unsigned char* v = ring + st * P::kTileBytes;
      const int valid = min(kTile, seg.p_hi + 1 - k0);
      __nv_bfloat162 bad = __float2bfloat162_rn(0.f);
      auto look = [&](const uint4& x) {   // 0 * x is 0, or NaN where x is not finite
        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, bad);
      };
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4* rows4 = reinterpret_cast<uint4*>(v + c * kBlk);   // eight chunks per row
#pragma unroll 8
        for (int i = lane; i < valid * 8; i += 32) look(rows4[i]);
        for (int i = valid * 8 + lane; i < kTile * 8; i += 32) rows4[i] = make_uint4(0, 0, 0, 0);
      }
      const float2 f = __bfloat1622float2(bad);
      if (__any_sync(0xffffffffu, !(f.x == 0.f) || !(f.y == 0.f)) && lane == 0) misc[1] = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA ------------------------------------------------------------------------
    if (nt > 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdO = idesc_bf16_f32(128, D, false, true);
      const uint32_t lead = lane == 0;
      // Descriptors of an operand differ in their start address alone (16-byte units).
      const uint32_t dq = (uint32_t)sw128_desc(smem_u32(qs), 16, 1024);
      const uint32_t dk = (uint32_t)sw128_desc(smem_u32(ring), 16, 1024);
      const uint32_t dv = (uint32_t)sw128_desc(smem_u32(ring), kBlk, 1024);
      auto all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      auto mma_s = [&](int t, int j, int st) {
        const uint32_t qd = dq + (uint32_t)(t * (P::kTileBytes >> 4));
        const uint32_t kd = dk + (uint32_t)(st * (P::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (uint32_t)(((kk >> 2) * kBlk + (kk & 3) * 32) >> 4);
          mma_ss(lead, tm + t * 128, qd + o, kd + o, kIdS, kk > 0 ? 1u : 0u);
        }
        if (lead) tc_commit(&sfull[4 * t + (j & 3)]);
      };
      auto mma_o = [&](int t, int st, int half, uint32_t acc) {
        const uint32_t vd = dv + (uint32_t)(st * (P::kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(lead, tm + 256 + t * D, tm + t * 128 + half * 32 + kk * 8,
                 vd + (uint32_t)((half * 4 + kk) * 128), kIdO, kk > 0 ? 1u : acc);
      };
      // Straight code for one query tile and for two: a branch around an instruction costs more than it.
      auto walk = [&](auto tiles) {
        constexpr int N = decltype(tiles)::value;
        bool ok = all(qfull, 0) && all(&full[0], 0);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < N; ++t) mma_s(t, 0, 0);
        }
        int sv = 1 % S, sk = 2 % S;           // stages of V_j and K_(j+1)
        uint32_t pv = 0, pk = 2 / S;          // and their parities
        for (int j = 0; j < nt && ok; ++j) {
          const bool last = j + 1 == nt;
          const uint32_t pj = (uint32_t)(j & 1);
          ok = all(&full[sv], pv);
#pragma unroll
          for (int t = 0; t < N; ++t) {
            ok = ok && all(&pfull[2 * t], pj);
            if (!ok) break;
            tc_fence_after();
            mma_o(t, sv, 0, j > 0 ? 1u : 0u);
            if (t == 0 && !last) ok = all(&full[sk], pk);
            ok = ok && all(&pfull[2 * t + 1], pj);
            if (!ok) break;
            tc_fence_after();
            mma_o(t, sv, 1, 1u);
            if (!last) mma_s(t, j + 1, sk);
            else if (lead) tc_commit(&ofull[t]);
          }
          sv += 2;
          if (sv >= S) {
            sv -= S;
            pv ^= 1u;
          }
          sk += 2;
          if (sk >= S) {
            sk -= S;
            pk ^= 1u;
          }
        }
        return ok;
      };
      const bool ok = nq == 2 ? walk(std::integral_constant<int, 2>{}) : walk(std::integral_constant<int, 1>{});
      if (!ok && lead) {   // MMAs in flight end before the tensor memory is given back
        tc_commit(qfull);
        (void)mbar_wait_bounded(qfull, 1);
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarp && (warp - kSoftWarp) >> 2 < nq) {
    // ---- softmax ----------------------------------------------------------------------
    const int t = (warp - kSoftWarp) >> 2;
    const int rr0 = t * kTile + (warp & 3) * 32;   // the warp's first row in the segment
    const bool live = rr0 + lane < rows;
    const int pos = live ? last_seen(a, seg.prefix, seg.b0 + ((rr0 + lane) >> gs)) : -1;
    const uint32_t ts = tm + t * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tm + 256 + t * D + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = a.scale_log2;
    float m = kNegInf, l = 0.f;   // the row's maximum (log2) and sum
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      ok = __all_sync(0xffffffffu, wait(&sfull[4 * t + (j & 3)], (uint32_t)((j >> 2) & 1)));
      if (!ok) break;
      tc_fence_after();
      float x[kTile];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
      tmem_wait_ld();
      if (j >= clear) {
        const int hi = pos - (seg.first + j) * kTile;
#pragma unroll
        for (int c0 = 0; c0 < kTile; c0 += 32)   // 32 keys that all rows of the warp see stay as they are
          if (__any_sync(0xffffffffu, c0 + 31 > hi)) {
#pragma unroll
            for (int i = c0; i < c0 + 32; ++i)
              if (i > hi) x[i] = kNegInf;
          }
      }
      float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < kTile; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e + 4 < kTile) top[e] = max3(top[e], x[i + e], x[i + e + 4]);
          else top[e] = fmaxf(top[e], x[i + e]);
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
      // O_t holds no product yet at j = 0; later, every product before S_t is done.
      if (__any_sync(0xffffffffu, mx > m + kGrow)) {
        const float mn = fmaxf(m, mx);
        const float f = mn == kNegInf ? 1.f : ex2(m - mn);
        m = mn;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            float o[16];
            tmem_ld16(to + 16 * i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= f;
            tmem_st16(to + 16 * i, reinterpret_cast<const uint32_t*>(o));
          }
        }
      }
      const float mu = m == kNegInf ? 0.f : m;
      const uint64_t cc = pair(c, c), mm = pair(-mu, -mu);
      uint64_t sum[2] = {0ull, 0ull};   // two pairs of zeros
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float u, w;
          unpair(fma_pair(pair(x[64 * h + 2 * i], x[64 * h + 2 * i + 1]), cc, mm), &u, &w);
          u = ex2(u);
          w = ex2(w);
          sum[i & 1] = add_pair(sum[i & 1], pair(u, w));
          p[i] = pack_bf16(u, w);
        }
        tmem_st32(ts + 32 * h, p);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * t + h]);
      }
      float u, w;
      unpair(add_pair(sum[0], sum[1]), &u, &w);
      l += u + w;
    }

    // ---- shares out --------------------------------------------------------------------
    // A thread puts its row into the ring, which is done with once the last products are, and copies it out from
    // there: rows lie 16 bytes more than their length apart, so that eight lanes' chunks fall into eight bank groups.
    for (int i = 0; i < nq; ++i) ok = ok && (nt == 0 || __all_sync(0xffffffffu, wait(&ofull[i], 0)));
    tc_fence_after();
    if (ok && !misc[1]) {   // (otherwise nothing is right, or the rows are computed again below)
      static_assert(2 * kTile * (D * 4 + 16) <= S * P::kTileBytes, "rows fit the ring");
      unsigned char* mine = ring + (rr0 + lane) * (D * 4 + 16);
#pragma unroll
      for (int h = 0; h < D / 32; ++h) {
        float o[32];
        tmem_ld32(to + 32 * h, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(mine + 128 * h + 16 * e) =
              nt > 0 ? make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      fence_proxy_async_smem();
      if (live) {
        bulk_s2g(a.part_o + (seg.row + rr0 + lane) * D, mine, D * 4);
        *reinterpret_cast<float2*>(a.part_ml + 2 * (seg.row + rr0 + lane)) = make_float2(m, l);
      }
      bulk_wait_read();   // before the ring is filled again
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (misc[0]) break;   // a wait ran out
  if (misc[1])
    for (int r = warp; r < rows; r += kThreadsTc / 32)
      shared_row_by_hand<__nv_bfloat16, D>(a, *s_seg, kTile, r, last_seen(a, seg.prefix, seg.b0 + (r >> gs)), lane);
  __syncthreads();   // misc has been read
  }
  if (warp >= kSoftWarp) bulk_wait();
  if (warp == kMmaWarp) {
    tmem_dealloc(*tmem_slot, 512);
    if (lane == 0 && misc[0] && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_TIMEOUT);
  }
}

template <int D, int G>
cudaError_t launch(const SharedTcArgs& ta, int64_t grid, cudaStream_t stream) {
  using C = Walk<D, G>;
  constexpr int kWalk = C::kWarps * warp_bytes<C, D, G>() + 1024;
  constexpr int kSmem = SharedPlanTc<D>::kSmem > kWalk ? SharedPlanTc<D>::kSmem : kWalk;
  static_assert(kSmem + 1024 <= 232448, "with the lists' own");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_shared_tc_kernel<D, G>), kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreadsTc, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_shared_tc_kernel<D, G>, ta);
}

template <int D>
cudaError_t launch_group(const SharedTcArgs& ta, int64_t grid, cudaStream_t stream) {
  switch (ta.a.group) {
    case 1: return launch<D, 1>(ta, grid, stream);
    case 2: return launch<D, 2>(ta, grid, stream);
    case 4: return launch<D, 4>(ta, grid, stream);
    default: return launch<D, 8>(ta, grid, stream);
  }
}

}  // namespace

cudaError_t paged_shared_tc_launch(const PagedSharedArgs& a, const PagedDecodeArgs& rest, int head_dim, int grid,
                                   cudaStream_t stream) {
  const int ps = a.pool.page_size;
  if (!encoder()) return cudaErrorNotSupported;
  SharedTcArgs ta;
  ta.a = a;
  ta.rest = rest;
  ta.box_rows = ps < kTile ? ps : kTile;
  ta.group_shift = a.group == 1 ? 0 : a.group == 2 ? 1 : a.group == 4 ? 2 : 3;
  if (!encode_maps(a.pool, a.q, a.q_heads, a.group, a.pool.batch, head_dim, ta.box_rows, &ta.q, &ta.k, &ta.v))
    return cudaErrorInvalidValue;
  return head_dim == 64 ? launch_group<64>(ta, grid, stream) : launch_group<128>(ta, grid, stream);
}

}  // namespace lf
