// Causal attention of the last tokens of every sequence over a paged bf16 cache
// on the tensor cores (tcgen05), head_dim 64 and 128, with an optional sliding
// window and sinks.  The formula is lf_paged_prompt.cu's.
//
// Work.  A CTA takes 256 rows of one KV head's queries, (token, head of the group)
// pairs with the head inner, as two tiles of 128: every key and value it loads
// serves both tiles and all heads of the group.  Key tiles of 128 tokens that no
// row sees are not visited.  A sequence's last rows, which see the most keys, start first.
//
// Roles (12 warps, of which one rests: the softmax groups start at a multiple of four):
//   loader   gathers K and V tiles by page with TMA (one box per page and 64
//            columns, one lane each; a page past the end is a box outside the
//            tensor, which the hardware fills with zeros) into a ring;
//   scrubber where some row does not see some key of a tile, a weight of 0 must
//            take nothing of the value, but 0 * NaN is NaN on the tensor cores: it
//            zeroes the rows behind the last key that a row of the CTA sees and
//            looks for values that are not finite in the others.  If it finds any where
//            no row looks (between sinks and window), it zeroes these too; if any are
//            left, the CTA's rows are computed again, one by one, at the end;
//   MMA      S_t = Q_t K^T into tensor memory, then O_t += P_t V with P_t read from
//            tensor memory; the two tiles take turns, so that one's softmax runs
//            under the other's products;
//   softmax  two groups of four warps, a thread per row: S from tensor memory, the
//            running maximum, P = 2^(s - m) rounded to bf16 back over S, the sum in
//            fp32.  O is scaled down only when a row's maximum has grown by more
//            than 2^8 (P and the sum stay far from fp32's range, and the division
//            at the end makes any m right), so nearly never after the first tiles.
//
// Rounding P to bf16 (half a step is 2^-8 of a weight) is what the tensor cores
// take; a second product for the remainder would double the P V work.
//
// Bound by the MMAs and by what keeps them waiting.  Both query tiles'
// products with a key tile are 2048 clocks of the tensor cores; a CTA takes 2700, 2590 with the
// softmax left out.
// Around its key tiles a CTA spends about 10 thousand clocks: barriers, lookups and
// the first tiles' way in, the rows' way out, the next launch on the SM, and with one CTA per SM (all
// of the tensor memory, 200 KB) nothing runs meanwhile.  Measured, bf16, heads of 128, the same inputs
// again and again (other inputs every time): one prompt of 8192 tokens, 32 / 8 heads, 350 us, 1.57
// PFLOP/s, 82 % of the library's dense product (375 us, 1.46, 76 %); 12000 with a window of 1000,
// 16 / 8 heads, 117 us (120); chunks of 1 to 512 of 24 sequences behind up to 2048, 32 / 8 heads, 119 us
// (131).  Heads of 64 have half the products under the same softmax: 8192 tokens 293 us, 0.94 PFLOP/s.
// The scrubber's reads are 2 us of the window's 117 (measured without them).
#include "lf_paged_tc.cuh"
#include "longflow.h"

namespace lf {

namespace {

struct PromptTcArgs {
  CUtensorMap q, k, v;
  PagedPromptArgs a;
  int box_rows;      // tokens of one TMA box: min(page_size, 128)
  int group_shift;
};

struct Work {
  int p_lo, p_hi, sink, gap, first, last, q0, g;
  int64_t r0, rows;
};

template <int D>
__global__ void __launch_bounds__(kThreadsTc, 1) paged_prompt_tc_kernel(const __grid_constant__ PromptTcArgs ta) {
  using P = TcPlan<D>;
  constexpr int S = P::kStages;
  const PagedPromptArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform for the compiler too
  const int G = a.group, gs = ta.group_shift;
  int number;
  const int b = locate(a, blockIdx.x, &number);

  // The loader's lookups for the first key tile, before it is known whether that is
  // tile 0 (it is unless a window without sinks starts behind it).
  const int boxes = kTile / ta.box_rows, box = lane % boxes, blk = lane / boxes;
  int guess = -1;
  if (warp == kLoadWarp) {
    if (lane < 3) tma_prefetch_desc(lane == 0 ? &ta.q : lane == 1 ? &ta.k : &ta.v);
    int pi, slot;
    paged_split(a.pool, box * ta.box_rows, &pi, &slot);
    if (pi < a.pool.max_pages) guess = a.pool.table[(int64_t)b * a.pool.max_pages + pi];
  }
  Piece piece;
  if (!take_piece(a, blockIdx.x, b, number, 2 * kTile, tid == kRestWarp * 32 && blockIdx.y == 0, &piece)) return;
  const int g = piece.g, q0 = piece.q0, first_pos = piece.first_pos, p_lo = piece.p_lo, p_hi = piece.p_hi;
  const int64_t r0 = piece.r0, rows = piece.rows;
  const Tiles tiles(a, p_lo, p_hi, kTile, blockIdx.y);
  const int nt = tiles.count();
  // Does some row of the CTA not see some key of the tile at k0?
  const int behind = behind_window(a, p_lo);
  auto masked = [&](int k0) { return some_hidden(a, p_lo, p_hi, k0, kTile); };

  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);   // [S] a tile is ready for the MMAs
  uint64_t* raw = full + S;                             // [S] V landed, to be scrubbed
  uint64_t* qfull = raw + S;
  uint64_t* sfull = qfull + 1;                          // [t][j & 3] S_t of key tile j ready, and
                                                        // every MMA before it done
  uint64_t* pfull = sfull + 8;                          // [2][2] half of P_t written (O_t scaled)
  uint64_t* ofull = pfull + 4;                          // [2] O_t final
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + 528);   // [0] a wait expired, [1] by hand
  // The piece as the softmax threads read it, which have no registers to spare.
  volatile Work* work = reinterpret_cast<volatile Work*>(smem + 768);
  if (tid == kRestWarp * 32) {
    work->p_lo = p_lo;
    work->p_hi = p_hi;
    work->sink = tiles.sink;
    work->gap = tiles.gap;
    work->first = tiles.first;
    work->last = tiles.last;
    work->q0 = q0;
    work->g = g;
    work->r0 = r0;
    work->rows = rows;
  }
  unsigned char* qs = smem + P::kOffQ;
  unsigned char* ring = smem + P::kOffRing;

  // The loader sets up the barriers and starts on the queries and the first key tile
  // at once; the others meet it behind.
  auto page_of = [&](int tile, int first, int* slot) {   // of this lane's box; num_pages: zeros
    const int p = tile * kTile + box * ta.box_rows;
    *slot = 0;
    if (lane >= boxes * (D / 64) || p > p_hi) return a.pool.num_pages;
    int pi;
    paged_split(a.pool, p, &pi, slot);
    const int page = tile == 0 ? first : a.pool.table[(int64_t)b * a.pool.max_pages + pi];
    const bool unseen = p >= a.sinks && p + ta.box_rows <= behind;   // by all rows of the CTA
    if (page >= 0 && page < a.pool.num_pages && !unseen) return page;
    if (a.pool.err && !unseen) atomicOr(a.pool.err, LF_DEVERR_STATE);
    return a.pool.num_pages;
  };
  auto load = [&](int i, bool scrub, int page, int slot) {   // K (i even) or V of key tile i / 2
    const int st = i % S;
    uint64_t* bar = (i & 1) && scrub ? &raw[st] : &full[st];
    if (lane == 0) mbar_arrive_expect_tx(bar, P::kTileBytes);
    __syncwarp();
    if (lane < boxes * (D / 64))
      tma_load_4d(ring + st * P::kTileBytes + blk * kBlk + box * ta.box_rows * 128, (i & 1) ? &ta.v : &ta.k,
                  blk * 64, slot, g, page, bar);
  };
  int page = 0, slot = 0;
  if (warp == kLoadWarp) {
    if (lane == 0) {
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
    __syncwarp();
    if (nt > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(qfull, 2 * P::kTileBytes);
        for (int t = 0; t < 2; ++t)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(qs + t * P::kTileBytes + c * kBlk, &ta.q, c * 64, g * G,
                        q0 + (int)(r0 >> gs) + t * (kTile >> gs), qfull);
      }
      const bool scrub = masked(tiles.at(0) * kTile);
      page = page_of(tiles.at(0), guess, &slot);
      load(0, scrub, page, slot);
      load(1, scrub, page, slot);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // The first try costs a few tens of clocks, which the MMA warp's products hide; the
  // limit and the flag that ends everyone's waits come after it.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_longer(bar, parity, misc);
  };

  float m = kNegInf, l = 0.f;   // softmax threads: their row's maximum (log2) and sum

  if (warp == kLoadWarp) {
    // ---- loader ---------------------------------------------------------------------
    bool ok = true;
    if (nt > 1) page = page_of(tiles.at(1), guess, &slot);
    for (int j = 1; j < nt && ok; ++j) {
      const int cur_page = page, cur_slot = slot;
      if (j + 1 < nt) page = page_of(tiles.at(j + 1), guess, &slot);   // a tile ahead
      const bool scrub = masked(tiles.at(j) * kTile);
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        // The stage held load i - S, K or V of key tile u: K_u has been read once S_1
        // of tile u is there, V_u once S_1 of tile u + 1 is.  (u >= j - 4, and S_1 of
        // tile j waits for this load: of four barriers in turn none is a lap ahead.)
        const int u = (i - S + 1) >> 1;
        static_assert(S <= 8, "sfull barriers");
        if (i >= S) ok = wait(&sfull[4 + (u & 3)], (uint32_t)((u >> 2) & 1));
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
    for (int j = 0; j < nt; ++j) {
      const int k0 = tiles.at(j) * kTile;
      if (!masked(k0)) continue;
      const int st = (2 * j + 1) % S;
      const bool ok = wait(&raw[st], (phase >> st) & 1u);
      if (!__all_sync(0xffffffffu, ok)) break;
      phase ^= 1u << st;
      unsigned char* v = ring + st * P::kTileBytes;
      const int valid = min(kTile, p_hi + 1 - k0);
      __nv_bfloat162 bad = __float2bfloat162_rn(0.f);
      auto look = [&](const uint4& x) {   // 0 * x is 0, or NaN where x is not finite
        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, bad);
        bad = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, bad);
      };
      auto found = [&] {
        const float2 f = __bfloat1622float2(bad);
        return __any_sync(0xffffffffu, !(f.x == 0.f) || !(f.y == 0.f));
      };
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4* rows4 = reinterpret_cast<uint4*>(v + c * kBlk);   // eight chunks per row
#pragma unroll 8
        for (int i = lane; i < valid * 8; i += 32) look(rows4[i]);
        for (int i = valid * 8 + lane; i < kTile * 8; i += 32) rows4[i] = make_uint4(0, 0, 0, 0);
      }
      // Rows front .. back - 1 lie behind every row's window.  Only where something was found it
      // is asked whether it lies there: those rows become zeros, the others are looked at again.
      // (Every such tile's rows told apart from the start: 12000 tokens with a window of 1000, 118 us against 116.)
      bool any = found();
      const int front = max(a.sinks - k0, 0), back = min(behind - k0, valid);
      if (any && front < back) {
        bad = __float2bfloat162_rn(0.f);
#pragma unroll 1
        for (int i = lane; i < D / 64 * valid * 8; i += 32) {
          const int c = i / (valid * 8), j = i - c * valid * 8;
          uint4* row = reinterpret_cast<uint4*>(v + c * kBlk) + j;
          if ((j >> 3) >= front && (j >> 3) < back) *row = make_uint4(0, 0, 0, 0);
          else look(*row);
        }
        any = found();
      }
      if (any && lane == 0) misc[1] = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA ------------------------------------------------------------------------
    // The tensor cores take an instruction every 64 clocks, so what stands between
    // two of them counts: the warp walks the tiles together, one lane's predicate is
    // on the instructions, descriptors are uniform values, and the two commits of a
    // key tile serve the softmax and the loader both.
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
      bool ok = all(qfull, 0) && all(&full[0], 0);
      if (ok) {
        tc_fence_after();
        mma_s(0, 0, 0);
        mma_s(1, 0, 0);
      }
      int sv = 1 % S, sk = 2 % S;           // stages of V_j and K_(j+1)
      uint32_t pv = 0, pk = 2 / S;          // and their parities
      for (int j = 0; j < nt && ok; ++j) {
        const bool last = j + 1 == nt;
        const uint32_t pj = (uint32_t)(j & 1);
        ok = all(&full[sv], pv);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
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
      if (!ok && lead) {   // MMAs in flight end before the tensor memory is given back
        tc_commit(qfull);
        (void)mbar_wait_bounded(qfull, 1);
      }
    }
    __syncwarp();
  } else if (warp >= kSoftWarp) {
    // ---- softmax ----------------------------------------------------------------------
    const int t = (warp - kSoftWarp) >> 2;
    const int rr0 = t * kTile + (warp & 3) * 32;   // the warp's first row in the piece
    const bool live = work->r0 + rr0 + lane < work->rows;
    const int pos = live ? work->p_lo + ((rr0 + lane) >> gs) : -1;
    const uint32_t ts = tm + t * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tm + 256 + t * D + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = a.scale_log2;
    bool ok = true;
    const int n = work->last - work->first;
    for (int j = 0; j < n; ++j) {
      const int at = work->first + j;
      const int k0 = (at < work->sink ? at : at + work->gap) * kTile;
      const bool hidden = some_hidden(a, work->p_lo, work->p_hi, k0, kTile);
      ok = __all_sync(0xffffffffu, wait(&sfull[4 * t + (j & 3)], (uint32_t)((j >> 2) & 1)));
      if (!ok) break;
      tc_fence_after();
      float x[kTile];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x + 32 * i);
      tmem_wait_ld();
      if (hidden) {
        const int hi = pos - k0, sk = a.sinks - k0;
        const int lo = a.window > 0 && pos >= 0 ? pos - a.window + 1 - k0 : -1;
#pragma unroll
        for (int c0 = 0; c0 < kTile; c0 += 32)   // 32 keys that all rows of the warp see stay as they are
          if (__any_sync(0xffffffffu, !(c0 + 31 <= hi && (c0 >= lo || c0 + 31 < sk)))) {
#pragma unroll
            for (int i = c0; i < c0 + 32; ++i)
              if (!(i <= hi && (i >= lo || i < sk))) x[i] = kNegInf;
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

    // ---- rows out --------------------------------------------------------------------
    ok = ok && (n == 0 || __all_sync(0xffffffffu, wait(&ofull[t], 0)));
    tc_fence_after();
    if (!ok || misc[1]) {
      // nothing is right, or the rows are computed again below: leave them
    } else if (a.splits > 1) {   // a share of the row: few rows, stored as they lie
      float* part = part_row<D>(a, blockIdx.x, blockIdx.y, 2 * kTile, rr0 + lane, m, l, live);
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        float o[32];
        tmem_ld32(to + 32 * i, o);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + 32 * i + e) =
                n > 0 ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      unsigned char* stage = smem + P::kOffOut + (warp - kSoftWarp) * 4096;   // 32 rows x 64 columns
      // Row rr of the warp's 32 is head rr % G of token rr / G from its first.
      const int64_t first = work->r0 + rr0;
      const int left = (int)min((int64_t)32, work->rows - first);
      const int q0 = work->q0, g = work->g;
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) +
                           ((int64_t)(q0 + (first >> gs)) * a.q_heads + g * G) * D + (lane & 7) * 8;
      const int64_t token = (int64_t)a.q_heads * D;
#pragma unroll 1
      for (int h = 0; h < D / 64; ++h) {   // through shared memory: whole lines of global memory
        __syncwarp();   // the half before has been read
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          float o[32];   // (without keys nothing is there; l is 0 then)
          tmem_ld32(to + 64 * h + 32 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = l == 0.f ? 0u : pack_bf16(o[8 * e + 2 * i] * inv, o[8 * e + 2 * i + 1] * inv);
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * q + e) ^ (lane & 7)) << 4)) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          if (rr < left)
            *reinterpret_cast<uint4*>(out + (rr >> gs) * token + (rr & (G - 1)) * D + h * 64) =
                *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
        }
      }
      if (live) {
        write_row_stats(a, (int64_t)(q0 + ((first + lane) >> gs)) * a.q_heads + g * G + (lane & (G - 1)), m, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
    if (lane == 0 && misc[0] && a.pool.err) atomicOr(a.pool.err, LF_DEVERR_TIMEOUT);
  }
  if (misc[1] && !misc[0]) {
    constexpr int kEach = (2 * kTile + kThreadsTc / 32 - 1) / (kThreadsTc / 32);   // rows of a warp
    rows_by_hand<__nv_bfloat16, D>(a, blockIdx.x, blockIdx.y, kTile, 2 * kTile, warp * kEach,
                                   min(kEach, 2 * kTile - warp * kEach), lane);
  }
}

template <int D>
cudaError_t launch(const PromptTcArgs& ta, dim3 grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&paged_prompt_tc_kernel<D>), TcPlan<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  paged_prompt_tc_kernel<D><<<grid, kThreadsTc, TcPlan<D>::kSmem, stream>>>(ta);
  return cudaGetLastError();
}

}  // namespace

bool paged_prompt_tc_takes(const PagedPool& pool, int head_dim) {
  // A key tile is whole boxes of whole pages (or a page is whole tiles), and a box
  // is whole groups of the eight rows that the swizzle repeats over.
  const int ps = pool.page_size;
  const bool pages = ps >= 8 && (ps < kTile ? kTile % ps == 0 : ps % kTile == 0);
  // A tensor map has no stride of zero, and none from 2^40 bytes on.
  const cuuint64_t st[3] = {legal_stride(pool.token_stride, ps), legal_stride(pool.head_stride, pool.kv_heads),
                            legal_stride(pool.page_stride, pool.num_pages)};
  for (cuuint64_t x : st)
    if (x < 16 || x >= 1ull << 40) return false;
  return (head_dim == 64 || head_dim == 128) && pages;
}

cudaError_t paged_prompt_tc_launch(const PagedPromptArgs& a, const PromptPlan& plan, int head_dim, cudaStream_t stream) {
  const int ps = a.pool.page_size;
  if (!encoder()) return cudaErrorNotSupported;
  PromptTcArgs ta;
  ta.a = a;
  ta.box_rows = ps < kTile ? ps : kTile;
  ta.group_shift = a.group == 1 ? 0 : a.group == 2 ? 1 : a.group == 4 ? 2 : 3;
  if (!encode_maps(a.pool, a.q, a.q_heads, a.group, a.total_q, head_dim, ta.box_rows, &ta.q, &ta.k, &ta.v))
    return cudaErrorInvalidValue;
  const dim3 grid((unsigned)plan.pieces, plan.splits);
  return head_dim == 64 ? launch<64>(ta, grid, stream) : launch<128>(ta, grid, stream);
}

}  // namespace lf
