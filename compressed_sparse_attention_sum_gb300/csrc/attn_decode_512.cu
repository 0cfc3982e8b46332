// csa_attn_decode on the tensor cores at d = 512 with 33 to 64 columns (the
// production width: 64 heads).
//
// As in attn_decode_tc.cu, O^T[channels, columns] += KV^T P^T with the (query,
// head) columns as N.  At this width an expanded tile of 128 slots is 128 KB, so a
// second one does not fit beside it, and a tile's steps (expand, S, softmax, O)
// follow one another.  Here a tile is 64 slots, three times, and eight warps
// expand, eight run the softmax and one issues the products, each on a tile of
// its own.
//
// To fill 128 rows with 64 slots, a tile's rows are (channel half, slot): row s
// holds channels 0-255 of slot s, row 64 + s its channels 256-511.  Q lies in
// TMEM, whose lanes are likewise (channel half, column), so that one product of
// K = 256
//   S' [128, 128] = Q' . KV'^T
// has in its two diagonal quarters the halves of S, which the softmax adds (the
// other quarters are not used; 128 columns take the tensor core no longer than
// 64 do).  With Q in TMEM, S' reads only the tile from shared memory: products
// with both operands there left too little of its bandwidth to the expansion.  A
// row of S' is a column of the softmax: its maximum and sum stay within a thread
// but for the four that share a row.
//
// 128 queries of 64 heads, 1152 slots each (18 tiles), 4 bits: 41.4 us in a graph
// that finds the rows in L2 (45.8 us where it does not), of which 9 are the prologue
// and the end.  40.4 us with one sum of P instead of two (attn_decode_tc.cu).
// Compared with that, one tile of 128 slots and its chain: 52.7 us; two tiles of 64,
// Q in shared memory and slots as the rows of S': 49.9 us (16 expanding warps
// instead of 8: 50.7 us).  What bounds it: 3.6k cycles a tile,
// of which the tensor core takes 2.1k (16 products of N = 128 and 16 of N = 64);
// shared memory moves 224 KB, 1.75k cycles, and its queue delays the expansion
// and the softmax, whose instructions fill about half of the issue slots.
#include "attn_decode.h"
#include "attn_decode_join.cuh"
#include "cache_expand.cuh"
#include "smem_once.h"

namespace csa {
namespace adt {

constexpr int kD5 = 512;
constexpr int kNC5 = 64;
constexpr int kTile5 = 64;                     // slots
constexpr int kConv5 = 8, kSoft5 = 8;          // warps that expand, warps of the softmax

struct Cfg512 {
  static constexpr int kThreads = (kConv5 + kSoft5 + 1) * 32;
  static constexpr uint32_t kBlk = 128 * 128;              // 64 channels of 128 rows
  static constexpr uint32_t kBuf = 4 * kBlk;               // a tile: 256 channels of 128 rows
  // TMEM: S' 128 columns, Q' 128, O^T 4 x 64
  static constexpr uint32_t kColS = 0, kColQ = 128, kColO = 256;
  static constexpr uint32_t KV = 0;                        // [3] tiles
  static constexpr uint32_t P = KV + 3 * kBuf;             // [64 columns][128 B: 64 slots]
  static constexpr uint32_t XCH = P + kNC5 * 128;          // [8 warps][32 lanes][16] halves of S to be added; at the
                                                           // end [64][4] sums as rounded
  static constexpr uint32_t BARS = XCH + kSoft5 * 2048;    // kv[3], o[3], s, sfree, p, q, end
  static constexpr uint32_t MISC = BARS + 11 * 8;          // TMEM slot, dead
  static constexpr uint32_t RED = (MISC + 8 + 15) / 16 * 16;   // [2][64][4] column maxima
  static constexpr uint32_t MRUN = RED + 8 * kNC5 * 4;     // [64] at the end
  static constexpr uint32_t ML = MRUN + kNC5 * 4;          // [64] (maximum, sum, O's factor) of this CTA
  static constexpr uint32_t SINK = ML + kNC5 * 16;         // [64] sink logits of the heads (log2 units)
  static constexpr uint32_t OKS = SINK + kNC5 * 4;         // [3][8] bits of the slots
  static constexpr uint32_t kBytes = OKS + 3 * 8;
  static constexpr uint32_t STAGE = KV;                    // O after the last tile
};

template <int BITS>
__global__ void __launch_bounds__(640, 1) attn_decode_512_kernel(
    const AttnDecodeArgs a, int per_group, int groups, int head_groups, int cs, int splits) {
  using C = Cfg512;
  constexpr int D = kD5, NC = kNC5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_kv = reinterpret_cast<uint64_t*>(sm + C::BARS);   // [3] tile expanded
  uint64_t* bar_o = bar_kv + 3;                                   // [3] O^T of the tile complete
  uint64_t* bar_s = bar_kv + 6;                                   // S' complete, oks of the tile
  uint64_t* bar_sfree = bar_kv + 7;                               // S' read
  uint64_t* bar_p = bar_kv + 8;                                   // P written
  uint64_t* bar_q = bar_kv + 9;                                   // Q written
  uint64_t* bar_end = bar_kv + 10;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::MISC);
  volatile int* dead = reinterpret_cast<int*>(sm + C::MISC + 4);
  float* red = reinterpret_cast<float*>(sm + C::RED);
  float* m_run = reinterpret_cast<float*>(sm + C::MRUN);
  float4* ml = reinterpret_cast<float4*>(sm + C::ML);
  unsigned char* oks = sm + C::OKS;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // blockIdx.x: group of queries (per_group of one sequence) and of heads, and
  // its split of the slots (the cs CTAs of a cluster are neighbours)
  const int group = (int)blockIdx.x / splits, split = (int)blockIdx.x - group * splits;
  const int rank = split % cs;
  const int hg = group % head_groups, qg = group / head_groups;
  const int bi = qg / groups, i0 = (qg - bi * groups) * per_group;
  const int nq = min(per_group, a.s_q - i0);
  const int h0 = hg * NC, heads = min(a.H - h0, per_group > 1 ? a.H : NC);   // heads of a query
  const long long row0 = (long long)bi * a.s_q + i0;

  const bool conv = warp < kConv5;
  // TMEM lane quarter of this thread in the softmax and at the end
  const int qd = warp & 3;
  const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
  // Q: column c is query i0 + c / H, head h0 + c % H; columns past them are zero.
  // Read by the softmax warps, 128 channels of a row of Q' each, in two batches;
  // the first leaves before anything is waited for.
  const int hq = (warp >> 2) & 1, upper = qd >> 1;
  const int c1 = (qd & 1) * 32 + lane;                     // column of this thread's row of S'
  uint4 qv[8];
  auto read_q = [&](int x0) {
    const int qi = per_group > 1 ? c1 / a.H : 0, h = per_group > 1 ? c1 - qi * a.H : c1;
    const bool live = qi < nq && h < heads;
    const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                                      ((row0 + (live ? qi : 0)) * a.H + h0 +
                                                       (live ? h : 0)) * D) +
                       upper * 32 + hq * 16 + x0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint4 v = __ldg(src + x);
      qv[x] = live ? v : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto store_q = [&](uint32_t taddr) {
    uint32_t w[32];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint4 v = permute8<BITS>(qv[x]);
      w[4 * x] = v.x;
      w[4 * x + 1] = v.y;
      w[4 * x + 2] = v.z;
      w[4 * x + 3] = v.w;
    }
    CSA_TMEM_ST32(taddr, w);
  };
  if (!conv && warp < kConv5 + kSoft5) read_q(0);
  float sink_v = -INFINITY;
  if (tid < heads && tid < NC && a.sink != nullptr) sink_v = sink_log2(__ldg(a.sink + h0 + tid));

  // The slots: the union window of the group's queries, then the index
  // entries (one query) or the blocks the last query sees.
  const DecodeRow last = decode_row(a, bi, i0 + nq - 1);
  const int wext = a.window + nq - 1;
  const int w0 = last.t - wext + 1;
  const int ring = a.P_raw * a.cs.page_size;
  const int ring0 = w0 >= 0 ? w0 % ring : ring - 1 - (int)((unsigned)(-1 - w0) % (unsigned)ring);
  const int slots = last.t < 0 ? 0 : wext + (a.idx != nullptr ? a.K : last.vis);
  const int tiles = (slots + kTile5 - 1) / kTile5;
  const int it0 = (unsigned)tiles * (unsigned)split / (unsigned)splits;   // tiles <= 2^19, splits <= 152
  const int n = (int)((unsigned)tiles * (unsigned)(split + 1) / (unsigned)splits) - it0;

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar_kv[i], kConv5);
      mbar_init(&bar_o[i], 1);
    }
    mbar_init(bar_s, 2);
    mbar_init(bar_sfree, kSoft5);
    mbar_init(bar_p, kSoft5);
    mbar_init(bar_q, kSoft5);
    mbar_init(bar_end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *dead = 0;
  }
  if (warp == kConv5 + kSoft5 && n > 0) tmem_alloc(tmem_slot, 512);
  if (tid < NC) {
    ml[tid] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    reinterpret_cast<float*>(sm + C::SINK)[tid] = sink_v;
  }

  // ---- the expanding side's reads: index entry, page id, codes ------------------
  const int cgr = lane >> 3;                               // scale group of every 128 channels
  const int cslot = warp * 8 + (lane & 7);
  const int32_t* raw_pages = a.raw_table + (long long)bi * a.P_raw;
  const int32_t* cmp_pages = a.cmp_table + (long long)bi * a.P_cmp;
  int jraw = 0, lslot = -1, page = 0;
  Codes<BITS> cd[4];
  auto slot_of = [&](int it) {                             // -1: past the tiles or the list
    const int s = (it0 + it) * kTile5 + cslot;
    return it < n && s < slots ? s : -1;
  };
  auto read_index = [&](int it) {
    const int s = slot_of(it);
    jraw = s - wext;
    if (a.idx != nullptr) jraw = __ldg(a.idx + row0 * a.K + max(s - wext, 0));
  };
  auto read_page = [&](int it) {
    const int s = slot_of(it);
    const bool raw = s < wext;
    const int rs = ring0 + s >= ring ? ring0 + s - ring : ring0 + s;
    int x = raw ? (w0 + s >= 0 ? rs : -1) : (jraw < last.vis ? jraw : -1);
    if (s < 0) x = -1;
    lslot = max(x, -1);
    page = __ldg((raw || x < 0 ? raw_pages : cmp_pages) + (x < 0 ? 0 : page_index(a.cs, x)));
  };
  // Addresses of the row that read_page found; masked: a row of zeros.
  const uint8_t *code_p = nullptr, *scale_p = nullptr;
  bool next_ok = false;
  auto locate = [&]() {
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
    const bool inside = (unsigned)page < (unsigned)a.cs.n_pages;
    if (lslot >= 0 && !inside) set_status(a.status, kDevCheck, kSiteCachePage);
    next_ok = lslot >= 0 && inside;
    const int r = lslot - page_index(a.cs, lslot) * a.cs.page_size;
    const uint8_t* base = a.cache + page_base(a.cs, page);
    code_p = (next_ok ? base + row_code(a.cs, r) : zero) + cgr * (4 * BITS);
    scale_p = next_ok ? base + row_scale(a.cs, r) : zero;
  };
  auto read_codes = [&](int m) {
#pragma unroll
    for (int e = 0; e < BITS / 4; ++e)
      cd[m].w[e] = __ldg(reinterpret_cast<const uint4*>(code_p + m * (16 * BITS)) + e);
  };
  if (conv && n > 0) read_index(0);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = n > 0 ? *tmem_slot : 0u;

  // A wait that gives up ends every later wait of the CTA.
  bool gone = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (gone) return false;
    if (mbar_try(bar, parity) || (!*dead && mbar_wait(bar, parity))) return true;
    *dead = 1;
    gone = true;
    return false;
  };
  // The same for a whole warp, with one answer.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };
  // One arrival a warp.
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  // Buffer and phase of a tile
  auto next = [](int& buf, uint32_t& ph) {
    if (++buf == 3) {
      buf = 0;
      ph ^= 1u;
    }
  };
  // Of column c1 over this thread's slots: the maximum, and the sum of P as computed
  // and as rounded to bf16 (attn_decode_tc.cu).
  float m1 = -INFINITY, l1 = 0.f, lr1 = 0.f;

  if (n == 0) {
  } else if (warp == kConv5 + kSoft5) {
    // ---- the issuing warp ------------------------------------------------------
    // S' of a tile goes ahead of O^T of the tile before.  The proxy fences stand on
    // this side of the barriers (attn_decode_tc.cu).
    constexpr uint32_t idesc_s = idesc_bf16_f32_major(128, 128, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16_f32_major(128, NC, 1, 0);
    const uint32_t td = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t kvd = sw128_desc(smem_addr(sm + C::KV)), pd = sw128_desc(smem_addr(sm + C::P));
    const uint64_t kvd_mn = sw128_desc_mn(smem_addr(sm + C::KV), C::kBlk);
    const int armed = armed_fault(a.status);               // test hook (attn_decode_tc.cu)
    bool up = wait_warp(bar_q, 0) && (armed != kSiteDecode || split != splits - 1);
    int buf = 0, bo = 0;                                   // of tile it, of tile it - 1
    uint32_t ph = 0;
    for (int it = 0; up && it <= n; ++it) {
      if (it < n) {
        up = wait_warp(&bar_kv[buf], ph);
        if (it > 0) up = up && wait_warp(bar_sfree, (it - 1) & 1);
        fence_proxy_async_smem();
        fence_after();
        const uint64_t ka = kvd + buf * (C::kBuf >> 4);
        if (up && elect_one()) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            mma_bf16_ts(td + C::kColS, td + C::kColQ + k * 8,
                        ka + (((k >> 2) * C::kBlk + (k & 3) * 32) >> 4), idesc_s, k > 0 ? 1u : 0u);
          mma_commit(bar_s);
          mbar_arrive(bar_s);                              // hands on what the expanding warps wrote
        }
        __syncwarp();
      }
      if (it > 0) {
        up = up && wait_warp(bar_p, (it - 1) & 1);
        fence_proxy_async_smem();
        fence_after();
        const uint64_t ka = kvd_mn + bo * (C::kBuf >> 4);
        if (up && elect_one()) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            // channels 128 m ..: two blocks, the rows of their half
#pragma unroll
            for (int k = 0; k < kTile5 / 16; ++k)
              mma_bf16_ss(td + C::kColO + m * NC,
                          ka + ((2 * (m & 1) * C::kBlk + (m >> 1) * (64 * 128) + k * 2048) >> 4),
                          pd + ((k * 32) >> 4), idesc_o, (it > 1 || k > 0) ? 1u : 0u);
          }
          mma_commit(&bar_o[bo]);
        }
        __syncwarp();
      }
      bo = buf;
      next(buf, ph);
    }
  } else if (conv) {
    // ---- the expanding warps -----------------------------------------------------
    read_page(0);
    read_index(1);
    locate();
    uint4 sc = __ldg(reinterpret_cast<const uint4*>(scale_p));
#pragma unroll
    for (int m = 0; m < 4; ++m) read_codes(m);
    read_page(1);
    read_index(2);
    int buf = 0;
    uint32_t ph = 0;
    for (int it = 0; it < n; ++it) {
      const unsigned oks8 = __ballot_sync(0xffffffffu, next_ok) & 255u;
      const uint32_t scales[4] = {sc.x, sc.y, sc.z, sc.w};
      locate();                                            // of the next tile
      sc = __ldg(reinterpret_cast<const uint4*>(scale_p));
      read_page(it + 2);
      read_index(it + 3);
      unsigned char* dst = sm + C::KV + buf * C::kBuf + cslot * 128;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t o[16];
        cd[m].scale = (scales[m] >> (8 * cgr)) & 255u;
        expand_words<BITS>(cd[m], o);
        read_codes(m);                                     // in flight until the next tile
        if (m == 0) {
          if (it > 2) wait(&bar_o[buf], ph ^ 1u);          // the buffer is free
          if (lane == 0) oks[buf * 8 + warp] = (unsigned char)oks8;
        }
        // group m * 4 + cgr: half m / 2, block of the half
        store_words(o, dst + (uint32_t)((m & 1) * 2 + (cgr >> 1)) * C::kBlk + (m >> 1) * (64 * 128),
                    (cgr & 1) * 4, cslot & 7);
      }
      arrive(&bar_kv[buf]);
      next(buf, ph);
    }
  } else {
    // ---- the softmax warps --------------------------------------------------------
    store_q(tmem + lane_base + C::kColQ + hq * 64);
    read_q(8);
    store_q(tmem + lane_base + C::kColQ + hq * 64 + 32);
    tmem_wait_st();
    fence_before();
    arrive(bar_q);
    // Lane (channel half, column) of S' has the half's part of its column at all
    // slots, in the columns of the same half.  A thread reads 32 of them, keeps 16
    // and exchanges the others with the thread that has the other half.
    const int sw = warp - kConv5;
    const int s0 = hq * 32 + upper * 16;                   // this thread's 16 slots
    const float sc2 = a.scale * kLog2e;
    const int my_q = per_group > 1 ? c1 / a.H : 0;         // query of column c1
    const int my_t = last.t - (nq - 1) + my_q;
    const int my_vis = min(my_t >= 0 ? (int)((unsigned)(my_t + 1) / (unsigned)a.ratio) : 0, last.vis);
    // its slots: [lo, hi) of the window, [wext, end)
    const int lo = my_t - a.window + 1 - w0, hi = my_t + 1 - w0;
    const int end = a.idx != nullptr ? slots : wext + my_vis;
    float m2 = -INFINITY;                                  // maximum of column hq * 32 + lane of O^T
    // of this thread, and of the warp with the other half (quarter qd ^ 2)
    unsigned char* xput = sm + C::XCH + (sw * 32 + lane) * 64;
    const unsigned char* xget = sm + C::XCH + ((hq * 4 + (qd ^ 2)) * 32 + lane) * 64;
    const int xs = (lane >> 1) & 3;                        // 16-byte chunks rotated against bank conflicts
    const int pair = 2 + hq * 2 + (qd & 1);                // barrier of those two warps
    const uint32_t ts = tmem + lane_base + C::kColS + upper * 64 + hq * 32;
    unsigned char* prow = sm + C::P + c1 * 128;
    // whether any of the softmax threads has it; orders their shared memory
    auto any_of_soft = [&](bool x) {
      int any;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.b32 q, %1, 0;\n\t"
          "bar.red.or.pred p, 1, %2, q;\n\t"
          "selp.b32 %0, 1, 0, p;\n\t}"
          : "=r"(any)
          : "r"((int)x), "n"(kSoft5 * 32)
          : "memory");
      return any != 0;
    };
    int buf = 0, bo = 0;                                   // of tile it, of tile it - 1
    uint32_t ph = 0, pho = 0;
    for (int it = 0; it < n; ++it) {
      wait(bar_s, it & 1);
      fence_after();
      // the slots that count, as bits
      const int s = (it0 + it) * kTile5 + s0;
      auto below = [&](int e) {                            // slots before e
        return (1u << min(max(e - s, 0), 16)) - 1u;
      };
      const unsigned live = *reinterpret_cast<const uint16_t*>(oks + buf * 8 + s0 / 8) &
                            ((below(hi) & ~below(lo)) | (below(end) & ~below(wext)));
      float x[16];
      uint32_t v[16], y[16];
      tmem_ld16_pair_wait(ts + upper * 16, v, ts + (upper ^ 1) * 16, y);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(xput + ((c ^ xs) << 4)) =
            make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
      fence_before();
      arrive(bar_sfree);
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 z = *reinterpret_cast<const float4*>(xget + ((c ^ xs) << 4));
        x[4 * c] = (__uint_as_float(v[4 * c]) + z.x) * sc2;
        x[4 * c + 1] = (__uint_as_float(v[4 * c + 1]) + z.y) * sc2;
        x[4 * c + 2] = (__uint_as_float(v[4 * c + 2]) + z.z) * sc2;
        x[4 * c + 3] = (__uint_as_float(v[4 * c + 3]) + z.w) * sc2;
      }
      if (__any_sync(0xffffffffu, live != 0xffffu)) {
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = (live >> c) & 1u ? x[c] : -INFINITY;
      }
      float mx = x[0];
#pragma unroll
      for (int c = 1; c < 16; ++c) mx = fmaxf(mx, x[c]);
      // P = 2^(x - m), masked slots 2^-inf = 0; a column without an unmasked
      // slot so far has m = -inf and takes 0 instead
      uint32_t pk[8];
      float lt, lrt;
      auto weights = [&]() {
        const float m_use = m1 == -INFINITY ? 0.f : m1;
        float l0 = 0.f, l2 = 0.f, r0 = 0.f, r2 = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float p0 = ex2(x[e] - m_use), p1 = ex2(x[e + 1] - m_use);
          l0 += p0;
          l2 += p1;
          pk[e / 2] = pack_bf16x2(p0, p1);
          r0 += __uint_as_float(pk[e / 2] << 16);
          r2 += __uint_as_float(pk[e / 2] & 0xffff0000u);
        }
        lt = l0 + l2;
        lrt = r0 + r2;
      };
      // A maximum moves where it grows by more than 2^kRescale, or from nothing.  Few
      // tiles have one that does: P is formed with the present ones beforehand, and
      // again, with the columns' new maxima, where any does.
      weights();
      const bool grow = any_of_soft(mx > m1 + kRescale);
      unsigned left = 0;                                   // columns of O^T to be rescaled
      float f2 = 1.f;
      if (grow) {
        float* rd = red + (it & 1) * 4 * NC;
        rd[c1 * 4 + hq * 2 + upper] = mx;
        asm volatile("bar.sync 1, %0;" ::"n"(kSoft5 * 32) : "memory");
        const float4 r1 = *reinterpret_cast<const float4*>(rd + c1 * 4);
        const float4 r2 = *reinterpret_cast<const float4*>(rd + (hq * 32 + lane) * 4);
        const float t1 = fmaxf(fmaxf(r1.x, r1.y), fmaxf(r1.z, r1.w));
        const float t2 = fmaxf(fmaxf(r2.x, r2.y), fmaxf(r2.z, r2.w));
        if (t1 > m1 + kRescale) {
          const float f1 = ex2(m1 - t1);                   // 0 when m1 = -inf
          l1 *= f1;
          lr1 *= f1;
          m1 = t1;
        }
        const bool g2 = t2 > m2 + kRescale;
        if (g2) {
          f2 = ex2(m2 - t2);
          m2 = t2;
        }
        left = __ballot_sync(0xffffffffu, g2);
        weights();
      }
      if (it > 0) {
        // P and, where a maximum grew, O^T are free once the tile before is done
        wait(&bar_o[bo], pho);
        fence_after();
        if (left != 0) {
          // the warp's lane quarter of O^T, all M tiles, its 32 columns
#pragma unroll 1
          for (; left != 0; left &= left - 1) {
            const int c = __ffs(left) - 1;
            const float fc = __shfl_sync(0xffffffffu, f2, c);
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              const uint32_t ta = tmem + lane_base + C::kColO + m * NC + hq * 32 + c;
              const uint32_t o = tmem_ld1_wait(ta);
              tmem_st1(ta, __float_as_uint(__uint_as_float(o) * fc));
            }
          }
          tmem_wait_st();
        }
      }
#pragma unroll
      for (int c8 = 0; c8 < 2; ++c8)
        *reinterpret_cast<uint4*>(prow + (((s0 / 8 + c8) ^ (c1 & 7)) << 4)) =
            make_uint4(pk[4 * c8], pk[4 * c8 + 1], pk[4 * c8 + 2], pk[4 * c8 + 3]);
      l1 += lt;
      lr1 += lrt;
      fence_before();
      arrive(bar_p);
      bo = buf;
      pho = ph;
      next(buf, ph);
    }
    red[((n & 1) * NC + c1) * 4 + hq * 2 + upper] = l1;
    // XCH was last read before the last tile's any_of_soft
    reinterpret_cast<float*>(sm + C::XCH)[c1 * 4 + hq * 2 + upper] = lr1;
    if (hq == 0 && upper == 0) m_run[c1] = m1;
  }
  // ---- the end: O^T to o or into shared memory as [column][channel] ------------------
  __syncthreads();
  if (n > 0) {
    if (warp < kConv5 + kSoft5) {
      wait(&bar_o[(n - 1) % 3], (unsigned)((n - 1) / 3) & 1u);
      fence_after();
    }
    if (tid < NC) {
      const float* rl = red + ((n & 1) * NC + tid) * 4;
      const float2 mine = make_float2(m_run[tid], (rl[0] + rl[1]) + (rl[2] + rl[3]));
      const float4 rr = *reinterpret_cast<const float4*>(sm + C::XCH + tid * 16);
      const float lr = (rr.x + rr.y) + (rr.z + rr.w);
      const float even = lr > 0.f ? __fdividef(mine.y, lr) : 1.f;   // sum as computed over sum as rounded
      if (cs == 1) {
        // the whole query: its sums with the sink, and each column's factor
        const int qi = per_group > 1 ? tid / a.H : 0, h = per_group > 1 ? tid - qi * a.H : tid;
        const bool live = qi < nq && h < heads;
        const float sink2 = live ? reinterpret_cast<const float*>(sm + C::SINK)[h] : -INFINITY;
        const float m = fmaxf(mine.x, sink2);
        float f = 0.f, out = -INFINITY;
        if (m > -INFINITY) {
          const float fm = ex2(mine.x - m), total = fmaf(mine.y, fm, ex2(sink2 - m));
          f = __fdividef(fm, total) * even;
          out = sink2 > -INFINITY && mine.y * fm == 0.f ? a.sink[h0 + h] : (m + log2f(total)) * kLn2;
        }
        m_run[tid] = f;
        if (live && !*dead) a.lse[(row0 + qi) * a.H + h0 + h] = out;
      } else {
        ml[tid] = make_float4(mine.x, mine.y, even, 0.f);
      }
    }
    __syncthreads();
    if (warp < kConv5 + kSoft5 && !*dead) {
      const int c0 = (warp >> 2) * 16, r = qd * 32 + lane; // 16 columns, channel of the M tile
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        uint32_t v[16];
        tmem_ld16_wait(tmem + lane_base + C::kColO + m * NC + c0, v);
        if (cs == 1) {
          store_o16<D, BITS>(v, m_run, c0, nq * heads,
                             (__nv_bfloat16*)a.o + (row0 * a.H + h0) * D, m * 128 + r);
        } else {
          const int ch = channel_of<BITS>(m * 128 + r);
          float* stage = reinterpret_cast<float*>(sm + C::STAGE);
#pragma unroll
          for (int c = 0; c < 16; ++c) stage[(c0 + c) * D + ch] = __uint_as_float(v[c]);
        }
      }
    }
    fence_before();
  }
  if (cs > 1) cg::this_cluster().sync();
  else __syncthreads();
  finish_decode<C, D, NC>(a, sm, *dead != 0, n, cs, rank, split, per_group, nq, heads, h0, row0);
  if (warp == kConv5 + kSoft5 && n > 0) free_tmem(tmem, 512, *dead != 0, bar_end);
  if (cs > 1) cg::this_cluster().sync();                   // no CTA leaves while another reads it
}

}  // namespace adt

namespace {

template <int BITS>
cudaError_t launch_512(const AttnDecodeArgs& a, const DecodePlan& p, cudaStream_t st) {
  using C = adt::Cfg512;
  const size_t smem = 1024 + C::kBytes;
  auto k = adt::attn_decode_512_kernel<BITS>;
  static SmemOnce once;
  const cudaError_t e = once(k, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int splits = p.cluster * p.parts;
  cfg.gridDim = dim3((unsigned)splits * (unsigned)(a.b * p.groups * p.head_groups));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, k, a, p.per_group, p.groups, p.head_groups, p.cluster, splits);
}

}  // namespace

cudaError_t launch_attn_decode_512(const AttnDecodeArgs& a, const DecodePlan& p, int bits,
                                   cudaStream_t st) {
  return bits == 4 ? launch_512<4>(a, p, st) : launch_512<8>(a, p, st);
}

}  // namespace csa
