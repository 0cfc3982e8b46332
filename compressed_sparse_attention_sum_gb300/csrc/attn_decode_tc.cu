// csa_attn_decode on the 5th-generation tensor cores (tcgen05 + TMEM): bf16
// queries, d in {64, 128, 256, 512}, cache of 4 or 8 bits (d = 512 with more than
// 32 columns: attn_decode_512.cu).
//
// Of one query, H rows of Q meet a few hundred to a thousand cached rows: the
// heads alone would fill a quarter to half of an M = 128 tile, so the products
// are formed transposed, with the slots (and then the channels) as M and the
// (query, head) columns as N:
//   S^T [slots, cols] = KV [slots, d] . Q^T          M = 128, N = NC, K = d
//   O^T [d, cols]    += KV^T [d, slots] . P^T        M = 128 channels a tile
// A CTA takes NC = 32 or 64 columns: the heads of one query or, when the
// queries of a sequence share their slots (no index list), of several.  Its
// slots come in tiles of 128; a query's tiles are split over the CTAs of a
// cluster, which join their results through each other's shared memory, and
// over several clusters where a row is long (attn_decode.cu joins those).
//
// The codes of a tile are fetched into registers while the tile before is in
// the softmax (its index entries and page ids one and two tiles earlier: each
// is a dependent read of global memory), expanded to bf16 (exact: a code has
// at most four significant bits) and stored once, 128-byte swizzled: read
// K-major the tile is the A operand of S^T, read MN-major that of O^T.  The
// expansion leaves a row's channels permuted within each eight
// (cache_expand.cuh): Q is permuted alike, and O is put back where it is
// stored.
//
// What bounds it: the latency of the chain index - page - codes - S - softmax -
// O - join (64 queries of 32 x 128, 8 bits, 5 tiles each: 12.2 us in a graph that
// finds its rows in L2, 14.4 us where it does not).
//
// The arithmetic is that of attn_tc512.cu: probabilities rounded to bf16 for the
// product with the values (the tensor core takes them so; each errs by at most
// 2^-8 of itself), two sums of them in fp32 and the running maximum in fp32,
// rescaling only when a column's maximum grows by more than 2^8.  LSE takes the
// sum as computed; O is divided by the sum as rounded, so that its weights add
// up to the rows' share and rounding errors that the slots have in common
// cancel.  The tensor core forms that sum: a product of P with ones, in the time
// in which the next tile is expanded (100 queries of 32 x 512 over 8 bits: 38.2 us
// with one sum, 38.7 with both; 41.7 with the second summed by the softmax
// threads, which takes 16 more registers).
#include "attn_decode.h"
#include "attn_decode_join.cuh"
#include "cache_expand.cuh"
#include "smem_once.h"

namespace csa {
namespace adt {

constexpr int kSlots = 128;
constexpr uint32_t kKvBlk = kSlots * 128;     // 64 channels of 128 slots

template <int D, int NC>
struct Cfg {
  static constexpr int kWarps = NC / 4;                    // lane quarter x 16 columns
  static constexpr int kCompute = kWarps * 32;
  static constexpr int kThreads = kCompute + 32;           // one more warp issues the MMAs
  static constexpr int kBound = (kThreads + 127) / 128 * 128;   // registers are given out to four warps at a time
  static constexpr int kBlocks = D < 128 ? 2 : D / 64;     // 64-channel blocks of the KV tile
  static constexpr int kMT = D < 128 ? 1 : D / 128;        // M tiles of O^T
  static constexpr int kPart = kMT < 2 ? 1 : 2;            // M tiles whose channels are handed over at once
  static constexpr int kParts = kMT / kPart;
  static constexpr int kGroups = D < 128 ? D / 32 : 4;     // scale groups of a row in one M tile
  static constexpr int kLanes = 8 * kGroups;               // lanes of eight slots
  static constexpr int kPerWarp = 8 * (32 / kLanes);       // slots a warp converts at once
  static constexpr int kPass = kPerWarp * kWarps;          // slots of one pass of all warps
  static constexpr int kSpt = kPass >= kSlots ? 1 : kSlots / kPass;   // slots of a thread
  static constexpr uint32_t kQBlk = NC * 128;
  static constexpr uint32_t kColO = 64;
  static constexpr uint32_t kColR = kColO + kMT * NC;      // sums of the rounded probabilities, alike in all lanes
  static constexpr uint32_t kColA = kColR + NC;            // ones: 16 elements of K
  static constexpr uint32_t kNeed = kColA + 8;
  static constexpr uint32_t kTmem = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t KV = (D / 64) * kQBlk;
  static constexpr uint32_t P = KV + kBlocks * kKvBlk;
  static constexpr uint32_t BARS = P + kSlots * 128;       // s, p, kv[kParts], o[kParts], end
  static constexpr uint32_t MISC = BARS + (3 + 2 * kParts) * 8;   // TMEM slot, dead
  static constexpr uint32_t RED = (MISC + 8 + 15) / 16 * 16;   // [2][4][NC] column maxima
  static constexpr uint32_t MRUN = RED + 8 * NC * 4;       // [2][NC]
  static constexpr uint32_t ML = MRUN + 2 * NC * 4;        // [NC] (maximum, sum, O's factor) of this CTA
  static constexpr uint32_t SINK = ML + NC * 16;           // [NC] sink logits of the heads (log2 units)
  static constexpr uint32_t OKS = SINK + NC * 4;           // [2][kSlots] bytes
  static constexpr uint32_t kBytes = OKS + 2 * kSlots;
  static constexpr uint32_t STAGE = KV;                    // [NC][D] O after the last tile
};

template <int D, int NC, int BITS>
__global__ void __launch_bounds__(Cfg<D, NC>::kBound, 1) attn_decode_tc_kernel(
    const AttnDecodeArgs a, int per_group, int groups, int cs) {
  using C = Cfg<D, NC>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* bar_p = bar_s + 1;
  uint64_t* bar_kv = bar_s + 2;
  uint64_t* bar_o = bar_kv + C::kParts;
  uint64_t* bar_end = bar_o + C::kParts;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::MISC);
  volatile int* dead = reinterpret_cast<int*>(sm + C::MISC + 4);
  float* red = reinterpret_cast<float*>(sm + C::RED);
  float* m_run = reinterpret_cast<float*>(sm + C::MRUN);
  float4* ml = reinterpret_cast<float4*>(sm + C::ML);
  unsigned char* oks = sm + C::OKS;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // blockIdx.x: split of the slots (the cs CTAs of a cluster are neighbours), y:
  // group of queries (per_group of one sequence), z: group of heads.  Divisions
  // only where there is something to divide: this code runs once, and fetching it
  // takes longer than its arithmetic (one query 7.3 -> 7.0 us).
  const int splits = gridDim.x, split = blockIdx.x, rank = split & (cs - 1);
  const int hg = blockIdx.z, qg = blockIdx.y;
  const int bi = groups == 1 ? qg : qg / groups, i0 = (qg - bi * groups) * per_group;
  const int nq = min(per_group, a.s_q - i0);
  const int h0 = hg * NC, heads = min(a.H - h0, per_group > 1 ? a.H : NC);   // heads of a query
  const long long row0 = (long long)bi * a.s_q + i0;

  // Q: column c is query i0 + c / H, head h0 + c % H; columns past them are zero.
  // The first reads leave before anything is waited for.
  constexpr int kQIter = (NC * (D / 8) + C::kThreads - 1) / C::kThreads;
  constexpr int kQBatch = kQIter < 8 ? kQIter : 8;
  uint4 qv[kQBatch];
  auto read_q = [&](int x0) {
#pragma unroll
    for (int x = 0; x < kQBatch; ++x) {
      const int e = tid + (x0 + x) * C::kThreads, c = e / (D / 8), ch = e - c * (D / 8);
      const int qi = per_group > 1 ? c / a.H : 0, h = per_group > 1 ? c - qi * a.H : c;
      qv[x] = make_uint4(0u, 0u, 0u, 0u);
      if (c < NC && qi < nq && h < heads)
        qv[x] = __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                                     ((row0 + qi) * a.H + h0 + h) * D + ch * 8));
    }
  };
  auto store_q = [&](int x0) {
#pragma unroll
    for (int x = 0; x < kQBatch; ++x) {
      const int e = tid + (x0 + x) * C::kThreads, c = e / (D / 8), ch = e - c * (D / 8);
      if (c < NC)
        *reinterpret_cast<uint4*>(sm + C::Q + (ch >> 3) * C::kQBlk + c * 128 +
                                  (((ch & 7) ^ (c & 7)) << 4)) = permute8<BITS>(qv[x]);
    }
  };
  read_q(0);
  // Test hook (csa_debug_arm_fault): with kSiteDecode armed the last split of each
  // query issues no product, so that the waits for the first run out with none in
  // flight.
  int armed = 0;
  if (warp == C::kWarps) armed = armed_fault(a.status);
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
  const int tiles = (slots + kSlots - 1) / kSlots;
  int it0 = 0, n = tiles;
  if (splits > 1) {                                        // tiles <= 2^18, splits <= 152
    it0 = (unsigned)tiles * (unsigned)split / (unsigned)splits;
    n = (int)((unsigned)tiles * (unsigned)(split + 1) / (unsigned)splits) - it0;
  }

  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_p, C::kWarps);
    mbar_init(bar_end, 1);
    for (int m = 0; m < C::kParts; ++m) {
      mbar_init(&bar_kv[m], C::kWarps);
      mbar_init(&bar_o[m], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *dead = 0;
  }
  if (warp == C::kWarps && n > 0) tmem_alloc(tmem_slot, C::kTmem);
  if (tid < NC) {
    m_run[tid] = -INFINITY;
    ml[tid] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    reinterpret_cast<float*>(sm + C::SINK)[tid] = sink_v;
  }

  // ---- the converting side's reads: index entry, page id, codes -----------------
  const int cgr = (lane >> 3) % C::kGroups;                // scale group this thread converts
  const int cslot = warp * C::kPerWarp + (lane / C::kLanes) * 8 + (lane & 7);
  const bool conv = warp < C::kWarps;
  int jraw[C::kSpt], lslot[C::kSpt], page[C::kSpt];
  Codes<BITS> cd[C::kSpt * C::kMT];
  const int32_t* raw_pages = a.raw_table + (long long)bi * a.P_raw;
  const int32_t* cmp_pages = a.cmp_table + (long long)bi * a.P_cmp;
  auto slot_of = [&](int it, int k) {                      // -1: past the tiles or the list
    const int s = (it0 + it) * kSlots + cslot + k * C::kPass;
    return it < n && cslot + k * C::kPass < kSlots && s < slots ? s : -1;
  };
  auto read_index = [&](int it) {
#pragma unroll
    for (int k = 0; k < C::kSpt; ++k) {
      const int s = slot_of(it, k);
      jraw[k] = s - wext;
      if (a.idx != nullptr) jraw[k] = __ldg(a.idx + row0 * a.K + max(s - wext, 0));
    }
  };
  auto read_page = [&](int it) {
#pragma unroll
    for (int k = 0; k < C::kSpt; ++k) {
      const int s = slot_of(it, k);
      const bool raw = s < wext;
      const int rs = ring0 + s >= ring ? ring0 + s - ring : ring0 + s;
      int x = raw ? (w0 + s >= 0 ? rs : -1) : (jraw[k] < last.vis ? jraw[k] : -1);
      if (s < 0) x = -1;
      lslot[k] = max(x, -1);
      page[k] = __ldg((raw || x < 0 ? raw_pages : cmp_pages) + (x < 0 ? 0 : page_index(a.cs, x)));
    }
  };
  auto fetch = [&](int it) {
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
#pragma unroll
    for (int k = 0; k < C::kSpt; ++k) {
      const bool inside = (unsigned)page[k] < (unsigned)a.cs.n_pages;
      const bool ok = lslot[k] >= 0 && inside;
      if (lslot[k] >= 0 && !inside) set_status(a.status, kDevCheck, kSiteCachePage);
      if (cgr == 0 && cslot + k * C::kPass < kSlots)
        oks[(it & 1) * kSlots + cslot + k * C::kPass] = ok;
      const int r = lslot[k] - page_index(a.cs, lslot[k]) * a.cs.page_size;
      const uint8_t* base = a.cache + page_base(a.cs, page[k]);
      const uint8_t* code = (ok ? base + row_code(a.cs, r) : zero) + cgr * (4 * BITS);
      const uint8_t* scale = ok ? base + row_scale(a.cs, r) : zero;
      uint32_t sw[C::kMT];                                 // the row's scale bytes, four a word
      if constexpr (C::kMT == 4) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(scale));
        sw[0] = w.x;
        sw[1] = w.y;
        sw[2] = w.z;
        sw[3] = w.w;
      } else if constexpr (C::kMT == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(scale));
        sw[0] = w.x;
        sw[1] = w.y;
      } else if constexpr (C::kGroups == 4) {
        sw[0] = __ldg(reinterpret_cast<const uint32_t*>(scale));
      } else {
        sw[0] = __ldg(reinterpret_cast<const uint16_t*>(scale));
      }
#pragma unroll
      for (int m = 0; m < C::kMT; ++m) {
        Codes<BITS>& c = cd[k * C::kMT + m];
#pragma unroll
        for (int e = 0; e < BITS / 4; ++e)
          c.w[e] = __ldg(reinterpret_cast<const uint4*>(code + m * (16 * BITS)) + e);
        c.scale = sw[m];                                   // this thread's byte is taken in convert
      }
    }
  };
  if (conv && n > 0) read_index(0);

  if (conv && n > 0) {
    read_page(0);
    read_index(1);
  }
  store_q(0);
#pragma unroll 1
  for (int x0 = kQBatch; x0 < kQIter; x0 += kQBatch) {
    read_q(x0);
    store_q(x0);
  }
  if (conv && n > 0) {
    fetch(0);
    read_page(1);
    read_index(2);
  }
  fence_proxy_async_smem();
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

  if (!conv) {
    // ---- the issuing warp ------------------------------------------------------
    // The tiles are written through the generic proxy and read through the async
    // one.  The proxy fence between stands on this side of the barriers, where one
    // thread executes it: it has to lie on the path from the write to the read, and
    // executed by all 16 writing warps it takes about 600 cycles each time.
    constexpr uint32_t idesc_s = idesc_bf16_f32_major(kSlots, NC, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16_f32_major(128, NC, 1, 1);
    constexpr uint32_t idesc_r = idesc_bf16_f32_major(128, NC, 0, 1);
    const uint64_t kvd = sw128_desc(smem_addr(sm + C::KV)), qd_s = sw128_desc(smem_addr(sm + C::Q));
    const uint64_t kvd_mn = sw128_desc_mn(smem_addr(sm + C::KV), kKvBlk);
    const uint64_t pd_mn = sw128_desc_mn(smem_addr(sm + C::P), kKvBlk);
    const uint32_t td = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    constexpr int kSteps = D < 128 ? D / 16 : 8;          // K steps of S^T in one M tile
    auto sum_p = [&](int it) {
#pragma unroll
      for (int k = 0; k < kSlots / 16; ++k)
        mma_bf16_ts(td + C::kColR, td + C::kColA, pd_mn + ((k * 2048) >> 4), idesc_r,
                    (it > 0 || k > 0) ? 1u : 0u);
    };
    bool up = armed != kSiteDecode || split != splits - 1;
    for (int it = 0; up && it < n; ++it) {
#pragma unroll
      for (int x = 0; x < C::kParts; ++x) {
        up = up && wait_warp(&bar_kv[x], it & 1);
        fence_proxy_async_smem();
        fence_after();
        if (up && elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kSteps * C::kPart; ++kk) {
            const int k = x * 8 * C::kPart + kk;
            mma_bf16_ss(td, kvd + (((k >> 2) * kKvBlk + (k & 3) * 32) >> 4),
                        qd_s + (((k >> 2) * C::kQBlk + (k & 3) * 32) >> 4), idesc_s,
                        k > 0 ? 1u : 0u);
          }
          if (x == C::kParts - 1) mma_commit(bar_s);
        }
        __syncwarp();
      }
      up = up && wait_warp(bar_p, it & 1);
      fence_proxy_async_smem();
      fence_after();
      if (up && elect_one()) {
#pragma unroll
        for (int x = 0; x < C::kParts; ++x) {
#pragma unroll
          for (int mm = 0; mm < C::kPart; ++mm) {
            const int m = x * C::kPart + mm;
#pragma unroll
            for (int k = 0; k < kSlots / 16; ++k)
              mma_bf16_ss(td + C::kColO + m * NC, kvd_mn + ((2 * m * kKvBlk + k * 2048) >> 4),
                          pd_mn + ((k * 2048) >> 4), idesc_o, (it > 0 || k > 0) ? 1u : 0u);
          }
          if (x == C::kParts - 1 && it == n - 1) sum_p(it);
          mma_commit(&bar_o[x]);
        }
        if (it < n - 1) sum_p(it);                         // complete with the next tile's S
      }
      __syncwarp();
    }
    __syncwarp();
  } else if (n > 0) {
    // ---- the converting and softmax warps --------------------------------------
    const int qd = warp & 3, hq = warp >> 2;
    const int r = qd * 32 + lane;                          // slot of S^T, channel of O^T
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    const float sc2 = a.scale * kLog2e;
    const int my_q = per_group > 1 ? (hq * 16) / a.H : 0;  // query of this thread's columns
    const int my_t = last.t - (nq - 1) + my_q;
    const int my_vis = min(my_t >= 0 ? (int)((unsigned)(my_t + 1) / (unsigned)a.ratio) : 0, last.vis);

    // One arrival a warp: 512 on one barrier take a thousand cycles.
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // Expands the fetched codes of tile it into the KV buffer, two M tiles at a
    // time; their channels are free once O^T of the tile before has read them.
    auto convert = [&](int it) {
#pragma unroll
      for (int x = 0; x < C::kParts; ++x) {
        // expanded in registers before the wait
        uint32_t o[C::kPart * C::kSpt][16];
#pragma unroll
        for (int e = 0; e < C::kPart * C::kSpt; ++e) {
          Codes<BITS> c = cd[(e % C::kSpt) * C::kMT + x * C::kPart + e / C::kSpt];
          c.scale = (c.scale >> (8 * cgr)) & 255u;
          expand_words<BITS>(c, o[e]);
        }
        if (it > 0) wait(&bar_o[x], (it - 1) & 1);
#pragma unroll
        for (int e = 0; e < C::kPart * C::kSpt; ++e) {
          const int m = x * C::kPart + e / C::kSpt, s = cslot + (e % C::kSpt) * C::kPass;
          if (s < kSlots)
            store_words(o[e], sm + C::KV + (uint32_t)(m * 2 + (cgr >> 1)) * kKvBlk + s * 128,
                        (cgr & 1) * 4, s & 7);
        }
        arrive(&bar_kv[x]);
      }
    };
    auto sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(C::kCompute) : "memory"); };

    float l_part[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) l_part[c] = 0.f;

    if (hq == 0) {
#pragma unroll 1
      for (int c = 0; c < 8; ++c) tmem_st1(tmem + lane_base + C::kColA + c, 0x3f803f80u);
      tmem_wait_st();
      fence_before();
    }

    convert(0);
    for (int it = 0; it < n; ++it) {
      const bool more = it + 1 < n;
      if (more) {
        fetch(it + 1);
        read_page(it + 2);
        read_index(it + 3);
      }
      wait(bar_s, it & 1);
      fence_after();
      // ---- softmax over the tile's slots, per column --------------------------
      // oks of this tile was written before the barrier of the tile before
      const int s = (it0 + it) * kSlots + r;
      bool ok = oks[(it & 1) * kSlots + r] != 0;
      if (s < wext) {
        const int pos = w0 + s;
        ok = ok && pos <= my_t && pos > my_t - a.window;
      } else {
        ok = ok && (a.idx != nullptr || s - wext < my_vis);
      }
      float x[16];
      {
        uint32_t v[16];
        tmem_ld16_wait(tmem + lane_base + hq * 16, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = ok ? __uint_as_float(v[c]) * sc2 : -INFINITY;
      }
      {
        float mx[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) mx[c] = x[c];
        const float m = lane_reduce16<true>(mx);
        if (lane < 16) red[((it & 1) * 4 + qd) * NC + hq * 16 + lane] = m;
      }
      sync();
      // lane c of every warp takes the new maximum of the warp's column c from the
      // four quarters; quarter 0 keeps it for the next tile
      float mt = -INFINITY, mo = -INFINITY;
      if (lane < 16) {
        const float* rq = red + (it & 1) * 4 * NC + hq * 16 + lane;
        mt = fmaxf(fmaxf(rq[0], rq[NC]), fmaxf(rq[2 * NC], rq[3 * NC]));
        mo = m_run[(it & 1) * NC + hq * 16 + lane];
      }
      const bool g = mt > mo + kRescale || (mo == -INFINITY && mt != -INFINITY);
      const float m_new = g ? mt : mo;
      if (qd == 0 && lane < 16) m_run[((it & 1) ^ 1) * NC + hq * 16 + lane] = m_new;
      const unsigned grow = __ballot_sync(0xffffffffu, g);
      if (grow != 0) {                                     // warp-uniform
        const float f = g ? ex2(mo - mt) : 1.f;            // 0 when mo = -inf
#pragma unroll
        for (int c = 0; c < 16; ++c) l_part[c] *= __shfl_sync(0xffffffffu, f, c);
        if (it > 0) {
#pragma unroll 1
          for (int m = 0; m <= C::kMT; ++m) {              // and the sums behind them
            const uint32_t ta = tmem + lane_base + C::kColO + m * NC + hq * 16;
#pragma unroll 1
            for (int c = 0; c < 16; ++c) {
              if (grow >> c & 1) {
                const uint32_t o = tmem_ld1_wait(ta + c);
                tmem_st1(ta + c, __float_as_uint(__uint_as_float(o) * __shfl_sync(0xffffffffu, f, c)));
              }
            }
          }
          tmem_wait_st();
        }
      }
      // P = 2^(x - m), masked slots 2^-inf = 0; a column without an unmasked
      // slot so far has m = -inf and takes 0 instead
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      unsigned char* prow = sm + C::P + r * 128;
#pragma unroll
      for (int c8 = 0; c8 < 2; ++c8) {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int c = c8 * 8 + e;
          const float p0 = ex2(x[c] - __shfl_sync(0xffffffffu, m_use, c));
          const float p1 = ex2(x[c + 1] - __shfl_sync(0xffffffffu, m_use, c + 1));
          l_part[c] += p0;
          l_part[c + 1] += p1;
          pk[e / 2] = pack_bf16x2(p0, p1);
        }
        *reinterpret_cast<uint4*>(prow + (((hq * 2 + c8) ^ (r & 7)) << 4)) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      fence_before();
      arrive(bar_p);
      if (more) convert(it + 1);
    }
#pragma unroll
    for (int x = 0; x < C::kParts; ++x) wait(&bar_o[x], (n - 1) & 1);
    fence_after();
    {
      const float l = lane_reduce16<false>(l_part);
      if (lane < 16) red[((n & 1) * 4 + qd) * NC + hq * 16 + lane] = l;
    }
    if (qd == 0) {
      uint32_t v[16];
      tmem_ld16_wait(tmem + C::kColR + hq * 16, v);
      // in the place of the last tile's maxima, which were read before bar_p of it
      float4* rr = reinterpret_cast<float4*>(red + ((n & 1) ^ 1) * 4 * NC + hq * 16);
      if (lane == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          rr[c] = make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]),
                              __uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
      }
    }
    sync();
    float2 mine = make_float2(-INFINITY, 0.f);
    float even = 1.f;                                      // sum as computed over sum as rounded
    if (tid < NC) {
      const float* rl = red + (n & 1) * 4 * NC + tid;
      mine = make_float2(m_run[(n & 1) * NC + tid], (rl[0] + rl[NC]) + (rl[2 * NC] + rl[3 * NC]));
      const float lr = red[((n & 1) ^ 1) * 4 * NC + tid];
      if (lr > 0.f) even = __fdividef(mine.y, lr);
    }
    if (cs == 1) {
      // the whole query: its sums with the sink, and each column's factor
      if (tid < NC) {
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
      }
      sync();
    } else if (tid < NC) {
      ml[tid] = make_float4(mine.x, mine.y, even, 0.f);
    }
    // O^T to o or into shared memory as [column][channel]: the KV tile's place
    if (!*dead) {
#pragma unroll 1
      for (int m = 0; m < C::kMT; ++m) {
        const int p = m * 128 + r;
        uint32_t v[16];
        tmem_ld16_wait(tmem + lane_base + C::kColO + m * NC + hq * 16, v);
        if (p < D) {
          if (cs == 1) {
            store_o16<D, BITS>(v, m_run, hq * 16, nq * heads,
                               (__nv_bfloat16*)a.o + (row0 * a.H + h0) * D, p);
          } else {
            const int ch = channel_of<BITS>(p);
            float* stage = reinterpret_cast<float*>(sm + C::STAGE);
#pragma unroll
            for (int c = 0; c < 16; ++c) stage[(hq * 16 + c) * D + ch] = __uint_as_float(v[c]);
          }
        }
      }
    }
    fence_before();
  }
  // ---- join ----------------------------------------------------------------------
  if (cs > 1) cg::this_cluster().sync();
  else __syncthreads();
  finish_decode<C, D, NC>(a, sm, *dead != 0, n, cs, rank, split, per_group, nq, heads, h0, row0);
  if (warp == C::kWarps && n > 0) free_tmem(tmem, C::kTmem, *dead != 0, bar_end);
  if (cs > 1) cg::this_cluster().sync();                   // no CTA leaves while another reads it
}

}  // namespace adt

namespace {

template <int D, int NC, int BITS>
cudaError_t launch_tc(const AttnDecodeArgs& a, const DecodePlan& p, cudaStream_t st) {
  using C = adt::Cfg<D, NC>;
  const size_t smem = 1024 + C::kBytes;
  auto k = adt::attn_decode_tc_kernel<D, NC, BITS>;
  static SmemOnce once;
  const cudaError_t e = once(k, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.cluster * p.parts), (unsigned)(a.b * p.groups), (unsigned)p.head_groups);
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
  return cudaLaunchKernelEx(&cfg, k, a, p.per_group, p.groups, p.cluster);
}

template <int D, int NC>
cudaError_t launch_tc_bits(const AttnDecodeArgs& a, int bits, const DecodePlan& p,
                           cudaStream_t st) {
  return bits == 4 ? launch_tc<D, NC, 4>(a, p, st) : launch_tc<D, NC, 8>(a, p, st);
}

template <int NC>
cudaError_t launch_tc_width(const AttnDecodeArgs& a, int bits, const DecodePlan& p,
                            cudaStream_t st) {
  switch (a.d) {
    case 64: return launch_tc_bits<64, NC>(a, bits, p, st);
    case 128: return launch_tc_bits<128, NC>(a, bits, p, st);
    case 256: return launch_tc_bits<256, NC>(a, bits, p, st);
    default:
      if constexpr (NC == 64) return launch_attn_decode_512(a, p, bits, st);
      else return launch_tc_bits<512, NC>(a, bits, p, st);
  }
}

}  // namespace

cudaError_t launch_attn_decode_tc(const AttnDecodeArgs& a, const DecodePlan& p, int bits,
                                  cudaStream_t st) {
  const cudaError_t e = p.cols == 32 ? launch_tc_width<32>(a, bits, p, st)
                                     : launch_tc_width<64>(a, bits, p, st);
  if (e != cudaSuccess || p.parts == 1) return e;
  return launch_attn_decode_combine(a, true, st);
}

}  // namespace csa
