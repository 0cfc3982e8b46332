// Indexer scores of csa_indexer_topk_decode on the 5th-generation tensor
// cores (tcgen05 + TMEM): bf16 queries, d_I 64 or 128.
//
// One token meets thousands of keys, so the keys are M:
//   S^T [keys, (query, head)] = K [128, d_I] . Q^T [cols, d_I]
// A CTA keeps the Q of up to 128 columns of one sequence (all heads of one
// query, or of several) in shared memory and walks every gridDim.x-th tile of
// 128 keys.  The codes of the next tile are fetched into registers while the
// present one is multiplied; a tile is expanded to bf16 once for all heads
// (exactly, cache_expand.cuh).  Two threads then own a key: each reads half of
// its row of S^T from TMEM and adds w_h ReLU(s) over those heads.
//
// What bounds it: expanding the codes and the weighted ReLU, in instructions
// issued; four CTAs on an SM hide each other's latency.  The tile's largest |k|
// and its range of scores go to the select.  Counting all tiles through and
// dealing them out evenly was slower (16 sequences 36 -> 42 us with the select:
// the count costs every CTA more than the uneven lengths do), as was a CTA of
// 128 threads, one a key.
#include "cache_expand.cuh"
#include "indexer_decode.h"
#include "smem_once.h"
#include "tcgen05.cuh"

namespace csa {
namespace idt {

using namespace csa::umma;

constexpr int kThreads = 256;            // two threads a key
constexpr int kSiteIndex = 0x74;
constexpr uint32_t kBlk = kIdxTile * 128;
constexpr float kNormSlack = 1.05f;       // the squares are summed 16 at a time in bf16

// Floats as signed integers of the same order (NaN beyond the infinities), and back.
__device__ __forceinline__ int float_order(float x) {
  const int u = __float_as_int(x);
  return u ^ ((u >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_float(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

template <int D, int NC>
struct Cfg {
  static constexpr int kGpt = D / 64;                    // scale groups of a thread: every other of a key
  static constexpr uint32_t kQBlk = NC * 128;
  static constexpr uint32_t K = (D / 64) * kQBlk;
  static constexpr uint32_t W = K + (D / 64) * kBlk;     // [NC] head weights
  static constexpr uint32_t BAR = W + NC * 4;
  static constexpr uint32_t MISC = BAR + 16;             // after the tiles' barrier and the end's: TMEM slot, dead
  static constexpr uint32_t BND = MISC + 8;              // [2][8], by tile parity
  static constexpr uint32_t RNG = BND + 64;              // [NC / 16][4] score ranges of the warps
  static constexpr uint32_t SUM = RNG + NC / 16 * 32;    // [2][NC / 16][128] half the heads' sums
  static constexpr uint32_t kBytes = SUM + 2 * (NC / 16) * kIdxTile * 4;
};

template <int D, int NC, int BITS>
__global__ void __launch_bounds__(kThreads, NC == 64 ? 4 : 3) index_scores_tc_kernel(const IndexDecodeArgs a,
                                                                   int per_group, int hpad) {
  using C = Cfg<D, NC>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* w_s = reinterpret_cast<float*>(sm + C::W);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::MISC);
  volatile int* dead = reinterpret_cast<int*>(sm + C::MISC + 4);
  int2* rng = reinterpret_cast<int2*>(sm + C::RNG);
  float* sums = reinterpret_cast<float*>(sm + C::SUM);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bi = blockIdx.y, i0 = blockIdx.z * per_group;
  const int nq = min(per_group, a.s_q - i0);
  const long long row0 = (long long)bi * a.s_q + i0;
  int most = 0;                                          // keys any query needs scores of
  for (int i = 0; i < nq; ++i) {
    const int v = index_vis(a, bi, i0 + i);
    if (v > a.topk) most = max(most, v);
  }
  const int tiles = (most + kIdxTile - 1) / kIdxTile;
  if ((int)blockIdx.x >= tiles) return;                  // CTA-uniform

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 1, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *dead = 0;
  }
  if (warp == 0) tmem_alloc(tmem_slot, NC);
  // Test hook (csa_debug_arm_fault): with kSiteIndex armed the first CTA of each
  // sequence issues no product, so that the wait for it runs out with none in flight.
  int armed = 0;
  if (tid == 0) armed = armed_fault(a.status);

  const int32_t* pages = a.table + (long long)bi * a.P;
  // Two threads expand a key: lane l and l + 16 of a warp, 16 keys a warp.
  const int cl = lane >> 4, ckey = warp * 16 + (lane & 15);
  // Page ids are read two tiles ahead and codes one, all of a step at once: a
  // dependent read of global memory takes as long as a tile's arithmetic.
  Codes<BITS> cd[C::kGpt];
  uint32_t scales = 0;                                   // of the key's groups, a byte each
  int page = 0;
  auto fetch_pages = [&](int tile) {
    page = __ldg(pages + page_index(a.cs, min(tile * kIdxTile + ckey, most - 1)));
  };
  auto fetch_codes = [&](int tile) {
    const int j = tile * kIdxTile + ckey;
    const bool ok = (unsigned)page < (unsigned)a.cs.n_pages;
    if (!ok) set_status(a.status, kDevCheck, kSiteCachePage);
    const int r = j - page_index(a.cs, j) * a.cs.page_size;
    const uint8_t* base = a.cache + page_base(a.cs, page);
    const bool live = ok && j < most;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
    const uint8_t* code = (live ? base + row_code(a.cs, r) : zero) + cl * (4 * BITS);
    const uint8_t* scale = live ? base + row_scale(a.cs, r) : zero;
#pragma unroll
    for (int k = 0; k < C::kGpt; ++k)
#pragma unroll
      for (int e = 0; e < BITS / 4; ++e)
        cd[k].w[e] = __ldg(reinterpret_cast<const uint4*>(code + k * (8 * BITS)) + e);
    if constexpr (D == 128) scales = __ldg(reinterpret_cast<const uint32_t*>(scale));
    else scales = __ldg(reinterpret_cast<const uint16_t*>(scale));
  };
  // Q: column c is query c / hpad, head c % hpad; the others are zero
  constexpr int kQChunks = NC * (D / 8) / kThreads;
  uint4 qv[kQChunks];
  float wv = 0.f;
  if (tid < NC) {
    const int qi = tid / hpad, h = tid - qi * hpad;
    if (qi < nq && h < a.H) wv = __ldg(a.w + (row0 + qi) * a.H + h);
  }
#pragma unroll
  for (int x = 0; x < kQChunks; ++x) {
    const int e = tid + x * kThreads, c = e / (D / 8), ch = e - c * (D / 8);
    const int qi = c / hpad, h = c - qi * hpad;
    qv[x] = make_uint4(0u, 0u, 0u, 0u);
    if (qi < nq && h < a.H)
      qv[x] = __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                                   ((row0 + qi) * a.H + h) * D + ch * 8));
  }
  fetch_pages(blockIdx.x);
  fetch_codes(blockIdx.x);
  fetch_pages(blockIdx.x + gridDim.x);
#pragma unroll
  for (int x = 0; x < kQChunks; ++x) {
    const int e = tid + x * kThreads, c = e / (D / 8), ch = e - c * (D / 8);
    *reinterpret_cast<uint4*>(sm + (ch >> 3) * C::kQBlk + c * 128 + (((ch & 7) ^ (c & 7)) << 4)) =
        permute8<BITS>(qv[x]);
  }
  if (tid < NC) w_s[tid] = wv;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const int half = warp >> 2, key_t = tid & 127;         // TMEM lane quarter: warp % 4
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;

  uint32_t parity = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    // ---- expand ----------------------------------------------------------------
    float norm2 = 0.f;                                   // |k|^2
#pragma unroll
    for (int k = 0; k < C::kGpt; ++k) {                  // group 2 k + cl
      uint32_t o[16];
      cd[k].scale = (scales >> (16 * k + 8 * cl)) & 255u;
      expand_words<BITS>(cd[k], o);
      store_words(o, sm + C::K + k * kBlk + ckey * 128, cl * 4, ckey & 7);
      float s = words_norm2(o);
      // squares of groups below 2^-40 may underflow
      if (cd[k].scale < 87u) s = fmaxf(s, 32.f * (BITS == 4 ? 36.f : 448.f * 448.f) * 0x1p-80f);
      norm2 += s;
    }
    norm2 += __shfl_xor_sync(0xffffffffu, norm2, 16);
    norm2 = warp_max(norm2);
    // by parity: the tile before is still read after its last barrier
    float* bnd = reinterpret_cast<float*>(sm + C::BND) + parity * 8;
    if (lane == 0) bnd[warp] = norm2;
    fence_proxy_async_smem();
    fence_before();
    __syncthreads();
    if (tid == 0 && (armed != kSiteIndex || blockIdx.x != 0)) {
      fence_after();
      constexpr uint32_t idesc = idesc_bf16_f32_major(kIdxTile, NC, 0, 0);
      const uint32_t ka = smem_addr(sm + C::K), qa = smem_addr(sm);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_bf16_ss(tmem, sw128_desc(ka + (k >> 2) * kBlk + (k & 3) * 32),
                    sw128_desc(qa + (k >> 2) * C::kQBlk + (k & 3) * 32), idesc, k > 0 ? 1u : 0u);
      mma_commit(bar);
    }
    if (tile + (int)gridDim.x < tiles) {
      fetch_codes(tile + gridDim.x);
      fetch_pages(tile + 2 * gridDim.x);
    }
    if (!mbar_wait(bar, parity)) *dead = 1;
    fence_after();
    // ---- sum_h w_h ReLU(s_h) for this thread's key, every other 16 heads ---------
#pragma unroll 1
    for (int q = 0; q < nq; ++q) {
      float t0 = 0.f, t1 = 0.f, t2 = 0.f, t3 = 0.f;
#pragma unroll 1
      for (int c0 = q * hpad + half * 16; c0 < (q + 1) * hpad; c0 += 32) {
        uint32_t v[16];
        tmem_ld16_wait(tmem + lane_base + c0, v);
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 w4 = *reinterpret_cast<const float4*>(w_s + c0 + c);
          fma_f32x2(t0, t1, pack_f32x2(w4.x, w4.y), fmaxf(__uint_as_float(v[c]), 0.f),
                    fmaxf(__uint_as_float(v[c + 1]), 0.f));
          fma_f32x2(t2, t3, pack_f32x2(w4.z, w4.w), fmaxf(__uint_as_float(v[c + 2]), 0.f),
                    fmaxf(__uint_as_float(v[c + 3]), 0.f));
        }
      }
      sums[(half * (NC / 16) + q) * kIdxTile + key_t] = (t0 + t1) + (t2 + t3);
    }
    fence_before();
    __syncthreads();                                     // sums; K and S are free
    const int j = tile * kIdxTile + key_t;
    for (int q = half; q < nq; q += 2) {
      float score = sums[q * kIdxTile + key_t] + sums[(NC / 16 + q) * kIdxTile + key_t];
      if (score != score) score = -INFINITY;             // the select's order has no NaN
      if (j < most && !*dead) a.scores[(row0 + q) * a.slots + j] = score;
      // the tile's range of scores, as ordered integers
      const int key = float_order(score);
      const int mn = __reduce_min_sync(0xffffffffu, j < most ? key : 0x7fffffff);
      const int mx = __reduce_max_sync(0xffffffffu, j < most ? key : (int)0x80000000);
      if (lane == 0) rng[q * 4 + (warp & 3)] = make_int2(mn, mx);
    }
    __syncthreads();                                     // rng
    if (tid < nq) {
      int2 r = rng[tid * 4];
#pragma unroll
      for (int k = 1; k < 4; ++k) {
        r.x = min(r.x, rng[tid * 4 + k].x);
        r.y = max(r.y, rng[tid * 4 + k].y);
      }
      float n2 = bnd[0];
#pragma unroll
      for (int k = 1; k < kThreads / 32; ++k) n2 = fmaxf(n2, bnd[k]);
      a.tile_info[(row0 + tid) * a.tiles + tile] =
          make_float4(sqrtf(n2) * kNormSlack, order_float(r.x), order_float(r.y), 0.f);
    }
    parity ^= 1;
    if (*dead) break;
  }
  if (tid == 0 && *dead) {
    set_status(a.status, kDevTimeout, kSiteIndex);
    // products may still run: wait for them, again with a limit, before TMEM is freed
    mma_commit(bar + 1);
    mbar_wait(bar + 1, 0);
  }
  __syncwarp();
  if (warp == 0) {
    fence_after();
    tmem_dealloc(tmem, NC);
  }
}

template <int D, int NC, int BITS>
cudaError_t launch(const IndexDecodeArgs& a, int per_group, int hpad, cudaStream_t st) {
  using C = Cfg<D, NC>;
  const size_t smem = 1024 + C::kBytes;
  auto k = index_scores_tc_kernel<D, NC, BITS>;
  static SmemOnce once;
  const cudaError_t e = once(k, smem);
  if (e != cudaSuccess) return e;
  const int groups = (a.s_q + per_group - 1) / per_group;
  // CTAs of a sequence: over all sequences half again as many as the four that
  // fit an SM, as those of shorter sequences find no tile
  long long g = (6ll * 152 + (long long)a.b * groups - 1) / ((long long)a.b * groups);
  g = g > a.tiles ? a.tiles : g;
  k<<<dim3((unsigned)g, a.b, groups), kThreads, smem, st>>>(a, per_group, hpad);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace idt

bool index_decode_tc_supported(int H, int d) { return (d == 64 || d == 128) && H <= 128; }

cudaError_t launch_index_scores_tc(const IndexDecodeArgs& a, int bits, cudaStream_t st) {
  const int hpad = (a.H + 15) / 16 * 16;
  // as many queries of a sequence as fit 128 columns share the expanded keys
  int pg = 128 / hpad;
  pg = pg > a.s_q ? a.s_q : pg;
  const bool wide = pg * hpad > 64;
#define CSA_IDX(D, NC)                                                                           \
  return bits == 4 ? idt::launch<D, NC, 4>(a, pg, hpad, st) : idt::launch<D, NC, 8>(a, pg, hpad, st)
  if (a.d == 64) {
    if (wide) CSA_IDX(64, 128);
    CSA_IDX(64, 64);
  }
  if (wide) CSA_IDX(128, 128);
  CSA_IDX(128, 64);
#undef CSA_IDX
}

}  // namespace csa
