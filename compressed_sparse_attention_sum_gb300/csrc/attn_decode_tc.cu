// csa_attn_decode on the 5th-generation tensor cores (tcgen05 + TMEM): bf16
// queries, d in {64, 128, 256, 512}, cache of 4 or 8 bits.
//
// Of one query, H rows of Q meet a few hundred to a thousand cached rows: the
// heads alone would fill a quarter to half of an M = 128 tile, so the products
// are formed transposed, with the slots (and then the channels) as M and the
// (query, head) columns as N:
//   S^T [slots, cols] = KV [slots, d] . Q^T          M = 128, N = NC, K = d
//   O^T [d, cols]    += KV^T [d, slots] . P^T        M = 128 channels a tile
// A CTA takes NC = 32 or 64 columns: the heads of one query or, when the
// queries of a sequence share their slots (no index list), of several.  Its
// slots come in tiles of 128; the split of a query's tiles over CTAs and their
// combination are those of attn_decode.cu.
//
// The codes of a tile are fetched into registers while the tile before is in
// the softmax, expanded to bf16 (exact: a code has at most four significant
// bits) and stored once, 128-byte swizzled: read K-major the tile is the A
// operand of S^T, read MN-major that of O^T.  The expansion leaves a row's
// channels permuted within each eight (cache_expand.cuh): Q is permuted alike,
// and O is put back where it is stored.
//
// What bounds it: at 64 heads x 512 the conversion of the codes (about three
// instructions a value) and the tensor core are alike in cost; at 32 x 128 the
// latency of the chain fetch - convert - S - softmax - O, which several CTAs
// on an SM overlap.  The arithmetic follows attn_fwd_tc512: probabilities in
// bf16, their sum and the running maximum in fp32, rescaling only when a
// column's maximum grows by more than 2^8.
#include "attn_decode.h"
#include "cache_expand.cuh"
#include "tcgen05.cuh"

namespace csa {
namespace adt {

using namespace csa::umma;

constexpr int kSlots = 128;
constexpr float kRescale = 8.f;
constexpr int kSiteDecode = 0x73;
constexpr uint32_t kKvBlk = kSlots * 128;     // 64 channels of 128 slots

template <int D, int NC>
struct Cfg {
  static constexpr int kWarps = NC / 4;                    // lane quarter x 16 columns
  static constexpr int kCompute = kWarps * 32;
  static constexpr int kThreads = kCompute + 32;           // one more warp issues the MMAs
  static constexpr int kBlocks = D < 128 ? 2 : D / 64;     // 64-channel blocks of the KV tile
  static constexpr int kMT = D < 128 ? 1 : D / 128;        // M tiles of O^T
  static constexpr int kGroups = D < 128 ? D / 32 : 4;     // scale groups of a row in one M tile
  static constexpr int kLanes = 8 * kGroups;               // lanes of eight slots
  static constexpr int kPerWarp = 8 * (32 / kLanes);       // slots a warp converts at once
  static constexpr int kPass = kPerWarp * kWarps;          // slots of one pass of all warps
  static constexpr int kSpt = kPass >= kSlots ? 1 : kSlots / kPass;   // slots of a thread
  static constexpr uint32_t kQBlk = NC * 128;
  static constexpr uint32_t kColO = 64;
  static constexpr uint32_t kNeed = kColO + kMT * NC;
  static constexpr uint32_t kTmem = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t KV = (D / 64) * kQBlk;
  static constexpr uint32_t P = KV + kBlocks * kKvBlk;
  static constexpr uint32_t BARS = P + kSlots * 128;       // s, p, kv[kMT], o[kMT]
  static constexpr uint32_t MISC = BARS + (2 + 2 * kMT) * 8;   // TMEM slot, dead, rescale
  static constexpr uint32_t RED = MISC + 16;               // [4][NC]
  static constexpr uint32_t MRUN = RED + 4 * NC * 4;
  static constexpr uint32_t FAC = MRUN + NC * 4;
  static constexpr uint32_t OKS = FAC + NC * 4;            // [2][kSlots] bytes
  static constexpr uint32_t kBytes = OKS + 2 * kSlots;
};

// Transposing butterfly: v[c] holds this lane's value of column c; afterwards
// lanes l and l + 16 hold op over all 32 lanes of column l % 16.
template <bool kMax>
__device__ __forceinline__ float lane_reduce16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 8, n = 8; off >= 1; off >>= 1, n >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      const float keep = up ? v[i + n] : v[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, off);
      v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  const float other = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return kMax ? fmaxf(v[0], other) : v[0] + other;
}

template <int D, int NC, int BITS>
__global__ void __launch_bounds__(Cfg<D, NC>::kThreads) attn_decode_tc_kernel(
    const AttnDecodeArgs a, int per_group, int groups, int head_groups) {
  using C = Cfg<D, NC>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* bar_p = bar_s + 1;
  uint64_t* bar_kv = bar_s + 2;
  uint64_t* bar_o = bar_kv + C::kMT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::MISC);
  volatile int* dead = reinterpret_cast<int*>(sm + C::MISC + 4);
  int* rescale = reinterpret_cast<int*>(sm + C::MISC + 8);
  float* red = reinterpret_cast<float*>(sm + C::RED);
  float* m_run = reinterpret_cast<float*>(sm + C::MRUN);
  float* fac = reinterpret_cast<float*>(sm + C::FAC);
  unsigned char* oks = sm + C::OKS;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // group of queries (per_group of one sequence) and of heads
  const int hg = (int)blockIdx.x % head_groups;
  const int qg = (int)blockIdx.x / head_groups;
  const int bi = qg / groups, i0 = (qg - bi * groups) * per_group;
  const int nq = min(per_group, a.s_q - i0);
  const int h0 = hg * NC, heads = min(a.H - h0, per_group > 1 ? a.H : NC);   // heads of a query
  const long long row0 = (long long)bi * a.s_q + i0;
  const int split = blockIdx.y;

  // The slots: the union window of the group's queries, then the index
  // entries (one query) or the blocks the last query sees.
  const DecodeRow last = decode_row(a, bi, i0 + nq - 1);
  const int wext = a.window + nq - 1;
  const int w0 = last.t - wext + 1;
  const int ring = a.P_raw * a.cs.page_size;
  const int ring0 = w0 >= 0 ? w0 % ring : ring - 1 - (int)((unsigned)(-1 - w0) % (unsigned)ring);
  const int slots = last.t < 0 ? 0 : wext + (a.idx != nullptr ? a.K : last.vis);
  const int tiles = (slots + kSlots - 1) / kSlots;
  const int it0 = (int)((long long)tiles * split / a.splits);
  const int n = (int)((long long)tiles * (split + 1) / a.splits) - it0;

  if (tid == 0) {
    mbar_init(bar_s, 1);
    mbar_init(bar_p, C::kCompute);
    for (int m = 0; m < C::kMT; ++m) {
      mbar_init(&bar_kv[m], C::kCompute);
      mbar_init(&bar_o[m], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *dead = 0;
  }
  if (warp == C::kWarps && n > 0) tmem_alloc(tmem_slot, C::kTmem);
  if (tid < NC) m_run[tid] = -INFINITY;
  // Q: column c is query i0 + c / H, head h0 + c % H; columns past them are zero
  for (int e = tid; e < NC * (D / 8); e += C::kThreads) {
    const int c = e / (D / 8), ch = e - c * (D / 8);
    const int qi = per_group > 1 ? c / a.H : 0, h = per_group > 1 ? c - qi * a.H : c;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (qi < nq && h < heads)
      v = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                          ((row0 + qi) * a.H + h0 + h) * D + ch * 8);
    *reinterpret_cast<uint4*>(sm + C::Q + (ch >> 3) * C::kQBlk + c * 128 +
                              (((ch & 7) ^ (c & 7)) << 4)) = permute8<BITS>(v);
  }
  fence_proxy_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = n > 0 ? *tmem_slot : 0u;

  // A wait that gives up ends every later wait of the CTA at once.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*dead) return false;
    if (mbar_wait(bar, parity)) return true;
    *dead = 1;
    return false;
  };

  if (warp == C::kWarps) {
    // ---- the issuing warp ------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32_major(kSlots, NC, 0, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32_major(128, NC, 1, 1);
      const uint32_t kva = smem_addr(sm + C::KV), qa = smem_addr(sm + C::Q);
      const uint32_t pa = smem_addr(sm + C::P);
      constexpr int kSteps = D < 128 ? D / 16 : 8;        // K steps of S^T in one M tile
      for (int it = 0; it < n; ++it) {
#pragma unroll 1
        for (int m = 0; m < C::kMT; ++m) {
          if (!wait(&bar_kv[m], it & 1)) break;
          fence_after();
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
            const int k = m * 8 + kk;
            mma_bf16_ss(tmem, sw128_desc(kva + (k >> 2) * kKvBlk + (k & 3) * 32),
                        sw128_desc(qa + (k >> 2) * C::kQBlk + (k & 3) * 32), idesc_s,
                        k > 0 ? 1u : 0u);
          }
        }
        if (*dead) break;
        mma_commit(bar_s);
        if (!wait(bar_p, it & 1)) break;
        fence_after();
#pragma unroll 1
        for (int m = 0; m < C::kMT; ++m) {
#pragma unroll
          for (int k = 0; k < kSlots / 16; ++k)
            mma_bf16_ss(tmem + C::kColO + m * NC, sw128_desc_mn(kva + 2 * m * kKvBlk + k * 2048, kKvBlk),
                        sw128_desc_mn(pa + k * 2048, kKvBlk), idesc_o, (it > 0 || k > 0) ? 1u : 0u);
          mma_commit(&bar_o[m]);
        }
      }
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
    const int cg = (lane >> 3) % C::kGroups;               // scale group this thread converts
    const int cslot = warp * C::kPerWarp + (lane / C::kLanes) * 8 + (lane & 7);

    const uint8_t* code_p[C::kSpt];
    const uint8_t* scale_p[C::kSpt];                       // null: masked
    Codes<BITS> cd[C::kSpt * C::kMT];

    auto locate = [&](int it) {
#pragma unroll
      for (int k = 0; k < C::kSpt; ++k) {
        const int s = (it0 + it) * kSlots + cslot + k * C::kPass;
        long long code = 0, scale = 0;
        bool ok = false;
        if (it < n && cslot + k * C::kPass < kSlots && s < slots) {
          if (s < wext) {
            const int pos = w0 + s;
            int slot = ring0 + s;                          // ring0 + s < 2 ring
            slot -= slot >= ring ? ring : 0;
            if (pos >= 0)
              ok = cache_row(a.cs, a.raw_table + (long long)bi * a.P_raw, slot, &code, &scale,
                             a.status);
          } else {
            const int j = a.idx != nullptr ? a.idx[row0 * a.K + s - wext] : s - wext;
            if (j >= 0 && j < last.vis)
              ok = cache_row(a.cs, a.cmp_table + (long long)bi * a.P_cmp, j, &code, &scale,
                             a.status);
          }
        }
        code_p[k] = a.cache + code + cg * (4 * BITS);
        scale_p[k] = ok ? a.cache + scale + cg : nullptr;
      }
    };
    auto fetch = [&]() {
#pragma unroll
      for (int k = 0; k < C::kSpt; ++k)
#pragma unroll
        for (int m = 0; m < C::kMT; ++m) {
          Codes<BITS>& c = cd[k * C::kMT + m];
          c.clear();
          if (scale_p[k] != nullptr) c.load(code_p[k] + m * (16 * BITS), scale_p[k] + m * 4);
        }
    };
    // Expands the fetched codes of tile it into the KV buffer; M tile m's
    // channels are free once O^T of the tile before has read them.
    auto convert = [&](int it) {
      if (cg == 0) {
#pragma unroll
        for (int k = 0; k < C::kSpt; ++k)
          if (cslot + k * C::kPass < kSlots)
            oks[(it & 1) * kSlots + cslot + k * C::kPass] = scale_p[k] != nullptr;
      }
#pragma unroll
      for (int m = 0; m < C::kMT; ++m) {
        if (it > 0) wait(&bar_o[m], (it - 1) & 1);
#pragma unroll
        for (int k = 0; k < C::kSpt; ++k) {
          const int s = cslot + k * C::kPass;
          if (s >= kSlots) continue;
          const Codes<BITS>& c = cd[k * C::kMT + m];
          unsigned char* dst = sm + C::KV + (uint32_t)(m * 2 + (cg >> 1)) * kKvBlk + s * 128;
          expand_group<BITS>(c, dst, (cg & 1) * 4, s & 7);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar_kv[m]);
      }
    };
    auto sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(C::kCompute) : "memory"); };

    float l_part[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) l_part[c] = 0.f;

    locate(0);
    fetch();
    convert(0);
    locate(1);
    for (int it = 0; it < n; ++it) {
      const bool more = it + 1 < n;
      if (more) fetch();
      sync();                                              // oks of this tile, rescale flag free
      if (tid == 0) *rescale = 0;
      wait(bar_s, it & 1);
      fence_after();
      // ---- softmax over the tile's slots, per column --------------------------
      const int s = (it0 + it) * kSlots + r;
      bool ok = oks[(it & 1) * kSlots + r] != 0;
      if (s < wext) {
        const int pos = w0 + s;
        ok = ok && pos <= my_t && pos > my_t - a.window;
      } else {
        ok = ok && (a.idx != nullptr || s - wext < my_vis);
      }
      const float bias = ok ? 0.f : -INFINITY;
      float x[16];
      {
        uint32_t v[16];
        tmem_ld16_wait(tmem + lane_base + hq * 16, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = fmaf(__uint_as_float(v[c]), sc2, bias);
      }
      {
        float mx[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) mx[c] = x[c];
        const float m = lane_reduce16<true>(mx);
        if (lane < 16) red[qd * NC + hq * 16 + lane] = m;
      }
      sync();
      if (tid < NC) {
        const float mt = fmaxf(fmaxf(red[tid], red[NC + tid]), fmaxf(red[2 * NC + tid], red[3 * NC + tid]));
        const float mo = m_run[tid];
        float f = 1.f;
        if (mt > mo + kRescale || (mo == -INFINITY && mt != -INFINITY)) {
          f = ex2(mo - mt);                                // 0 when mo = -inf
          m_run[tid] = mt;
          if (it > 0) *rescale = 1;
        }
        fac[tid] = f;
      }
      sync();
      if (*rescale) {
#pragma unroll
        for (int c = 0; c < 16; ++c) l_part[c] *= fac[hq * 16 + c];
#pragma unroll 1
        for (int m = 0; m < C::kMT; ++m) {
          const uint32_t ta = tmem + lane_base + C::kColO + m * NC + hq * 16;
          uint32_t v[16];
          tmem_ld16_wait(ta, v);
#pragma unroll
          for (int c = 0; c < 16; ++c)
            tmem_st1(ta + c, __float_as_uint(__uint_as_float(v[c]) * fac[hq * 16 + c]));
        }
        tmem_wait_st();
      }
      unsigned char* prow = sm + C::P + r * 128;
#pragma unroll
      for (int c8 = 0; c8 < 2; ++c8) {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int c = c8 * 8 + e;
          // a column without an unmasked slot so far has m = -inf: no mass
          const float m0 = m_run[hq * 16 + c], m1 = m_run[hq * 16 + c + 1];
          const float p0 = ok ? ex2(x[c] - m0) : 0.f;
          const float p1 = ok ? ex2(x[c + 1] - m1) : 0.f;
          l_part[c] += p0;
          l_part[c + 1] += p1;
          pk[e / 2] = pack_bf16x2(p0, p1);
        }
        *reinterpret_cast<uint4*>(prow + (((hq * 2 + c8) ^ (r & 7)) << 4)) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      fence_proxy_async_smem();
      fence_before();
      mbar_arrive(bar_p);
      if (more) {
        convert(it + 1);
        locate(it + 2);
      }
    }
#pragma unroll
    for (int m = 0; m < C::kMT; ++m) wait(&bar_o[m], (n - 1) & 1);
    fence_after();
    {
      const float l = lane_reduce16<false>(l_part);
      if (lane < 16) red[qd * NC + hq * 16 + lane] = l;
    }
    sync();
    if (tid < NC) {
      const float l = (red[tid] + red[NC + tid]) + (red[2 * NC + tid] + red[3 * NC + tid]);
      const int qi = per_group > 1 ? tid / a.H : 0, h = per_group > 1 ? tid - qi * a.H : tid;
      const bool live = qi < nq && h < heads && !*dead;
      const long long row = row0 + qi;
      if (a.splits > 1) {
        if (live) a.part_ml[(row * a.splits + split) * a.H + h0 + h] = make_float2(m_run[tid], l);
        fac[tid] = 1.f;
      } else {
        const float sink2 = a.sink != nullptr && live ? a.sink[h0 + h] * kLog2e : -INFINITY;
        const float m = m_run[tid], mm = fmaxf(m, sink2);
        float f = 0.f, out = -INFINITY;
        if (mm > -INFINITY) {
          const float fm = exp2f(m - mm), total = fmaf(l, fm, exp2f(sink2 - mm));
          f = fm / total;
          out = (mm + log2f(total)) * kLn2;
        }
        fac[tid] = f;
        if (live) a.lse[row * a.H + h0 + h] = out;
      }
    }
    sync();
    if (!*dead) {
#pragma unroll 1
      for (int m = 0; m < C::kMT; ++m) {
        const int p = m * 128 + r;
        uint32_t v[16];
        tmem_ld16_wait(tmem + lane_base + C::kColO + m * NC + hq * 16, v);
        if (p < D) {
          const int ch = channel_of<BITS>(p);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int col = hq * 16 + c;
            const int h = per_group > 1 ? col - my_q * a.H : col;
            if (my_q < nq && h < heads) {
              const float val = __uint_as_float(v[c]) * fac[col];
              const long long row = row0 + my_q;
              if (a.splits > 1)
                a.part_o[((row * a.splits + split) * a.H + h0 + h) * D + ch] = val;
              else
                ((__nv_bfloat16*)a.o)[(row * a.H + h0 + h) * D + ch] = __float2bfloat16_rn(val);
            }
          }
        }
      }
    }
    fence_before();
  } else {
    // no tile: an empty part of a split, or a query with nothing to attend to
    for (int c = tid; c < NC; c += C::kCompute) {
      const int qi = per_group > 1 ? c / a.H : 0, h = per_group > 1 ? c - qi * a.H : c;
      if (qi >= nq || h >= heads) continue;
      const long long rh = (row0 + qi) * a.H + h0 + h;
      if (a.splits > 1)
        a.part_ml[((row0 + qi) * a.splits + split) * a.H + h0 + h] = make_float2(-INFINITY, 0.f);
      else
        a.lse[rh] = a.sink != nullptr ? a.sink[h0 + h] : -INFINITY;
    }
    if (a.splits == 1) {
      for (int e = tid; e < nq * heads * (D / 8); e += C::kCompute) {
        const int c = e / (D / 8), qi = c / heads, h = c - qi * heads;
        *reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + ((row0 + qi) * a.H + h0 + h) * D +
                                  (e - c * (D / 8)) * 8) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *dead) set_status(a.status, kDevTimeout, kSiteDecode);
  if (warp == C::kWarps && n > 0) {
    fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

}  // namespace adt

namespace {

template <int D, int NC, int BITS>
cudaError_t launch_tc(const AttnDecodeArgs& a, int per_group, int groups, int head_groups,
                      cudaStream_t st) {
  using C = adt::Cfg<D, NC>;
  const size_t smem = 1024 + C::kBytes;
  auto k = adt::attn_decode_tc_kernel<D, NC, BITS>;
  const cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k<<<dim3((unsigned)(a.b * groups * head_groups), a.splits), C::kThreads, smem, st>>>(
      a, per_group, groups, head_groups);
  count_launches(1);
  return cudaGetLastError();
}

template <int D, int NC>
cudaError_t launch_tc_bits(const AttnDecodeArgs& a, int bits, int pg, int g, int hg,
                           cudaStream_t st) {
  return bits == 4 ? launch_tc<D, NC, 4>(a, pg, g, hg, st) : launch_tc<D, NC, 8>(a, pg, g, hg, st);
}

template <int NC>
cudaError_t launch_tc_width(const AttnDecodeArgs& a, int bits, int pg, int g, int hg,
                            cudaStream_t st) {
  switch (a.d) {
    case 64: return launch_tc_bits<64, NC>(a, bits, pg, g, hg, st);
    case 128: return launch_tc_bits<128, NC>(a, bits, pg, g, hg, st);
    case 256: return launch_tc_bits<256, NC>(a, bits, pg, g, hg, st);
    default: return launch_tc_bits<512, NC>(a, bits, pg, g, hg, st);
  }
}

}  // namespace

cudaError_t launch_attn_decode_tc(const AttnDecodeArgs& a, int bits, cudaStream_t st) {
  const DecodePlan p = decode_plan_tc(a.b, a.s_q, a.H, a.d, a.window, a.idx != nullptr ? a.K : 0,
                                      a.idx == nullptr, (long long)a.P_cmp * a.cs.page_size);
  const cudaError_t e = p.cols == 32
                            ? launch_tc_width<32>(a, bits, p.per_group, p.groups, p.head_groups, st)
                            : launch_tc_width<64>(a, bits, p.per_group, p.groups, p.head_groups, st);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_attn_decode_combine(a, true, st);
}

}  // namespace csa
