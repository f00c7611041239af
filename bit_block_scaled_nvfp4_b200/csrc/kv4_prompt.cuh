// Attention of many query rows per KV head over the 4-bit cache: prompts and chunks of prompts.
//
// Mathematics as in kv4_split.cuh (exact products of Q with K, FP32 scores, online softmax,
// P = fp16(2^(s - m + 6)), FP32 O and l) on the 16-bit tensor cores of tcgen05. Q is taken as it is and K
// decoded into Q's type, fp16 or bf16, exactly either way; V is decoded to fp16. The running maximum that P and O refer to follows the true one only when it
// has risen by more than 2^8 (so P stays below 2^14): O in tensor memory is rarely rescaled.
//
// A work item is a KV head of a sequence and up to 256 query rows of it, rows being (token, head of
// the group): two units of 128 rows (128 / g tokens, rounded down), one softmax warpgroup each,
// which share every decoded K and V tile of 128 keys. Bound: tensor cores and exponentials, 2048
// cycles a tile each (16.8 MFLOP; 32768 exponentials at 16 a cycle), and next to them shared
// memory: 3 x 64 KB read by the products and 64 KB written by the decoding, 2048 cycles at 128
// bytes a cycle. P stays in tensor memory (as the A operand, over its own scores).
//
// The key tiles of all items form one line, cut into equal ranges, one a CTA (kv4_range), whatever
// the lengths and however few the rows; an item that crosses CTAs leaves partials.
//
// Roles (512 threads): warp 0 issues the products, warps 1-3 bring in Q, warps 4-7 decode K and V
// pages from global memory (prefetched into registers a tile ahead) into the tensor cores'
// 128-byte-swizzled layout, warps 8-11 and 12-15 are the units' softmax.
// TMEM (512 columns): S_0, S_1 (P_u in the first 64 columns of S_u), O_0, O_1.
#pragma once
#include "kv4_split.cuh"

namespace qk4v8 {

constexpr float kRiseLimit = 8.f;                        // log2 of how far the maximum may rise unfollowed
constexpr int kPromptPartFloats = 256 * (kKv4D + 2);     // a partial: O, then m, then l of 256 rows

// sum over i < n of floor((a i + b) / 128)
__device__ __forceinline__ int64_t floor_sum128(int64_t n, int64_t a, int64_t b) {
  int64_t m = 128, ans = 0;
  while (true) {
    if (a >= m) { ans += (n - 1) * n / 2 * (a / m); a %= m; }
    if (b >= m) { ans += n * (b / m); b %= m; }
    const int64_t y = a * n + b;
    if (y < m) return ans;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
}
// A sequence's items per KV head: T2 tokens each, and the key tiles (128 keys) each of them sees.
struct PromptSeq {
  Kv4Seq q;
  int T2;
  __device__ __forceinline__ int items() const { return (q.n + T2 - 1) / T2; }
  __device__ __forceinline__ int tiles_to(int tok) const { return (q.ctx - q.n + tok + 127) >> 7; }  // seen by tokens < tok
  __device__ __forceinline__ int tiles(int i) const { return tiles_to(min(q.n, (i + 1) * T2)); }
  __device__ __forceinline__ int64_t before(int i) const {          // tiles of the items before item i
    const int last = items();
    const int64_t k = i < last ? i : last - 1;
    const int64_t s = k > 0 ? floor_sum128(k, T2, static_cast<int64_t>(q.ctx - q.n) + T2 + 127) : 0;
    return i < last ? s : s + tiles(last - 1);
  }
};

// A CTA's part of an item, as the scheduling warp hands it to the others.
struct PromptSeg {
  int s, h, q0, n, ctx;                                  // sequence, KV head; its first row, tokens, context
  int tok;                                               // the item's first token
  int j0, len;                                           // its key tiles j0 .. j0 + len - 1
  int mine0, mine1;                                      // how many of them unit 0 and 1 see
  int whole, first;                                      // the whole item; it begins here
};                                                       // (s = -1: no more)
struct PromptLayout {
  static constexpr int OFF_Q = 0;                        // [unit] 2 x 16 KB (64 channels each)
  static constexpr int OFF_K = 65536;                    // [stage] 2 x 16 KB (64 channels each)
  static constexpr int OFF_V = OFF_K + 65536;            // [stage] 2 x 16 KB (64 tokens each)
  static constexpr int OFF_MAP = OFF_V + 65536;          // [128] a row's token and head within the unit
  static constexpr int OFF_FLAG = OFF_MAP + 256;        // [8] pages missing, by tile
  static constexpr int OFF_RANGE = OFF_FLAG + 32;
  static constexpr int OFF_BAR = OFF_RANGE + (sizeof(Kv4Range) + 7) / 8 * 8;
  static constexpr int NSEG = 4;                         // segments handed out ahead
  static constexpr int N_BARS = 17 + 2 * NSEG;
  static constexpr int OFF_SEG = (OFF_BAR + N_BARS * 8 + 16 + 15) / 16 * 16;
  static constexpr int SMEM_BYTES = OFF_SEG + NSEG * 64;
  static_assert(sizeof(PromptSeg) <= 64, "a segment's slot");
  static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
  static constexpr uint32_t T_S = 0, T_O = 256;          // + 128 for unit 1
  static constexpr int THREADS = 512;
  static constexpr int REGS_LAUNCH = 128, REGS_ISSUE = 80, REGS_DECODE = 80, REGS_SOFTMAX = 176;
  static_assert(REGS_ISSUE + REGS_DECODE + 2 * REGS_SOFTMAX <= 4 * REGS_LAUNCH, "register split");
};
struct PromptWalk {
  PromptSeq sq;
  int s, h, i, j, left;
  __device__ __forceinline__ void find(const Kv4AttnArgs& a) {
    const int group = a.Hq / a.c.Hkv;
    for (; s < a.S; ++s) {
      sq.q = kv4_seq(a, s, false);
      if (sq.q.n * group > a.rows_max) return;
    }
    left = 0;
  }
  __device__ __forceinline__ void start(const Kv4AttnArgs& a, const Kv4Range* r) {
    sq.T2 = 2 * (128 / (a.Hq / a.c.Hkv));
    s = r->s;
    left = r->left;
    h = i = j = 0;
    find(a);
    if (left <= 0) return;
    const int64_t head = sq.before(sq.items());
    h = static_cast<int>(r->first / head);
    int64_t at = r->first - h * head;
    int lo = 0, hi = sq.items() - 1;                     // the last item with before(item) <= at
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (sq.before(m) <= at) lo = m; else hi = m - 1;
    }
    i = lo;
    j = static_cast<int>(at - sq.before(lo));
  }
  __device__ __forceinline__ bool next(const Kv4AttnArgs& a, PromptSeg& g) {
    if (left <= 0) return false;
    const int nt = sq.tiles(i), j1 = min(nt, j + left), TU = sq.T2 / 2;
    g.s = s; g.h = h; g.q0 = sq.q.q0; g.n = sq.q.n; g.ctx = sq.q.ctx;
    g.tok = i * sq.T2;
    g.j0 = j; g.len = j1 - j;
    const int nt0 = sq.tiles_to(min(sq.q.n, g.tok + TU));
    const int nt1 = g.tok + TU < sq.q.n ? nt : 0;
    g.mine0 = max(0, min(j1, nt0) - j);
    g.mine1 = max(0, min(j1, nt1) - j);
    g.whole = j == 0 && j1 == nt;
    g.first = j == 0;
    left -= j1 - j;
    j = 0;
    if (left > 0 && ++i == sq.items()) {
      i = 0;
      if (++h == a.c.Hkv) {
        h = 0;
        ++s;
        find(a);
      }
    }
    return true;
  }
};

// A block's scale times pairs of E2M1 values (as half2) in Q's type, exactly: in bf16 as
// (value 2^-112) (scale 2^112), both and the product normal.
template <typename T> struct KScale;
template <> struct KScale<__half> {
  __half2 f;
  __device__ __forceinline__ explicit KScale(float s) : f(__float2half2_rn(s)) {}
  __device__ __forceinline__ uint32_t times(uint32_t h) const { return hmul2(h, f); }
};
template <> struct KScale<__nv_bfloat16> {
  __nv_bfloat162 f;
  __device__ __forceinline__ explicit KScale(float s) : f(__float2bfloat162_rn(s * 0x1p112f)) {}
  __device__ __forceinline__ uint32_t times(uint32_t h) const {
    // the exponent field kept, fp16's bias of 15 read as bf16's of 127
    const uint32_t b = ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), f);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
// 16-byte asynchronous copy, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(copy ? 16 : 0)
               : "memory");
}
template <typename T>
__global__ void __launch_bounds__(512, 1) kv4_prompt_kernel(Kv4AttnArgs a) {
  using L = PromptLayout;
  extern __shared__ __align__(128) unsigned char kv4_smem[];
  unsigned char* sm = kv4_smem + ((1024u - (smem_u32(kv4_smem) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
  uint64_t* q_full = bars;                               // Q of the segment is in place
  uint64_t* q_empty = bars + 1;                          // its last QK^T is done
  uint64_t* k_full = bars + 2;                           // [2]
  uint64_t* k_empty = bars + 4;                          // [2]
  uint64_t* v_full = bars + 6;                           // [2]
  uint64_t* v_empty = bars + 8;                          // [2]
  uint64_t* s_full = bars + 10;                          // [unit] scores ready; all PVs before them done
  uint64_t* p_full = bars + 12;                          // [unit] P written, S read, O ready to add to
  uint64_t* o_full = bars + 14;                          // [unit] the segment's last PV is done
  uint64_t* mma_final = bars + 16;
  uint64_t* seg_full = bars + 17;                        // [NSEG]
  uint64_t* seg_empty = seg_full + L::NSEG;              // [NSEG]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Kv4Range* rng = reinterpret_cast<Kv4Range*>(sm + L::OFF_RANGE);
  volatile int* missing = reinterpret_cast<volatile int*>(sm + L::OFF_FLAG);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.Hq / a.c.Hkv;

  uchar2* row_map = reinterpret_cast<uchar2*>(sm + L::OFF_MAP);
  if (threadIdx.x < 128) row_map[threadIdx.x] = make_uchar2(threadIdx.x / group, threadIdx.x % group);
  if (threadIdx.x == 0) {
    mbar_init(q_full, 2);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_full + i, 1);
    }
    mbar_init(mma_final, 1);
    for (int i = 0; i < L::NSEG; ++i) {
      mbar_init(seg_full + i, 1);
      mbar_init(seg_empty + i, 1 + 2 + 4 + 8);           // products, Q, decoding, softmax
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  kv4_range<L::THREADS>(
      [&](int i) -> int64_t {
        PromptSeq s;
        s.q = kv4_seq(a, i, blockIdx.x == 0);
        s.T2 = 2 * (128 / group);
        return s.q.n * group > a.rows_max ? s.before(s.items()) * a.c.Hkv : 0;
      },
      a.S, 2, a.prompt_plan, rng);
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  auto seg_at = [&](int seg) -> const PromptSeg& {
    return *reinterpret_cast<const PromptSeg*>(sm + L::OFF_SEG + (seg % L::NSEG) * 64);
  };
  const int TU = 128 / group;                            // tokens of a unit
  const uint32_t role = warp == 0 ? kRoleMma : warp < 8 ? kRoleProducer : kRoleSoftmax;
  auto site = [&](uint64_t* bar, int tile) {
    return wait_site(kKernelKv4Prompt, role, static_cast<uint32_t>(bar - bars), tile);
  };
  auto waitw = [&](uint64_t* bar, uint32_t parity, int tile) -> bool {
    return bounded_wait_warp(bar, parity, abort_flag, site(bar, tile));
  };

  if (warp < 4) {
    setmaxnreg_to<L::REGS_ISSUE, L::REGS_LAUNCH>();
    if (warp == 0) {
      // ======================= products (one thread) =======================
      if (lane == 0) {
        auto wait1 = [&](uint64_t* bar, uint32_t parity, int tile) -> bool {
          return bounded_wait(bar, parity, abort_flag, site(bar, tile));
        };
        constexpr uint32_t idesc_qk = idesc_f16(128, 128, std::is_same<T, __nv_bfloat16>::value);
        constexpr uint32_t idesc_pv = idesc_f16(128, 128);
        // descriptors of the first blocks; an offset of n bytes adds n / 16
        const uint64_t dQ = make_sdesc(smem_u32(sm + L::OFF_Q), 16, 1024, kSw128);
        const uint64_t dK = make_sdesc(smem_u32(sm + L::OFF_K), 16, 1024, kSw128);
        const uint64_t dV = make_sdesc(smem_u32(sm + L::OFF_V), 16, 1024, kSw128);
        auto qk = [&](int u, int tile) {                 // S_u = Q_u K^T
          const uint64_t q = dQ + u * 2048, k = dK + (tile & 1) * 2048;
          const uint32_t tS = tbase + L::T_S + u * 128;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16(tS, q + (kk >> 2) * 1024 + (kk & 3) * 2, k + (kk >> 2) * 1024 + (kk & 3) * 2, idesc_qk, kk > 0 ? 1u : 0u);
          mma_commit(s_full + u);
        };
        auto pv = [&](int u, int tile, bool first) {     // O_u += P_u V
          const uint64_t v = dV + (tile & 1) * 2048;
          const uint32_t tS = tbase + L::T_S + u * 128, tO = tbase + L::T_O + u * 128;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ta(tO, tS + kk * 8, v + (kk >> 2) * 1024 + (kk & 3) * 2, idesc_pv, (first && kk == 0) ? 0u : 1u);
        };
        int tile = 0;
        uint32_t odd = 0;                                // bit u: unit u's tiles so far, odd or even
        bool ok = true;
        for (int seg = 0;; ++seg) {
          ok = wait1(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1, tile);
          if (!ok) break;
          const int len = seg_at(seg).len, mine0 = seg_at(seg).mine0, mine1 = seg_at(seg).mine1;
          const bool end = seg_at(seg).s < 0;
          mbar_arrive(seg_empty + seg % L::NSEG);
          if (end) break;
          ok = wait1(q_full, seg & 1, tile) && wait1(k_full + (tile & 1), (tile >> 1) & 1, tile);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < 2; ++u)
            if ((u ? mine1 : mine0) > 0) qk(u, tile);
          mma_commit(k_empty + (tile & 1));
          if (len == 1) mma_commit(q_empty);
          for (int t = 0; t < len && ok; ++t, ++tile) {
            bool v_in = false, k_in = false;
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
              const int mine = u ? mine1 : mine0;
              if (t < mine) {
                ok = wait1(p_full + u, (odd >> u) & 1, tile) &&
                     (v_in || wait1(v_full + (tile & 1), (tile >> 1) & 1, tile));
                if (!ok) break;
                v_in = true;
                tc_fence_after();
                pv(u, tile, t == 0);
                odd ^= 1u << u;
                if (t + 1 == mine) mma_commit(o_full + u);
              }
              if (t + 1 < mine) {
                ok = k_in || wait1(k_full + ((tile + 1) & 1), ((tile + 1) >> 1) & 1, tile);
                if (!ok) break;
                k_in = true;
                tc_fence_after();
                qk(u, tile + 1);
              }
            }
            if (!ok) break;
            if (t + 1 < len) mma_commit(k_empty + ((tile + 1) & 1));
            if (t + 2 == len) mma_commit(q_empty);
            mma_commit(v_empty + (tile & 1));
          }
          if (!ok) break;
        }
        mma_commit(mma_final);
        mbar_wait(mma_final, 0);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ============================ segments (one thread) ============================
      if (lane == 0) {
        PromptWalk walk;
        walk.start(a, rng);
        bool more = true;
        for (int seg = 0; more; ++seg) {
          if (seg >= L::NSEG && !bounded_wait(seg_empty + seg % L::NSEG, (seg / L::NSEG - 1) & 1, abort_flag,
                                              site(seg_empty + seg % L::NSEG, seg)))
            break;
          PromptSeg g;
          more = walk.next(a, g);
          if (!more) g.s = -1;
          *reinterpret_cast<PromptSeg*>(sm + L::OFF_SEG + (seg % L::NSEG) * 64) = g;
          mbar_arrive(seg_full + seg % L::NSEG);
        }
      }
      __syncwarp();
    } else {
      // ================================ Q ================================
      // Copied as it is, half a warp a row, 16 bytes a thread; rows without a token are zero. The
      // eights of channels are stored in K's order (see the decoding).
      const int hw = lane >> 4, ch = lane & 15;
      const int pos = ((ch & 8) << 11) | (((ch & 7) ^ ((ch & 8) >> 2)) << 4);
      for (int seg = 0;; ++seg) {
        if (!waitw(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1, seg)) break;
        const PromptSeg& g = seg_at(seg);
        if (g.s < 0) break;
        const int left = g.n - g.tok;                    // tokens from the item's first on
        const T* q = static_cast<const T*>(a.q) + (g.q0 + g.tok) * a.q_stride + g.h * group * kKv4D + ch * 8;
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + seg % L::NSEG);
        // the last segment's products have read Q
        if (seg > 0 && !waitw(q_empty, (seg - 1) & 1, seg)) break;
#pragma unroll 4
        for (int r = (warp - 1) * 2 + hw; r < 256; r += 4) {
          const int ru = r & 127;
          const uchar2 at = row_map[ru];
          const int tok = (r >> 7) * TU + at.x;
          const bool real = ru < TU * group && tok < left;
          cp_async16_or_zero(sm + L::OFF_Q + (r >> 7) * 32768 + ru * 128 + (pos ^ ((ru & 7) << 4)),
                             real ? q + tok * a.q_stride + at.y * kKv4D : q, real);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
    }
  } else if (warp < 8) {
    setmaxnreg_to<L::REGS_DECODE, L::REGS_LAUNCH>();
    // ============================ K and V decoding ============================
    // K: thread (token row, quarter of the channels): four words of eight channels become four
    // 16-byte chunks. Of the upper 64 channels, chunks 2 c and 2 c + 1 trade places with
    // 2 (c ^ 1) and 2 (c ^ 1) + 1, so that the eight threads of two rows write eight different
    // 16-byte banks; Q has the same order.
    // V: thread (page, eight tokens, 16 channels): four token pairs of a channel are a chunk.
    const int tid = threadIdx.x - 128;
    const int kr = tid >> 2, kq = tid & 3;
    const int vp = tid >> 6, vt = tid & 7, vb = (tid >> 3) & 7;
    bool ok = true;
    int tile = 0;
    // prefetched: the next tile's page ids, its K and (after K) its V
    uint4 kc[4], vc[4];
    uint32_t ks[4];
    uint2 vs;
    int v_left;                                          // this thread's V slots that lie in the context
    // the tile at hand, and the next one's segment and place
    int id0 = -1, id1 = -1, h = 0, ctx = 0, j = 0;
    int seg = -1, jn = 0, j_end = 0;
    // steps to the next tile: its page ids; false when there is none
    auto next_tile = [&](int& p0, int& p1) -> bool {
      if (++jn >= j_end) {
        if (seg >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(seg_empty + seg % L::NSEG);
        }
        ++seg;
        if (!waitw(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1, tile) || seg_at(seg).s < 0) return false;
        jn = seg_at(seg).j0;
        j_end = jn + seg_at(seg).len;
      }
      // the second page may lie behind the context: the first again then, with no slot that counts
      const int32_t* row = a.table + static_cast<int64_t>(seg_at(seg).s) * a.max_pages;
      const int np = (seg_at(seg).ctx + 63) >> 6;
      p0 = __ldg(row + 2 * jn);
      p1 = __ldg(row + min(2 * jn + 1, np - 1));
      return true;
    };
    auto valid = [&](int id) { return id >= 0 && id < a.c.num_pages; };
    auto load_k = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int id = i < 2 ? id0 : id1, row = (i & 1) * 32 + kr;
        kc[i] = make_uint4(0, 0, 0, 0);
        ks[i] = 0;
        if (valid(id)) {
          const int64_t tok = (static_cast<int64_t>(id) * a.c.Hkv + h) * 64 + row;
          kc[i] = __ldg(reinterpret_cast<const uint4*>(a.c.k_pages + tok * 64 + kq * 16));
          ks[i] = __ldg(reinterpret_cast<const uint16_t*>(a.c.k_scales + tok * 8 + kq * 2));
        }
      }
    };
    auto load_v = [&]() {
      const int id = vp ? id1 : id0;
#pragma unroll
      for (int i = 0; i < 4; ++i) vc[i] = make_uint4(0, 0, 0, 0);
      vs = make_uint2(0, 0);
      if (valid(id)) {
        const int64_t head = static_cast<int64_t>(id) * a.c.Hkv + h;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vc[i] = __ldg(reinterpret_cast<const uint4*>(a.c.v_pages + (head * 32 + vt * 4 + i) * 128 + vb * 16));
        vs = __ldg(reinterpret_cast<const uint2*>(a.c.v_scales + (head * 8 + vb) * 64 + vt * 8));
      }
      v_left = ctx - (j * 128 + vp * 64 + vt * 8);
    };
    int n0 = -1, n1 = -1;                                // page ids of the tile after
    bool more = next_tile(id0, id1);
    if (more) {
      h = seg_at(seg).h; ctx = seg_at(seg).ctx; j = jn;
      load_k();
    }
    while (more && ok) {
      const int stg = tile & 1;
      const bool after = next_tile(n0, n1);
      // ---- K ----
      if (tile >= 2 && !waitw(k_empty + stg, ((tile >> 1) - 1) & 1, tile)) { ok = false; break; }
      load_v();
      if (tid == 0) {
        const int gone = (valid(id0) ? 0 : 1) | (valid(id1) ? 0 : 2);
        missing[tile & 7] = gone;
        if (gone) flag_error(kStatusBounds);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 32 + kr;
        const __half2 sc = e4m3x2_to_half2(ks[i]);
        const KScale<T> f0(__low2float(sc)), f1(__high2float(sc));
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&kc[i]);
        unsigned char* row = sm + L::OFF_K + stg * 32768 + (kq >> 1) * 16384 + r * 128;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t d[4];
          e2m1x8_to_half2(w[e], d);
#pragma unroll
          for (int x = 0; x < 4; ++x) d[x] = e < 2 ? f0.times(d[x]) : f1.times(d[x]);
          const int chunk = ((kq & 1) * 4 + (e ^ (kq & 2))) ^ (r & 7);
          *reinterpret_cast<uint4*>(row + chunk * 16) = make_uint4(d[0], d[1], d[2], d[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + stg);
      // ---- V, with the next tile's K on its way ----
      id0 = n0; id1 = n1;
      if (after) {
        h = seg_at(seg).h; ctx = seg_at(seg).ctx; j = jn;
        load_k();
      }
      if (tile >= 2 && !waitw(v_empty + stg, ((tile >> 1) - 1) & 1, tile)) { ok = false; break; }
      {
        if (v_left < 8) {                                // slots behind it: value 0 (weight 0 x NaN is not 0)
          const uint64_t keep = v_left <= 0 ? 0 : (1ull << (8 * v_left)) - 1;
          vs.x &= static_cast<uint32_t>(keep);
          vs.y &= static_cast<uint32_t>(keep >> 32);
        }
        const __half2 f[4] = {e4m3x2_to_half2(vs.x & 0xFFFFu), e4m3x2_to_half2(vs.x >> 16),
                              e4m3x2_to_half2(vs.y & 0xFFFFu), e4m3x2_to_half2(vs.y >> 16)};
        unsigned char* base = sm + L::OFF_V + stg * 32768 + vp * 16384 + vb * 16 * 128;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t d[4][4];                              // [token pair][channel]
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e2m1x8_to_half2(reinterpret_cast<const uint32_t*>(&vc[i])[e], d[i]);
#pragma unroll
            for (int x = 0; x < 4; ++x) d[i][x] = hmul2(d[i][x], f[i]);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int cc = e * 4 + x;
            *reinterpret_cast<uint4*>(base + cc * 128 + ((vt ^ (cc & 7)) << 4)) = make_uint4(d[0][x], d[1][x], d[2][x], d[3][x]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full + stg);
      more = after;
      ++tile;
    }
  } else {
    setmaxnreg_to<L::REGS_SOFTMAX, L::REGS_LAUNCH>();
    // ================================ softmax ================================
    const int wq = warp & 3, unit = (warp - 8) >> 2, row = wq * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + L::T_S + unit * 128 + lane_addr, tO = tbase + L::T_O + unit * 128 + lane_addr;
    const float C = *a.c.k_ts * a.softmax_scale * kLog2e;
    bool ok = true;
    int tile = 0, n = 0, n_o = 0;                        // tiles; of this unit; segments with any
    for (int seg = 0;; ++seg) {
      if (!waitw(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1, tile)) break;
      const PromptSeg& g = seg_at(seg);
      if (g.s < 0) break;
      const int mine = unit == 0 ? g.mine0 : g.mine1;
      const int t0 = g.tok + unit * TU;
      const int lim = g.ctx - g.n + t0 + row_map[row].x - g.j0 * 128;   // the last key seen, from the segment's first
      const int lim_min = g.ctx - g.n + t0 - g.j0 * 128; // the last key that every row of the unit sees, likewise
      float m_ref = -INFINITY;
      float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      for (int t = 0; t < mine; ++t, ++n) {
        if (!waitw(s_full + unit, n & 1, n)) { ok = false; break; }
        tc_fence_after();
        float x[128];
        {
          uint32_t* xr = reinterpret_cast<uint32_t*>(x);
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32(tS + c, xr + c);
          tmem_wait_ld();
        }
        const int gone = missing[(tile + t) & 7];
        if (t * 128 + 127 > lim_min) {
          const int last = lim - t * 128;
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = c <= last ? x[c] : -INFINITY;
        }
        if (gone) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (gone & (c < 64 ? 1 : 2)) x[c] = -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], x[c + 2 * k], x[c + 2 * k + 1]);
        }
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * C;
        // a row's first keys, or a rise past the limit: the reference follows
        if (__any_sync(0xffffffffu, mt > m_ref + kRiseLimit)) {
          const float m_new = fmaxf(m_ref, mt);
          if (t > 0) {
            const float al = m_new == -INFINITY ? 1.f : ex2_approx(m_ref - m_new);
            const float2 A = make_float2(al, al);
            l2[0] = __fmul2_rn(l2[0], A);
            l2[1] = __fmul2_rn(l2[1], A);
#pragma unroll
            for (int c = 0; c < 128; c += 8) {            // a few columns at a time: the scores are live
              uint32_t o[8];
              tmem_ld8(tO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; k += 2) {
                const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), A);
                o[k] = __float_as_uint(v.x);
                o[k + 1] = __float_as_uint(v.y);
              }
              tmem_st8(tO + c, o);
            }
          }
          m_ref = m_new;
        }
        const float bias = kPShift - (m_ref == -INFINITY ? 0.f : m_ref);
        const float2 C2 = make_float2(C, C), B2 = make_float2(bias, bias);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float2 e = __ffma2_rn(make_float2(x[c + k], x[c + k + 1]), C2, B2);
            e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            l2[(k >> 1) & 1] = __fadd2_rn(l2[(k >> 1) & 1], e);
            p[k >> 1] = pack_half2(e.x, e.y);
          }
          tmem_st16(tS + c / 2, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + unit);
      }
      if (!ok) break;
      tile += g.len;
      // ---- O of the segment ----
      const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
      if (mine > 0) {
        if (!waitw(o_full + unit, n_o & 1, n)) { ok = false; break; }
        ++n_o;
        tc_fence_after();
      }
      const uchar2 at = row_map[row];
      const int tok = t0 + at.x;
      const bool real = row < TU * group && tok < g.n;
      const bool whole = g.whole;
      float* part = a.prompt_part + static_cast<int64_t>(2 * blockIdx.x + (g.first ? 1 : 0)) * kPromptPartFloats;
      const int64_t orow = static_cast<int64_t>(g.q0 + tok) * a.Hq + g.h * group + at.y;
      __syncwarp();
      if (lane == 0) mbar_arrive(seg_empty + seg % L::NSEG);
      const float f = l == 0.f ? 0.f : *a.c.v_ts / l;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_ld32(tO + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (!real) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * kKv4D + c);
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            dst[k >> 3] = make_uint4(pack2<T>(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f),
                                     pack2<T>(__uint_as_float(o[k + 2]) * f, __uint_as_float(o[k + 3]) * f),
                                     pack2<T>(__uint_as_float(o[k + 4]) * f, __uint_as_float(o[k + 5]) * f),
                                     pack2<T>(__uint_as_float(o[k + 6]) * f, __uint_as_float(o[k + 7]) * f));
        } else {
          uint4* dst = reinterpret_cast<uint4*>(part + (unit * 128 + row) * kKv4D + c);
#pragma unroll
          for (int k = 0; k < 32; k += 4) dst[k >> 2] = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      if (real) {
        if (!whole) {
          part[256 * kKv4D + unit * 128 + row] = m_ref;
          part[256 * (kKv4D + 1) + unit * 128 + row] = l;
        } else if (a.lse != nullptr) {
          a.lse[orow] = l == 0.f ? -INFINITY : (m_ref + log2f(l) - kPShift) * kLn2;
        }
      }
      tc_fence_before();                                 // O's reads precede the next segment's first P
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the partials of items that cross CTAs. CTA (i, y) takes the item that CTA i - 1 of the prompt
// kernel began and CTA i went on with, if any, and rows 32 y ..; a warp takes four rows, a lane four
// channels.
template <typename T>
__global__ void __launch_bounds__(256) kv4_prompt_merge_kernel(Kv4AttnArgs a) {
  const int cta = blockIdx.x + 1, group = a.Hq / a.c.Hkv;
  const int64_t per = a.prompt_plan[0], at = per * cta;
  int lo = 0, hi = a.S - 1;                              // the last sequence that begins at or before `at`
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (a.prompt_plan[1 + m] <= at) lo = m; else hi = m - 1;
  }
  PromptSeq sq;
  sq.T2 = 2 * (128 / group);
  sq.q = kv4_seq(a, lo, false);
  if (sq.q.n * group <= a.rows_max) return;              // `at` is behind the last unit
  const int64_t head = sq.before(sq.items()), in = at - a.prompt_plan[1 + lo];
  const int h = static_cast<int>(in / head);
  if (h >= a.c.Hkv) return;
  const int64_t r = in - h * head;
  int i0 = 0, i1 = sq.items() - 1;
  while (i0 < i1) {
    const int m = (i0 + i1 + 1) >> 1;
    if (sq.before(m) <= r) i0 = m; else i1 = m - 1;
  }
  const int64_t first = at - (r - sq.before(i0));        // the item's first unit
  if (first == at || first / per != cta - 1) return;     // not cut here, or not here first
  const int c1 = static_cast<int>((first + sq.tiles(i0) - 1) / per);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, TU = sq.T2 / 2;
  auto part = [&](int c) {
    return a.prompt_part + static_cast<int64_t>(2 * c + (c == cta - 1 ? 1 : 0)) * kPromptPartFloats;
  };
  for (int k = 0; k < 4; ++k) {
    const int row = blockIdx.y * 32 + warp * 4 + k, ru = row & 127;
    const int tok = i0 * sq.T2 + (row >> 7) * TU + ru / group;
    if (ru >= TU * group || tok >= sq.q.n) continue;
    float M = -INFINITY;
    for (int c = cta - 1; c <= c1; ++c) M = fmaxf(M, part(c)[256 * kKv4D + row]);
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = cta - 1; c <= c1; ++c) {
      const float* p = part(c);
      const float w = ex2_approx(p[256 * kKv4D + row] - mu);
      const float4 v = *reinterpret_cast<const float4*>(p + row * kKv4D + lane * 4);
      l += w * p[256 * (kKv4D + 1) + row];
      acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    }
    const float f = l == 0.f ? 0.f : *a.c.v_ts / l;
    const int64_t orow = static_cast<int64_t>(sq.q.q0 + tok) * a.Hq + h * group + ru % group;
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + orow * kKv4D + lane * 4) =
        make_uint2(pack2<T>(acc.x * f, acc.y * f), pack2<T>(acc.z * f, acc.w * f));
    if (a.lse != nullptr && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l) - kPShift) * kLn2;
  }
}

}  // namespace qk4v8
