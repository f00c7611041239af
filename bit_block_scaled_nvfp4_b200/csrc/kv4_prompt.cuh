// Attention of many query rows per KV head over the 4-bit cache: prompts and chunks of prompts.
//
// Mathematics as in kv4_split.cuh (Q to fp16 by a power of two per row, K and V decoded exactly to
// fp16, FP32 scores, online softmax, P = fp16(2^(s - m + 6)), FP32 O and l) on the fp16 tensor cores of
// tcgen05. The running maximum that P and O refer to follows the true one only when it
// has risen by more than 2^8 (so P stays below 2^14): O in tensor memory is rarely rescaled.
//
// A work item is a KV head of a sequence and up to 256 query rows of it, rows being (token, head of
// the group): two units of 128 rows (128 / g tokens, rounded down), one softmax warpgroup each,
// which share every decoded K and V tile of 128 keys. Bound: tensor cores and exponentials, 2048
// cycles a tile each (16.8 MFLOP; 32768 exponentials at 16 a cycle), and next to them shared
// memory: 3 x 64 KB read by the products and 64 KB written by the decoding, 2048 cycles at 128
// bytes a cycle. P stays in tensor memory (as the A operand).
//
// The key tiles of all items form one line, cut into equal ranges, one a CTA (kv4_range), whatever
// the lengths and however few the rows; an item that crosses CTAs leaves partials.
//
// Measured as graphs, 32 query and 8 KV heads: 16384 tokens 2.19 ms (1.00 PFLOP/s, 61 % of the measured bf16 rate), 512
// tokens after 32000 cached 279 us (0.97 PFLOP/s). A tile of two units takes about 3900 cycles: the
// softmax warps are busy for 1690 of a half tile's 1930 (exponentials of two warps an SM quarter, 1024, behind them
// the maximum, the packing and the decoding warps' share of the issue slots). With one unit of rows (a few proposed
// tokens) a tile still takes about 3300: the decoding of its pages, by one pair of warps for K and one for V, is then
// what takes longest.
//
// Roles (512 threads): warps 0 and 2 issue the products of unit 0 and 1 (one warp for both left the tensor
// cores waiting while it waited: 323 us a chunk of 512 tokens at 32512, 293 with two), warp 1 hands out
// the work and loads Q (TMA), warps 4 and 5 decode K and 6 and 7 V, page by page, into the tensor cores'
// 128-byte-swizzled layout, warps 8-11 and 12-15 are the units' softmax; warp 3 has none.
// TMEM (512 columns): S_0, S_1 (two half tiles of 64 keys each; P of a half over its first 32 columns), O_0, O_1. The
// scores of a half are issued as soon as the product with the P in its place is, so that a unit always has
// one half's scores waiting while its softmax works on the other's.
#pragma once
#include "kv4_split.cuh"

namespace qk4v8 {

constexpr float kRiseLimit = 8.f;                        // log2 of how far the maximum may rise unfollowed
constexpr int kPromptPartFloats = 256 * (kKv4D + 2);     // a partial: O, then m, then l of 256 rows

// sum over i < n of floor((a i + b) / 128), n < 2^31: the published floor-sum algorithm (whole parts taken out, then
// the roles of a and the modulus exchanged, as Euclid's algorithm goes on (a, 128)). Divisions are in
// 32 bits where the numbers allow it: 64-bit ones made the search for a CTA's place take 10 us.
__device__ __forceinline__ int64_t floor_sum128(uint32_t n, uint32_t a, uint64_t b64) {
  uint32_t m = 128, b = static_cast<uint32_t>(b64 & 127);
  int64_t ans = static_cast<int64_t>(n) * static_cast<int64_t>(b64 >> 7);
  while (true) {
    const uint32_t q = a / m;
    a -= q * m;
    ans += static_cast<int64_t>(n) * (n - 1) / 2 * q + static_cast<int64_t>(n) * (b / m);
    b %= m;
    const uint64_t y = static_cast<uint64_t>(a) * n + b;
    if (y < m) return ans;
    if (y >> 32) {
      n = static_cast<uint32_t>(y / m);
      b = static_cast<uint32_t>(y % m);
    } else {
      n = static_cast<uint32_t>(y) / m;
      b = static_cast<uint32_t>(y) - n * m;
    }
    const uint32_t t = m;
    m = a;
    a = t;
  }
}
// A sequence's items per KV head: T2 tokens each, the key tiles (128 keys) each of them sees, and the units of
// work they count: its tiles, after one for the item itself (its Q, its O, filling the pipeline).
struct PromptSeq {
  Kv4Seq q;
  int T2;
  __device__ __forceinline__ int items() const { return (q.n + T2 - 1) / T2; }
  __device__ __forceinline__ int tiles_to(int tok) const { return (q.ctx - q.n + tok + 127) >> 7; }  // seen by tokens < tok
  __device__ __forceinline__ int tiles(int i) const { return tiles_to(min(q.n, (i + 1) * T2)); }
  __device__ __forceinline__ int units(int i) const { return tiles(i) + 1; }
  __device__ __forceinline__ int64_t before(int i) const {          // units of the items before item i
    const int last = items();
    const int64_t k = i < last ? i : last - 1;
    const int64_t s = k > 0 ? floor_sum128(static_cast<uint32_t>(k), T2, static_cast<uint64_t>(q.ctx - q.n) + T2 + 127) : 0;
    return i + (i < last ? s : s + tiles(last - 1));
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
// Where a CTA's range begins inside an item: for the kernel that joins the partials.
struct PromptCut {
  int j, units;                                          // units of the item before the range (0: no cut), in all
  int tok, h, q0, n;                                     // its first token, KV head; its sequence's first row, tokens
  int pad[2];
};
struct PromptLayout {
  static constexpr int OFF_Q = 0;                        // [unit] 2 x 16 KB (64 channels each)
  static constexpr int OFF_K = 65536;                    // [4] pages, 2 x 8 KB (64 channels each)
  static constexpr int OFF_V = OFF_K + 65536;            // [4] pages, 16 KB
  static constexpr int OFF_CODES = OFF_V + 65536;        // codes and scales of the next two pages, K's and V's
  static constexpr int OFF_MAP = OFF_CODES + 2 * 9216;   // [128] a row's token and head within the unit
  static constexpr int OFF_FLAG = OFF_MAP + 256;        // [16] whether the page is missing
  static constexpr int OFF_RANGE = OFF_FLAG + 64;
  static constexpr int OFF_BAR = OFF_RANGE + (sizeof(Kv4Range) + 7) / 8 * 8;
  static constexpr int NSEG = 4;                         // segments handed out ahead
  static constexpr int N_BARS = 32 + 2 * NSEG;
  static constexpr int OFF_SEG = (OFF_BAR + N_BARS * 8 + 16 + 15) / 16 * 16;
  static constexpr int OFF_WALK = OFF_SEG + NSEG * 64;
  static constexpr int OFF_NAN = OFF_WALK + 64;          // [NSEG][8] first key with a NaN in these 16 V channels
  static constexpr int SMEM_BYTES = OFF_NAN + NSEG * 32;
  static_assert(OFF_NAN % 16 == 0, "reset in words of 16 bytes");
  static_assert(sizeof(PromptSeg) <= 64, "a segment's slot");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static constexpr uint32_t T_S = 0, T_O = 256;          // + 128 for unit 1; S + 64 for a tile's second half
  static constexpr int THREADS = 512;
};
struct PromptWalk {                                      // (in OFF_WALK's 64 bytes)
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
    if (left == 1 && j == 0) left = 0;                   // an item's first unit alone: no tile, nothing to do
    if (left <= 0) return false;
    // j counts units: tiles j - 1 on, from 0
    const int nt = sq.tiles(i), u1 = min(nt + 1, j + left), TU = sq.T2 / 2;
    const int j0 = max(0, j - 1), j1 = u1 - 1;
    g.s = s; g.h = h; g.q0 = sq.q.q0; g.n = sq.q.n; g.ctx = sq.q.ctx;
    g.tok = i * sq.T2;
    g.j0 = j0; g.len = j1 - j0;
    const int nt0 = sq.tiles_to(min(sq.q.n, g.tok + TU));
    const int nt1 = g.tok + TU < sq.q.n ? nt : 0;
    g.mine0 = max(0, min(j1, nt0) - j0);
    g.mine1 = max(0, min(j1, nt1) - j0);
    g.whole = j0 == 0 && j1 == nt;
    g.first = j == 0;
    left -= u1 - j;
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

// Largest magnitude of eight packed 16-bit values.
template <typename T> __device__ __forceinline__ float amax8_packed(const uint4& u);
template <> __device__ __forceinline__ float amax8_packed<__nv_bfloat16>(const uint4& u) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
  const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
  return fmaxf(__low2float(m), __high2float(m));
}
template <> __device__ __forceinline__ float amax8_packed<__half>(const uint4&) { return 0.f; }

// A page id: a read-only load that stays where it is written, ahead of its use.
__device__ __forceinline__ int prefetch_id(const int32_t* p) {
  int v;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
template <typename T>
__global__ void __launch_bounds__(512, 1)
kv4_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, Kv4AttnArgs a) {
  using L = PromptLayout;
  constexpr bool kConvertQ = std::is_same<T, __nv_bfloat16>::value;
  // at a fixed, 1024-byte aligned address (there is no other shared memory): every address in it is a
  // constant and takes no register
  extern __shared__ __align__(1024) unsigned char kv4_prompt_smem[];
  unsigned char* const sm = kv4_prompt_smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
  uint64_t* q_full = bars;                               // Q of the segment is in place
  uint64_t* q_empty = bars + 1;                          // its last QK^T is done
  uint64_t* k_full = bars + 2;                           // [4] a page of K, of V: decoded, used
  uint64_t* k_empty = bars + 6;
  uint64_t* v_full = bars + 10;
  uint64_t* v_empty = bars + 14;
  uint64_t* s_full = bars + 18;                          // [unit][half tile] its scores are ready
  uint64_t* p_full = bars + 22;                          // [unit][half tile] P written over its scores
  uint64_t* pv_done = bars + 26;                         // [unit][half tile] its product with V is done
  // (Barriers for each half: a softmax may be two halves ahead of the products, and nobody may wait two
  // phases behind. It is never further ahead: a half's scores are issued after its last product.)
  uint64_t* mma_final = bars + 30;
  uint64_t* q_raw = bars + 31;                           // Q has been copied in, to be converted
  uint64_t* seg_full = bars + 32;                        // [NSEG]
  uint64_t* seg_empty = seg_full + L::NSEG;              // [NSEG]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::N_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Kv4Range* rng = reinterpret_cast<Kv4Range*>(sm + L::OFF_RANGE);
  volatile int* missing = reinterpret_cast<volatile int*>(sm + L::OFF_FLAG);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.Hq / a.c.Hkv;

  uchar2* row_map = reinterpret_cast<uchar2*>(sm + L::OFF_MAP);
  if ((smem_u32(sm) & 1023u) != 0) {                     // cannot happen; the tensor cores would read other rows
    if (threadIdx.x == 0) {
      flag_error(kStatusBounds);
      a.prompt_cut[blockIdx.x] = {};
    }
    return;
  }
  if (threadIdx.x < 128) row_map[threadIdx.x] = make_uchar2(threadIdx.x / group, threadIdx.x % group);
  if (threadIdx.x == 0) {
    mbar_init(q_raw, 1);
    mbar_init(q_full, kConvertQ ? 8 : 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(k_full + i, 2);
      mbar_init(k_empty + i, 2);
      mbar_init(v_full + i, 2);
      mbar_init(v_empty + i, 2);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
    }
    mbar_init(mma_final, 2);
    for (int i = 0; i < L::NSEG; ++i) {
      mbar_init(seg_full + i, 1);
      mbar_init(seg_empty + i, 2 + 1 + 4 + 8);           // products, Q, decoding, softmax
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
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_slot, 0);   // (uniform for the compiler too)
  auto seg_at = [&](int seg) -> const PromptSeg& {
    return *reinterpret_cast<const PromptSeg*>(sm + L::OFF_SEG + (seg % L::NSEG) * 64);
  };
  const int TU = 128 / group;                            // tokens of a unit
  // A wait gives up when it has passed its limit, or when another one has (abort_flag: 1 + its barrier |
  // role << 8); the place is reported at the end.
  const int role = warp < 4 && warp != 1 ? kRoleMma : warp < 8 ? kRoleProducer : kRoleSoftmax;
  auto gave_up = [&](uint64_t* bar, long long t0) -> bool {
    if (clock64() - t0 > kWaitLimitCycles) *abort_flag = 1 + static_cast<int>(bar - bars) + (role << 8);
    return *abort_flag != 0;
  };
  auto waitw = [&](uint64_t* bar, uint32_t parity) -> bool {        // by a whole warp
    if (__any_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__any_sync(0xffffffffu, mbar_try_wait(bar, parity)))
      if (__any_sync(0xffffffffu, gave_up(bar, t0))) return false;
    return true;
  };
  auto wait1 = [&](uint64_t* bar, uint32_t parity) -> bool {        // by one thread
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
      if (gave_up(bar, t0)) return false;
    return true;
  };

  if (warp < 4) {
    if ((warp & 1) == 0) {
      // ======================= products =======================
      {
        constexpr uint32_t idesc_qk = idesc_f16(128, 64), idesc_pv = idesc_f16(128, 128);
        // descriptors of the first blocks: an offset of n bytes adds n / 16
        const uint64_t dQ = make_sdesc(smem_u32(sm + L::OFF_Q), 16, 1024, kSw128);
        const uint64_t dK = make_sdesc(smem_u32(sm + L::OFF_K), 16, 1024, kSw128);
        const uint64_t dV = make_sdesc(smem_u32(sm + L::OFF_V), 16, 1024, kSw128);
        int tile = 0;
        uint32_t odd = 0;                                // the unit's tiles so far, odd or even
        bool ok = true;
        for (int seg = 0;; ++seg) {
          ok = waitw(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1);
          if (!ok) break;
          const int len = __shfl_sync(0xffffffffu, seg_at(seg).len, 0);
          const int mine0 = __shfl_sync(0xffffffffu, seg_at(seg).mine0, 0);
          const int mine1 = __shfl_sync(0xffffffffu, seg_at(seg).mine1, 0);
          const bool end = __shfl_sync(0xffffffffu, seg_at(seg).s, 0) < 0;
          if (lane == 0) mbar_arrive(seg_empty + seg % L::NSEG);
          __syncwarp();
          if (end || !(ok = waitw(q_full, seg & 1))) break;
          // x counts half tiles. Rounds -2 and -1: the first tile's scores. Round x: the product of half x with V,
          // and the scores of half x + 2 in its place.
          const int u = warp >> 1, mine = 2 * (u ? mine1 : mine0);
#pragma unroll 1
          for (int x = -2; x < 2 * len; ++x) {
            const int h = x & 1, now = 2 * tile + x, nx = now + 2;        // pages of halves x and x + 2
            const uint32_t tS = tbase + L::T_S + u * 128 + h * 64;
            if (x >= 0) {
              if (!(ok = waitw(v_full + (now & 3), (now >> 2) & 1))) break;
              if (x < mine) {
                if (!(ok = waitw(p_full + 2 * u + h, odd))) break;
                odd ^= h;
                tc_fence_after();
                mma_f16_ta_k64_elect(tbase + L::T_O + u * 128, tS, dV + (now & 3) * 1024, idesc_pv, x == 0 ? 0u : 1u);   // O_u += P_u V
                mma_commit_elect(pv_done + 2 * u + h);
              }
              mma_commit_elect(v_empty + (now & 3));
            }
            if (x + 2 < 2 * len) {
              if (!(ok = waitw(k_full + (nx & 3), (nx >> 2) & 1))) break;
              if (x + 2 < mine) {
                tc_fence_after();
                mma_f16_k128_elect<8192>(tS, dQ + u * 2048, dK + (nx & 3) * 1024, idesc_qk);                  // S_u = Q_u K^T
                mma_commit_elect(s_full + 2 * u + h);
              }
              mma_commit_elect(k_empty + (nx & 3));
              if (x + 3 == 2 * len) mma_commit_elect(q_empty);
            }
          }
          if (!ok) break;
          tile += len;
        }
        mma_commit_elect(mma_final);
        mbar_wait(mma_final, 0);
        __syncwarp();
      }
      __syncwarp();
    } else if (warp == 1 && lane == 0) {
      // ======================= segments and Q (one thread) =======================
      // Hands out the segments, two ahead of the one whose Q is brought in, and loads Q: per unit two boxes of
      // 64 channels x the group's heads x TU tokens, rows being (token, head). (Tokens of another sequence
      // behind this one's are loaded too and nobody's rows; behind the last token: zeros.)
      prefetch_tmap(&tm_q);
      PromptWalk* const walk = reinterpret_cast<PromptWalk*>(sm + L::OFF_WALK);   // (no registers for it)
      int handed = 0;
      auto hand_out = [&]() {
        PromptSeg* g = reinterpret_cast<PromptSeg*>(sm + L::OFF_SEG + (handed % L::NSEG) * 64);
        if (!walk->next(a, *g)) g->s = -1;
        int4* nans = reinterpret_cast<int4*>(sm + L::OFF_NAN + (handed % L::NSEG) * 32);
        nans[0] = nans[1] = make_int4(INT_MAX, INT_MAX, INT_MAX, INT_MAX);
        mbar_arrive(seg_full + handed % L::NSEG);
        ++handed;
      };
      walk->start(a, rng);
      {
        PromptCut cut = {};
        if (walk->left > 0 && walk->j > 0)
          cut = {walk->j, walk->sq.units(walk->i), walk->i * walk->sq.T2, walk->h, walk->sq.q.q0, walk->sq.q.n, {0, 0}};
        a.prompt_cut[blockIdx.x] = cut;
      }
      hand_out();
      hand_out();
      int seg = 0;
      for (;; ++seg) {
        const PromptSeg& g = seg_at(seg);
        if (g.s < 0) break;
        // the last segment's products have read Q
        if (seg > 0 && !wait1(q_empty, (seg - 1) & 1)) break;
        uint64_t* bar = kConvertQ ? q_raw : q_full;
        mbar_arrive_expect_tx(bar, 4 * 128 * TU * group);
#pragma unroll 1
        for (int b = 0; b < 4; ++b)
          tma_load_3d(sm + L::OFF_Q + b * 16384, &tm_q, bar, (b & 1) * 64, g.h * group, g.q0 + g.tok + (b >> 1) * TU);
        mbar_arrive(seg_empty + seg % L::NSEG);
        // the slot's last user: the segment two before this one
        if (handed >= L::NSEG && !wait1(seg_empty + handed % L::NSEG, (handed / L::NSEG - 1) & 1)) { ++seg; break; }
        hand_out();
      }
      // never leave a copy in flight into this CTA's shared memory
      if (seg > 0) mbar_wait(kConvertQ ? q_raw : q_full, (seg - 1) & 1);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ============================ K and V decoding ============================
    // Warps 4 and 5 decode K, warps 6 and 7 V, page by page into rings of four. Codes and scales come
    // two pages ahead, by asynchronous copies that each thread makes for itself; the page's id has been
    // read a page before that. A page that does not exist leaves what was there (codes are always
    // finite) and counts with scale 0. (Loops stay loops: with all roles unrolled the code of a tile
    // passes the instruction cache, and a decoded word cost five times its instructions.)
    const bool is_v = warp >= 6;
    struct Page {
      int id, h, left;                                   // -1: none; KV head, segment's slot << 16; slots in the context
    };
    int seg = -1, pages = 0, seg_h = 0, left = 0;
    const int32_t* ids = nullptr;
    bool end = false;
    auto next_page = [&]() -> Page {
      if (end) return Page{-1, 0, 0};
      if (--pages < 0) {
        if (seg >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(seg_empty + seg % L::NSEG);
        }
        ++seg;
        if (!waitw(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1) || seg_at(seg).s < 0) {
          end = true;
          return Page{-1, 0, 0};
        }
        const PromptSeg& g = seg_at(seg);
        pages = 2 * g.len - 1;
        seg_h = g.h | (seg % L::NSEG) << 16;
        left = g.ctx - g.j0 * 128;
        ids = a.table + static_cast<int64_t>(g.s) * a.max_pages + 2 * g.j0;
      }
      Page p = {-1, seg_h, left};
      if (left > 0) p.id = prefetch_id(ids);
      left -= 64;
      ++ids;
      return p;
    };
    auto valid = [&](int id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(a.c.num_pages); };
    // pages p0 (being decoded), p1, p2 (to be loaded), and the one whose id is being read; count: pages that
    // there are in all, known at the end. Three rounds without a page fill the pipeline.
    Page p0 = {-1, 0, 0}, p1 = p0, p2 = p0;
    int have = 0;                                        // pages handed out so far
    const int tid = threadIdx.x & 63;
    // K: a thread has half the channels of two rows: eight words of eight channels become eight 16-byte
    // chunks, four at a time. The threads of the upper half begin with the last four, so that the eight threads
    // of four rows write to eight different banks of 16 bytes.
    // V: a thread has eight tokens of 16 channels: four token pairs of a channel are a chunk.
    const int kr = tid >> 1, kh = tid & 1, vt = tid & 7, vb = tid >> 3;
    unsigned char* codes = sm + L::OFF_CODES + (is_v ? 9216 : 0) + tid * 16;   // [slot][4][64]
    unsigned char* scales = sm + L::OFF_CODES + 8192 + (is_v ? 9216 + tid * 8 : tid * 4);
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    for (int g = -3;; ++g) {
      const int stg = g & 3, slot = g & 1;
      const Page p3 = next_page();
      if (!end) ++have;
      if (g >= 0) {
        if (g >= have) break;
        if (g >= 4 && !waitw(empty + stg, ((g >> 2) - 1) & 1)) break;
        cp_async_wait<1>();
        const bool there = valid(p0.id);
        if (!is_v) {
          if (tid == 0) {
            const int gone = !there && p0.left > 0;
            missing[g & 15] = gone;
            if (gone) flag_error(kStatusBounds);
          }
          unsigned char* row = sm + L::OFF_K + stg * 16384 + kh * 8192 + kr * 128;
#pragma unroll 1
          for (int it = 0; it < 4; ++it) {               // rows kr and kr + 32
            const int o = (it & 1) ^ kh, r = it >> 1;    // which four of the row's words
            const uint32_t sc = *reinterpret_cast<const uint16_t*>(scales + slot * 512 + r * 256 + o * 2);
            const __half2 s2 = e4m3x2_to_half2(there ? sc : 0u);
            const uint4 c = *reinterpret_cast<const uint4*>(codes + slot * 4096 + (r * 2 + o) * 1024);
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&c);
            const uint32_t pos = static_cast<uint32_t>(((kr & 7) << 4) ^ (o << 6));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 f = e < 2 ? __low2half2(s2) : __high2half2(s2);
              uint32_t d[4];
              e2m1x8_to_half2(w[e], d);
#pragma unroll
              for (int x = 0; x < 4; ++x) d[x] = hmul2(d[x], f);
              *reinterpret_cast<uint4*>(row + r * 4096 + (pos ^ (e << 4))) = make_uint4(d[0], d[1], d[2], d[3]);
            }
          }
        } else {
          uint2 sc = *reinterpret_cast<const uint2*>(scales + slot * 512);
          const int in = there ? p0.left - vt * 8 : 0;   // of the thread's slots, those in the context
          if (in < 8) {                                  // the others: value 0 (weight 0 x NaN is not 0)
            const uint64_t keep = in <= 0 ? 0 : (1ull << (8 * in)) - 1;
            sc.x &= static_cast<uint32_t>(keep);
            sc.y &= static_cast<uint32_t>(keep >> 32);
          }
          // A NaN would reach the rows that do not see it too (0 x NaN): value 0, and NaN for those that do at the end
          const uint32_t nx = e4m3_nans(sc.x), ny = e4m3_nans(sc.y);
          if (nx | ny) {
            const int at = vt * 8 + (nx ? (__ffs(nx) >> 3) - 1 : (__ffs(ny) >> 3) + 3);
            atomicMin(reinterpret_cast<int*>(sm + L::OFF_NAN) + (p0.h >> 16) * 8 + vb, at - p0.left);
            sc.x &= ~((nx >> 7) * 0xFFu);
            sc.y &= ~((ny >> 7) * 0xFFu);
          }
          const __half2 f[4] = {e4m3x2_to_half2(sc.x & 0xFFFFu), e4m3x2_to_half2(sc.x >> 16),
                                e4m3x2_to_half2(sc.y & 0xFFFFu), e4m3x2_to_half2(sc.y >> 16)};
          unsigned char* row = sm + L::OFF_V + stg * 16384 + vb * 16 * 128;
#pragma unroll 1
          for (int e = 0; e < 4; ++e, row += 512) {
            uint32_t d[4][4];                            // [token pair][channel 4 e + x]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              e2m1x8_to_half2(*reinterpret_cast<const uint32_t*>(codes + slot * 4096 + k * 1024 + e * 4), d[k]);
#pragma unroll
              for (int x = 0; x < 4; ++x) d[k][x] = hmul2(d[k][x], f[k]);
            }
            const uint32_t pos = static_cast<uint32_t>(vt ^ ((e & 1) * 4)) << 4;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *reinterpret_cast<uint4*>(row + x * 128 + (pos ^ (x << 4))) = make_uint4(d[0][x], d[1][x], d[2][x], d[3][x]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + stg);
      }
      if (valid(p2.id)) {                                // into the place of the page just decoded
        const int64_t head = static_cast<int64_t>(p2.id) * a.c.Hkv + (p2.h & 0xFFFF);
        if (!is_v) {
          const uint8_t* k = a.c.k_pages + head * 4096 + kr * 64 + kh * 32;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            cp_async16(codes + slot * 4096 + r * 2048, k + r * 2048);
            cp_async16(codes + slot * 4096 + r * 2048 + 1024, k + r * 2048 + 16);
            cp_async4(scales + slot * 512 + r * 256, a.c.k_scales + head * 512 + (kr + r * 32) * 8 + kh * 4, true);
          }
        } else {
          const uint8_t* v = a.c.v_pages + head * 4096 + vt * 512 + vb * 16;
#pragma unroll
          for (int k = 0; k < 4; ++k) cp_async16(codes + slot * 4096 + k * 1024, v + k * 128);
          cp_async8(scales + slot * 512, a.c.v_scales + head * 512 + vb * 64 + vt * 8);
        }
      }
      cp_async_commit();
      p0 = p1;
      p1 = p2;
      p2 = p3;
    }
    cp_async_wait<0>();                                  // a wait that gave up leaves copies on their way
  } else {
    // ================================ softmax ================================
    const int wq = warp & 3, unit = (warp - 8) >> 2, row = wq * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tbase + L::T_S + unit * 128 + lane_addr, tO = tbase + L::T_O + unit * 128 + lane_addr;
    bool ok = true;
    int tile = 0, n = 0;                                 // tiles; half tiles of this unit
    for (int seg = 0;; ++seg) {
      if (!waitw(seg_full + seg % L::NSEG, (seg / L::NSEG) & 1)) break;
      const PromptSeg& g = seg_at(seg);
      if (g.s < 0) break;
      const int mine = unit == 0 ? g.mine0 : g.mine1;
      const int t0 = g.tok + unit * TU;
      // (rows that are nobody's, with another sequence's Q or none: factor 0, so that they never raise the
      // maximum and what they hold does not show in the rounding of the warp's others)
      const bool somebodys = row < TU * group && t0 + row_map[row].x < g.n;
      float C = somebodys ? *a.c.k_ts * a.softmax_scale * kLog2e : 0.f;
      if constexpr (kConvertQ) {
        // the thread's row of Q to fp16 under a power of two (kv4_row_factor), which goes into its C
        if (!waitw(q_raw, seg & 1)) break;
        unsigned char* q = sm + L::OFF_Q + unit * 32768 + row * 128;
        float m = 0.f;
#pragma unroll 4
        for (int c = 0; c < 16; ++c)
          m = fmaxf(m, amax8_packed<T>(*reinterpret_cast<const uint4*>(q + (c >> 3) * 16384 + (((c ^ row) & 7) << 4))));
        const float2 fac = kv4_row_factor<T>(m), f2 = make_float2(fac.x, fac.x);
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          uint4* at = reinterpret_cast<uint4*>(q + (c >> 3) * 16384 + (((c ^ row) & 7) << 4));
          uint4 u = *at;
          uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __fmul2_rn(to_float2<T>(w[e]), f2);
            w[e] = pack_half2(f.x, f.y);
          }
          *at = u;
        }
        C *= fac.y;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      if (somebodys) C = kv4_score_factor(C);
      const int lim_min = g.ctx - g.n + t0 - g.j0 * 128; // the last key that every row of the unit sees, from the segment's first
      float m_ref = -INFINITY;
      float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
      for (int x = 0; x < 2 * mine; ++x, ++n) {           // half tiles
        const int h = x & 1;
        const uint32_t tSh = tS + h * 64;
        if (!waitw(s_full + 2 * unit + h, (n >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const bool gone = missing[(2 * tile + x) & 15] != 0;
        if (x * 64 + 63 > lim_min || gone) {             // keys that not every row sees: masked in place
          const int last = gone ? -1 : lim_min + row_map[row].x - x * 64;
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t y[16];
            tmem_ld16(tSh + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = c + k <= last ? y[k] : 0xFF800000u;
            tmem_st16(tSh + c, y);
          }
          tmem_wait_st();
        }
        uint32_t y[64];
        tmem_ld32(tSh, y);
        tmem_ld32(tSh + 32, y + 32);
        tmem_wait_ld();
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 64; k += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmax3(m4[i], __uint_as_float(y[k + 2 * i]), __uint_as_float(y[k + 2 * i + 1]));
        }
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * C;
        // a row's first keys, or a rise past the limit: the reference follows
        if (__any_sync(0xffffffffu, mt > m_ref + kRiseLimit)) {
          const float m_new = fmaxf(m_ref, mt);
          if (x > 0) {
            const float al = m_new == -INFINITY ? 1.f : ex2_approx(m_ref - m_new);
            const float2 A = make_float2(al, al);
            l2[0] = __fmul2_rn(l2[0], A);
            l2[1] = __fmul2_rn(l2[1], A);
            if (!waitw(pv_done + 2 * unit + (h ^ 1), ((n - 1) >> 1) & 1)) { ok = false; break; }   // the last half's is in O
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              uint32_t o[16];
              tmem_ld16(tO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), A);
                o[k] = __float_as_uint(v.x);
                o[k + 1] = __float_as_uint(v.y);
              }
              tmem_st16(tO + c, o);
            }
          }
          m_ref = m_new;
        }
        const float bias = kPShift - (m_ref == -INFINITY ? 0.f : m_ref);
        const float2 C2 = make_float2(C, C), B2 = make_float2(bias, bias);
        uint32_t p[4][8];                                // P takes the place of the scores' first columns
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          float2 e = __ffma2_rn(make_float2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), C2, B2);
          e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
          l2[(k >> 1) & 1] = __fadd2_rn(l2[(k >> 1) & 1], e);
          p[k >> 4][(k >> 1) & 7] = pack_half2(e.x, e.y);
          if ((k & 15) == 14) tmem_st8(tSh + (k >> 4) * 8, p[k >> 4]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 2 * unit + h);
      }
      if (!ok) break;
      tile += g.len;
      // ---- O of the segment ----
      const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
      if (mine > 0) {
        if (!waitw(pv_done + 2 * unit + 1, ((n - 1) >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
      }
      // (thread's place read afresh: addresses computed from it before the tiles would stay in registers)
      int me;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(me));
      const int my_row = me & 127, my_unit = (me >> 7) & 1;
      const uchar2 at = row_map[my_row];
      const int tok = g.tok + my_unit * TU + at.x;
      const bool real = my_row < TU * group && tok < g.n;
      const bool whole = g.whole;
      float* part = a.prompt_part + static_cast<int64_t>(2 * blockIdx.x + (g.first ? 1 : 0)) * kPromptPartFloats;
      const int64_t orow = static_cast<int64_t>(g.q0 + tok) * a.Hq + g.h * group + at.y;
      uint32_t nans = 0;                                 // bit b: the row sees a NaN in V channels 16 b ..
      {
        const volatile int* first = reinterpret_cast<const volatile int*>(sm + L::OFF_NAN) + (seg % L::NSEG) * 8;
#pragma unroll
        for (int b = 0; b < 8; ++b) nans |= (first[b] <= tok - g.n ? 1u : 0u) << b;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(seg_empty + seg % L::NSEG);
      const float f = l == 0.f ? 0.f : *a.c.v_ts / l;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_ld32(tO + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (nans) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (nans >> ((c + k) >> 4) & 1) o[k] = 0x7FFFFFFF;
        }
        if (real && whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * kKv4D + c);
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            dst[k >> 3] = make_uint4(pack2<T>(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f),
                                     pack2<T>(__uint_as_float(o[k + 2]) * f, __uint_as_float(o[k + 3]) * f),
                                     pack2<T>(__uint_as_float(o[k + 4]) * f, __uint_as_float(o[k + 5]) * f),
                                     pack2<T>(__uint_as_float(o[k + 6]) * f, __uint_as_float(o[k + 7]) * f));
        } else if (real) {
          uint4* dst = reinterpret_cast<uint4*>(part + (my_unit * 128 + my_row) * kKv4D + c);
#pragma unroll
          for (int k = 0; k < 32; k += 4) dst[k >> 2] = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
        __syncwarp();
      }
      if (real) {
        if (!whole) {
          part[256 * kKv4D + my_unit * 128 + my_row] = m_ref;
          part[256 * (kKv4D + 1) + my_unit * 128 + my_row] = l;
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
  if (threadIdx.x == 0 && *abort_flag != 0) {
    flag_error(kStatusTimeout);
    record_timeout(wait_site(kKernelKv4Prompt, *abort_flag >> 8, (*abort_flag & 0xFF) - 1, 0));
  }
}

// Joins the partials of items that cross CTAs. CTA (i, y) takes the item that CTA i of the prompt
// kernel began and CTA i + 1 went on with, if any, and rows 8 y ..; a warp takes a row, a lane four
// channels.
template <typename T>
__global__ void __launch_bounds__(256) kv4_prompt_merge_kernel(Kv4AttnArgs a) {
  const int cta = blockIdx.x + 1, group = a.Hq / a.c.Hkv, TU = 128 / group;
  const PromptCut cut = a.prompt_cut[cta];
  const int per = static_cast<int>(a.prompt_plan[0]);    // units a CTA
  if (cut.j == 0 || cut.j > per) return;                 // not cut here, or not here first
  const int c1 = cta + (cut.units - cut.j - 1) / per;
  // (a first unit alone at the end of a CTA's range has left no partial)
  const int c0 = cut.j == 1 ? cta : cta - 1;
  if (c0 == c1) return;                                  // written by the prompt kernel
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto part = [&](int c) {
    return a.prompt_part + static_cast<int64_t>(2 * c + (c == cta - 1 ? 1 : 0)) * kPromptPartFloats;
  };
  const int row = blockIdx.y * 8 + warp, ru = row & 127;
  const int tok = cut.tok + (row >> 7) * TU + ru / group;
  if (ru >= TU * group || tok >= cut.n) return;
  float M = -INFINITY;
  for (int c = c0; c <= c1; ++c) M = fmaxf(M, part(c)[256 * kKv4D + row]);
  const float mu = M == -INFINITY ? 0.f : M;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; ++c) {
    const float* p = part(c);
    const float w = ex2_approx(p[256 * kKv4D + row] - mu);
    const float4 v = *reinterpret_cast<const float4*>(p + row * kKv4D + lane * 4);
    l += w * p[256 * (kKv4D + 1) + row];
    acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
  }
  const float f = l == 0.f ? 0.f : *a.c.v_ts / l;
  const int64_t orow = static_cast<int64_t>(cut.q0 + tok) * a.Hq + cut.h * group + ru % group;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + orow * kKv4D + lane * 4) =
      make_uint2(pack2<T>(acc.x * f, acc.y * f), pack2<T>(acc.z * f, acc.w * f));
  if (a.lse != nullptr && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l) - kPShift) * kLn2;
}

}  // namespace qk4v8
