// Attention of few query rows per KV head over the 4-bit cache (decoding steps, two tokens of few heads):
// split over the keys, plus the merge of the splits.
//
// Mathematics: for the n query tokens of a sequence and one KV head, the R = n g rows (token,
// head of the group) see the same keys. S^T = K Q^T and O^T += V^T P^T on 16-bit tensor cores with
// FP32 accumulators; K and V are E2M1 x E4M3 products of at most six significant bits between
// 2^-10 and 2688, exact in fp16. Q is scaled per row by a power of two into fp16's range (exact
// but for elements more than 2^27 times below the row's largest) and the factor goes into the softmax constant.
// P = 2^(s - m + 6) is rounded to fp16 (2^-11 relative; the 2^6 keeps weights down to 2^-20
// of the largest out of the subnormals); m, l and O are FP32, l sums the unrounded weights.
//
// Bound: with up to eight rows a KV head, HBM: the cache is read once, 144 bytes a token and KV head. With 9 to 16
// rows (NT = 2) it is not: 24 sequences of two tokens of 8 heads take 95 us, 21 % of the HBM rate, with half the tokens
// in flight and twice the softmax and products for each decoded word. Everything is laid out so
// that codes go from shared memory into tensor-core operands without being moved between threads:
//   * keys are the M dimension of both products (16 tokens or 16 channels a tile), rows the N
//     dimension (8 a tile), so a decoding step of g <= 8 wastes nothing on padding rows to 16;
//   * a thread of the K operand needs pairs of neighbouring channels of a token: a byte of the
//     page. The order of channels is free as long as Q has the same one: thread t of four takes
//     channels 32 t .. 32 t + 31, one 16-byte load;
//   * a thread of the V^T operand needs pairs of neighbouring tokens of a channel: a byte of the
//     page too, since V's bytes pair tokens. Thread c of eight takes channels 16 c .. 16 c + 15, one
//     16-byte load and one scale block;
//   * P^T has to change from accumulator to operand layout: one 8x8 transpose a tile (movmatrix).
// The tensor-core form is mma.sync: operands come from registers, where the decoding leaves
// them; through shared or tensor memory every decoded byte would be written and read again.
//
// Work split: the pages of all (sequence, KV head) pairs form one line, cut into equal
// consecutive ranges, one a CTA and one CTA an SM, whatever the lengths. The CTA's warps take
// pages in turn, each with its own running maximum, and are joined through shared memory where a
// pair ends. A pair inside one CTA is written out; one that crosses CTAs leaves partials
// (O, m, l) that the merge kernel joins. Each warp loads its own pages, two stages of one page,
// by 16-byte asynchronous copies, with no barrier between warps until a pair ends. (One warp
// issuing bulk copies for all of them reached 1 page in 1020 cycles, 4 copies of 4096 + 4096 +
// 512 + 512 bytes: 33 % of the HBM rate.)
// Measured as graphs: 64 sequences of 8192 to 32768 tokens, 32 query and 8 KV heads, one token each: 274 us with
// the join, 5.6 TB/s (86 % of the measured 6.5; planned calls whose inputs change from pass to pass: 295 to 312 us); one
// sequence of 1001 tokens: 12 us, two launches.
#pragma once
#include <climits>
#include <type_traits>
#include "kv4.cuh"
#include "attn_fwd.cuh"

namespace qk4v8 {

struct PromptCut;
struct Kv4AttnArgs {
  Kv4Cache c;
  const void* q;
  int64_t q_stride;
  const int32_t* cu_q;       // or null: one token a sequence
  const int32_t* lens;
  const int32_t* table;
  int32_t total_q, S, max_pages, Hq, max_q, max_context;
  int32_t rows_max;          // the split kernel takes sequences of at most this many rows a KV head
  float softmax_scale;
  void* out;
  float* lse;
  int64_t* plan;             // workspace: the split kernel's kv4_range plan
  float* part;               // workspace: its partials, two a CTA
  int64_t* prompt_plan;      // the same of the prompt kernel
  PromptCut* prompt_cut;   // one a CTA
  float* prompt_part;
};

constexpr float kPShift = 6.f;

struct Kv4Seq {
  int q0, n, ctx;            // first query row, query tokens, context
};
// Sequence s as the caller gave it; n = 0 when it has no query tokens or is out of range.
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4AttnArgs& a, int s, bool flag) {
  Kv4Seq q;
  q.q0 = a.cu_q ? a.cu_q[s] : s;
  q.n = a.cu_q ? a.cu_q[s + 1] - q.q0 : 1;
  q.ctx = a.lens[s];
  if (q.n == 0) return q;
  if (q.n < 0 || q.n > a.max_q || q.q0 < 0 || q.q0 > a.total_q - q.n || q.ctx < q.n ||
      q.ctx > a.max_context || ((q.ctx - 1) >> 6) >= a.max_pages) {
    if (flag) flag_error(kStatusBounds);
    q.n = 0;
  }
  return q;
}

// A CTA's part of a line of units that the sequences fill one after another: from unit `first` of
// sequence s on, `left` units.
struct Kv4Range {
  int64_t sums[16];          // of the warps, while it is found
  int64_t first;
  int s, left;
};
// Cuts the line into equal parts of at least `least` units, one a CTA, and finds this CTA's. weight(i):
// units of sequence i. plan[0] gets the units a CTA, plan[1 + i] the first unit of sequence i (for
// the kernels that join partials). Two passes over the sequences: the total, then the place.
template <int THREADS, typename W>
__device__ __forceinline__ void kv4_range(W weight, int S, int least, int64_t* plan, Kv4Range* r) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t w = 0, before = 0, total = 0, first = 0, per = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t run = 0;
    if (pass == 1) {
      per = (total + gridDim.x - 1) / gridDim.x;
      if (per < least) per = least;
      first = per * blockIdx.x;
      if (first > total) first = total;
      if (tid == 0) {
        r->s = S;
        r->first = 0;
        r->left = static_cast<int>(per < total - first ? per : total - first);
        if (blockIdx.x == 0) plan[0] = per;
      }
      __syncthreads();
    }
    for (int i0 = 0; i0 < S; i0 += THREADS) {
      const int i = i0 + tid;
      if (pass == 0 || S > THREADS) {                    // a single chunk is kept from pass 0
        w = i < S ? weight(i) : 0;
        int64_t x = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) r->sums[warp] = x;
        __syncthreads();
        before = x - w;
        int64_t sum = 0;
#pragma unroll
        for (int k = 0; k < THREADS / 32; ++k) {
          if (k < warp) before += r->sums[k];
          sum += r->sums[k];
        }
        if (pass == 0) total += sum;
        else { before += run; run += sum; }
      }
      if (pass == 1 && i < S) {
        if (blockIdx.x == 0) plan[1 + i] = before;
        if (w > 0 && first >= before && first < before + w) { r->s = i; r->first = first - before; }
      }
    }
  }
  __syncthreads();
}

// A position in the line of units (a unit: one page of one KV head of a sequence; sequence by
// sequence, head by head), and the units left from there in the CTA's range.
struct Kv4Walk {
  int s, h, p, np, left;
  Kv4Seq q;
  // the first sequence from s on that the split kernel takes
  __device__ __forceinline__ void find(const Kv4AttnArgs& a) {
    const int group = a.Hq / a.c.Hkv;
    for (; s < a.S; ++s) {
      q = kv4_seq(a, s, false);
      if (q.n > 0 && q.n * group <= a.rows_max) {
        np = (q.ctx + 63) >> 6;
        return;
      }
    }
    left = 0;
  }
  __device__ __forceinline__ void next_pair(const Kv4AttnArgs& a) {
    if (++h == a.c.Hkv) {
      h = 0;
      ++s;
      find(a);
    }
  }
  __device__ __forceinline__ void advance(const Kv4AttnArgs& a, int units) {
    p += units;
    left -= units;
    while (left > 0 && p >= np) {
      p -= np;
      next_pair(a);
    }
  }
};

// NT: tiles of eight rows, 1 or 2.
template <int NT>
struct Kv4SplitLayout {
  static constexpr int WARPS = 12, THREADS = WARPS * 32;
  static constexpr int NS = 2;                          // stages a warp, of one page
  static constexpr int MT = NT == 1 ? 4 : 2;            // tiles of 16 tokens taken at once
  static constexpr int ROWS = NT * 8;
  static constexpr int STAGE = 9216, OFF_V = 4096, OFF_KS = 8192, OFF_VS = 8704;
  static constexpr int Q_LD = 272;                      // bytes of a Q row (256 + 16)
  static constexpr int M_LD = 132;                      // floats of a row in the join (128 + 4)
  static constexpr int OFF_Q = WARPS * NS * STAGE;
  static constexpr int OFF_ML = OFF_Q + ROWS * Q_LD;    // [warp][8 rows] (m, l)
  static constexpr int OFF_ROW = OFF_ML + WARPS * 8 * 8;        // [ROWS] C, then [ROWS] limit
  static constexpr int OFF_RANGE = OFF_ROW + ROWS * 8;
  static constexpr int OFF_AT = OFF_RANGE + sizeof(Kv4Range);   // [warp] where its O lies in the join
  static constexpr int SMEM = OFF_AT + WARPS * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(8 * M_LD * 4 <= STAGE, "a stage holds a warp's O of eight rows");
};
constexpr int kKv4PartRows = 16;                        // rows of a partial (the larger layout's)
constexpr int kKv4PartFloats = kKv4PartRows * (kKv4D + 2);

// 16-byte asynchronous copy past L1.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B, 16x8x16, fp16 operands, FP32 accumulators.
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit elements over the warp (thread i: row i / 4, columns 2 (i % 4) ..).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return pack2<__half>(lo, hi); }

// The power of two that brings a row with largest magnitude `amax` to [2^10, 2^11) (1 for a row
// of zeros, infinities or NaN), and its inverse. bf16 rows need it to become fp16; fp16 rows keep 1.
template <typename T>
__device__ __forceinline__ float2 kv4_row_factor(float amax) {
  if (!std::is_same<T, __nv_bfloat16>::value || !(amax > 0.f) || amax > 3.4e38f) return make_float2(1.f, 1.f);
  int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu) - 127 - 10;
  e = max(-126, min(126, e));
  return make_float2(__uint_as_float(static_cast<uint32_t>(127 - e) << 23),
                     __uint_as_float(static_cast<uint32_t>(127 + e) << 23));
}

// A row's factor from products to scores in base 2. One that has left FP32's range at the bottom becomes the
// smallest normal number: products stay below 2^35, so every score is still as good as 0, while 0 times a hidden
// key's -inf would be NaN.
__device__ __forceinline__ float kv4_score_factor(float c) { return c == 0.f ? 0x1p-126f : c; }

template <int NT, typename T>
__global__ void __launch_bounds__(Kv4SplitLayout<NT>::THREADS, 1)
kv4_split_kernel(Kv4AttnArgs a) {
  using L = Kv4SplitLayout<NT>;
  extern __shared__ __align__(128) unsigned char kv4_smem[];
  unsigned char* sm = kv4_smem;
  Kv4Range* rng = reinterpret_cast<Kv4Range*>(sm + L::OFF_RANGE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.Hq / a.c.Hkv;

  kv4_range<L::THREADS>(
      [&](int i) -> int64_t {
        const Kv4Seq q = kv4_seq(a, i, blockIdx.x == 0);
        return (q.n > 0 && q.n * group <= a.rows_max) ? static_cast<int64_t>((q.ctx + 63) >> 6) * a.c.Hkv : 0;
      },
      a.S, 4, a.plan, rng);
  Kv4Walk walk;                                         // the pair at hand
  walk.s = rng->s;
  walk.left = rng->left;
  walk.h = walk.p = 0;
  walk.find(a);
  if (walk.left > 0) {
    walk.h = static_cast<int>(rng->first / walk.np);
    walk.p = static_cast<int>(rng->first % walk.np);
  }
  Kv4Walk ahead = walk;                                 // the next page this warp loads
  ahead.advance(a, warp);
  unsigned char* ring = sm + warp * (L::NS * L::STAGE);
  auto page_of = [&](const Kv4Walk& w) {
    return w.left > 0 ? a.table[static_cast<int64_t>(w.s) * a.max_pages + w.p] : -1;
  };
  // Starts the loads of a page into a stage and moves on; whether there was one.
  auto load_page = [&](int st, int page) -> bool {
    const bool mine = ahead.left > 0;
    const bool good = mine && page >= 0 && page < a.c.num_pages;
    if (good) {
      const int64_t head = static_cast<int64_t>(page) * a.c.Hkv + ahead.h;
      unsigned char* d = ring + st * L::STAGE + lane * 16;
      const uint8_t* k = a.c.k_pages + head * 4096 + lane * 16;
      const uint8_t* v = a.c.v_pages + head * 4096 + lane * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) cp_async16(d + i * 512, k + i * 512);
      cp_async16(d + L::OFF_KS, a.c.k_scales + head * 512 + lane * 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) cp_async16(d + L::OFF_V + i * 512, v + i * 512);
      cp_async16(d + L::OFF_VS, a.c.v_scales + head * 512 + lane * 16);
    } else if (mine && lane == 0) {
      flag_error(kStatusBounds);
    }
    cp_async_commit();
    if (mine) ahead.advance(a, L::WARPS);
    return good;
  };
  bool ok0 = load_page(0, page_of(ahead));              // stage `st` holds the warp's next page
  bool ok1 = load_page(1, page_of(ahead));
  int st = 0, gi = 0;                                   // gi: units of this CTA before the pair

  // ================================ attention ================================
  constexpr int MT = L::MT;
  const int c = lane >> 2, t = lane & 3;
  float* row_c = reinterpret_cast<float*>(sm + L::OFF_ROW);
  int* row_lim = reinterpret_cast<int*>(sm + L::OFF_ROW) + L::ROWS;
  bool owed = false;                                    // a stage to be loaded after the join
  while (walk.left > 0) {
    struct { Kv4Seq q; int h, p0, p1, np; } g = {walk.q, walk.h, walk.p, min(walk.np, walk.p + walk.left), walk.np};
    walk.left -= g.p1 - g.p0;
    walk.p = 0;
    if (walk.left > 0) walk.next_pair(a);
    const int rows = g.q.n * group;
    // ---- Q: rows to fp16, zeros past the last; constants of each row ----
    __syncthreads();                                    // the last pair's rows and join are done with
    if (owed) {
      const bool good = load_page(st ^ 1, page_of(ahead));
      (st ? ok0 : ok1) = good;
      owed = false;
    }
    for (int r = warp; r < L::ROWS; r += L::WARPS) {
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < rows) {
        const T* src = static_cast<const T*>(a.q) + (g.q.q0 + r / group) * a.q_stride +
                       (g.h * group + r % group) * kKv4D + lane * 4;
        const uint2 u = *reinterpret_cast<const uint2*>(src);
        const float2 x = to_float2<T>(u.x), y = to_float2<T>(u.y);
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
      }
      float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float2 fac = kv4_row_factor<T>(m);
      *reinterpret_cast<uint2*>(sm + L::OFF_Q + r * L::Q_LD + lane * 8) =
          make_uint2(pack_half2(f[0] * fac.x, f[1] * fac.x), pack_half2(f[2] * fac.x, f[3] * fac.x));
      if (lane == 0) {
        row_c[r] = kv4_score_factor(fac.y * (*a.c.k_ts * a.softmax_scale * kLog2e));
        row_lim[r] = r < rows ? g.q.ctx - g.q.n + r / group : -1;
      }
    }
    __syncthreads();
    // a thread's rows of a tile: 2 t and 2 t + 1, in the halves of its pairs
    uint32_t q[NT][16];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        reinterpret_cast<uint4*>(q[nt])[k] =
            *reinterpret_cast<const uint4*>(sm + L::OFF_Q + (nt * 8 + c) * L::Q_LD + t * 64 + k * 16);
    float2 m[NT], l[NT];
    float o[NT][8][4];
    int nan_at = INT_MAX;                               // the first key with a NaN in this thread's V channels
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = make_float2(-INFINITY, -INFINITY);
      l[nt] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    for (int p = g.p0 + (warp + L::WARPS - gi % L::WARPS) % L::WARPS; p < g.p1; p += L::WARPS) {
      const int next = page_of(ahead);
      cp_async_wait<1>();
      __syncwarp();
      if (st ? ok1 : ok0) {
        const unsigned char* sp = ring + st * L::STAGE;
#pragma unroll 1
        for (int first = 0; first < 64; first += MT * 16) {
          // ---- S^T = K Q^T: MT tiles of 16 tokens ----
          float s[MT][NT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
            const int tok = first + mt * 16 + c;
            const uint4 ka = *reinterpret_cast<const uint4*>(sp + tok * 64 + t * 16);
            const uint4 kb = *reinterpret_cast<const uint4*>(sp + (tok + 8) * 64 + t * 16);
            const __half2 sa = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sp + L::OFF_KS + tok * 8 + t * 2));
            const __half2 sb = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sp + L::OFF_KS + (tok + 8) * 8 + t * 2));
            const uint32_t* kaw = reinterpret_cast<const uint32_t*>(&ka);
            const uint32_t* kbw = reinterpret_cast<const uint32_t*>(&kb);
#pragma unroll
            for (int w = 0; w < 4; ++w) {                  // a word: 8 channels, two k-steps' halves
              const __half2 fa = w < 2 ? __low2half2(sa) : __high2half2(sa);
              const __half2 fb = w < 2 ? __low2half2(sb) : __high2half2(sb);
              uint32_t ha[4], hb[4];
              e2m1x8_to_half2(kaw[w], ha);
              e2m1x8_to_half2(kbw[w], hb);
#pragma unroll
              for (int k = 0; k < 4; ++k) { ha[k] = hmul2(ha[k], fa); hb[k] = hmul2(hb[k], fb); }
              const uint32_t a0[4] = {ha[0], hb[0], ha[1], hb[1]}, a1[4] = {ha[2], hb[2], ha[3], hb[3]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(s[mt][nt], a0, q[nt][4 * w], q[nt][4 * w + 1]);
                mma16816(s[mt][nt], a1, q[nt][4 * w + 2], q[nt][4 * w + 3]);
              }
            }
          }
          // ---- softmax over the MT * 16 tokens; this thread has tokens c + 8 j ----
          uint32_t pb[MT][NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + 2 * t;
            if (p * 64 + 63 > g.q.ctx - g.q.n) {            // keys that not every row sees
              const int lim0 = row_lim[r] - p * 64 - first - c, lim1 = row_lim[r + 1] - p * 64 - first - c;
#pragma unroll
              for (int j = 0; j < 2 * MT; ++j) {
                if (8 * j > lim0) s[j >> 1][nt][(j & 1) * 2] = -INFINITY;
                if (8 * j > lim1) s[j >> 1][nt][(j & 1) * 2 + 1] = -INFINITY;
              }
            }
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mx0 = fmax3(mx0, s[mt][nt][0], s[mt][nt][2]);
              mx1 = fmax3(mx1, s[mt][nt][1], s[mt][nt][3]);
            }
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) {
              mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
              mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
            }
            const float2 C = *reinterpret_cast<const float2*>(row_c + r);
            const float n0 = fmaxf(m[nt].x, mx0 * C.x), n1 = fmaxf(m[nt].y, mx1 * C.y);
            const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
            if (__any_sync(0xffffffffu, n0 != m[nt].x || n1 != m[nt].y)) {
              const float2 al = make_float2(ex2_approx(m[nt].x - u0), ex2_approx(m[nt].y - u1));
              m[nt] = make_float2(n0, n1);
              l[nt] = __fmul2_rn(l[nt], al);
#pragma unroll
              for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                  const float2 v = __fmul2_rn(make_float2(o[nt][i][k], o[nt][i][k + 1]), al);
                  o[nt][i][k] = v.x;
                  o[nt][i][k + 1] = v.y;
                }
            }
            const float2 bias = make_float2(kPShift - u0, kPShift - u1);
#pragma unroll
            for (int j = 0; j < 2 * MT; ++j) {
              float2 x = __ffma2_rn(make_float2(s[j >> 1][nt][(j & 1) * 2], s[j >> 1][nt][(j & 1) * 2 + 1]), C, bias);
              x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
              l[nt] = __fadd2_rn(l[nt], x);
              pb[j >> 1][nt][j & 1] = transpose8x8(pack_half2(x.x, x.y));
            }
          }
          // ---- O^T += V^T P^T: MT steps of 16 tokens ----
#pragma unroll
          for (int kt = 0; kt < MT; ++kt) {
            const int r0 = first / 2 + kt * 8 + t;                     // this thread's token pairs: r0, r0 + 4
            const uint4 va = *reinterpret_cast<const uint4*>(sp + L::OFF_V + r0 * 128 + c * 16);
            const uint4 vb = *reinterpret_cast<const uint4*>(sp + L::OFF_V + (r0 + 4) * 128 + c * 16);
            uint32_t sca = *reinterpret_cast<const uint16_t*>(sp + L::OFF_VS + c * 64 + r0 * 2);
            uint32_t scb = *reinterpret_cast<const uint16_t*>(sp + L::OFF_VS + c * 64 + (r0 + 4) * 2);
            if (p * 64 + 63 > g.q.ctx - g.q.n) {           // slots behind the context: weight 0, value 0
              const int left = g.q.ctx - p * 64;           // valid slots of the page
              if (2 * r0 >= left) sca = 0; else if (2 * r0 + 1 >= left) sca &= 0xFFu;
              if (2 * r0 + 8 >= left) scb = 0; else if (2 * r0 + 9 >= left) scb &= 0xFFu;
              // A NaN would reach the rows that do not see it too (0 x NaN): value 0, and NaN for those that do in the end
              const uint32_t na = e4m3_nans(sca), nb = e4m3_nans(scb);
              if (na | nb) {
                const int at = na ? 2 * r0 + ((na & 0x80u) ? 0 : 1) : 2 * r0 + 8 + ((nb & 0x80u) ? 0 : 1);
                nan_at = min(nan_at, p * 64 + at);
                sca &= ~((na >> 7) * 0xFFu);
                scb &= ~((nb >> 7) * 0xFFu);
              }
            }
            const __half2 fa = e4m3x2_to_half2(sca), fb = e4m3x2_to_half2(scb);
            const uint32_t* vaw = reinterpret_cast<const uint32_t*>(&va);
            const uint32_t* vbw = reinterpret_cast<const uint32_t*>(&vb);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t ha[4], hb[4];
              e2m1x8_to_half2(vaw[w], ha);
              e2m1x8_to_half2(vbw[w], hb);
#pragma unroll
              for (int k = 0; k < 4; ++k) { ha[k] = hmul2(ha[k], fa); hb[k] = hmul2(hb[k], fb); }
              const uint32_t a0[4] = {ha[0], ha[1], hb[0], hb[1]}, a1[4] = {ha[2], ha[3], hb[2], hb[3]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(o[nt][2 * w], a0, pb[kt][nt][0], pb[kt][nt][1]);
                mma16816(o[nt][2 * w + 1], a1, pb[kt][nt][0], pb[kt][nt][1]);
              }
            }
          }
        }
      }
      __syncwarp();                                      // the stage has been read
      if (p + L::WARPS < g.p1) {
        const bool good = load_page(st, next);
        (st ? ok1 : ok0) = good;
      } else {
        owed = true;                                     // its O goes there first
      }
      st ^= 1;
    }
    gi += g.p1 - g.p0;

    // ---- the warps' results joined, eight rows at a time ----
    const bool whole = g.p0 == 0 && g.p1 == g.np;
    float* mbuf = reinterpret_cast<float*>(ring + (st ^ 1) * L::STAGE);
    if (__any_sync(0xffffffffu, nan_at != INT_MAX)) {
#pragma unroll
      for (int x = 1; x <= 2; x <<= 1) nan_at = min(nan_at, __shfl_xor_sync(0xffffffffu, nan_at, x));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (nan_at <= row_lim[nt * 8 + 2 * t + k]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[nt][i][k] = o[nt][i][2 + k] = __int_as_float(0x7FFFFFFF);
          }
    }
    int* at = reinterpret_cast<int*>(sm + L::OFF_AT);
    if (lane == 0) at[warp] = owed ? static_cast<int>(reinterpret_cast<unsigned char*>(mbuf) - sm) : -1;
    float2* mlbuf = reinterpret_cast<float2*>(sm + L::OFF_ML);
    float* part = a.part + static_cast<int64_t>(2 * blockIdx.x + (g.p0 > 0 ? 0 : 1)) * kKv4PartFloats;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0) __syncthreads();
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1) {
        l[nt].x += __shfl_xor_sync(0xffffffffu, l[nt].x, x);
        l[nt].y += __shfl_xor_sync(0xffffffffu, l[nt].y, x);
      }
      if (c == 0) {
        mlbuf[warp * 8 + 2 * t] = make_float2(m[nt].x, l[nt].x);
        mlbuf[warp * 8 + 2 * t + 1] = make_float2(m[nt].y, l[nt].y);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!owed) break;                                // no page of this pair: nothing to join
        float* dst = mbuf + (2 * t + k) * L::M_LD + c * 16;   // channels 16 c + 2 i, + 1
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[nt][i][k], o[nt][i][2 + k], o[nt][i + 1][k], o[nt][i + 1][2 + k]);
      }
      __syncthreads();
      for (int rr = warp; rr < 8; rr += L::WARPS) {       // a warp joins a row, a lane four channels
        const int r = nt * 8 + rr;
        if (r >= rows) break;
        float M = -INFINITY, ls = 0.f;
#pragma unroll
        for (int k = 0; k < L::WARPS; ++k) M = fmaxf(M, mlbuf[k * 8 + rr].x);
        const float mu = M == -INFINITY ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < L::WARPS; ++k) {
          if (at[k] < 0) continue;
          const float2 ml = mlbuf[k * 8 + rr];
          const float wgt = ex2_approx(ml.x - mu);
          const float4 v = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(sm + at[k]) + rr * L::M_LD + lane * 4);
          ls += wgt * ml.y;
          acc.x += wgt * v.x; acc.y += wgt * v.y; acc.z += wgt * v.z; acc.w += wgt * v.w;
        }
        if (whole) {
          const float f = ls == 0.f ? 0.f : *a.c.v_ts / ls;
          const int64_t orow = static_cast<int64_t>(g.q.q0 + r / group) * a.Hq + g.h * group + r % group;
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + orow * kKv4D + lane * 4) =
              make_uint2(pack2<T>(acc.x * f, acc.y * f), pack2<T>(acc.z * f, acc.w * f));
          if (a.lse != nullptr && lane == 0)
            a.lse[orow] = ls == 0.f ? -INFINITY : (M + log2f(ls) - kPShift) * kLn2;
        } else {
          *reinterpret_cast<float4*>(part + r * kKv4D + lane * 4) = acc;
          if (lane == 0) *reinterpret_cast<float2*>(part + kKv4PartRows * kKv4D + 2 * r) = make_float2(M, ls);
        }
      }
    }
  }
}

// Joins the partials of the pairs that cross CTAs. One CTA per (sequence, KV head) and row; a thread
// per channel.
template <typename T>
__global__ void __launch_bounds__(128) kv4_merge_kernel(Kv4AttnArgs a) {
  const int s = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv, r = blockIdx.y;
  const int group = a.Hq / a.c.Hkv;
  const Kv4Seq q = kv4_seq(a, s, false);
  if (q.n <= 0 || q.n * group > a.rows_max || r >= q.n * group) return;
  const int np = (q.ctx + 63) >> 6;
  const int64_t per = a.plan[0], first = a.plan[1 + s] + static_cast<int64_t>(h) * np;
  const int c0 = static_cast<int>(first / per), c1 = static_cast<int>((first + np - 1) / per);
  if (c0 == c1) return;                                 // written by the split kernel
  const int tid = threadIdx.x;
  auto part = [&](int cta) {
    return a.part + static_cast<int64_t>(2 * cta + (cta == c0 ? 1 : 0)) * kKv4PartFloats;
  };
  float M = -INFINITY;
  for (int k = c0 + (tid & 31); k <= c1; k += 32) M = fmaxf(M, part(k)[kKv4PartRows * kKv4D + 2 * r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float mu = M == -INFINITY ? 0.f : M;
  float acc = 0.f, ls = 0.f;
#pragma unroll 4
  for (int k = c0; k <= c1; ++k) {
    const float* p = part(k);
    const float2 ml = *reinterpret_cast<const float2*>(p + kKv4PartRows * kKv4D + 2 * r);
    const float w = ex2_approx(ml.x - mu);
    ls += w * ml.y;
    acc += w * p[r * kKv4D + tid];
  }
  const int64_t orow = static_cast<int64_t>(q.q0 + r / group) * a.Hq + h * group + r % group;
  const float f = ls == 0.f ? 0.f : *a.c.v_ts / ls;
  static_cast<T*>(a.out)[orow * kKv4D + tid] = static_cast<T>(acc * f);
  if (a.lse != nullptr && tid == 0) a.lse[orow] = ls == 0.f ? -INFINITY : (M + log2f(ls) - kPShift) * kLn2;
}

}  // namespace qk4v8
