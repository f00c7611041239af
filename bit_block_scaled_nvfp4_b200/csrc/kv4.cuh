// The 4-bit paged cache: tokens quantized into it and read back. K and V in NVFP4, every token on
// its own (quantize.cuh's block arithmetic with the cache's fixed tensor scales); layout in
// include/qk4v8.h.
//
// One thread per (token, KV head, 16-channel block). V bytes hold two tokens, so the thread of
// an even position writes both tokens' nibbles when the odd one is new too, and a token whose
// neighbour is not part of the call keeps the neighbour's nibble; no two threads write one byte.
// A CTA's 256 threads cover consecutive rows; the first row's sequence is found by counting the
// offsets not past it (all threads, one pass over cu), later rows walk on from there.
//
// Bound: HBM; stored are 512 bytes of K and V in and 144 out a token and head, read back the reverse. 30000
// tokens of 8 heads stored and read back take 97 us on the device, 3.3 TB/s of 6.5: what is left is the
// encoder's arithmetic (about 115 instructions a block) and V's scales, one or two bytes a 64-byte row
// apart. 64 tokens, one a sequence, take 8.4 us for both calls: two launches.
#pragma once
#include "quantize.cuh"

namespace qk4v8 {

struct Kv4Cache {
  uint8_t* k_pages;
  uint8_t* k_scales;
  const float* k_ts;
  uint8_t* v_pages;
  uint8_t* v_scales;
  const float* v_ts;
  int32_t num_pages, Hkv;
};

struct Kv4TokensArgs {
  Kv4Cache c;
  void* k;
  void* v;
  int64_t k_stride, v_stride;
  const int32_t* cu;
  const int32_t* start;
  const int32_t* page_table;
  int32_t total, S, max_pages;
};

constexpr int kKv4D = 128, kKv4Blocks = kKv4D / 16;   // head dimension; scale blocks a token

// Number of cu[1..S] not past `row` = the sequence of that row (S when it is behind the last),
// by every thread of the CTA.
__device__ __forceinline__ int kv4_seq_of_row(const int32_t* cu, int S, int row) {
  int n = 0;
  for (int i0 = 0; i0 < S; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    n += __syncthreads_count(i < S && cu[i + 1] <= row);
  }
  return n;
}

// A token's place in the cache: physical page and slot. false (and the status word set) when it
// has none.
struct Kv4Place {
  int page, slot;
};
__device__ __forceinline__ bool kv4_place(const Kv4TokensArgs& a, int s, int pos, bool flag,
                                          Kv4Place& pl) {
  if (a.start[s] < 0 || pos < 0 || (pos >> 6) >= a.max_pages) {
    if (flag) flag_error(kStatusBounds);
    return false;
  }
  pl.page = a.page_table[static_cast<int64_t>(s) * a.max_pages + (pos >> 6)];
  pl.slot = pos & 63;
  if (pl.page < 0 || pl.page >= a.c.num_pages) {
    if (flag) flag_error(kStatusBounds);
    return false;
  }
  return true;
}

// Eight nibbles -> the low nibbles of eight bytes.
__device__ __forceinline__ uint2 nibbles_to_bytes(uint32_t w) {
  uint32_t lo = w & 0xFFFFu, hi = w >> 16;
  lo = (lo | (lo << 8)) & 0x00FF00FFu;
  hi = (hi | (hi << 8)) & 0x00FF00FFu;
  return make_uint2((lo | (lo << 4)) & 0x0F0F0F0Fu, (hi | (hi << 4)) & 0x0F0F0F0Fu);
}

// The row of this thread, its sequence and position; false when it has none.
struct Kv4Job {
  int row, s, pos, last, h, b;      // last: the row is its sequence's last
};
__device__ __forceinline__ bool kv4_job(const Kv4TokensArgs& a, Kv4Job& j) {
  // item blockIdx * 256 + threadIdx = row * per_row + rest, in 32-bit divisions (a 64-bit one takes
  // longer than the encoding of a block): 256 (x per_row + y) = 256 x rows and 256 y items
  const uint32_t per_row = a.c.Hkv * kKv4Blocks;
  const uint32_t x = blockIdx.x / per_row, y = 256 * (blockIdx.x - x * per_row);
  const uint32_t first = y / per_row, at = y - first * per_row + threadIdx.x, more = at / per_row;
  const uint32_t row0 = 256 * x + first, row = row0 + more, rest = at - more * per_row;
  int s = kv4_seq_of_row(a.cu, a.S, static_cast<int>(row0));
  if (row >= static_cast<uint32_t>(a.total)) return false;
  j.row = static_cast<int>(row);
  j.h = rest / kKv4Blocks;
  j.b = rest % kKv4Blocks;
  while (s < a.S && a.cu[s + 1] <= j.row) ++s;
  if (s >= a.S || a.cu[s] > j.row) return false;      // behind the last sequence
  j.s = s;
  // 64 bits: a start near the top of 32 bits must not wrap to a valid position
  const int64_t pos = static_cast<int64_t>(a.start[s]) + (j.row - a.cu[s]);
  j.pos = pos > 0x7fffffff ? -1 : static_cast<int>(pos);
  j.last = j.row + 1 >= a.cu[s + 1] || j.row + 1 >= a.total;
  return true;
}

template <typename T>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4TokensArgs a) {
  __shared__ float2 tab[2][128];                       // nvfp4_den_table of K's and V's tensor scale
  // (scales are positive; a negative one must not lead past the tables)
  const float k_ts = fabsf(*a.c.k_ts), v_ts = fabsf(*a.c.v_ts);
  nvfp4_den_table(k_ts, tab[0]);
  nvfp4_den_table(v_ts, tab[1]);
  Kv4Job j;
  const bool mine = kv4_job(a, j);
  __syncthreads();
  if (!mine) return;
  Kv4Place pl;
  if (!kv4_place(a, j.s, j.pos, true, pl)) return;
  const bool odd = pl.slot & 1, pair = !odd && !j.last;
  const bool v_too = !odd || j.row == a.cu[j.s];       // else written by the even token's thread
  const int64_t head = static_cast<int64_t>(pl.page) * a.c.Hkv + j.h;
  const int64_t in = j.h * kKv4D + j.b * 16;
  const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + j.row * a.k_stride + in);
  const T* vr = static_cast<const T*>(a.v) + j.row * a.v_stride + in;
  const uint4* vs = reinterpret_cast<const uint4*>(vr);
  const uint4* vs1 = reinterpret_cast<const uint4*>(vr + a.v_stride);
  uint4* dst = reinterpret_cast<uint4*>(a.c.v_pages + (head * 32 + (pl.slot >> 1)) * kKv4D + j.b * 16);
  uint4 k[2], v[2], v1[2], old;                        // all loads before the first use
  k[0] = __ldg(ks);
  k[1] = __ldg(ks + 1);
  if (v_too) {
    v[0] = __ldg(vs);
    v[1] = __ldg(vs + 1);
    if (pair) {
      v1[0] = __ldg(vs1);
      v1[1] = __ldg(vs1 + 1);
    } else {
      old = *dst;                                      // the pair's other token is not new
    }
  }
  uint32_t w[2];
  const int64_t tok = head * 64 + pl.slot;
  const uint32_t sc = nvfp4_encode16_packed<T, false>(k, k_ts, __frcp_rn(k_ts), tab[0], w, nullptr);
  *reinterpret_cast<uint2*>(a.c.k_pages + tok * (kKv4D / 2) + j.b * 8) = make_uint2(w[0], w[1]);
  a.c.k_scales[tok * kKv4Blocks + j.b] = static_cast<uint8_t>(sc);
  if (!v_too) return;
  const float y_t = __frcp_rn(v_ts);
  uint8_t* sdst = a.c.v_scales + (head * kKv4Blocks + j.b) * 64 + pl.slot;
  const uint32_t s0 = nvfp4_encode16_packed<T, false>(v, v_ts, y_t, tab[1], w, nullptr);
  const uint2 c0 = nibbles_to_bytes(w[0]), c1 = nibbles_to_bytes(w[1]);
  uint32_t o[4] = {c0.x, c0.y, c1.x, c1.y};
  if (pair) {
    const uint32_t s1 = nvfp4_encode16_packed<T, false>(v1, v_ts, y_t, tab[1], w, nullptr);
    const uint2 d0 = nibbles_to_bytes(w[0]), d1 = nibbles_to_bytes(w[1]);
    o[0] |= d0.x << 4; o[1] |= d0.y << 4; o[2] |= d1.x << 4; o[3] |= d1.y << 4;
    *reinterpret_cast<uint16_t*>(sdst) = static_cast<uint16_t>(s0 | (s1 << 8));
  } else {
    const uint32_t* ow = reinterpret_cast<const uint32_t*>(&old);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = odd ? (ow[i] & 0x0F0F0F0Fu) | (o[i] << 4) : (ow[i] & 0xF0F0F0F0u) | o[i];
    *sdst = static_cast<uint8_t>(s0);
  }
  *dst = make_uint4(o[0], o[1], o[2], o[3]);
}

// E2M1 pairs of a word's four bytes -> half2 each (low half: low nibble).
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// Bit 7 of each byte that is one of E4M3's two NaN codes.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Two values v0, v1 -> one packed word of T (16-bit types).
template <typename T> __device__ __forceinline__ uint32_t pack2(float v0, float v1);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float v0, float v1) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(v0, v1);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float v0, float v1) {
  const __half2 t = __floats2half2_rn(v0, v1);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <typename T>
__device__ __forceinline__ void store16(T* dst, const float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(dst)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4TokensArgs a) {
  Kv4Job j;
  if (!kv4_job(a, j)) return;
  Kv4Place pl;
  if (!kv4_place(a, j.s, j.pos, true, pl)) return;
  const int64_t head = static_cast<int64_t>(pl.page) * a.c.Hkv + j.h;
  const int64_t in = j.h * kKv4D + j.b * 16;
  const int64_t tok = head * 64 + pl.slot;
  const uint2 kc = *reinterpret_cast<const uint2*>(a.c.k_pages + tok * (kKv4D / 2) + j.b * 8);
  const uint4 vc = *reinterpret_cast<const uint4*>(a.c.v_pages + (head * 32 + (pl.slot >> 1)) * kKv4D + j.b * 16);
  // code * scale has at most six significant bits: exact; one rounding by the tensor scale
  const __half2 ks = e4m3x2_to_half2(a.c.k_scales[tok * kKv4Blocks + j.b] * 0x101u);
  const __half2 vs = e4m3x2_to_half2(a.c.v_scales[(head * kKv4Blocks + j.b) * 64 + pl.slot] * 0x101u);
  const float kt = *a.c.k_ts, vt = *a.c.v_ts;
  float f[16];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t d[4];
    e2m1x8_to_half2(i ? kc.y : kc.x, d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t t = hmul2(d[e], ks);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&t));
      f[8 * i + 2 * e] = __fmul_rn(x.x, kt);
      f[8 * i + 2 * e + 1] = __fmul_rn(x.y, kt);
    }
  }
  store16<T>(static_cast<T*>(a.k) + j.row * a.k_stride + in, f);
  const uint32_t* vw = reinterpret_cast<const uint32_t*>(&vc);
  const uint32_t half = (pl.slot & 1) ? 0x7632u : 0x5410u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t d[4];                                     // a channel's two tokens each
    e2m1x8_to_half2(vw[i], d);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const uint32_t t = hmul2(__byte_perm(d[e], d[e + 1], half), vs);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&t));
      f[4 * i + e] = __fmul_rn(x.x, vt);
      f[4 * i + e + 1] = __fmul_rn(x.y, vt);
    }
  }
  store16<T>(static_cast<T*>(a.v) + j.row * a.v_stride + in, f);
}

}  // namespace qk4v8
