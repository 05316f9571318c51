// Cached tokens and a chunk's own tokens as fp16 tensor-core operands: one warp
// turns 16 tokens (a subtile) of one (sequence, kv head) into rows of a
// 128-token key tile and value tile in shared memory.
//
// Both tiles are [128 token rows][128 channels] fp16 in two blocks of 64
// channels (128-byte rows, 128-byte swizzle: 16-byte piece p of row r is at
// piece p ^ (r % 8)).  Two free orders are used so that codes become operands
// without moving halves about:
//  * key channels: 8-channel pieces in the order (0,4,1,5,2,6,3,7) (the query
//    tile alike): masking a word of codes yields channels k and k + 4 together;
//  * token rows: row = token with its two lowest bits swapped (keys and values
//    alike): the value stores of eight lanes fall into eight different banks.
#pragma once

#include "kvq_chunk.cuh"
#include "kvq_rows.cuh"

namespace kvq {

constexpr int kKeys = 128;                       // tokens per key / value tile
constexpr int kSubs = kKeys / kTile;             // subtiles per tile
constexpr int kBlockBytes = kKeys * 128;         // one block of 64 channels
constexpr int kTileBytes16 = 2 * kBlockBytes;    // one key or value tile

__host__ __device__ constexpr int row_of_token(int t) { return (t & ~3) | ((t & 1) << 1) | ((t >> 1) & 1); }

// What the softmax has to know about a tile, one entry per subtile.
// kind 0: codes in the cache format's standard scaling; kind 1: fp16 rows in
// their own scaling; kind 2: the arrays say.  score = kmul * (row product),
// value = 2^vlog * (row); vinv = 2^-vlog.  bad: bit r, the token of row r
// holds a value that is not finite (its row is zero here); bit 16, the
// subtile's page id is out of range.
struct TileInfo {
  float kmul[kSubs], vlog[kSubs], vinv[kSubs];
  uint32_t bad[kSubs];
  uint8_t kind[kSubs];
};

__device__ __forceinline__ uint32_t f16_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// (w & mask) holds codes at 2^log2F of two halves -> the codes as exact halves
// (1024 + F * code, then x / F - 1024 / F in one exact fma).
template <int LOG2F>
__device__ __forceinline__ uint32_t codes_h2(uint32_t w, uint32_t mask) {
  constexpr uint32_t inv = (15u - LOG2F) << 10, off = 0x8000u | ((25u - LOG2F) << 10);
  return f16_fma(lop_or(w, mask, 0x64006400u), inv | (inv << 16), off | (off << 16));
}
// Bytes `sel` of w (nibbles 0 and 2 of sel; 1 and 3 are 4) -> exact halves.
__device__ __forceinline__ uint32_t bytes_h2(uint32_t w, uint32_t sel) {
  return f16_fma(prmt(w, 0x64646464u, sel), 0x3C003C00u, 0xE400E400u);
}
__device__ __forceinline__ void e4m3x4_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Address of 16-byte piece p (0..15: channels [8p, 8p + 8)) of row r of a tile at shared address `tile`.
__device__ __forceinline__ uint32_t piece_at(uint32_t tile, int r, int p) {
  return tile + (p >> 3) * kBlockBytes + r * 128 + (((p & 7) ^ (r & 7)) << 4);
}
// Eight channels of a key (or query) row, in the tile's channel order.
__device__ __forceinline__ void put_key8(uint32_t tile, int r, int p, const float (&x)[8]) {
  st_shared16(piece_at(tile, r, p), pack_h2(x[0], x[4]), pack_h2(x[1], x[5]), pack_h2(x[2], x[6]), pack_h2(x[3], x[7]));
}
__device__ __forceinline__ void put_value8(uint32_t tile, int r, int p, const float (&x)[8]) {
  st_shared16(piece_at(tile, r, p), pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]), pack_h2(x[6], x[7]));
}

// Largest finite magnitude of a subtile's rows -> the power e they are divided
// by (2^e): 0 unless fp16 would overflow or lose bits of the largest numbers,
// which otherwise come to [2^8, 2^9).  A bf16 number of 2^(e - 17) or more is
// then a half as it is; smaller ones are off by 2^(e - 25) at most.  (No less
// than 2^-90, whose inverse times a row's weights stays in fp32.)
constexpr int kLeastPower = -90;
__device__ __forceinline__ int tile_exponent(float amax) {
  if (amax == 0.f || (amax >= 0x1p-6f && amax < 0x1p15f)) return 0;
  return max((int)(__float_as_uint(amax) >> 23) - 127 - 8, kLeastPower);
}
// The same for values, whose power is a factor of the softmax weights too: P
// carries 2^e, so pieces of one row should not differ in e for no reason.
// Nothing is taken out of [2^-8, 2^15); smaller ones come to [2^-2, 2^-1), only
// so far up that a half holds them, larger ones to [2^8, 2^9); zeros hold back
// nobody's weights.  (With packed pieces always at e = 0 and small raw ones
// brought to 2^8, an INT cache whose values were all about 2^-13 gave its new
// tokens' weights 2^-21 of their size, in halves.)
constexpr float kLeastValue = 0x1p-8f;
__device__ __forceinline__ int value_exponent(float amax) {
  if (amax == 0.f) return kLeastPower;
  if (amax >= kLeastValue && amax < 0x1p15f) return 0;
  const int lg = (int)(__float_as_uint(amax) >> 23) - 127;
  return lg > 0 ? lg - 8 : max(lg + 2, kLeastPower);
}
// x * 2^e for |e| <= 252, in two steps so that neither factor overflows.
__device__ __forceinline__ float scale_by(float x, int e) {
  const int a = e / 2, b = e - a;
  return x * __uint_as_float((uint32_t)(a + 127) << 23) * __uint_as_float((uint32_t)(b + 127) << 23);
}
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;                 // NaN and infinities count as nothing
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}
// ---------------------------------------------------------------------------
// Whole quantized subtiles: codes -> exact halves -> one fma per pair
// ---------------------------------------------------------------------------

// The packed regions of one (sequence, kv head), for addresses of subtiles.
template <int FMT>
struct UnitSrc {
  const uint8_t *k, *v;        // contiguous: the unit's first row and tile; paged: the head's part of page 0
  const __half *km, *vm;
  const int32_t* pages;        // paged: the sequence's table row
  const uint8_t* widths;       // MIXED: the sequence's group widths
  size_t page_codes, page_km, page_vm;         // paged: steps from page to page
  int lg_group, num_pages;
  __device__ __forceinline__ void init(const kvq_cache& c, int b, int h) {
    const kvq_shape& s = c.shape;
    pages = nullptr;
    widths = nullptr;
    lg_group = 31 - __clz(s.group | 1);
    num_pages = s.num_pages;
    page_codes = page_km = page_vm = 0;
    if (s.page_size != 0) {
      pages = c.page_table + (size_t)b * s.max_pages_per_seq;
      page_codes = (size_t)s.num_kv_heads * tile_bytes(FMT);
      page_km = (size_t)s.num_kv_heads * 2 * kHeadDim;
      page_vm = (size_t)s.num_kv_heads * 2 * kTile;
      k = (const uint8_t*)c.k_codes + Addr::pg_k_codes(s, 0, h);
      km = (const __half*)c.k_meta + Addr::pg_k_meta(s, 0, h);
      v = (const uint8_t*)c.v_codes + Addr::pg_v_codes(s, 0, h);
      vm = (const __half*)c.v_meta + Addr::pg_v_meta(s, 0, h);
      return;
    }
    k = (const uint8_t*)c.k_codes + Addr::k_codes_unit(s, b, h);
    v = (const uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, 0);
    vm = FMT == 8 ? nullptr : (const __half*)c.v_meta + Addr::v_meta_token(s, b, h, 0);
    km = FMT == 8 ? nullptr
                  : (const __half*)c.k_meta + (FMT == 16 ? Addr::k_meta_token(s, b, h, 0) : Addr::k_meta_group(s, b, h, 0));
    if (FMT == 6) widths = c.group_bits + (size_t)b * (s.capacity / s.group);
  }
};

// Where the packed words of one subtile are.
struct SubSrc {
  const uint8_t *k, *v;
  const __half *km, *vm;
  bool two;                    // codes of 2 bits
};
// False if its page id is out of range.
template <int FMT>
__device__ __forceinline__ bool sub_src(const UnitSrc<FMT>& u, int tile, SubSrc& d) {
  d.two = FMT == 2;
  if (u.pages) {
    const int page = u.pages[tile];
    if (page < 0 || page >= u.num_pages) return false;
    d.k = u.k + page * u.page_codes;
    d.v = u.v + page * u.page_codes;
    d.km = u.km + page * u.page_km;
    d.vm = u.vm + page * u.page_vm;
    return true;
  }
  d.k = u.k + (size_t)tile * tile_bytes(FMT);
  d.v = u.v + (size_t)tile * tile_bytes(FMT);
  d.vm = u.vm + (size_t)tile * 2 * kTile;
  d.km = u.km;
  if constexpr (FMT == 16) {
    d.km = u.km + (size_t)tile * 2 * kTile;
  } else if constexpr (FMT != 8) {
    const int g = tile * kTile >> u.lg_group;
    d.km = u.km + (size_t)g * 2 * kHeadDim;
    if constexpr (FMT == 6) {
      d.two = u.widths[g] != 4;
      // a 2-bit group's key rows are packed from the start of its INT4 slot
      if (d.two) d.k -= (size_t)(tile * kTile - (g << u.lg_group)) * (kHeadDim / 4);
    }
  }
  return true;
}

// A subtile's packed words as one warp's lanes hold them.
template <int FMT> struct SubWords {
  static constexpr int kBits = FMT == 6 ? 4 : (FMT == 16 ? 8 : FMT);
  static constexpr int kKW = kBits == 8 ? 16 : 8;            // key words: 8 rows of one or two
  static constexpr int kVW = 2 * kBits;
  static constexpr int kKM = FMT == 8 ? 0 : (FMT == 2 || FMT == 6) ? 16 : 8;
  uint32_t k[kKW], v[kVW];
  uint32_t km[kKM ? kKM : 1];                                // key scales, then zeros, of the lane's channels (INT8: per row)
  uint32_t vm[FMT == 8 ? 1 : 4];                             // value (scale, zero) of the lane's four tokens
  uint32_t probe;                                            // that of token lane % 16, loaded with the keys (FP8: none)
};

// The value (scale, zero) of token lane % 16.
__device__ __forceinline__ uint32_t value_probe(const SubSrc& d) {
  return *reinterpret_cast<const uint32_t*>(d.vm + 2 * (threadIdx.x & 15));
}

template <int FMT>
__device__ __forceinline__ void load_keys(const SubSrc& d, SubWords<FMT>& w) {
  const int lane = threadIdx.x & 31, j = lane & 15, half = lane >> 4;
  const bool two = FMT == 2 || (FMT == 6 && d.two);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 2 * i + half;
    if constexpr (SubWords<FMT>::kBits == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(d.k + r * kHeadDim + 8 * j);
      w.k[2 * i] = x.x; w.k[2 * i + 1] = x.y;
    } else if (two) {
      w.k[i] = *reinterpret_cast<const uint16_t*>(d.k + r * (kHeadDim / 4) + 2 * j);
    } else {
      w.k[i] = *reinterpret_cast<const uint32_t*>(d.k + r * (kHeadDim / 2) + 4 * j);
    }
  }
  if constexpr (FMT != 8) w.probe = value_probe(d);
  if constexpr (FMT == 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w.km[i] = *reinterpret_cast<const uint32_t*>(d.km + 2 * (2 * i + half));
  } else if constexpr (FMT != 8) {
    // the words that hold this lane's 8 channels: scales, then zeros
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half* m = d.km + i * kHeadDim;
      if (two) {
        // word r of 8 holds channels (r, r + 8) of 16
        const uint4 a = *reinterpret_cast<const uint4*>(m + 16 * (j >> 1));
        const uint4 b = *reinterpret_cast<const uint4*>(m + 16 * (j >> 1) + 8);
        uint32_t* k = w.km + 8 * i;
        k[0] = a.x; k[1] = a.y; k[2] = a.z; k[3] = a.w;
        k[4] = b.x; k[5] = b.y; k[6] = b.z; k[7] = b.w;
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(m + 8 * j);   // pairs (0,2) (1,3) (4,6) (5,7)
        w.km[4 * i] = a.x; w.km[4 * i + 1] = a.y; w.km[4 * i + 2] = a.z; w.km[4 * i + 3] = a.w;
      }
    }
  }
}

template <int FMT>
__device__ __forceinline__ void load_values(const SubSrc& d, SubWords<FMT>& w) {
  const int lane = threadIdx.x & 31, l = lane & 3;
#pragma unroll
  for (int i = 0; i < SubWords<FMT>::kVW / 4; ++i) {
    if (FMT == 6 && d.two && i > 0) break;
    const uint4 x = *reinterpret_cast<const uint4*>(d.v + 512 * i + 16 * lane);
    w.v[4 * i] = x.x; w.v[4 * i + 1] = x.y; w.v[4 * i + 2] = x.z; w.v[4 * i + 3] = x.w;
  }
  if constexpr (FMT != 8) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w.vm[q] = *reinterpret_cast<const uint32_t*>(d.vm + 2 * (2 * l + (q & 1) + 8 * (q >> 1)));
  }
}

// Key rows of subtile `sub` into the key tile.  BITS: 2, 4 or 8.
template <int FMT, int BITS>
__device__ __forceinline__ void keys_to_tile(const SubWords<FMT>& w, uint32_t tile, int sub) {
  const int lane = threadIdx.x & 31, j = lane & 15, half = lane >> 4;
  const uint32_t base = tile + (j >> 3) * kBlockBytes + (kTile * sub + 2 * half) * 128;
  const uint32_t p = (uint32_t)((j & 7) ^ (2 * half));
  uint32_t sc[4], zc[4];                         // scales and zeros of channels (k, k + 4)
  if constexpr (FMT != 8 && FMT != 16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BITS == 2) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        sc[k] = prmt(w.km[k], w.km[4 + k], sel);
        zc[k] = prmt(w.km[8 + k], w.km[12 + k], sel);
      } else {
        sc[k] = prmt(w.km[k & 1], w.km[2 + (k & 1)], k < 2 ? 0x5410u : 0x7632u);
        zc[k] = prmt(w.km[4 + (k & 1)], w.km[6 + (k & 1)], k < 2 ? 0x5410u : 0x7632u);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {                  // token row 2i + half -> tile row 4 (i / 2) + 2 half + i % 2
    const uint32_t at = base + (4 * (i >> 1) + (i & 1)) * 128 + ((p ^ (4 * ((i >> 1) & 1) + (i & 1))) << 4);
    uint32_t x[4];
    if constexpr (BITS == 4) {
      const uint32_t a = w.k[i], b = a >> 8;     // nibble k = channel k
      x[0] = codes_h2<0>(a, 0x000F000Fu); x[1] = codes_h2<4>(a, 0x00F000F0u);
      x[2] = codes_h2<0>(b, 0x000F000Fu); x[3] = codes_h2<4>(b, 0x00F000F0u);
    } else if constexpr (BITS == 2) {
      const uint32_t a = prmt(w.k[i], 0u, 0x4140u);          // channels 0-3 low half, 4-7 high half
      x[0] = codes_h2<0>(a, 0x00030003u); x[1] = codes_h2<2>(a, 0x000C000Cu);
      x[2] = codes_h2<4>(a, 0x00300030u); x[3] = codes_h2<6>(a, 0x00C000C0u);
    } else {
      const uint32_t a = prmt(w.k[2 * i], w.k[2 * i + 1], 0x5140u);   // bytes of channels 0, 4, 1, 5
      const uint32_t b = prmt(w.k[2 * i], w.k[2 * i + 1], 0x7362u);   // 2, 6, 3, 7
      if constexpr (FMT == 8) {
        e4m3x4_h2(a, x[0], x[1]);
        e4m3x4_h2(b, x[2], x[3]);
      } else {
        x[0] = bytes_h2(a, 0x4140u); x[1] = bytes_h2(a, 0x4342u);
        x[2] = bytes_h2(b, 0x4140u); x[3] = bytes_h2(b, 0x4342u);
      }
    }
    if constexpr (FMT == 16) {
      const uint32_t s = prmt(w.km[i], 0u, 0x1010u), z = prmt(w.km[i], 0u, 0x3232u);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = f16_fma(x[k], s, z);
    } else if constexpr (FMT != 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = f16_fma(x[k], sc[k], zc[k]);
    }
    st_shared16(at, x[0], x[1], x[2], x[3]);
  }
}

// Value rows of subtile `sub` into the value tile: lane (n, l) has channels
// [16n, 16n + 16) of tokens 2l, 2l + 1, 2l + 8, 2l + 9.
template <int FMT, int BITS>
__device__ __forceinline__ void values_to_tile(const SubWords<FMT>& w, uint32_t tile, int sub) {
  const int lane = threadIdx.x & 31, n = lane >> 2, l = lane & 3;
  const int r0 = 4 * (l >> 1) + (l & 1);         // tile row of token 2l; 2l + 1 is two rows on, 2l + 8 eight
  const uint32_t base = tile + (n >> 2) * kBlockBytes + (kTile * sub + r0) * 128;
  const uint32_t p = (uint32_t)((2 * (n & 3)) ^ r0);
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    uint32_t x[4][4];                            // [token 2l + q % 2 + 8 (q / 2)][channel pair]
    if constexpr (BITS == 8) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t w0 = w.v[8 * hh + 2 * c], w1 = w.v[8 * hh + 2 * c + 1];   // byte q = token q
        const uint32_t a = prmt(w0, w1, 0x5140u), b = prmt(w0, w1, 0x7362u);
        if constexpr (FMT == 8) {
          e4m3x4_h2(a, x[0][c], x[1][c]);
          e4m3x4_h2(b, x[2][c], x[3][c]);
        } else {
          x[0][c] = bytes_h2(a, 0x4140u);
          x[1][c] = bytes_h2(a, 0x4342u);
          x[2][c] = bytes_h2(b, 0x4140u);
          x[3][c] = bytes_h2(b, 0x4342u);
        }
      }
      if constexpr (FMT == 16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t s = prmt(w.vm[q], 0u, 0x1010u), z = prmt(w.vm[q], 0u, 0x3232u);
#pragma unroll
          for (int c = 0; c < 4; ++c) x[q][c] = f16_fma(x[q][c], s, z);
        }
      }
    } else {
#pragma unroll
      for (int o = 0; o < 2; ++o) {              // the pair of tokens (2l + o, 2l + o + 8) sits in one word's halves
        const uint32_t s = prmt(w.vm[o], w.vm[o + 2], 0x5410u), z = prmt(w.vm[o], w.vm[o + 2], 0x7632u);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t e, f;                         // channels 8hh + 2c and 8hh + 2c + 1
          if constexpr (BITS == 4) {
            const uint32_t a = o ? w.v[4 * hh + c] >> 8 : w.v[4 * hh + c];
            e = codes_h2<0>(a, 0x000F000Fu);
            f = codes_h2<4>(a, 0x00F000F0u);
          } else {
            const uint32_t v = w.v[2 * hh + (c >> 1)];
            if (o == 0) {
              e = (c & 1) ? codes_h2<4>(v, 0x00300030u) : codes_h2<0>(v, 0x00030003u);
              f = (c & 1) ? codes_h2<6>(v, 0x00C000C0u) : codes_h2<2>(v, 0x000C000Cu);
            } else {
              const uint32_t a = v >> 8;
              e = (c & 1) ? codes_h2<4>(a, 0x00300030u) : codes_h2<0>(a, 0x00030003u);
              f = (c & 1) ? codes_h2<6>(a, 0x00C000C0u) : codes_h2<2>(a, 0x000C000Cu);
            }
          }
          e = f16_fma(e, s, z);
          f = f16_fma(f, s, z);
          x[o][c] = prmt(e, f, 0x5410u);
          x[o + 2][c] = prmt(e, f, 0x7632u);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st_shared16(base + (2 * (q & 1) + 8 * (q >> 1)) * 128 + ((p ^ hh ^ (2 * (q & 1))) << 4), x[q][0], x[q][1], x[q][2],
                  x[q][3]);
  }
}

// ---------------------------------------------------------------------------
// Any other subtile
// ---------------------------------------------------------------------------

// Rows of a subtile that are not quantized: token t = base + r from the window
// ring (t < n), from the chunk (t < total) or none (zero).
struct RawRows {
  const uint16_t* ring;        // slot 0 of the unit's ring
  const uint16_t* fresh;       // the chunk's row of token n for this head
  int64_t stride;              // between chunk rows
  int n, total, slots;         // (slots >= 16)
  int slot0;                   // slot of token base
  // Piece p (8 channels) of row r; t = base + r.
  __device__ __forceinline__ uint4 load(int t, int r, int p) const {
    int slot = slot0 + r;
    if (slot >= slots) slot -= slots;
    const uint16_t* src = t < n ? ring + (size_t)slot * kHeadDim : fresh + (t - n) * stride;
    return t < total ? *reinterpret_cast<const uint4*>(src + 8 * p) : make_uint4(0u, 0u, 0u, 0u);
  }
};

// Largest of two packed pairs of bf16 magnitudes (sign bits cleared; the bit
// patterns are in order, infinities and NaN on top).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t abs_max8(uint32_t m, const uint4& w) {
  return abs_max2(abs_max2(abs_max2(abs_max2(m, w.x), w.y), w.z), w.w);
}
__device__ __forceinline__ uint32_t larger_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// A largest bf16 magnitude that fp16 takes as it is: 0, or in [2^-6, 2^15).
__device__ __forceinline__ bool ordinary(uint32_t m) { return m == 0u || (m >= 0x3C80u && m < 0x4700u); }
// The same for values: in [2^-8, 2^15).
__device__ __forceinline__ bool ordinary_value(uint32_t m) { return m >= 0x3B80u && m < 0x4700u; }

// Eight bf16 numbers -> four fp16 pairs, in the key tiles' channel order or in order.
__device__ __forceinline__ void put_raw8(uint32_t at, const uint4& w, bool key) {
  const float x0 = bf16_lo(w.x), x1 = bf16_hi(w.x), x2 = bf16_lo(w.y), x3 = bf16_hi(w.y);
  const float x4 = bf16_lo(w.z), x5 = bf16_hi(w.z), x6 = bf16_lo(w.w), x7 = bf16_hi(w.w);
  st_shared16(at, pack_h2(x0, key ? x4 : x1), pack_h2(key ? x1 : x2, key ? x5 : x3),
              pack_h2(key ? x2 : x4, key ? x6 : x5), pack_h2(key ? x3 : x6, x7));
}

// Sixteen bf16 rows, as loaded (piece lane % 16 of rows 2i + lane / 16), into a
// tile.  False, and nothing written, if a number is not finite or the
// magnitudes need a power of two taken out.  gone: none of the rows is a token.
struct RawWords {
  uint4 w[8];
};
__device__ __forceinline__ void load_rows(const RawRows& raw, int base, RawWords& x) {
  const int lane = threadIdx.x & 31, p = lane & 15, half = lane >> 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) x.w[i] = raw.load(base + 2 * i + half, 2 * i + half, p);
}
__device__ __forceinline__ bool rows_to_tile(const RawWords& x, uint32_t tile, int sub, bool key, bool gone) {
  const int lane = threadIdx.x & 31, p = lane & 15, half = lane >> 4;
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = abs_max8(m, x.w[i]);
  m = __reduce_max_sync(0xffffffffu, larger_half(m));
  if (!(key ? ordinary(m) : ordinary_value(m) || (gone && m == 0u))) return false;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    put_raw8(piece_at(tile, kTile * sub + 4 * (i >> 1) + 2 * half + (i & 1), p), x.w[i], key);
  return true;
}

// Non-zero if code * scale + zero may leave fp16's range for a (scale, zero)
// pair: |zero| >= 2^15, or scale >= 2^11 (INT8: 2^7); below both it is less
// than 65504.
template <int FMT>
__device__ __forceinline__ uint32_t past_half(uint32_t m) {
  constexpr uint32_t top = FMT == 16 ? 0x5800u : 0x6800u;
  return ((m & 0x7FFF7FFFu) + (((0x8000u - 0x7800u) << 16) | (0x8000u - top))) & 0x80008000u;
}

// Values of the subtile's tokens from `quant` on -> zero.
template <int FMT>
__device__ __forceinline__ void drop_values(SubWords<FMT>& w, int quant) {
  const int l = threadIdx.x & 3;
  uint32_t keep = 0u;                            // byte q of every 8-bit word is token 2l + q % 2 + 8 (q / 2)
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bool in = 2 * l + (q & 1) + 8 * (q >> 1) < quant;
    if (in) keep |= 0xFFu << (8 * q);
    if constexpr (FMT != 8)
      if (!in) w.vm[q] = 0u;
  }
#pragma unroll
  for (int i = 0; i < SubWords<FMT>::kVW; ++i)
    if (SubWords<FMT>::kBits == 8) w.v[i] &= keep;
}

// Whether a value of the subtile could be anything but a finite half (its
// scale and zero are large, or it holds an e4m3 NaN): to be looked at closely
// where a row may not see it, since 0 times such a value is NaN.
template <int FMT>
__device__ __forceinline__ bool values_odd(const SubWords<FMT>& w) {
  uint32_t odd = 0u;
  if constexpr (FMT == 8) {
#pragma unroll
    for (int i = 0; i < SubWords<FMT>::kVW; ++i) odd |= ((w.v[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) odd |= past_half<FMT>(w.vm[q]);
  }
  return __any_sync(0xffffffffu, odd != 0u);
}

// The most that code * scale + zero can be in magnitude (infinities and NaN
// come out on top as bit patterns, sign aside).
template <int FMT>
__device__ __forceinline__ float most_of(uint32_t m, bool two) {
  const float top = FMT == 16 ? 255.f : FMT == 2 || (FMT == 6 && two) ? 3.f : 15.f;
  return fmaf(top, __low2float(u32_as_h2(m)), fabsf(__high2float(u32_as_h2(m))));
}

// The scales and zeros of the lane's values times 2^e, 0 <= e <= 15 (exact).
template <int FMT>
__device__ __forceinline__ void scale_values(SubWords<FMT>& w, int e) {
  const uint32_t f = (uint32_t)(15 + e) << 10;
#pragma unroll
  for (int q = 0; q < 4; ++q) asm("mul.rn.f16x2 %0, %0, %1;\n" : "+r"(w.vm[q]) : "r"(f | (f << 16)));
}

// Non-zero if a key of the lane could be anything but a finite half: code *
// scale + zero is taken in halves on the way to the tiles, and may pass 65504
// where scale and zero do not (minimum 0 and maximum 100000 make an INT4 scale
// of 6668).  FP8 codes are halves as they are.
template <int FMT>
__device__ __forceinline__ uint32_t keys_past(const SubWords<FMT>& w, bool two) {
  uint32_t odd = 0u;
  if constexpr (FMT == 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) odd |= past_half<FMT>(w.km[i]);
  } else if constexpr (FMT != 8) {
    auto larger = [](uint32_t a, uint32_t b) {               // of the magnitudes; NaN stays
      return h2_as_u32(__hmax2_nan(__habs2(u32_as_h2(a)), __habs2(u32_as_h2(b))));
    };
    uint32_t sc, ze;
    if (FMT == 2 || (FMT == 6 && two)) {
      constexpr int z = SubWords<FMT>::kKM / 2;
      sc = larger(larger(larger(w.km[0], w.km[1]), larger(w.km[2], w.km[3])),
                  larger(larger(w.km[4], w.km[5]), larger(w.km[6], w.km[7])));
      ze = larger(larger(larger(w.km[z], w.km[z + 1]), larger(w.km[z + 2], w.km[z + 3])),
                  larger(larger(w.km[z + 4], w.km[z + 5]), larger(w.km[z + 6], w.km[z + 7])));
    } else {
      sc = larger(larger(w.km[0], w.km[1]), larger(w.km[2], w.km[3]));
      ze = larger(larger(w.km[4], w.km[5]), larger(w.km[6], w.km[7]));
    }
    odd |= past_half<FMT>(prmt(sc, ze, 0x5410u)) | past_half<FMT>(prmt(sc, ze, 0x7632u));
  }
  return odd;
}

// Non-zero unless code * scale + zero stays below kLeastValue: |zero| < 2^-9 and
// scale < 2^-13 (INT2: 2^-11, INT8: 2^-17).
template <int FMT>
__device__ __forceinline__ uint32_t not_small(uint32_t m) {
  constexpr uint32_t least = FMT == 16 ? 0x0080u : FMT == 2 ? 0x1000u : 0x0800u;
  return ((m & 0x7FFF7FFFu) + (((0x8000u - 0x1800u) << 16) | (0x8000u - least))) & 0x80008000u;
}

// Whether a subtile needs a closer look, from the words that load_keys has: a
// key or value may not be a finite half, or all values are small, and a power
// of two is taken out.  Cost: 1 % of 2048 tokens over 16384 (760 us), 3 % of
// MIXED, whose producers are the bound (836 us).
template <int FMT>
__device__ __forceinline__ bool words_odd(const SubWords<FMT>& w, bool two) {
  if constexpr (FMT == 8) {
    return false;
  } else {
    return __any_sync(0xffffffffu, (keys_past<FMT>(w, two) | past_half<FMT>(w.probe)) != 0u) ||
           !__any_sync(0xffffffffu, not_small<FMT>(w.probe) != 0u);
  }
}

__device__ __forceinline__ void rope8(float (&x)[8], int t, int ch, const double* freq) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float c, s;
    rope_cos_sin(t, freq[ch / 2 + i], c, s);
    const float a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = a * c - b * s;
    x[2 * i + 1] = a * s + b * c;
  }
}

// Keys of a subtile from token `base` on: the first `quant` rows from the
// packed tile d, the others raw.  Two passes (largest magnitude, then the
// rows), so that any range of numbers fits.  Returns the power of two taken out.
template <int FMT>
__device__ __noinline__ int keys_any(const TileSrc& d, int quant, const RawRows& raw, int base, const double* freq,
                                     uint32_t tile, int sub) {
  const int lane = threadIdx.x & 31, p = lane & 15, half = lane >> 4;
  float amax = 0.f;
  int e = 0;
  for (int pass = 0; pass < 2; ++pass) {
    auto one = [&](int r, int ch, const float (&x)[8]) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
      if (pass == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(y[i]));
        return;
      }
      if (freq) rope8(y, base + r, ch, freq);
      if (e != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = scale_by(y[i], -e);
      }
      put_key8(tile, kTile * sub + row_of_token(r), ch / 8, y);
    };
    if (quant > 0) key_rows<FMT>(d, 0, quant, one);
    for (int r = quant + half; r < kTile; r += 2) {
      float x[8];
      unpack8(raw.load(base + r, r, p), x);
      one(r, 8 * p, x);
    }
    if (pass == 0) e = tile_exponent(warp_max(amax) * (freq ? 1.5f : 1.f));   // a rotation grows a pair by sqrt 2 at most
  }
  return e;
}

// Values alike; rows with a value that is not finite become zero and set
// their tile row's bit in `bad`.
template <int FMT>
__device__ __noinline__ int values_any(const TileSrc& d, int quant, const RawRows& raw, int base, uint32_t tile, int sub,
                                       uint32_t& bad) {
  const int lane = threadIdx.x & 31, p = lane & 15, half = lane >> 4;
  float amax = 0.f;
  uint32_t mine = 0u;                            // bad tokens this lane has seen
  int e = 0;
  for (int pass = 0; pass < 2; ++pass) {
    auto one = [&](int r, int ch, const float (&x)[8]) {
      float y[8];
      const bool zero = pass == 1 && (mine >> r & 1u);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = zero ? 0.f : x[i];
      if (pass == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          amax = fmaxf(amax, finite_abs(y[i]));
          if (!(fabsf(y[i]) < INFINITY)) mine |= 1u << r;
        }
        return;
      }
      if (e != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = scale_by(y[i], -e);
      }
      put_value8(tile, kTile * sub + row_of_token(r), ch / 8, y);
    };
    if (quant > 0)
      value_rows<FMT>(d, 0, quant, [&](int r, int ch, const float (&x)[16]) {
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = x[i];
          b[i] = x[8 + i];
        }
        one(r, ch, a);
        one(r, ch + 8, b);
      });
    for (int r = quant + half; r < kTile; r += 2) {
      float x[8];
      unpack8(raw.load(base + r, r, p), x);
      one(r, 8 * p, x);
    }
    if (pass == 0) {
      e = value_exponent(warp_max(amax));
      mine = __reduce_or_sync(0xffffffffu, mine);
    }
  }
  bad = 0u;
  for (int r = 0; r < kTile; ++r) bad |= (mine >> r & 1u) << row_of_token(r);
  return e;
}

__device__ __forceinline__ void zero_rows(uint32_t tile, int sub) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 8; ++i) st_shared16(piece_at(tile, kTile * sub + 2 * i + (lane >> 4), lane & 15), 0u, 0u, 0u, 0u);
}

}  // namespace kvq
