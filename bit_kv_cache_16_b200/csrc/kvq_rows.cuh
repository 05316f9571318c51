// Reading quantized tokens back, one 16-token tile of one (sequence, kv head)
// per warp: x^ = code * scale + zero in fp32 (e4m3 code * scale for FP8), for
// the kernels that need rows of numbers rather than tensor-core fragments.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

// Where tile `tile` (tokens [16 tile, 16 tile + 16)) of a unit is stored.
struct TileSrc {
  const uint8_t* k;        // key row of the tile's token 0
  const __half* km;        // INT2/INT4: [2][128] of the tile's group; INT8: [16][2]
  const uint8_t* v;        // the value tile
  const __half* vm;        // [16][2] (unused for FP8)
  const uint32_t* ksp;     // dense-and-sparse: [128] kept keys of the group, else null
  const uint32_t* vsp;     // dense-and-sparse: [16] kept values, else null
  float ks, vs;            // FP8: the head's static scales
  int bits;                // width of the codes: 2, 4 or 8
  int t0;                  // the tile's first token within its group
};

// False if the tile's page id is out of range.
template <int FMT>
__device__ __forceinline__ bool tile_src(const kvq_cache& c, int b, int h, int tile, TileSrc& d) {
  const kvq_shape& s = c.shape;
  d.ksp = d.vsp = nullptr;
  d.ks = d.vs = 1.f;
  d.bits = FMT == 16 ? 8 : FMT;
  d.t0 = 0;
  if (s.page_size != 0) {
    const int page = c.page_table[(size_t)b * s.max_pages_per_seq + tile];
    if (page < 0 || page >= s.num_pages) return false;
    d.k = (const uint8_t*)c.k_codes + Addr::pg_k_codes(s, page, h);
    d.km = (const __half*)c.k_meta + Addr::pg_k_meta(s, page, h);
    d.v = (const uint8_t*)c.v_codes + Addr::pg_v_codes(s, page, h);
    d.vm = (const __half*)c.v_meta + Addr::pg_v_meta(s, page, h);
    return true;
  }
  const size_t unit = (size_t)b * s.num_kv_heads + h;
  d.k = (const uint8_t*)c.k_codes + Addr::k_codes_unit(s, b, h) + (size_t)tile * tile_bytes(FMT);
  d.v = (const uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, tile);
  d.km = nullptr;
  d.vm = (const __half*)c.v_meta + Addr::v_meta_token(s, b, h, tile * kTile);
  if constexpr (FMT == 8) {
    d.ks = c.fp8_scale[h];
    d.vs = c.fp8_scale[s.num_kv_heads + h];
  } else if constexpr (FMT == 16) {
    d.km = (const __half*)c.k_meta + Addr::k_meta_token(s, b, h, tile * kTile);
  } else {
    const int g = tile * kTile / s.group;
    d.t0 = tile * kTile - g * s.group;
    d.km = (const __half*)c.k_meta + Addr::k_meta_group(s, b, h, g);
    if constexpr (FMT == 6) {
      d.bits = c.group_bits[(size_t)b * (s.capacity / s.group) + g] == 4 ? 4 : 2;
      // a 2-bit group's key rows are packed from the start of its INT4 slot
      if (d.bits == 2) d.k -= (size_t)d.t0 * (kHeadDim / 4);
    }
    if (s.sparse) {
      d.ksp = c.k_sparse + (unit * (size_t)(s.capacity / s.group) + g) * kHeadDim;
      d.vsp = c.v_sparse + unit * (size_t)s.capacity + (size_t)tile * kTile;
    }
  }
  return true;
}

// Codes -> numbers, two at a time, each rounded as the scalar steps would be:
// a code of `bits` bits at bit `pos` of w (pos + bits <= 23), OR-ed into the
// mantissa of 2^23, is 2^23 + 2^pos code; the difference is exact, and 2^-pos is
// taken up by the scale (a power of two: exact), so that x^ = code * s + z is
// one fp32 fma.
constexpr uint32_t kMagic = 0x4B000000u;     // 2^23
__device__ __forceinline__ pair_t magic_codes(uint32_t a, uint32_t b) {
  return pair_add(pair(__uint_as_float(a), __uint_as_float(b)), pair(-8388608.f, -8388608.f));
}
__device__ __forceinline__ float pow2_neg(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }
__device__ __forceinline__ float e4m3_f32(uint32_t byte) { return __half2float(u32_as_h2(e4m3x2_to_h2(byte)).x); }

// Key rows: lane owns channels [8j, 8j + 8), j = lane % 16, of the tile's rows
// 2i + lane / 16; emit(row, channel, x[8]) for each of rows [lo, hi).
// SP: dense-and-sparse.
template <int BITS, bool PER_TOKEN, bool SP, class Emit>
__device__ __forceinline__ void key_rows_bits(const TileSrc& d, int lo, int hi, Emit emit) {
  const int lane = threadIdx.x & 31, j = lane & 15, half = lane >> 4;
  float s[8], z[8];
  uint32_t kept[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = d.ks;                    // FP8: code * scale
    z[i] = 0.f;
  }
  if constexpr (BITS == 4 && !PER_TOKEN) {
    // the 8 channels' pairs are stored in the order (0,2) (1,3) (4,6) (5,7)
    const uint4 a = *reinterpret_cast<const uint4*>(d.km + 8 * j);
    const uint4 b = *reinterpret_cast<const uint4*>(d.km + kHeadDim + 8 * j);
    const uint32_t sw[4] = {a.x, a.y, a.z, a.w}, zw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int u = (r & 1) + 4 * (r >> 1);
      s[u] = __low2float(u32_as_h2(sw[r])) * pow2_neg(4 * (u & 3));
      s[u + 2] = __high2float(u32_as_h2(sw[r])) * pow2_neg(4 * ((u + 2) & 3));
      z[u] = __low2float(u32_as_h2(zw[r])); z[u + 2] = __high2float(u32_as_h2(zw[r]));
    }
  } else if constexpr (BITS == 2 && !PER_TOKEN) {
    // word r of a 16-channel block holds channels (r, r + 8)
    const uint4* sp = reinterpret_cast<const uint4*>(d.km + 16 * (j >> 1));
    const uint4* zp = reinterpret_cast<const uint4*>(d.km + kHeadDim + 16 * (j >> 1));
    const uint4 a = sp[0], b = sp[1], e = zp[0], f = zp[1];
    const uint32_t sw[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, zw[8] = {e.x, e.y, e.z, e.w, f.x, f.y, f.z, f.w};
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      s[r] = ((j & 1) ? __high2float(u32_as_h2(sw[r])) : __low2float(u32_as_h2(sw[r]))) * pow2_neg(2 * r);
      z[r] = (j & 1) ? __high2float(u32_as_h2(zw[r])) : __low2float(u32_as_h2(zw[r]));
    }
  }
  if constexpr (SP) {
#pragma unroll
    for (int i = 0; i < 8; ++i) kept[i] = d.ksp[8 * j + i];
  }
  constexpr int RB = kHeadDim * BITS / 8;
#pragma unroll
  for (int i = 0; i < kTile / 2; ++i) {
    const int r = 2 * i + half;
    if (r < lo || r >= hi) continue;
    float x[8];
    const uint8_t* row = d.k + r * RB;
    if constexpr (BITS == 8) {
      const uint2 w2 = *reinterpret_cast<const uint2*>(row + 8 * j);
      const uint32_t w[2] = {w2.x, w2.y};
      if constexpr (PER_TOKEN) {
        const uint32_t m = *reinterpret_cast<const uint32_t*>(d.km + 2 * r);
        const float st = __low2float(u32_as_h2(m)), zt = __high2float(u32_as_h2(m));
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const uint32_t sel = 0x7440u | (u & 3), sel2 = 0x7440u | ((u & 3) + 1);
          unpair(pair_fma(magic_codes(prmt(w[u >> 2], kMagic, sel), prmt(w[u >> 2], kMagic, sel2)), pair(st, st),
                          pair(zt, zt)), x[u], x[u + 1]);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = e4m3_f32((w[u >> 2] >> (8 * (u & 3))) & 0xFFu) * d.ks;
      }
    } else {
      uint32_t w = BITS == 4 ? *reinterpret_cast<const uint32_t*>(row + 4 * j)
                             : (uint32_t)*reinterpret_cast<const uint16_t*>(row + 2 * j);
#pragma unroll
      for (int u = 0; u < 8; u += 2) {
        if (BITS == 4 && u == 4) w >>= 16;
        const int p = BITS == 4 ? 4 * (u & 3) : 2 * u;
        constexpr uint32_t mask = (1u << BITS) - 1u;
        unpair(pair_fma(magic_codes(lop_or(w, mask << p, kMagic), lop_or(w, mask << (p + BITS), kMagic)),
                        pair(s[u], s[u + 1]), pair(z[u], z[u + 1])), x[u], x[u + 1]);
      }
    }
    if constexpr (SP) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if ((int)(kept[u] >> 16) == d.t0 + r) x[u] = bf16_lo(kept[u]);
    }
    emit(r, 8 * j, x);
  }
}

template <int FMT, class Emit>
__device__ __forceinline__ void key_rows(const TileSrc& d, int lo, int hi, Emit emit) {
  if constexpr (FMT == 8) key_rows_bits<8, false, false>(d, lo, hi, emit);
  else if constexpr (FMT == 16) key_rows_bits<8, true, false>(d, lo, hi, emit);
  else if constexpr (FMT == 6) {
    if (d.bits == 4) key_rows_bits<4, false, false>(d, lo, hi, emit);
    else key_rows_bits<2, false, false>(d, lo, hi, emit);
  } else if (d.ksp) key_rows_bits<FMT, false, true>(d, lo, hi, emit);
  else key_rows_bits<FMT, false, false>(d, lo, hi, emit);
}

// Value rows: lane (n, l) owns channels [16n, 16n + 16) of tokens 2l, 2l+1,
// 2l+8, 2l+9 (the tile's layout); emit(row, channel, x[16]) once per token.
template <int BITS, bool FP8, bool SP, class Emit>
__device__ __forceinline__ void value_rows_bits(const TileSrc& d, int lo, int hi, Emit emit) {
  constexpr int NW = 2 * BITS;         // words per lane
  const int lane = threadIdx.x & 31, n = lane >> 2, l = lane & 3;
  uint32_t w[NW];
#pragma unroll
  for (int i = 0; i < NW / 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(d.v + 512 * i + 16 * lane);
    w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {        // byte q of every word is this token's
    const int r = 2 * l + (q & 1) + 8 * (q >> 1);
    if (BITS < 8 && q == 2) {
#pragma unroll
      for (int i = 0; i < NW; ++i) w[i] >>= 16;
    }
    if (r < lo || r >= hi) continue;
    float s = d.vs, z = 0.f;
    if constexpr (!FP8) {
      const uint32_t m = *reinterpret_cast<const uint32_t*>(d.vm + 2 * r);
      s = __low2float(u32_as_h2(m));
      z = __high2float(u32_as_h2(m));
    }
    float x[16];
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < 16; ++u) x[u] = e4m3_f32((w[u] >> (8 * q)) & 0xFFu) * s;
    } else if constexpr (BITS == 8) {
#pragma unroll
      for (int u = 0; u < 16; u += 2)
        unpair(pair_fma(magic_codes(prmt(w[u], kMagic, 0x7440u | q), prmt(w[u + 1], kMagic, 0x7440u | q)), pair(s, s),
                        pair(z, z)), x[u], x[u + 1]);
    } else {
      constexpr int PW = 8 / BITS;     // channels per byte of a word
      constexpr uint32_t mask = (1u << BITS) - 1u;
#pragma unroll
      for (int c = 0; c < PW; c += 2) {
        const int p = 8 * (q & 1) + BITS * c;
        const pair_t s2 = pair(s * pow2_neg(p), s * pow2_neg(p + BITS)), z2 = pair(z, z);
#pragma unroll
        for (int i = 0; i < NW; ++i)
          unpair(pair_fma(magic_codes(lop_or(w[i], mask << p, kMagic), lop_or(w[i], mask << (p + BITS), kMagic)), s2, z2),
                 x[PW * i + c], x[PW * i + c + 1]);
      }
    }
    if constexpr (SP) {
      const uint32_t kept = d.vsp[r];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if ((int)(kept >> 16) == 16 * n + u) x[u] = bf16_lo(kept);
    }
    emit(r, 16 * n, x);
  }
}

template <int FMT, class Emit>
__device__ __forceinline__ void value_rows(const TileSrc& d, int lo, int hi, Emit emit) {
  if constexpr (FMT == 8) value_rows_bits<8, true, false>(d, lo, hi, emit);
  else if constexpr (FMT == 16) value_rows_bits<8, false, false>(d, lo, hi, emit);
  else if constexpr (FMT == 6) {
    if (d.bits == 4) value_rows_bits<4, false, false>(d, lo, hi, emit);
    else value_rows_bits<2, false, false>(d, lo, hi, emit);
  } else if (d.vsp) value_rows_bits<FMT, false, true>(d, lo, hi, emit);
  else value_rows_bits<FMT, false, false>(d, lo, hi, emit);
}

}  // namespace kvq
