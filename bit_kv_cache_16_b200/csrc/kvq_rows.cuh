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

// A code of up to 8 bits -> fp32: OR-ed into the mantissa of 2^23, exactly.
__device__ __forceinline__ float code_f32(uint32_t code) { return __uint_as_float(0x4B000000u | code) - 8388608.f; }

__device__ __forceinline__ float e4m3_f32(uint32_t byte) { return __half2float(u32_as_h2(e4m3x2_to_h2(byte)).x); }

// Key rows: lane owns channels [8j, 8j + 8), j = lane % 16, of the tile's rows
// 2i + lane / 16; emit(row, channel, x[8]) for each of rows [lo, hi).
template <int BITS, bool PER_TOKEN, class Emit>
__device__ __forceinline__ void key_rows_bits(const TileSrc& d, int lo, int hi, Emit emit) {
  const int lane = threadIdx.x & 31, j = lane & 15, half = lane >> 4;
  float s[8], z[8];
  uint32_t kept[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = d.ks;                    // FP8: code * scale
    z[i] = 0.f;
    kept[i] = 0xFFFFFFFFu;          // no token of a group has this index
  }
  if constexpr (BITS == 4 && !PER_TOKEN) {
    // the 8 channels' pairs are stored in the order (0,2) (1,3) (4,6) (5,7)
    const uint4 a = *reinterpret_cast<const uint4*>(d.km + 8 * j);
    const uint4 b = *reinterpret_cast<const uint4*>(d.km + kHeadDim + 8 * j);
    const uint32_t sw[4] = {a.x, a.y, a.z, a.w}, zw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int u = (r & 1) + 4 * (r >> 1);
      s[u] = __low2float(u32_as_h2(sw[r])); s[u + 2] = __high2float(u32_as_h2(sw[r]));
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
      s[r] = (j & 1) ? __high2float(u32_as_h2(sw[r])) : __low2float(u32_as_h2(sw[r]));
      z[r] = (j & 1) ? __high2float(u32_as_h2(zw[r])) : __low2float(u32_as_h2(zw[r]));
    }
  }
  if (d.ksp) {
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
      float st = d.ks, zt = 0.f;
      if constexpr (PER_TOKEN) {
        const uint32_t m = *reinterpret_cast<const uint32_t*>(d.km + 2 * r);
        st = __low2float(u32_as_h2(m));
        zt = __high2float(u32_as_h2(m));
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t code = (w[u >> 2] >> (8 * (u & 3))) & 0xFFu;
        x[u] = PER_TOKEN ? fmaf(code_f32(code), st, zt) : e4m3_f32(code) * st;
      }
    } else {
      const uint32_t w = BITS == 4 ? *reinterpret_cast<const uint32_t*>(row + 4 * j)
                                   : (uint32_t)*reinterpret_cast<const uint16_t*>(row + 2 * j);
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = fmaf(code_f32((w >> (BITS * u)) & ((1u << BITS) - 1u)), s[u], z[u]);
    }
    if (d.ksp) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if ((int)(kept[u] >> 16) == d.t0 + r) x[u] = bf16_lo(kept[u]);
    }
    emit(r, 8 * j, x);
  }
}

template <int FMT, class Emit>
__device__ __forceinline__ void key_rows(const TileSrc& d, int lo, int hi, Emit emit) {
  if constexpr (FMT == 8) key_rows_bits<8, false>(d, lo, hi, emit);
  else if constexpr (FMT == 16) key_rows_bits<8, true>(d, lo, hi, emit);
  else if constexpr (FMT == 6) {
    if (d.bits == 4) key_rows_bits<4, false>(d, lo, hi, emit);
    else key_rows_bits<2, false>(d, lo, hi, emit);
  } else key_rows_bits<FMT, false>(d, lo, hi, emit);
}

// Value rows: lane (n, l) owns channels [16n, 16n + 16) of tokens 2l, 2l+1,
// 2l+8, 2l+9 (the tile's layout); emit(row, channel, x[8]) twice per token.
template <int BITS, bool FP8, class Emit>
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
  for (int q = 0; q < 4; ++q) {
    const int r = 2 * l + (q & 1) + 8 * (q >> 1);
    if (r < lo || r >= hi) continue;
    float s = d.vs, z = 0.f;
    if constexpr (!FP8) {
      const uint32_t m = *reinterpret_cast<const uint32_t*>(d.vm + 2 * r);
      s = __low2float(u32_as_h2(m));
      z = __high2float(u32_as_h2(m));
    }
    const uint32_t kept = d.vsp ? d.vsp[r] : 0xFFFFFFFFu;
    constexpr int PW = 8 / BITS;       // channels per byte of a word
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int ch = 8 * hh + u;
        const uint32_t code = (w[ch / PW] >> (8 * q + BITS * (ch % PW))) & ((1u << BITS) - 1u);
        x[u] = FP8 ? e4m3_f32(code) * s : fmaf(code_f32(code), s, z);
        if ((int)(kept >> 16) == 16 * n + ch) x[u] = bf16_lo(kept);
      }
      emit(r, 16 * n + 8 * hh, x);
    }
  }
}

template <int FMT, class Emit>
__device__ __forceinline__ void value_rows(const TileSrc& d, int lo, int hi, Emit emit) {
  if constexpr (FMT == 8) value_rows_bits<8, true>(d, lo, hi, emit);
  else if constexpr (FMT == 16) value_rows_bits<8, false>(d, lo, hi, emit);
  else if constexpr (FMT == 6) {
    if (d.bits == 4) value_rows_bits<4, false>(d, lo, hi, emit);
    else value_rows_bits<2, false>(d, lo, hi, emit);
  } else value_rows_bits<FMT, false>(d, lo, hi, emit);
}

}  // namespace kvq
