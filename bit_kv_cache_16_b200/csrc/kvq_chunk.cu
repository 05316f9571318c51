// kvq_chunk_attention: a chunk's query rows against the packed cache and,
// causally, against the chunk's own tokens, on the tensor cores.
//
// Per (sequence, kv head) the query rows of all gq heads and new tokens form
// one matrix (row R = head R % gq of token R / gq).  For each tile of 128
// tokens: S = Q K^T (128 rows x 128 keys, fp16 operands, fp32 in TMEM), the
// online softmax with one thread per row (64 keys at a time), P = fp16 back
// into TMEM, O += P V with O in TMEM.  Packed tokens become fp16 operands once
// per CTA and tile (kvq_tiles.cuh); fp16 holds every code exactly and a
// dequantized number to 2^-11, eight times finer than bf16, and a power of two
// is taken out of 16-token pieces whose numbers would not fit.
//
// What bounds it: a stream's tile is a chain (scores, maximum, weights, P V,
// next scores) of about 2400 cycles of softmax and 1500 of products, and TMEM
// has room for two streams (S or P and O: 256 columns each).  Together a tile
// of 256 rows takes about 4500 cycles, of which the tensor pipe is busy 44 %,
// the exponential unit 44 %, the issue slots 48 %.  Measured alone with a cold
// L2: 2048 tokens over 32768 INT4 tokens, 32 / 8 heads, 1306 us (868 TFLOP/s);
// 1000 over 65536 INT2 tokens, 64 / 8 heads, 2175 us (995); 2 x 1024 in a
// window of 4096 + 4 over FP8, 525 us (524; 480 with a warm L2); 6 tokens over
// 8 x 8192 INT4, 70 us (1.2 TB/s of packed tokens: the paired form's chain of 33
// tiles a CTA).  Keys before RoPE and dense-and-sparse caches (keys_any /
// values_any for every piece): 2048 over 16384, 7160 and 6500 us, 785 without.
//
// Sixteen warps, because a seventeenth would leave 96 registers a thread, and
// a spilled register is a trip to L2 here (shared memory takes the whole L1):
// 2205 us with spills in the softmax, 1648 without.  Two softmax warpgroups
// per stream (24 warps, 80 registers) took 1446 us against 1290.
#include "kvq_tiles.cuh"

namespace kvq {

constexpr int kRows = 128;                   // query rows per stream: one TMEM lane and one softmax thread each
constexpr int kProducerWarp = 8;             // warps 0-3 and 4-7: softmax of streams 0 and 1; 8-14: producers
constexpr int kProducers = 7;                // (and the softmax warps none of whose rows is real)
constexpr int kMmaWarp = kProducerWarp + kProducers;            // issues every product
constexpr int kChunkThreads = 32 * (kMmaWarp + 1);              // four warps per scheduler: 128 registers each
constexpr int kHalf = kKeys / 2;             // a row's softmax takes 64 keys at a time
constexpr int kStages = 2;                   // key tiles in flight
// Value tiles in flight.  A producer may have two subtiles of one tile, and
// writes the values of the first before the keys of the second.  Paired
// streams ask for the keys of tile g + 2 while the values of tile g are still
// in use (and those of tile g - 1 are used up): the values of tile g + 2 need
// a third stage.  Shared keys: those of tile g + 1 while g - 1 is used up.
__host__ __device__ constexpr int value_stages(bool shared_keys) { return shared_keys ? 2 : 3; }
constexpr int kMaxValueStages = 3;
constexpr int kInfos = 4;                    // tile descriptions in flight
// A row's reference is its maximum at first, and stays while no weight passes
// 2^kTop (fp16 ends at 65504).  From the stream's half tile kSettle on, when
// the maximum has mostly been seen, it lies 2^kLift lower: fp16 loses what is
// below 2^-25, then 2^-31 of the largest weight; 131072 such tokens are 2^-14
// of a row, where they would be 2^-8.  The price is one more scaling of O, and
// a maximum that grows by 2^(kTop - kLift) moves the reference again: 2048
// tokens over 32768 take 1307 us, 1295 without a lift, 1316 with one of 8; lifted
// from the start, 2 x 1024 tokens in a window of 4096 + 4 (its first tile shows
// four keys) take 600, 520 so.
constexpr float kLift = 6.f, kTop = 15.f;
constexpr int kSettle = 6;
constexpr unsigned long long kWaitNs = 2000000000ull;

// Eight channels of a query row (16 lanes a row) whose magnitudes need a power
// of two taken out, or that is not finite throughout; returns the power.
__device__ __noinline__ float put_scaled8(uint32_t at, uint4 v) {
  float x[8], amax = 0.f;
  unpack8(v, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(x[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = tile_exponent(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = scale_by(x[i], -e);
  st_shared16(at, pack_h2(x[0], x[4]), pack_h2(x[1], x[5]), pack_h2(x[2], x[6]), pack_h2(x[3], x[7]));
  return scale_by(1.f, e);
}

// What every thread of a CTA knows about its work.
struct Work {
  ChunkSeq sq;
  int b, kv, gq, r0, rows, split;
  int first, tiles;                          // tiles [first, first + tiles) of the range
  TileRange range;
  int stream_tiles[2];
};

struct ChunkCtrl {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kMaxValueStages], v_empty[kMaxValueStages];
  uint64_t s_full[2], p_ready[2][2], o_done[2], finished[2], drained;   // [stream][half of the tile]
  uint32_t tmem;
  int abort;
  TileInfo info[kInfos];
  float qmul[2 * kRows];                     // 2^e of each query row
  float ml[kRows][2];                        // paired streams: (m, l) of stream 1
  double freq[kHeadDim / 2];                 // RoPE pair frequencies
  Work work;                                 // kept here, not in every thread's registers
  int clear;                                 // tokens from here on are hidden from no row of the CTA by the window
  int sinks;                                 // tiles that end here or below neither
  int straight;                              // quantized tokens whose codes go straight to halves (0: rotated or sparse keys)
  int2 seen[8];                              // the same for a softmax warp's rows, and its first row's position
};

__host__ __device__ constexpr int chunk_smem_bytes(bool shared_keys) {
  return 1024 + ((shared_keys ? 2 : 1) + kStages + value_stages(shared_keys)) * kTileBytes16 + (int)sizeof(ChunkCtrl);
}

// --- mbarriers, tcgen05 ---------------------------------------------------

__device__ __forceinline__ void bar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}
// False when the wait was given up (here or by another thread of the CTA):
// the caller leaves its loop, and the CTA ends with an error bit.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* abort) {
  if (bar_try(b, parity)) return true;
  const unsigned long long t0 = now_ns();
  while (!bar_try(b, parity)) {
    if (*abort) return false;
    if (now_ns() - t0 > kWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, bar_wait(b, parity, abort));
}
// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_u32(b))
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 32 columns of the thread's lane -> 32 registers, starting at r.
__device__ __forceinline__ void tc_ld32(float* r, uint32_t at) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(at));
}
__device__ __forceinline__ void tc_ld16(float* r, uint32_t at) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(at));
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t at, const uint32_t* u) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(at), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, 8-row groups 1024 bytes
// apart; `lead` = bytes between blocks of 64 elements along the major axis.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// fp16 x fp16 -> fp32, M = N = 128; the value operand is stored with channels (N) contiguous.
constexpr uint32_t kIdescQK = (1u << 4) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}

// TMEM columns: S of the streams, half by half (P over the start of its half), then O of the streams.
__device__ __forceinline__ uint32_t tm_s(uint32_t tmem, int i) { return tmem + 128 * i; }
__device__ __forceinline__ uint32_t tm_o(uint32_t tmem, int i) { return tmem + 256 + 128 * i; }

// --- the kernel -----------------------------------------------------------

// The scaling of subtiles of kinds 0 and 1.
struct Scaling {
  float kmul, vlog, vinv;
};
// FP8 codes stand for themselves in the tiles; the head's static scales come in
// here.  (A value scale below kLeastScale, whose inverse times a row's weights
// could pass fp32, does not: such a head's tokens go through values_any.)
constexpr float kLeastScale = 0x1p-90f;
__device__ __forceinline__ Scaling static_scaling(const kvq_cache& c, int kv) {
  const float vs = fmaxf(c.fp8_scale[c.shape.num_kv_heads + kv], kLeastScale);
  return Scaling{c.fp8_scale[kv], log2f(vs), 1.f / vs};
}

// A subtile that is not a whole quantized one, both tiles; its description
// goes into `info`.  Returns its kind.  (A function of its own with few
// arguments: its registers are not the fast path's.)
template <int FMT>
__device__ __noinline__ int produce_other(const ChunkAttnArgs& A, ChunkCtrl& C, const UnitSrc<FMT>& unit, int base,
                                          uint32_t kt, uint32_t vt, int sub, TileInfo& info) {
  const kvq_cache& c = A.c;
  const kvq_shape& s = c.shape;
  const ChunkSeq& sq = C.work.sq;
  const bool rope = s.rope_theta > 0.f;
  const int lane = threadIdx.x & 31;
  const int quant = min(max(sq.nq - base, 0), kTile);        // quantized rows come first
  bool codes = FMT == 8 && quant > 0;                        // (codes as they are: the static scales come in later)
  int ek = 0, ev = 0;
  uint32_t bad = 0u;
  TileSrc d;
  if constexpr (FMT == 8) d.vs = 1.f;
  if (quant > 0 && !tile_src<FMT>(c, C.work.b, C.work.kv, base / kTile, d)) {
    if (lane == 0) atomicOr(c.err_word, KVQ_DEVERR_PAGE_RANGE);
    zero_rows(kt, sub);
    zero_rows(vt, sub);
    bad = 1u << 16;
  } else {
    const size_t ring = is_token_cache(FMT) ? 0 : Addr::ring_row(s, C.work.b, C.work.kv, 0);
    const size_t at = ((size_t)sq.t0 * s.num_kv_heads + C.work.kv) * kHeadDim;
    RawRows raw;
    raw.stride = (int64_t)s.num_kv_heads * kHeadDim;
    raw.n = sq.n;
    raw.total = sq.total;
    raw.slots = max(window_slots(s), kTile);
    raw.slot0 = base % raw.slots;
    RawRows raw_v = raw;
    raw.ring = (const uint16_t*)c.k_res + ring;
    raw.fresh = A.k + at;
    raw_v.ring = (const uint16_t*)c.v_res + ring;
    raw_v.fresh = A.v + at;
    bool packed = quant > 0 && !rope && !s.sparse;
    if constexpr (FMT == 8) codes = packed = codes && d.vs >= kLeastScale;
    if (packed) {
      // packed words: a tile at the window's edge, or (8-bit formats) the
      // sequence's last one with the chunk's first tokens behind it
      SubSrc p;
      SubWords<FMT> w;
      sub_src<FMT>(unit, base / kTile, p);
      load_keys<FMT>(p, w);
      load_values<FMT>(p, w);
      if (quant < kTile) drop_values<FMT>(w, quant);         // (what lies behind the end is not data)
      // raw rows take the codes' scaling (FP8), so that the subtile has one
      const float k_inv = codes ? 1.f / d.ks : 1.f, v_inv = codes ? 1.f / d.vs : 1.f;
      bool fits = !__any_sync(0xffffffffu, keys_past<FMT>(w, p.two) != 0u) && !values_odd<FMT>(w) && k_inv < INFINITY && v_inv < INFINITY;
      float amax_k = 0.f, amax_v = 0.f;
      if constexpr (FMT != 8) {
#pragma unroll
        for (int q = 0; q < 4; ++q) amax_v = fmaxf(amax_v, most_of<FMT>(w.vm[q], p.two));
      }
      for (int r = quant + (lane >> 4); r < kTile; r += 2) {
        float x[8], y[8];
        unpack8(raw.load(base + r, r, lane & 15), x);
        unpack8(raw_v.load(base + r, r, lane & 15), y);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          amax_k = fmaxf(amax_k, fabsf(x[u] * k_inv));
          amax_v = fmaxf(amax_v, fabsf(y[u] * v_inv));
          fits = fits && fabsf(x[u]) < INFINITY && fabsf(y[u]) < INFINITY;
        }
      }
      amax_k = warp_max(amax_k);                             // (whole-warp shuffles: not behind a lane's own `fits`)
      amax_v = warp_max(amax_v);
      fits = fits && tile_exponent(amax_k) == 0;
      if (FMT == 8) {
        fits = fits && (amax_v == 0.f || value_exponent(amax_v) == 0);      // (codes have the head's scale)
      } else if (quant < kTile) {
        fits = fits && value_exponent(amax_v) == 0;
      } else if (amax_v < kLeastValue) {                     // small packed values: 2^ev out of their scales and zeros
        ev = amax_v == 0.f ? kLeastPower : max(value_exponent(amax_v), -15);
        if (amax_v > 0.f) scale_values<FMT>(w, -ev);
      }
      if (__all_sync(0xffffffffu, fits)) {
        if (FMT == 6 && p.two) {
          keys_to_tile<FMT, 2>(w, kt, sub);
          values_to_tile<FMT, 2>(w, vt, sub);
        } else {
          keys_to_tile<FMT, SubWords<FMT>::kBits>(w, kt, sub);
          values_to_tile<FMT, SubWords<FMT>::kBits>(w, vt, sub);
        }
        __syncwarp();
        for (int r = quant + (lane >> 4); r < kTile; r += 2) {
          float x[8], y[8];
          unpack8(raw.load(base + r, r, lane & 15), x);
          unpack8(raw_v.load(base + r, r, lane & 15), y);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            x[u] *= k_inv;
            y[u] *= v_inv;
          }
          put_key8(kt, kTile * sub + row_of_token(r), lane & 15, x);
          put_value8(vt, kTile * sub + row_of_token(r), lane & 15, y);
        }
        if (ev == 0) return 0;
        if (lane == 0) {
          info.kmul[sub] = 1.f;
          info.vlog[sub] = (float)ev;
          info.vinv[sub] = scale_by(1.f, -ev);
          info.bad[sub] = 0u;
        }
        return 2;
      }
      ev = 0;
    }
    bool k_done = false, v_done = false;
    if (quant == 0 && !rope) {
      RawWords x[2];                                         // both on their way at once
      load_rows(raw, base, x[0]);
      load_rows(raw_v, base, x[1]);
      const bool gone = base >= sq.total;
      k_done = rows_to_tile(x[0], kt, sub, true, gone);
      v_done = rows_to_tile(x[1], vt, sub, false, gone);
    }
    if (codes && quant == kTile) d.ks = d.vs = 1.f;          // (with raw rows: in natural scale, kind 1)
    if (!k_done) ek = keys_any<FMT>(d, quant, raw, base, rope ? C.freq : nullptr, kt, sub);
    if (!v_done) ev = values_any<FMT>(d, quant, raw_v, base, vt, sub, bad);
  }
  const bool scaled = codes && quant == kTile;
  if (ek == 0 && ev == 0 && bad == 0u) return FMT == 8 && !scaled ? 1 : 0;
  if (lane == 0) {
    const Scaling p = scaled ? static_scaling(c, C.work.kv) : Scaling{1.f, 0.f, 1.f};
    info.kmul[sub] = scale_by(p.kmul, ek);
    info.vlog[sub] = p.vlog + (float)ev;
    info.vinv[sub] = scale_by(p.vinv, -ev);
    info.bad[sub] = bad;
  }
  return 2;
}

// Producer pw of `step`: subtiles pw, pw + step, ... (subtile x is number x % 8
// of tile x / 8).  In a run of whole quantized subtiles the keys are one
// subtile ahead of the values, K(x) K(x + step) V(x) K(x + 2 step) V(x + step)
// ..., so that a tile's last keys do not wait for the stage of its first
// values, and packed words are on their way while others are turned into
// halves.  Any other subtile, and one whose numbers may not fit a half, is
// made on its own between two runs, when no word is held.
template <int FMT, bool SHARED>
__device__ __forceinline__ void produce(const ChunkAttnArgs& A, ChunkCtrl& C, const UnitSrc<FMT>& unit, uint32_t k_tiles, uint32_t v_tiles, int pw, int step) {
  constexpr int kValueStages = value_stages(SHARED);
  const int lane = threadIdx.x & 31;
  const volatile Work& W = C.work;           // read where it is used: registers are short
  const int last = C.work.tiles * kSubs;

  auto wait_keys = [&](int x) {
    const int g = x / kSubs;
    return warp_wait(&C.k_empty[g % kStages], ((g / kStages) & 1) ^ 1, &C.abort);
  };
  auto wait_values = [&](int x) {
    const int g = x / kSubs;
    return warp_wait(&C.v_empty[g % kValueStages], ((g / kValueStages) & 1) ^ 1, &C.abort);
  };
  auto hand_over = [&](uint64_t* bar) {
    fence_async();
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
  };
  auto tile = [&](int x) {
    const int y = W.first + x / kSubs, lead = W.range.lead;
    return y < lead ? y : W.range.skip + y - lead;
  };
  auto key_tile = [&](int x) { return k_tiles + (x / kSubs) % kStages * kTileBytes16; };
  auto value_tile = [&](int x) { return v_tiles + (x / kSubs) % kValueStages * kTileBytes16; };
  auto packed = [&](int x, SubSrc& d) {
    const int t0 = tile(x) * kKeys, base = t0 + kTile * (x % kSubs);
    const volatile ChunkCtrl& V = C;
    return V.straight - base >= kTile && (t0 >= V.clear || t0 + kKeys <= V.sinks) && sub_src<FMT>(unit, base / kTile, d);
  };

  int x = pw;
  while (x < last) {
    SubSrc d;
    if (packed(x, d)) {
      SubWords<FMT> w;
      load_keys<FMT>(d, w);
      bool more = true, two = false;         // two: the held values have 2-bit codes
      int y = -1;                            // whose values are held
      while (more && !words_odd<FMT>(w, d.two)) {
        // keys of x
        const int g = x / kSubs;
        if (!wait_keys(x)) return;
        const bool two_here = d.two;
        if (FMT == 6 && two_here) keys_to_tile<FMT, 2>(w, key_tile(x), x % kSubs);
        else keys_to_tile<FMT, SubWords<FMT>::kBits>(w, key_tile(x), x % kSubs);
        if (lane == 0) C.info[g % kInfos].kind[x % kSubs] = 0;
        hand_over(&C.k_full[g % kStages]);
        const SubSrc here = d;
        more = x + step < last && packed(x + step, d);
        if (more) load_keys<FMT>(d, w);
        // values of y, the subtile before
        if (y >= 0) {
          if (!wait_values(y)) return;
          if (FMT == 6 && two) values_to_tile<FMT, 2>(w, value_tile(y), y % kSubs);
          else values_to_tile<FMT, SubWords<FMT>::kBits>(w, value_tile(y), y % kSubs);
          hand_over(&C.v_full[(y / kSubs) % kValueStages]);
        }
        load_values<FMT>(here, w);
        two = two_here;
        y = x;
        x += step;
      }
      if (y >= 0) {
        if (!wait_values(y)) return;
        if (FMT == 6 && two) values_to_tile<FMT, 2>(w, value_tile(y), y % kSubs);
        else values_to_tile<FMT, SubWords<FMT>::kBits>(w, value_tile(y), y % kSubs);
        hand_over(&C.v_full[(y / kSubs) % kValueStages]);
      }
      if (!more) continue;                   // the next subtile is not a packed one
    }
    // The softmax reads the description when the scores are there, so it has
    // to be complete before the keys are handed over: rows that need a look
    // give their values first.
    if (!wait_keys(x) || !wait_values(x)) return;
    const int g = x / kSubs, sub = x % kSubs;
    const int kind = produce_other<FMT>(A, C, unit, tile(x) * kKeys + kTile * sub, key_tile(x), value_tile(x), sub,
                                        C.info[g % kInfos]);
    if (lane == 0) C.info[g % kInfos].kind[sub] = (uint8_t)kind;
    hand_over(&C.k_full[g % kStages]);
    hand_over(&C.v_full[g % kValueStages]);
    x += step;
  }
}

// The products, issued by one elected thread of the last warp (the whole warp
// waits; everything that addresses operands is warp-uniform).  P V of a tile's
// first half runs while the softmax does the second; the next scores follow
// the second P V, whose P they overwrite (the tensor core takes one thread's
// products in order), while the other stream's softmax runs.  (Scores in two
// blocks of 64 keys, each with its own next product, were slower: a product
// of N = 64 takes 58 cycles, one of N = 128 about 72, both bound by the query
// operand's way from shared memory.)  False: a wait was given up.
constexpr uint32_t kStageStep = kTileBytes16 >> 4;

template <bool SHARED>
__device__ __forceinline__ bool issue_all(ChunkCtrl& C, uint32_t q_tiles, uint32_t k_tiles, uint32_t v_tiles) {
  constexpr int kValueStages = value_stages(SHARED);
  const uint32_t tmem = __shfl_sync(0xffffffffu, C.tmem, 0);
  const int n0 = __shfl_sync(0xffffffffu, C.work.stream_tiles[0], 0), n1 = __shfl_sync(0xffffffffu, C.work.stream_tiles[1], 0);
  const uint64_t q0 = operand_desc(q_tiles, 16), k0 = operand_desc(k_tiles, 16), v0 = operand_desc(v_tiles, kBlockBytes);
  // scores of stream i's tile `it`; `done`: the last that read the keys
  auto scores = [&](int i, int it, bool done) {
    const int st = (SHARED ? it : i) & 1;
    const uint64_t q = q0 + (SHARED ? i : 0) * kStageStep, k = k0 + st * kStageStep;
    const uint32_t d = tm_s(tmem, i);
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint64_t off = ((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4;   // 16 channels on
        mma_ss(d, q + off, k + off, kIdescQK, kk > 0);
      }
      if (done) tc_commit(&C.k_empty[st]);
      tc_commit(&C.s_full[i]);
    }
    __syncwarp();
  };
  auto values = [&](int i, int it, int h, bool done, bool last) {
    const int st = (SHARED ? it : 2 * it + i) % kValueStages;
    const uint64_t v = v0 + st * kStageStep + ((h * kHalf * 128) >> 4);
    const uint32_t d = tm_o(tmem, i), p = tm_s(tmem, i) + kHalf * h, add = it > 0 || h > 0;
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)                       // 16 tokens on: 16 rows of 128 bytes
        mma_ts(d, p + 8 * kk, v + ((kk * 16 * 128) >> 4), kIdescPV, kk > 0 ? 1u : add);
      if (done) tc_commit(&C.v_empty[st]);
      tc_commit(&C.o_done[i]);
      if (last) tc_commit(&C.finished[i]);
    }
    __syncwarp();
  };
  // stage of a stream's tile: SHARED, tile it for both; else tile 2 it + i
  auto full = [&](uint64_t* bar, int stages, int i, int it) {
    const int g = SHARED ? it : 2 * it + i;
    return warp_wait(bar + g % stages, (g / stages) & 1, &C.abort);
  };
  const int closer = SHARED && n1 > 0 ? 1 : 0;             // SHARED: the stream that reads a tile last
  for (int i = 0; i < 2; ++i) {
    if ((i ? n1 : n0) == 0) continue;
    if (!full(C.k_full, kStages, i, 0)) return false;
    tc_after();
    scores(i, 0, !SHARED || i == closer);
  }
  for (int it = 0; it < n0; ++it)
    for (int i = 0; i < 2; ++i) {
      const int n = i ? n1 : n0;
      if (it >= n) continue;
      const bool done = !SHARED || i == closer;
      // (what the producers owe first: it is there as a rule)
      if (!full(C.v_full, kValueStages, i, it) || (it + 1 < n && !full(C.k_full, kStages, i, it + 1))) return false;
      if (!warp_wait(&C.p_ready[i][0], it & 1, &C.abort)) return false;
      tc_after();
      values(i, it, 0, false, false);
      if (!warp_wait(&C.p_ready[i][1], it & 1, &C.abort)) return false;
      tc_after();
      values(i, it, 1, done, it + 1 == n);
      if (it + 1 < n) scores(i, it + 1, done);
    }
  return true;
}
// After a wait that was given up: the products in flight end before TMEM is
// freed (again with a limit).
__device__ __forceinline__ void drain(ChunkCtrl& C) {
  tc_commit(&C.drained);
  const unsigned long long t0 = now_ns();
  while (!bar_try(&C.drained, 0) && now_ns() - t0 < kWaitNs) {}
}

struct RowState {
  float m, l;                                // reference (log2 units) and sum of this thread's row
};


// One stream's softmax state in a thread: it owns one row.
struct Row {
  RowState r;
  float cm;                                  // the row's factor: |softmax_scale| log2(e) 2^e
  uint32_t ts, to;                           // TMEM addresses of the warp's scores and output
};

// Moves the row's reference to cover `top` if it has to, and O with it;
// `turn` is the number of the half tile in the stream.  False: a wait was
// given up.
__device__ __forceinline__ bool raise(ChunkCtrl& C, int i, int turn, float top, Row& w) {
  RowState& r = w.r;
  const bool settle = turn == kSettle && r.m > -INFINITY;
  const bool up = settle || top > r.m + kTop || (r.m == -INFINITY && top > -INFINITY);
  if (!__any_sync(0xffffffffu, up)) return true;
  const float mn = up ? (settle ? fmaxf(top, r.m) : top) - (turn < kSettle ? 0.f : kLift) : r.m;
  const float f = r.m == -INFINITY ? (up ? 0.f : 1.f) : (up ? ex2(r.m - mn) : 1.f);
  if (turn > 0 && __any_sync(0xffffffffu, up && r.m != -INFINITY)) {
    // O is at rest once the P V of the half before this is done (the one
    // before that is: a parity tells one phase from the next only)
    if (!warp_wait(&C.o_done[i], (turn - 1) & 1, &C.abort)) return false;
    tc_after();
    const float fo = r.m == -INFINITY ? 1.f : f;               // O is zero then
#pragma unroll 1
    for (int c0 = 0; c0 < kHeadDim; c0 += 16) {
      float o[16];
      tc_ld16(o, w.to + c0);
      tc_wait_ld();
#pragma unroll
      for (int u = 0; u < 16; ++u) o[u] *= fo;
      tc_st16(w.to + c0, reinterpret_cast<uint32_t*>(o));
    }
    tc_wait_st();
  }
  r.l *= f;
  r.m = mn;
  return true;
}

__device__ __forceinline__ float most(float top, const float (&x)[32]) {
  float t4[4] = {top, x[0], x[1], x[2]};
#pragma unroll
  for (int c = 3; c + 1 < 32; c += 2) t4[(c >> 1) & 3] = fmaxf(fmaxf(t4[(c >> 1) & 3], x[c]), x[c + 1]);
  return fmaxf(fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])), x[31]);
}

// 32 scores -> P (fp16, TMEM column `at` on); adds their weights to `sum`.
__device__ __forceinline__ void weigh(const float (&x)[32], pair_t k2, pair_t off2, uint32_t at, pair_t (&sum)[2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float a, b;
      unpair(pair_fma(pair(x[16 * c + 2 * u], x[16 * c + 2 * u + 1]), k2, off2), a, b);
      a = ex2(a);
      b = ex2(b);
      sum[u & 1] = pair_add(sum[u & 1], pair(a, b));
      p[u] = pack_h2(a, b);
    }
    tc_st8(at + 8 * c, p);
  }
}
__device__ __forceinline__ float total(const pair_t (&sum)[2]) {
  float a, b;
  unpair(pair_add(sum[0], sum[1]), a, b);
  return a + b;
}

__device__ __forceinline__ void hand_over_p(ChunkCtrl& C, int i, int h) {
  tc_wait_st();
  tc_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(&C.p_ready[i][h]);
}

__device__ __forceinline__ int thread_id() {   // read again where it is used, not held over the loop
  int t;
  asm volatile("mov.u32 %0, %tid.x;" : "=r"(t));
  return t;
}

// Bits t - t0 of the tokens in [t0, t0 + 64) that the row at position p sees, in
// the tile's row order.
__device__ __forceinline__ uint2 visible64(int t0, int p, int window, int sinks) {
  auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
  unsigned long long m = below(p + 1 - t0);
  if (window > 0) m &= ~below(p - window + 1 - t0) | below(sinks - t0);
  m = (m & 0x9999999999999999ull) | ((m & 0x2222222222222222ull) << 1) | ((m & 0x4444444444444444ull) >> 1);
  return make_uint2((uint32_t)m, (uint32_t)(m >> 32));
}
__device__ __forceinline__ void hide(float (&x)[32], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < 32; ++c) x[c] = seen >> c & 1u ? x[c] : -INFINITY;
}

// A tile whose tokens have one scaling (all: every row of the warp sees every
// token).  Two halves of 64 keys: a row's scores of a half are held in
// registers, and the second half's are on their way while the first is weighed.
__device__ __forceinline__ bool soft_plain(const ChunkAttnArgs& A, ChunkCtrl& C, int i, int it, bool all, int t0,
                                           int first_row, const Scaling& sc, Row& w) {
  const float k = fmaxf(w.cm * sc.kmul, 0x1p-126f);           // (not 0: hidden scores are -inf, and stay it)
  const pair_t k2 = pair(k, k);
  float xa[32], xb[32];
  tc_ld32(xa, w.ts);
  tc_ld32(xb, w.ts + 32);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    tc_wait_ld();
    if (!all) {
      const int R = min(first_row + thread_id() % kRows, C.work.rows - 1);
      const uint2 seen = visible64(t0 + kHalf * h, C.work.sq.n + R / C.work.gq, A.window, A.sinks);
      hide(xa, seen.x);
      hide(xb, seen.y);
    }
    if (!raise(C, i, 2 * it + h, fmaf(most(most(-INFINITY, xa), xb), k, sc.vlog), w)) return false;
    const float off = sc.vlog - (w.r.m == -INFINITY ? 0.f : w.r.m);
    const pair_t off2 = pair(off, off);
    pair_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
    weigh(xa, k2, off2, w.ts + kHalf * h, sum);
    if (h == 0) tc_ld32(xa, w.ts + kHalf);
    weigh(xb, k2, off2, w.ts + kHalf * h + 16, sum);
    if (h == 0) tc_ld32(xb, w.ts + kHalf + 32);
    w.r.l = fmaf(total(sum), sc.vinv, w.r.l);
    hand_over_p(C, i, h);
  }
  return true;
}

// Any other tile: subtile by subtile with its own scaling, hidden and missing
// tokens left out.
__device__ __forceinline__ bool soft_any(const ChunkAttnArgs& A, ChunkCtrl& C, int i, int it, int slot, const Scaling& packed,
                                      int t0, int p_row, Row& w) {
  const TileInfo& info = C.info[slot];
  auto scaling = [&](int sub) {
    const int kind = info.kind[sub];
    return kind == 0 ? packed : kind == 1 ? Scaling{1.f, 0.f, 1.f} : Scaling{info.kmul[sub], info.vlog[sub], info.vinv[sub]};
  };
  auto bad_bits = [&](int sub) { return info.kind[sub] == 2 ? info.bad[sub] : 0u; };
  // scores (log2 units, with the value scale) less `ref`: the same steps as soft_plain's
  auto scores = [&](int sub, float ref, float (&x)[16]) {
    tc_ld16(x, w.ts + kTile * sub);
    tc_wait_ld();
    const Scaling sc = scaling(sub);
    const float k = w.cm * sc.kmul, off = sc.vlog - ref;
    const uint32_t seen = bad_bits(sub) >> 16 ? 0u : visible64(t0 + kTile * sub, p_row, A.window, A.sinks).x;
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = seen >> c & 1u ? fmaf(x[c], k, off) : -INFINITY;
  };
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const int s0 = kSubs / 2 * h;
    float top = -INFINITY;
#pragma unroll 1
    for (int j = 0; j < kSubs / 2; ++j) {
      float x[16];
      scores(s0 + j, 0.f, x);
#pragma unroll
      for (int c = 0; c < 16; ++c) top = fmaxf(top, x[c]);
    }
    if (!raise(C, i, 2 * it + h, top, w)) return false;
    const float ref = w.r.m == -INFINITY ? 0.f : w.r.m;
#pragma unroll 1
    for (int j = 0; j < kSubs / 2; ++j) {                      // P lies over scores that have been read
      float x[16], sum = 0.f;
      scores(s0 + j, ref, x);
      const uint32_t bad = bad_bits(s0 + j);
      uint32_t p[8];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if ((bad >> c & 1u) && x[c] != -INFINITY) sum = __int_as_float(0x7FC00000);   // the row sees such a value
        x[c] = ex2(x[c]);
        sum += x[c];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) p[u] = pack_h2(x[2 * u], x[2 * u + 1]);
      tc_st8(w.ts + kHalf * h + 8 * j, p);
      w.r.l = fmaf(sum, scaling(s0 + j).vinv, w.r.l);
    }
    hand_over_p(C, i, h);
  }
  return true;
}

// Row r (m, l, O) of stream i -> the caller's output, or this split's partial.
__device__ __forceinline__ void store_row(const ChunkAttnArgs& A, const Work& W, int R, const RowState& r, uint32_t to,
                                          bool any, const float* other, const float* f) {
  const kvq_shape& s = A.c.shape;
  const bool mine = R < W.rows;
  const size_t row = mine ? (size_t)(W.sq.t0 + R / W.gq) * s.num_q_heads + W.kv * W.gq + R % W.gq : 0;
  const bool partial = A.splits > 1;
  const float inv = partial ? 1.f : (r.l > 0.f ? 1.f / r.l : (r.l == 0.f ? 0.f : r.l));
  const size_t slot = (size_t)W.split * A.rows * s.num_q_heads + row;
#pragma unroll 1
  for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
    float o[32];
    if (any) {                               // warp-uniform
      tc_ld32(o, to + c0);
      tc_wait_ld();
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = any && r.l != 0.f ? o[i] * f[0] * inv : 0.f;
    if (other) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(other + 4 * (((c0 / 4) + i) ^ (threadIdx.x & 31)));
        o[4 * i] = fmaf(x.x, f[1] * inv, o[4 * i]); o[4 * i + 1] = fmaf(x.y, f[1] * inv, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(x.z, f[1] * inv, o[4 * i + 2]); o[4 * i + 3] = fmaf(x.w, f[1] * inv, o[4 * i + 3]);
      }
    }
    if (!mine) continue;
    if (partial) {
      float4* dst = reinterpret_cast<float4*>(A.ws_o + slot * kHeadDim + c0);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(A.out + row * kHeadDim + c0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = make_uint4(pack_bf2(o[8 * i], o[8 * i + 1]), pack_bf2(o[8 * i + 2], o[8 * i + 3]),
                            pack_bf2(o[8 * i + 4], o[8 * i + 5]), pack_bf2(o[8 * i + 6], o[8 * i + 7]));
    }
  }
  if (mine && partial) *reinterpret_cast<float2*>(A.ws_ml + 2 * slot) = make_float2(r.m, r.l);
}

// The softmax of stream i (its warps 4i ... 4i + 3; a thread has the row of its
// number), then the stream's part of the output.
template <int FMT, bool SHARED>
__device__ __forceinline__ void soften(const ChunkAttnArgs& A, ChunkCtrl& C, int i, float* o1_rows) {
  const Work& W = C.work;
  const int tiles = W.stream_tiles[i];
  bool ok = true;
  Row w;
  w.r = RowState{-INFINITY, 0.f};
  {
    const int row = thread_id() % kRows, lane = row & 31;
    const int R = W.r0 + (SHARED ? i * kRows : 0) + row, last = W.rows - 1, w0 = R - lane;
    const bool idle = w0 > last;                             // no row of this warp is real
    const uint32_t lanes = (uint32_t)(row & ~31) << 16;
    w.ts = tm_s(C.tmem, i) + lanes;
    w.to = tm_o(C.tmem, i) + lanes;
    // (not 0, so that -inf stays -inf: with a scale of 0 every score is the same all the same)
    w.cm = fmaxf(fabsf(A.scale_log2), 0x1p-100f) * C.qmul[SHARED ? i * kRows + row : row];
    if (lane == 0)
      C.seen[4 * i + row / 32] = make_int2(
          A.window > 0 ? W.sq.n + min(w0 + 31, last) / W.gq - A.window + 1 : 0, W.sq.n + min(w0, last) / W.gq);
    __syncwarp();
    const Scaling packed = FMT == 8 ? static_scaling(A.c, W.kv) : Scaling{1.f, 0.f, 1.f};
    for (int it = 0; it < tiles; ++it) {
      const int g = SHARED ? it : 2 * it + i, slot = g % kInfos;
      const int t0 = W.range.tile(W.first + g) * kKeys;
      const volatile int2& seen = C.seen[thread_id() / 32];
      const bool clear = t0 + kKeys - 1 <= seen.y && (t0 >= seen.x || t0 + kKeys <= A.sinks);
      if (!(ok = warp_wait(&C.s_full[i], it & 1, &C.abort))) break;
      if (idle) {
        if ((thread_id() & 31) == 0) {
          bar_arrive(&C.p_ready[i][0]);
          bar_arrive(&C.p_ready[i][1]);
        }
        continue;
      }
      tc_after();
      const uint2 kinds = *reinterpret_cast<const uint2*>(C.info[slot].kind);
      const bool one = kinds.x == kinds.y && kinds.x == (kinds.x & 0xFFu) * 0x01010101u && (kinds.x & 0xFFu) != 2u;
      const int first_row = W.r0 + (SHARED ? i * kRows : 0);
      if (one) {
        ok = soft_plain(A, C, i, it, clear, t0, first_row,
                        FMT != 8 || (kinds.x & 0xFFu) == 0u ? packed : Scaling{1.f, 0.f, 1.f}, w);
      } else {
        const int R = min(first_row + thread_id() % kRows, W.rows - 1);
        ok = soft_any(A, C, i, it, slot, packed, t0, W.sq.n + R / W.gq, w);
      }
      if (!ok) break;
    }
  }
  const bool any = tiles > 0;
  if (ok && any) ok = warp_wait(&C.finished[i], 0, &C.abort);
  const int row = thread_id() % kRows, lane = row & 31, R = W.r0 + (SHARED ? i * kRows : 0) + row;
  const bool idle = R - lane >= W.rows;
  tc_after();
  const float one[2] = {1.f, 0.f};
  if (SHARED) {
    if (ok && !idle) store_row(A, W, R, w.r, w.to, any, nullptr, one);
  } else {
    // join the streams: stream 1's row through shared memory (the tiles are used up)
    const int threads = 64 * min(4, (W.rows - W.r0 + 31) / 32);      // the softmax warps of both streams
    auto join = [&] { asm volatile("bar.sync 1, %0;\n" ::"r"(threads) : "memory"); };
    float* o1 = o1_rows + row * kHeadDim;
    join();
    if (i == 1) {
      C.ml[row][0] = w.r.m;
      C.ml[row][1] = w.r.l;
      if (ok && any && !idle) {
#pragma unroll 1
        for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
          float o[32];
          tc_ld32(o, w.to + c0);
          tc_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<float4*>(o1 + 4 * ((c0 / 4 + u) ^ lane)) =
                make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
    }
    join();
    if (i == 0 && ok && !idle) {
      const float m0 = w.r.m, m1 = C.ml[row][0], l1 = C.ml[row][1];
      const bool two = W.stream_tiles[1] > 0;
      const float M = fmaxf(m0, m1), ref = M == -INFINITY ? 0.f : M;
      const float f[2] = {ex2(m0 - ref), two && m1 != -INFINITY ? ex2(m1 - ref) : 0.f};
      const RowState j{M, w.r.l * f[0] + (two ? l1 * f[1] : 0.f)};
      store_row(A, W, R, j, w.to, any, two ? o1 : nullptr, f);
    }
  }
  tc_before();
}

// Grid (row blocks x splits, H_kv, B), 16 warps, one CTA per SM.
// SHARED: 256 query rows, a stream for each half, every key tile serves both.
// Otherwise 128 rows at most: both streams have the same rows, stream i takes
// the tiles of parity i, and the halves of the sum are joined at the end.
template <int FMT, bool SHARED>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_attention_kernel(const __grid_constant__ ChunkAttnArgs A) {
  extern __shared__ uint8_t smem_raw[];
  grid_dependents_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const kvq_shape& s = A.c.shape;
  constexpr int kBlockRows = (SHARED ? 2 : 1) * kRows;
  Work W;
  W.kv = blockIdx.y;
  W.b = blockIdx.z;
  W.gq = s.num_q_heads / s.num_kv_heads;
  W.split = blockIdx.x % A.splits;
  W.r0 = (int)(gridDim.x / A.splits - 1 - blockIdx.x / A.splits) * kBlockRows;   // the longest rows first
  W.sq = chunk_seq(A, W.b);
  W.rows = W.sq.m * W.gq;
  if (W.sq.err && blockIdx.x == 0 && W.kv == 0 && tid == 0) atomicOr(A.c.err_word, W.sq.err);
  if (W.r0 >= W.rows) return;
  const int block_rows = min(kBlockRows, W.rows - W.r0);
  const TileRange range(W.sq.n + W.r0 / W.gq, W.sq.n + (W.r0 + block_rows - 1) / W.gq, A.window, A.sinks, kKeys);
  W.range = range;
  W.first = (int)((int64_t)range.count * W.split / A.splits);
  W.tiles = (int)((int64_t)range.count * (W.split + 1) / A.splits) - W.first;
  if (SHARED) {
    W.stream_tiles[0] = W.tiles;
    W.stream_tiles[1] = block_rows > kRows ? W.tiles : 0;
  } else {
    W.stream_tiles[0] = (W.tiles + 1) / 2;
    W.stream_tiles[1] = W.tiles / 2;
  }

  const uint32_t q_tiles = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t k_tiles = q_tiles + (SHARED ? 2 : 1) * kTileBytes16, v_tiles = k_tiles + kStages * kTileBytes16;
  uint8_t* generic = smem_raw + (q_tiles - smem_u32(smem_raw));
  ChunkCtrl& C = *reinterpret_cast<ChunkCtrl*>(generic + (v_tiles + value_stages(SHARED) * kTileBytes16 - q_tiles));
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(&C.k_full[i], kSubs); bar_init(&C.k_empty[i], 1);
    }
    for (int i = 0; i < kMaxValueStages; ++i) { bar_init(&C.v_full[i], kSubs); bar_init(&C.v_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      bar_init(&C.s_full[i], 1); bar_init(&C.o_done[i], 1); bar_init(&C.finished[i], 1);
      const int busy = SHARED ? 4 : (block_rows + 31) / 32;
      bar_init(&C.p_ready[i][0], busy); bar_init(&C.p_ready[i][1], busy);
    }
    bar_init(&C.drained, 1);
    C.abort = 0;
    C.work = W;
    C.straight = s.rope_theta > 0.f || s.sparse ? 0 : W.sq.nq;
    C.sinks = A.sinks;
    C.clear = A.window > 0 ? W.sq.n + (W.r0 + block_rows - 1) / W.gq - A.window + 1 : 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kProducerWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&C.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  __shared__ UnitSrc<FMT> unit;              // read again for every tile: no registers held
  if (tid == 32 * kProducerWarp) unit.init(A.c, W.b, W.kv);
  if (s.rope_theta > 0.f && warp == kProducerWarp) {
    for (int i = lane; i < kHeadDim / 2; i += 32) C.freq[i] = pow((double)s.rope_theta, -2.0 * i / kHeadDim);
  }
  // Query rows -> fp16 in the key tiles' channel order, powers of two aside
  // (they go into the row's factor), negated for a negative scale; 16 threads
  // a row, rows past the end zero.
  {
    constexpr int kPer = kBlockRows * 16 / kChunkThreads;
    const int p = tid & 15;
    uint4 w[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int R = W.r0 + (tid >> 4) + u * (kChunkThreads / 16);
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (R < W.rows)
        w[u] = *reinterpret_cast<const uint4*>(
            A.q + ((size_t)(W.sq.t0 + R / W.gq) * s.num_q_heads + W.kv * W.gq + R % W.gq) * kHeadDim + 8 * p);
    }
    const uint32_t sign = A.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll 2
    for (int u = 0; u < kPer; ++u) {
      const int row = (tid >> 4) + u * (kChunkThreads / 16);
      uint4 v = w[0];
#pragma unroll
      for (int i = 0; i + 1 < kPer; ++i) w[i] = w[i + 1];
      v.x ^= sign; v.y ^= sign; v.z ^= sign; v.w ^= sign;
      uint32_t m = larger_half(abs_max8(0u, v));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t at = piece_at(q_tiles + (row / kRows) * kTileBytes16, row % kRows, p);
      float factor = 1.f;
      if (__all_sync(0xffffffffu, ordinary(m))) {
        put_raw8(at, v, true);
      } else {
        factor = put_scaled8(at, v);
      }
      if (p == 0) C.qmul[row] = factor;
    }
    fence_async();
  }
  if (FMT == 8 && tid == 0 && A.c.fp8_scale[s.num_kv_heads + W.kv] < kLeastScale) C.straight = 0;
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = C.tmem;

  if (warp == kMmaWarp) {
    if (!issue_all<SHARED>(C, q_tiles, k_tiles, v_tiles) && elect_one()) drain(C);
    __syncwarp();
  } else if (warp < kProducerWarp && (SHARED || 32 * (warp & 3) < block_rows)) {
    soften<FMT, SHARED>(A, C, __shfl_sync(0xffffffffu, warp >> 2, 0), reinterpret_cast<float*>(generic + kTileBytes16));
  } else {
    // with shared keys every softmax warp stays one; otherwise those without rows help
    const int busy = SHARED ? 4 : (block_rows + 31) / 32;    // softmax warps per stream
    const int pw = warp >= kProducerWarp ? warp - kProducerWarp
                                         : kProducers + (warp >> 2) * (4 - busy) + (warp & 3) - busy;
    // (with at most two tiles' subtiles between its own, a producer leaves out no
    // use of a stage that a barrier's parity could take for the next)
    static_assert(kProducers + 2 * 3 <= 2 * kSubs, "producers");
    produce<FMT, SHARED>(A, C, unit, k_tiles, v_tiles, pw, kProducers + 2 * (4 - busy));
  }
  __syncthreads();
  if (warp == kProducerWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
  if (tid == 0 && C.abort) atomicOr(A.c.err_word, KVQ_DEVERR_WAIT_TIMEOUT);
}

// Joins the splits' partials.  Grid (rows of a sequence / 8, B), one warp per
// (new token, query head) row, four channels per lane.
__global__ void __launch_bounds__(256) chunk_merge_kernel(ChunkAttnArgs A) {
  grid_dependency_wait();
  const kvq_shape& s = A.c.shape;
  const ChunkSeq sq = chunk_seq(A, blockIdx.y);
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= (int64_t)sq.m * s.num_q_heads) return;
  const size_t row = (size_t)sq.t0 * s.num_q_heads + i, rows = (size_t)A.rows * s.num_q_heads;
  float M = -INFINITY;
  for (int p = 0; p < A.splits; ++p) M = fmaxf(M, A.ws_ml[2 * (p * rows + row)]);
  const float ref = M == -INFINITY ? 0.f : M;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < A.splits; ++p) {
    const float2 ml = *reinterpret_cast<const float2*>(A.ws_ml + 2 * (p * rows + row));
    if (ml.y == 0.f) continue;               // nothing visible in this range (NaN goes on)
    const float f = ex2(ml.x - ref);
    const float4 x = *reinterpret_cast<const float4*>(A.ws_o + (p * rows + row) * kHeadDim + 4 * lane);
    l = fmaf(ml.y, f, l);
    o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y); o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
  *reinterpret_cast<uint2*>(A.out + row * kHeadDim + 4 * lane) = make_uint2(pack_bf2(o.x, o.y), pack_bf2(o.z, o.w));
}

// --- host -----------------------------------------------------------------

static bool shared_keys(const kvq_shape& s, int max_new) {
  return (long long)max_new * (s.num_q_heads / s.num_kv_heads) > kRows;
}
static long long row_blocks(const kvq_shape& s, int max_new) {
  const long long rows = (long long)max_new * (s.num_q_heads / s.num_kv_heads);
  const int block = shared_keys(s, max_new) ? 2 * kRows : kRows;
  return (rows + block - 1) / block;
}

size_t chunk_workspace_bytes(const kvq_shape& s, int num_splits, int rows) {
  if (num_splits <= 1) return 0;
  return (size_t)num_splits * rows * s.num_q_heads * (kHeadDim + 2) * sizeof(float);
}

// Key ranges per row block: the fewest rounds of CTAs over the SMs, counting
// what a CTA costs beside its tiles (set-up and output, worth about four
// tiles).  2048 tokens over 32768 (256 row blocks): 1 range 1317 us, 4 1316;
// 6 tokens over 8 x 8192: 1 range 104 us, 2 ranges 69, 4 77.
int chunk_default_splits(const kvq_shape& s, int rows, int max_new, int max_len, int window, int sinks) {
  const long long span = window > 0 ? min((long long)max_len + max_new, (long long)window + sinks + max_new)
                                    : (long long)max_len + max_new;
  const int tiles = (int)((span + kKeys - 1) / kKeys) + 1;
  const long long ctas = row_blocks(s, max_new) * s.num_kv_heads * min(s.batch, max(rows, 1));
  int best = 1;
  double least = 1e30;
  for (int n = 1; n <= 64 && n <= tiles; ++n) {
    const long long rounds = (ctas * n + 147) / 148;
    const double t = (double)rounds * ((tiles + n - 1) / n + 4 + (n > 1 ? 1 : 0));
    if (t < least * 0.97) {
      least = t;
      best = n;
    }
  }
  return best;
}

template <int FMT, bool SHARED>
static cudaError_t launch_form(const ChunkAttnArgs& A, cudaStream_t st) {
  const kvq_shape& s = A.c.shape;
  constexpr int kSmem = chunk_smem_bytes(SHARED);
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(chunk_attention_kernel<FMT, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmem);
  if (e != cudaSuccess) return e;
  const long long x = max(row_blocks(s, min(A.max_new, A.rows)), 1ll) * A.splits;   // (the kernel divides by the splits)
  if (x > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  dim3 grid((unsigned)x, s.num_kv_heads, s.batch);
  chunk_attention_kernel<FMT, SHARED><<<grid, kChunkThreads, kSmem, st>>>(A);
  return cudaGetLastError();
}

cudaError_t launch_chunk_attention(const ChunkAttnArgs& args, cudaStream_t st) {
  ChunkAttnArgs A = args;
  const kvq_shape& s = A.c.shape;
  const size_t rows = (size_t)A.rows * s.num_q_heads;
  A.ws_ml = A.ws_o ? A.ws_o + (size_t)A.splits * rows * kHeadDim : nullptr;
  const bool wide = shared_keys(s, min(A.max_new, A.rows));
  cudaError_t e;
#define KVQ_CHUNK_FORM(F) (wide ? launch_form<F, true>(A, st) : launch_form<F, false>(A, st))
  switch (s.format) {
    case KVQ_FORMAT_INT2: e = KVQ_CHUNK_FORM(2); break;
    case KVQ_FORMAT_INT4: e = KVQ_CHUNK_FORM(4); break;
    case KVQ_FORMAT_MIXED: e = KVQ_CHUNK_FORM(6); break;
    case KVQ_FORMAT_FP8_E4M3: e = KVQ_CHUNK_FORM(8); break;
    default: e = KVQ_CHUNK_FORM(16); break;
  }
#undef KVQ_CHUNK_FORM
  if (e != cudaSuccess || A.splits == 1) return e;
  const long long per_seq = (long long)min(A.max_new, A.rows) * s.num_q_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)max((per_seq + 7) / 8, 1ll), s.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel, A);
}

}  // namespace kvq
