// The NVFP4 key/value cache: head norms and position rotation in front of it,
// the quantizing write, and the read back to bf16.
//
// Cache layout (pages of ps tokens, H heads of D values; ps a power of two
// >= 16):
//   K codes  [page][head][token][D/2]        K scales [page][head][token][D/16]
//   V codes  [page][head][ps/16][D/2][16]    V scales [page][head][ps/16][D/16][16]
// K rows lie as the format has them.  V is grouped in fragments of 16 tokens
// with the token last: a lane of the attention kernels then finds the codes
// of one value pair for 16 consecutive tokens in one 16-byte load, which is
// the order the product with the softmax weights contracts over, so V needs
// no transposition on the read path.  One byte still belongs to one token,
// so appending a token is plain byte stores and never a read-modify-write.
#include "common.h"
#include "kv_cache.h"
#include "quant_block.h"

namespace nvfp4k {
namespace {

// Where slot s lives: token s % ps of page s / ps.
struct SlotPlace {
  int64_t page;
  int32_t at;
};
__device__ __forceinline__ SlotPlace place_of(int64_t slot, const KvCache& c) {
  return {slot >> c.ps_log2, (int32_t)(slot & ((1 << c.ps_log2) - 1))};
}
__device__ __forceinline__ bool slot_valid(int64_t slot, const KvCache& c) {
  return slot >= 0 && (slot >> c.ps_log2) < c.num_pages;
}

// Piece x of a workgroup whose pieces begin at `first`, `per_token` pieces a
// token: token t, piece r of it.  One 64-bit division for the workgroup.
struct Piece {
  int64_t t;
  int32_t r;
};
__device__ __forceinline__ Piece piece_of(int64_t first, uint32_t x, int per_token) {
  const int64_t t0 = first / per_token;
  const uint32_t y = (uint32_t)(first - t0 * per_token) + x, dt = y / (uint32_t)per_token;
  return {t0 + dt, (int32_t)(y - dt * per_token)};
}

// Workgroups go round the 8 XCDs in turn; with this each XCD takes a run of the
// n (a multiple of 8) places, so that neighbours, which share fragments and
// scale lines at their ends, share an L2: 65536 tokens x 8 heads of 128 read
// back fetch 77 MB instead of 128, 16381 written store 19 instead of 27.
__device__ __forceinline__ int64_t in_runs(uint32_t x, uint32_t n) { return (int64_t)(x & 7) * (n >> 3) + (x >> 3); }

// ---- quantizing write -----------------------------------------------------

// One thread quantizes one 16-block of one K row (the format's absmax rule)
// and stores its 8 code bytes and scale byte.
__device__ __forceinline__ void write_k_block(const KvCache& c, int64_t slot, int head, int blk,
                                              const uint32_t (&w)[8], float g, float rg) {
  if (!slot_valid(slot, c)) return;
  const SlotPlace p = place_of(slot, c);
  const int64_t row = ((p.page * c.heads + head) << c.ps_log2) + p.at;
  uint32_t sc;
  const uint2 codes = absmax_block<true>(w, g, rg, sc);
  *reinterpret_cast<uint2*>(c.k_codes + row * (c.head_dim >> 1) + blk * 8) = codes;
  c.k_scales[row * (c.head_dim >> 4) + blk] = (uint8_t)sc;
}

// The same for one V row: the 8 code bytes go to 8 value pairs of the
// token's fragment, 16 bytes apart.
__device__ __forceinline__ void write_v_block(const KvCache& c, int64_t slot, int head, int blk,
                                              const uint32_t (&w)[8], float g, float rg) {
  if (!slot_valid(slot, c)) return;
  const SlotPlace p = place_of(slot, c);
  const int64_t frag = ((p.page * c.heads + head) << (c.ps_log2 - 4)) + (p.at >> 4);
  const int tok = p.at & 15;
  uint32_t sc;
  const uint2 codes = absmax_block<true>(w, g, rg, sc);
  uint8_t* dst = c.v_codes + frag * (c.head_dim * 8) + blk * 128 + tok;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dst[i * 16] = (uint8_t)(codes.x >> (8 * i));
    dst[(i + 4) * 16] = (uint8_t)(codes.y >> (8 * i));
  }
  c.v_scales[frag * c.head_dim + blk * 16 + tok] = (uint8_t)sc;
}

__device__ __forceinline__ void load_block(const uint16_t* src, uint32_t (&w)[8]) {
  const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// V blocks of a unit: 16 tokens (the lane's low bits, so that consecutive
// slots give 16-byte stores) x 4 blocks of one head per wave.
__device__ __forceinline__ void write_v_unit(const KvCache& c, int64_t unit, const uint16_t* v, int64_t v_stride,
                                             const int64_t* slots, int64_t tokens) {
  const int lane = threadIdx.x & 63;
  const int quads = c.head_dim >> 6;                 // groups of 4 blocks in a row
  const int per_group = c.heads * quads;
  const int64_t tg = unit / per_group;
  const int r = (int)(unit - tg * per_group);
  const int head = r / quads, blk = (r - head * quads) * 4 + (lane >> 4);
  const int64_t t = tg * 16 + (lane & 15);
  if (t >= tokens) return;
  const float g = *c.v_gscale;
  uint32_t w[8];
  load_block(v + t * v_stride + head * c.head_dim + blk * 16, w);
  write_v_block(c, slots[t], head, blk, w, g, scale_recip(g));
}

// Grid: first the K blocks (one thread each), then the V units (one wave each).
// Bound by HBM: 16381 tokens x 8 heads of 128, 86 MB, in 20.5 us, 4.2 TB/s (a
// large copy reaches 5.1; two or four blocks a thread take as long); a few
// tokens by latency, 4 us.
__global__ __launch_bounds__(256) void kv_write_kernel(KvCache c, const uint16_t* k, int64_t k_stride,
                                                       const uint16_t* v, int64_t v_stride, const int64_t* slots,
                                                       int64_t tokens, int64_t k_groups) {
  if ((int64_t)blockIdx.x < k_groups) {
    const int blocks = c.head_dim >> 4;
    const Piece p = piece_of(in_runs(blockIdx.x, (uint32_t)k_groups) * 256, threadIdx.x, c.heads * blocks);
    if (p.t >= tokens) return;
    const int head = p.r / blocks, blk = p.r - head * blocks;
    const float g = *c.k_gscale;
    uint32_t w[8];
    load_block(k + p.t * k_stride + p.r * 16, w);
    write_k_block(c, slots[p.t], head, blk, w, g, scale_recip(g));
  } else {
    const int64_t unit = in_runs(blockIdx.x - (uint32_t)k_groups, gridDim.x - (uint32_t)k_groups) * 4 + (threadIdx.x >> 6);
    write_v_unit(c, unit, v, v_stride, slots, tokens);
  }
}

// ---- read back ------------------------------------------------------------

// A value pair, fl32(E2M1 * fl32(s g)) rounded once to bf16, of byte `sel` of
// the codes.
template <int sel>
__device__ __forceinline__ uint32_t value_pair(uint32_t codes, float d) {
  const half2v h = e2m1x2_to_f16<sel>(codes);
  return f32x2_to_bf16x2_rne((float)h.x * d, (float)h.y * d);
}

// K: a thread turns 8 values (a dword of codes) into one 16-byte store, kPieces
// of them a workgroup's width apart.
// V, long lists (kPieces > 1): a wave takes 16 tokens of one head (two heads
// with D = 64, half a head with D = 256), a lane one value pair; every
// token's row then leaves as 4 bytes a lane.  Where the 16 slots run on by
// one -- a stretch of a sequence -- their codes are the 16 bytes of a fragment
// or straddle two, so two 16-byte loads and a byte shift fetch all 16 tokens;
// other slot lists load a byte a token.
// V, short lists: a thread gathers one 16-block, the blocks laid out as in the
// write.  More requests, a shorter chain: 777 tokens x 4 heads of 64 take
// 3.4 us against 5.5, but 65536 x 8 heads of 128 take 102 against 69 (344 MB:
// 5.0 TB/s, the rate of a large copy).

// The V block a thread of a write_v_unit layout owns.
__device__ __forceinline__ void read_v_unit(const KvCache& c, int64_t unit, const int64_t* slots, int64_t tokens,
                                            uint16_t* v) {
  const int lane = threadIdx.x & 63, d = c.head_dim;
  const int quads = d >> 6, per_group = c.heads * quads;
  const int64_t tg = unit / per_group;
  const int r = (int)(unit - tg * per_group), head = r / quads, blk = (r - head * quads) * 4 + (lane >> 4);
  const int64_t t = tg * 16 + (lane & 15);
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  uint32_t lo = 0u, hi = 0u, sc = 0u;
  if (slot_valid(slot, c)) {
    const SlotPlace p = place_of(slot, c);
    const int64_t frag = ((p.page * c.heads + head) << (c.ps_log2 - 4)) + (p.at >> 4);
    const uint8_t* src = c.v_codes + frag * (d * 8) + blk * 128 + (p.at & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo |= (uint32_t)src[i * 16] << (8 * i);
      hi |= (uint32_t)src[(i + 4) * 16] << (8 * i);
    }
    sc = c.v_scales[frag * d + blk * 16 + (p.at & 15)];
  }
  const float s = e4m3_to_f32(sc) * *c.v_gscale;
  uint4* dst = reinterpret_cast<uint4*>(v + (t * c.heads + head) * d + blk * 16);
  dst[0] = make_uint4(value_pair<0>(lo, s), value_pair<1>(lo, s), value_pair<2>(lo, s), value_pair<3>(lo, s));
  dst[1] = make_uint4(value_pair<0>(hi, s), value_pair<1>(hi, s), value_pair<2>(hi, s), value_pair<3>(hi, s));
}

// Bytes o .. o + 15 of the 32 in (a, b).
__device__ __forceinline__ void shift_bytes(const uint4& a, const uint4& b, int o, uint32_t (&w)[4]) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = o >> 2;                                  // uniform over the wave
    const uint32_t lo = q == 0 ? x[i] : q == 1 ? x[i + 1] : q == 2 ? x[i + 2] : x[i + 3];
    const uint32_t hi = q == 0 ? x[i + 1] : q == 1 ? x[i + 2] : q == 2 ? x[i + 3] : x[i + 4];
    w[i] = __builtin_amdgcn_alignbyte(hi, lo, o & 3);
  }
}

template <int kPieces>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, const int64_t* slots, int64_t tokens, uint16_t* k,
                                                      uint16_t* v, int64_t k_groups) {
  const int d = c.head_dim;
  if ((int64_t)blockIdx.x < k_groups) {
    const int pieces = d >> 3, per_token = c.heads * pieces;
    const int64_t first = in_runs(blockIdx.x, (uint32_t)k_groups) * (256 * kPieces);
    const float g = *c.k_gscale;
    // slots, then codes and scales, of every piece at once; padding reads
    // slot 0 and drops what it gets
    Piece p[kPieces];
    int64_t slot[kPieces];
    uint32_t codes[kPieces], sc[kPieces];
    bool live[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      p[j] = piece_of(first, threadIdx.x + 256 * j, per_token);
      live[j] = p[j].t < tokens;
      slot[j] = slots[live[j] ? p[j].t : 0];
    }
    const bool pool = c.num_pages > 0;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const bool ok = slot_valid(slot[j], c);
      const SlotPlace at = place_of(ok ? slot[j] : 0, c);
      const int head = p[j].r / pieces, piece = p[j].r - head * pieces;
      const int64_t row = ((at.page * c.heads + head) << c.ps_log2) + at.at;
      codes[j] = pool ? *reinterpret_cast<const uint32_t*>(c.k_codes + row * (d >> 1) + piece * 4) : 0u;
      sc[j] = pool ? c.k_scales[row * (d >> 4) + (piece >> 1)] : 0u;
      if (!ok) codes[j] = sc[j] = 0u;
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (!live[j]) continue;
      const float s = e4m3_to_f32(sc[j]) * g;
      *reinterpret_cast<uint4*>(k + (first + threadIdx.x + 256 * j) * 8) =
          make_uint4(value_pair<0>(codes[j], s), value_pair<1>(codes[j], s), value_pair<2>(codes[j], s),
                     value_pair<3>(codes[j], s));
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t unit = in_runs(blockIdx.x - (uint32_t)k_groups, gridDim.x - (uint32_t)k_groups) * 4 + (threadIdx.x >> 6);
  if constexpr (kPieces == 1) {
    read_v_unit(c, unit, slots, tokens, v);
    return;
  }
  const int per_group = (c.heads * d + 127) >> 7;            // waves of 64 value pairs
  const int64_t tg = unit / per_group;
  const int64_t t0 = tg * 16;
  if (t0 >= tokens) return;
  const int value = ((int)(unit - tg * per_group) * 64 + lane) * 2;   // of the token's row
  const bool in_row = value < c.heads * d;                            // an odd count of heads of 64 leaves half a wave
  const int head = in_row ? value / d : 0, pair = in_row ? (value - head * d) >> 1 : 0;
  const int count = (int)min((int64_t)16, tokens - t0);
  const float g = *c.v_gscale;
  const int64_t mine = (lane & 15) < count ? slots[t0 + (lane & 15)] : -1;
  const int64_t slot0 = __shfl(mine, 0, 64);
  uint16_t* out = v + t0 * c.heads * d + value;
  const int64_t row_step = (int64_t)c.heads * d;
  auto fragment = [&](int64_t slot) {
    const SlotPlace p = place_of(slot, c);
    return ((p.page * c.heads + head) << (c.ps_log2 - 4)) + (p.at >> 4);
  };
  if (__all(mine == slot0 + (lane & 15) && slot_valid(mine, c))) {
    const int64_t fa = fragment(slot0), fb = fragment(slot0 + 15);
    const int o = (int)(slot0 & 15);
    const uint4 ca = *reinterpret_cast<const uint4*>(c.v_codes + fa * (d * 8) + pair * 16);
    const uint4 cb = *reinterpret_cast<const uint4*>(c.v_codes + fb * (d * 8) + pair * 16);
    const uint4 sa = *reinterpret_cast<const uint4*>(c.v_scales + fa * d + (pair >> 3) * 16);
    const uint4 sb = *reinterpret_cast<const uint4*>(c.v_scales + fb * d + (pair >> 3) * 16);
    uint32_t codes[4], sc[4];
    shift_bytes(ca, cb, __builtin_amdgcn_readfirstlane(o), codes);
    shift_bytes(sa, sb, __builtin_amdgcn_readfirstlane(o), sc);
    if (!in_row) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = e4m3_to_f32((sc[i] >> (8 * j)) & 0xFFu) * g;
        const uint32_t x = j == 0 ? value_pair<0>(codes[i], s) : j == 1 ? value_pair<1>(codes[i], s)
                         : j == 2 ? value_pair<2>(codes[i], s) : value_pair<3>(codes[i], s);
        *reinterpret_cast<uint32_t*>(out + (4 * i + j) * row_step) = x;
      }
    }
    return;
  }
  uint32_t codes[16], sc[16];
  const bool pool = c.num_pages > 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t slot = __shfl(mine, i, 64);
    const bool ok = slot_valid(slot, c);
    const int64_t f = fragment(ok ? slot : 0);
    const int at = ok ? (int)(slot & 15) : 0;
    codes[i] = pool ? c.v_codes[f * (d * 8) + pair * 16 + at] : 0u;
    sc[i] = pool ? c.v_scales[f * d + (pair >> 3) * 16 + at] : 0u;
    if (!ok) codes[i] = sc[i] = 0u;
  }
  if (!in_row) return;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < count) *reinterpret_cast<uint32_t*>(out + i * row_step) = value_pair<0>(codes[i], e4m3_to_f32(sc[i]) * g);
}

// ---- head norms and position rotation ---------------------------------------

// A row (one head of one token) belongs to D/8 lanes, 8 values each, held as
// two pieces of four so that a rotation pair never leaves its lane:
//   halves (i, i + rot/2): pieces 4 l and rot/2 + 4 l for l < rot/8, and
//     8 consecutive values past rot for the lanes that only pass through;
//   interleaved (2 i, 2 i + 1): 8 consecutive values.
// Either way lane l uses cos/sin entries 4 l .. 4 l + 3.
//
// Bound by HBM at many tokens (4 bytes a value); the vector unit is close
// behind, so the row sum runs on data-parallel-primitive adds, the root is the
// hardware's reciprocal square root (1 ulp of fp32 under a bf16 rounding) and
// nothing is divided per row: 16381 tokens x 72 heads of 128, 612 MB, in 118
// us, 5.2 TB/s, a large copy's rate.

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
  auto add = [](float x, int moved) { return x + __builtin_bit_cast(float, moved); };
#define NVFP4_DPP(x, ctrl) __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), ctrl, 0xF, 0xF, true)
  v = add(v, NVFP4_DPP(v, 0xB1));                       // quad_perm 1,0,3,2
  v = add(v, NVFP4_DPP(v, 0x4E));                       // quad_perm 2,3,0,1
  v = add(v, NVFP4_DPP(v, 0x141));                      // row_half_mirror: the other quad of 8
  if constexpr (kLanes >= 16) v = add(v, NVFP4_DPP(v, 0x140));   // row_mirror: the other 8 of 16
#undef NVFP4_DPP
  if constexpr (kLanes >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// The hardware's reciprocal root takes denormal numbers for zero.
__device__ __forceinline__ float rsqrt_of(float x) {
  const bool tiny = x < 0x1p-126f;
  return __builtin_amdgcn_rsqf(tiny ? x * 0x1p32f : x) * (tiny ? 0x1p16f : 1.0f);
}

template <int D, int kRows, bool kInter, bool kWrite>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope a, KvCache c, const int64_t* slots,
                                                        const uint16_t* v, int64_t v_stride, int64_t row_groups) {
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes;
  if (kWrite && (int64_t)blockIdx.x >= row_groups) {
    const int64_t group = in_runs(blockIdx.x - (uint32_t)row_groups, gridDim.x - (uint32_t)row_groups);
    write_v_unit(c, group * 4 + (threadIdx.x >> 6), v, v_stride, slots, a.tokens);
    return;
  }
  // K rows on their way to the cache, as bf16, for the 16-block quantizer
  __shared__ __align__(16) uint16_t stage[kWrite ? kRows * kGroups * D : 8];
  const int l = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const uint32_t heads = a.q_heads + a.k_heads;
  const int half = a.rot >> 1;
  const uint32_t row0 = blockIdx.x * (kRows * kGroups), t0 = row0 / heads, h0 = row0 - t0 * heads;
  const bool turn = kInter ? 8 * l < a.rot : 4 * l < half;
  const int at0 = kInter ? 8 * l : turn ? 4 * l : a.rot + 8 * (l - (a.rot >> 3));
  const int at1 = at0 + (turn && !kInter ? half : 4);
  // token and head of the workgroup's row x: a multiplication by 2^32 / heads
  // rounded up, exact while x * heads < 2^32 (heads <= 2^15 is checked)
  auto place = [&](uint32_t x, int64_t& t, int& h) {
    const uint32_t y = h0 + x, dt = heads == 1 ? y : __umulhi(y, a.heads_magic);
    t = (int64_t)t0 + dt;
    h = (int)(y - dt * heads);
  };
  // every load first: weights, the rows, their positions, their table entries
  uint2 qw0, qw1, kw0, kw1;
  qw0 = qw1 = kw0 = kw1 = make_uint2(0x3F803F80u, 0x3F803F80u);       // ones
  if (a.q_weight) {
    qw0 = *reinterpret_cast<const uint2*>(a.q_weight + at0);
    qw1 = *reinterpret_cast<const uint2*>(a.q_weight + at1);
  }
  if (a.k_weight) {
    kw0 = *reinterpret_cast<const uint2*>(a.k_weight + at0);
    kw1 = *reinterpret_cast<const uint2*>(a.k_weight + at1);
  }
  uint2 p0[kRows], p1[kRows];
  int64_t t[kRows];
  int h[kRows], pos[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    place(i * kGroups + grp, t[i], h[i]);
    p0[i] = p1[i] = make_uint2(0u, 0u);
    pos[i] = -1;
    if (t[i] < a.tokens) {
      const uint16_t* src = h[i] < a.q_heads ? a.q + t[i] * a.q_stride + h[i] * D
                                             : a.k + t[i] * a.k_stride + (h[i] - a.q_heads) * D;
      p0[i] = *reinterpret_cast<const uint2*>(src + at0);
      p1[i] = *reinterpret_cast<const uint2*>(src + at1);
      if (turn) pos[i] = a.positions[t[i]];
    }
  }
  float4 cs[kRows], sn[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float nan = __builtin_nanf("");                  // past the table: NaN, never a stray read
    cs[i] = sn[i] = make_float4(nan, nan, nan, nan);
    if ((uint32_t)pos[i] < (uint32_t)a.max_pos) {
      const float* tab = a.cos_sin + (int64_t)pos[i] * a.rot + 4 * l;
      cs[i] = *reinterpret_cast<const float4*>(tab);
      sn[i] = *reinterpret_cast<const float4*>(tab + half);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (t[i] >= a.tokens) continue;        // uniform over the lanes of a row
    const bool is_q = h[i] < a.q_heads;
    float y[8];
    const uint32_t xw[4] = {p0[i].x, p0[i].y, p1[i].x, p1[i].y};
    const uint32_t w[4] = {is_q ? qw0.x : kw0.x, is_q ? qw0.y : kw0.y, is_q ? qw1.x : kw1.x, is_q ? qw1.y : kw1.y};
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = __uint_as_float(xw[j] << 16);
      y[2 * j + 1] = __uint_as_float(xw[j] & 0xFFFF0000u);
      ss = __builtin_fmaf(y[2 * j], y[2 * j], ss);
      ss = __builtin_fmaf(y[2 * j + 1], y[2 * j + 1], ss);
    }
    const float r = rsqrt_of(row_sum<kLanes>(ss) * (1.0f / D) + a.eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = y[2 * j] * r * __uint_as_float(w[j] << 16);
      y[2 * j + 1] = y[2 * j + 1] * r * __uint_as_float(w[j] & 0xFFFF0000u);
    }
    if (turn) {
      const float cv[4] = {cs[i].x, cs[i].y, cs[i].z, cs[i].w}, sv[4] = {sn[i].x, sn[i].y, sn[i].z, sn[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float& u0 = y[kInter ? 2 * j : j];
        float& u1 = y[kInter ? 2 * j + 1 : j + 4];
        const float r0 = u0 * cv[j] - u1 * sv[j], r1 = u1 * cv[j] + u0 * sv[j];
        u0 = r0;
        u1 = r1;
      }
    }
    const uint2 o0 = make_uint2(f32x2_to_bf16x2_rne(y[0], y[1]), f32x2_to_bf16x2_rne(y[2], y[3]));
    const uint2 o1 = make_uint2(f32x2_to_bf16x2_rne(y[4], y[5]), f32x2_to_bf16x2_rne(y[6], y[7]));
    uint16_t* dst;
    if (is_q) dst = a.q_out + t[i] * a.q_out_stride + h[i] * D;
    else if (kWrite) dst = stage + (i * kGroups + grp) * D;
    else dst = a.k_out + t[i] * a.k_out_stride + (h[i] - a.q_heads) * D;
    *reinterpret_cast<uint2*>(dst + at0) = o0;
    *reinterpret_cast<uint2*>(dst + at1) = o1;
  }
  if (kWrite) {
    __syncthreads();
    constexpr int kBlocks = D / 16;
    const float g = *c.k_gscale, rg = scale_recip(g);
    for (int i = threadIdx.x; i < kRows * kGroups * kBlocks; i += 256) {
      const int row = i / kBlocks, blk = i % kBlocks;
      int64_t tok;
      int hd;
      place(row, tok, hd);
      hd -= a.q_heads;
      if (hd < 0 || tok >= a.tokens) continue;
      uint32_t w[8];
      load_block(stage + row * D + blk * 16, w);
      write_k_block(c, slots[tok], hd, blk, w, g, rg);
    }
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Workgroups, rounded up for in_runs (the added ones find no token).
int64_t run_groups(int64_t pieces, int64_t per_group) { return ceil_div(pieces, 8 * per_group) * 8; }
int64_t k_block_groups(const KvCache& c, int64_t tokens) { return run_groups(tokens * c.heads * (c.head_dim >> 4), 256); }
int64_t v_unit_groups(const KvCache& c, int64_t tokens) {
  return run_groups(ceil_div(tokens, 16) * c.heads * (c.head_dim >> 6), 4);
}

template <int D, int kRows, bool kInter>
void run_norm_rope(const NormRope& a, const KvCache* c, const int64_t* slots, const uint16_t* v, int64_t v_stride,
                   hipStream_t stream) {
  const int64_t per_group = (int64_t)kRows * (256 / (D / 8));
  const int64_t rows = ceil_div(a.tokens * (a.q_heads + a.k_heads), per_group);
  if (c)
    norm_rope_kernel<D, kRows, kInter, true>
        <<<dim3((uint32_t)(rows + v_unit_groups(*c, a.tokens))), 256, 0, stream>>>(a, *c, slots, v, v_stride, rows);
  else
    norm_rope_kernel<D, kRows, kInter, false>
        <<<dim3((uint32_t)rows), 256, 0, stream>>>(a, KvCache{}, nullptr, nullptr, 0, rows);
}

// Four rows a thread once that still leaves several workgroups for every
// compute unit: a call of 16381 tokens x 72 heads of 128 takes 121 us (118 of
// them the kernel) against 146 with one, with the cache 139 against 161, 8000
// x 20 heads of 256 36.0 against 38.4 (the row's chain of loads and its
// addresses are paid once for four); 32 tokens x 48 heads 4.5 us against 3.4,
// 1000 x 72 10.8 against 10.3.
template <int D, bool kInter>
void pick_norm_rope(const NormRope& a, const KvCache* c, const int64_t* slots, const uint16_t* v, int64_t v_stride,
                    hipStream_t stream) {
  if (a.tokens * (a.q_heads + a.k_heads) * D >= (int64_t)device_cus() * 4 * 4 * 2048)
    run_norm_rope<D, 4, kInter>(a, c, slots, v, v_stride, stream);
  else
    run_norm_rope<D, 1, kInter>(a, c, slots, v, v_stride, stream);
}

}  // namespace

hipError_t launch_kv_write(const KvCache& c, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int64_t* slots, int64_t tokens, hipStream_t stream) {
  const int64_t kg = k_block_groups(c, tokens), vg = v_unit_groups(c, tokens);
  kv_write_kernel<<<dim3((uint32_t)(kg + vg)), 256, 0, stream>>>(c, (const uint16_t*)k, k_stride, (const uint16_t*)v,
                                                                v_stride, slots, tokens, kg);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, void* k, void* v,
                          hipStream_t stream) {
  const int64_t pieces = tokens * c.heads * (c.head_dim >> 3);
  uint16_t *kp = (uint16_t*)k, *vp = (uint16_t*)v;
  if (pieces >= (int64_t)device_cus() * 4 * 1024) {
    const int64_t kg = run_groups(pieces, 1024);
    const int64_t vg = run_groups(ceil_div(tokens, 16) * ceil_div((int64_t)c.heads * c.head_dim, 128), 4);
    kv_read_kernel<4><<<dim3((uint32_t)(kg + vg)), 256, 0, stream>>>(c, slots, tokens, kp, vp, kg);
  } else {
    const int64_t kg = run_groups(pieces, 256), vg = v_unit_groups(c, tokens);
    kv_read_kernel<1><<<dim3((uint32_t)(kg + vg)), 256, 0, stream>>>(c, slots, tokens, kp, vp, kg);
  }
  return hipGetLastError();
}

hipError_t launch_norm_rope(const NormRope& a, int head_dim, const KvCache* c, const int64_t* slots, const void* v,
                            int64_t v_stride, hipStream_t stream) {
  const uint16_t* vp = (const uint16_t*)v;
  NormRope b = a;
  const uint32_t heads = a.q_heads + a.k_heads;
  b.heads_magic = heads > 1 ? (uint32_t)(((uint64_t(1) << 32) + heads - 1) / heads) : 0;
  if (head_dim == 64 && a.interleaved) pick_norm_rope<64, true>(b, c, slots, vp, v_stride, stream);
  else if (head_dim == 64) pick_norm_rope<64, false>(b, c, slots, vp, v_stride, stream);
  else if (head_dim == 128 && a.interleaved) pick_norm_rope<128, true>(b, c, slots, vp, v_stride, stream);
  else if (head_dim == 128) pick_norm_rope<128, false>(b, c, slots, vp, v_stride, stream);
  else if (a.interleaved) pick_norm_rope<256, true>(b, c, slots, vp, v_stride, stream);
  else pick_norm_rope<256, false>(b, c, slots, vp, v_stride, stream);
  return hipGetLastError();
}

}  // namespace nvfp4k
